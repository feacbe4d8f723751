"""Where the parts of smla_prompt_fwd's workspace lie (csrc/prompt_layout.h, compiled for the host)."""
import ctypes
import os
import subprocess

import pytest
import torch

import indexer_top_sparse_score_gb300 as smla

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "indexer_top_sparse_score_gb300", "csrc", "prompt_layout.h")
ROWS, VALUES, HEAD = 512, 128, 256
NAMES = ["plan", "cuts", "blocks", "line_at", "sorted", "block_at", "part_ml", "part_o"]
SOURCE = """
#include "%s"
extern "C" void parts(uintptr_t base, int max_blocks, int pairs, int n_seqs, int can_cut, size_t* o) {
  const smla::PromptParts w = smla::prompt_parts(base, 256, max_blocks, pairs, n_seqs, can_cut != 0);
  const size_t at[] = {w.plan, w.cuts, w.blocks, w.line_at, w.sorted, w.block_at, w.part_ml, w.part_o, w.bytes,
                       sizeof(smla::Plan), sizeof(smla::Cut), sizeof(smla::Block)};
  for (int i = 0; i < 12; ++i) o[i] = at[i];
}
"""


@pytest.fixture(scope="module")
def parts(tmp_path_factory):
    d = tmp_path_factory.mktemp("layout")
    (d / "parts.cpp").write_text(SOURCE % HEADER)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-o", str(d / "parts.so"), str(d / "parts.cpp")], check=True)
    f = ctypes.CDLL(str(d / "parts.so")).parts
    f.argtypes, f.restype = [ctypes.c_size_t] + [ctypes.c_int] * 4 + [ctypes.POINTER(ctypes.c_size_t)], None

    def call(base, max_blocks, pairs, n_seqs, can_cut):
        o = (ctypes.c_size_t * 12)()
        f(base, max_blocks, pairs, n_seqs, int(can_cut), o)
        return dict(zip(NAMES + ["bytes", "Plan", "Cut", "Block"], o))

    return call


SHAPES = [(1, 1, 1), (7, 76, 5), (300, 76, 37), (2501, 75, 2500), (33, 2, 1)]


@pytest.mark.parametrize("max_blocks,pairs,n_seqs", SHAPES)
@pytest.mark.parametrize("lead", range(0, 256, 16))
def test_parts_lie_on_the_boundaries_of_their_accesses(parts, lead, max_blocks, pairs, n_seqs):
    """Every workspace on a 16-byte boundary: partial values are written 32 bytes at a time, their maxima and sums 8,
    the plan's entries 8 and 4; the parts lie in order, none over another, and end within the size."""
    base = (1 << 20) + lead
    w = parts(base, max_blocks, pairs, n_seqs, True)
    assert (base + w["part_o"]) % 32 == 0
    for name, n in (("part_ml", 8), ("plan", 8), ("line_at", 8), ("cuts", 16), ("blocks", 16), ("sorted", 16), ("block_at", 4)):
        assert (base + w[name]) % n == 0, name
    rows = 2 * pairs * ROWS
    sizes = dict(plan=w["Plan"], cuts=pairs * w["Cut"], blocks=max_blocks * w["Block"], line_at=8 * max_blocks, sorted=max_blocks * w["Block"],
                 block_at=4 * (n_seqs + 1), part_ml=8 * rows, part_o=4 * VALUES * rows)
    end = HEAD
    for name in NAMES:
        assert w[name] >= end, name
        end = w[name] + sizes[name]
    assert end <= w["bytes"] == parts(0, max_blocks, pairs, n_seqs, True)["bytes"]


@pytest.mark.parametrize("max_blocks,pairs,n_seqs", SHAPES)
def test_without_pieces(parts, max_blocks, pairs, n_seqs):
    w = parts(1 << 20, max_blocks, pairs, n_seqs, False)
    assert w["part_ml"] == w["part_o"] == 0 and w["bytes"] >= w["block_at"] + 4 * (n_seqs + 1)


@pytest.mark.skipif(torch.cuda.is_available(), reason="one pair where there is no GPU")
@pytest.mark.parametrize("total_q,total_k,n_seqs", [(100, 300, 3), (100, 30000, 3), (16384, 16384, 1), (15, 45000, 5)])
def test_size_function_is_the_layouts(parts, total_q, total_k, n_seqs):
    smla.build()
    got = smla.lib().smla_prompt_fwd_workspace_size(total_q, total_k, n_seqs, 64, 64)
    assert got == parts(0, total_q // ROWS + n_seqs, 1, n_seqs, total_k > 1024)["bytes"]
