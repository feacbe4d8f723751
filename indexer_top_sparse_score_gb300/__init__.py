"""Indexer-selected sparse MLA for one GB300: thin Python binding of libsmla.so.

Every step of the layer (indexer, causal top-k, sparse MLA) runs in the CUDA
kernels of ``csrc/`` behind the C ABI declared in ``include/smla.h``. This
module only marshals torch tensors (device memory, the current stream) into
that ABI. There is no CPU fallback: if the library is not built, every call
raises.
"""
from __future__ import annotations

import ctypes
import os
import subprocess
import threading
from concurrent.futures import ThreadPoolExecutor
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
_CSRC = os.path.join(_HERE, "csrc")
_INCLUDE = os.path.join(os.path.dirname(_HERE), "include")
_BUILD = os.path.join(_HERE, "_build")
LIB_PATH = os.path.join(_BUILD, "libsmla.so")
SOURCES = ["api.cu", "indexer.cu", "mla.cu", "noalloc.cu", "prefix.cu", "serve.cu"]
NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC"]

SMLA_BF16, SMLA_FP8_E4M3, SMLA_FP8_DS_MLA = 0, 1, 2
STATUS = {0: "SMLA_OK", 1: "SMLA_ERR_INVALID_ARG", 2: "SMLA_ERR_UNSUPPORTED", 3: "SMLA_ERR_WORKSPACE",
          4: "SMLA_ERR_CUDA", 5: "SMLA_ERR_DEVICE_BOUNDS", 6: "SMLA_ERR_TIMEOUT"}
D_QK, D_V, PAGE = 576, 512, 64
STATUS_BYTES = 256  # the status word heads every workspace

_lock = threading.Lock()
_lib = None


class SmlaError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {STATUS.get(code, code)}")


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    deps = [os.path.join(_CSRC, f) for f in os.listdir(_CSRC)] + [os.path.join(_INCLUDE, f)
                                                                  for f in os.listdir(_INCLUDE)]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/*.cu for sm_103a into _build/libsmla.so (in-tree)."""
    if not force and not _stale():
        return LIB_PATH
    os.makedirs(_BUILD, exist_ok=True)
    nvcc = _nvcc()
    objs = [os.path.join(_BUILD, s.replace(".cu", ".o")) for s in SOURCES]

    def compile_one(i):
        cmd = [nvcc, *NVCC_FLAGS, "-c", os.path.join(_CSRC, SOURCES[i]), "-o", objs[i]]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {SOURCES[i]}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            print(r.stdout, r.stderr)

    with ThreadPoolExecutor(len(SOURCES)) as ex:
        list(ex.map(compile_one, range(len(SOURCES))))
    tmp = LIB_PATH + f".{os.getpid()}.tmp"
    cmd = [nvcc, "-shared", "-gencode", "arch=compute_103a,code=sm_103a", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


class PagedCache(ctypes.Structure):
    _fields_ = [("kv", ctypes.c_void_p), ("kv_scale", ctypes.c_void_p), ("k_idx", ctypes.c_void_p),
                ("k_idx_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
                ("idx_dtype", ctypes.c_int32), ("d_idx", ctypes.c_int32)]


_vp, _i32, _sz, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
_SIGS = {
    "smla_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "smla_version": (ctypes.c_int, []),
    "smla_indexer_topk_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32]),
    "smla_indexer_topk": (ctypes.c_int, [_vp, _vp, _i32, _i32, _vp, _i32, _i32, _vp, _vp, _i32, _i32, _vp,
                                          _vp, _vp, _sz, _vp]),
    "smla_sparse_mla_fwd_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32]),
    "smla_sparse_mla_fwd": (ctypes.c_int, [_vp, _vp, _i32, _i32, _vp, _i32, _i32, _vp, _i32, _vp, _i32, _f32,
                                            _vp, _vp, _vp, _sz, _vp]),
    "smla_sparse_mla_prefill_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32]),
    "smla_sparse_mla_prefill": (ctypes.c_int, [_vp, _vp, _i32, _i32, _vp, _i32, _vp, _vp, _i32, _i32, _f32,
                                                _vp, _vp, _vp, _vp, _sz, _vp]),
    "smla_sparse_mla_decode_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32]),
    "smla_sparse_mla_decode": (ctypes.c_int, [_vp, _vp, _i32, _i32, _vp, _i32, _i32, _vp, _i32, _vp, _vp, _i32,
                                               _i32, _f32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "smla_sparse_mla_prefill_noalloc": (ctypes.c_int, [_vp, _vp, _i32, _i32, _vp, _i32, _vp, _vp, _i32, _i32,
                                                        _f32, _vp, _vp, _vp]),
    "smla_noalloc_read_status": (ctypes.c_int, [_vp, ctypes.POINTER(ctypes.c_uint32)]),
    "smla_read_status": (ctypes.c_int, [_vp, _vp, ctypes.POINTER(ctypes.c_uint32)]),
}

class RopeTable(ctypes.Structure):
    """smla_rope: cos_sin [max_pos][64] and the pairing of the rotated values."""
    _fields_ = [("cos_sin", ctypes.c_void_p), ("max_pos", ctypes.c_int32), ("kv_interleaved", ctypes.c_int32),
                ("idx_interleaved", ctypes.c_int32)]


_i64 = ctypes.c_int64
# include/smla_serve.h
_SERVE_SIGS = {
    "smla_build_tables": (ctypes.c_int, [_vp, _vp, _i32, _vp, _i32, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp,
                                         _vp, _sz, _vp]),
    "smla_cache_append": (ctypes.c_int, [_vp, _vp, _i32, _vp, _vp, _vp, _i64, _vp, _vp, _i64, _vp, _vp, _f32, _vp,
                                         _sz, _vp]),
    "smla_query_prep": (ctypes.c_int, [_vp, _i32, _vp, _vp, _i64, _i64, _i32, _vp, _vp, _i64, _i32, _i32, _i32, _vp,
                                       _f32, _vp, _f32, _vp, _vp, _vp, _sz, _vp]),
    "smla_shared_prefix_fwd_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32]),
    "smla_shared_prefix_fwd": (ctypes.c_int, [_vp, _vp, _i32, _i32, _vp, _i32, _i32, _i32, _vp, _i32, _f32, _vp, _vp,
                                              _vp, _sz, _vp]),
}


def lib(build_if_missing: bool = False):
    """The loaded libsmla.so. Raises if it has not been built (no fallback)."""
    global _lib
    with _lock:
        if _lib is None:
            if build_if_missing:
                build()
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"libsmla.so is not built ({LIB_PATH}); run "
                                   "indexer_top_sparse_score_gb300.build() first")
            L = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in {**_SIGS, **_SERVE_SIGS}.items():
                f = getattr(L, name)
                f.restype = res
                f.argtypes = args
            _lib = L
    return _lib


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _check(rc: int, what: str):
    if rc != 0:
        raise SmlaError(rc, what)


def _dtype_code(name: str) -> int:
    return {"bf16": SMLA_BF16, "fp8": SMLA_FP8_E4M3, "fp8_ds_mla": SMLA_FP8_DS_MLA}[name]


def make_cache(cache) -> PagedCache:
    """C view of a paged cache object with kv / kv_scale / k_idx / k_idx_scale
    tensors and kv_dtype / idx_dtype names ("bf16" or "fp8")."""
    return PagedCache(kv=_p(cache.kv), kv_scale=_p(cache.kv_scale), k_idx=_p(cache.k_idx),
                      k_idx_scale=_p(cache.k_idx_scale), num_pages=cache.kv.shape[0],
                      page_size=cache.kv.shape[1], kv_dtype=_dtype_code(cache.kv_dtype),
                      idx_dtype=_dtype_code(cache.idx_dtype), d_idx=cache.k_idx.shape[-1])


# torch's current stream as an integer, without the Stream object that
# torch.cuda.current_stream() builds (where this torch has the call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    return torch.empty(max(256, (nbytes + 255) // 256 * 256), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------------------- entry points
def indexer_topk(cache, page_tables, seq_lens, max_seq_len, q_per_seq, q_idx, w, topk, out_idx=None,
                 out_scores=None, ws=None, stream=None, want_scores=False):
    """Steps 1-2 for n_seqs sequences of q_per_seq query rows (see smla_indexer_topk)."""
    L = lib()
    pt = page_tables if page_tables.dim() == 2 else page_tables[None]
    n_seqs, max_pages = pt.shape
    rows = n_seqs * q_per_seq
    h_idx = q_idx.shape[1]
    if out_idx is None:
        out_idx = torch.empty((rows, topk), dtype=torch.int32, device=q_idx.device)
    if want_scores and out_scores is None:
        out_scores = torch.empty((rows, topk), dtype=torch.float32, device=q_idx.device)
    need = L.smla_indexer_topk_workspace_size(n_seqs, max_seq_len, q_per_seq, h_idx, topk)
    if ws is None:
        ws = workspace(need, q_idx.device)
    c = make_cache(cache)
    rc = L.smla_indexer_topk(ctypes.byref(c), _p(pt), max_pages, n_seqs, _p(seq_lens), max_seq_len,
                             q_per_seq, _p(q_idx), _p(w), h_idx, topk, _p(out_idx), _p(out_scores),
                             _p(ws), ws.numel(), _stream(stream))
    _check(rc, "smla_indexer_topk")
    return (out_idx, out_scores, ws) if want_scores else (out_idx, ws)


def sparse_mla_fwd(cache, page_tables, q, idx, sm_scale, *, prefix_len=0, seq_lens=None, q_per_seq=None,
                   out=None, lse=None, ws=None, stream=None):
    """Step 3 over given index lists (see smla_sparse_mla_fwd)."""
    L = lib()
    pt = page_tables if page_tables.dim() == 2 else page_tables[None]
    n_seqs, max_pages = pt.shape
    rows, H, _ = q.shape
    topk = idx.shape[1]
    if q_per_seq is None:
        q_per_seq = rows // n_seqs
    if out is None:
        out = torch.empty((rows, H, D_V), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((rows, H), dtype=torch.float32, device=q.device)
    if ws is None:
        max_keys = prefix_len + q_per_seq if seq_lens is None else 0
        ws = workspace(L.smla_sparse_mla_fwd_workspace_size(max_keys, rows, H, topk, _dtype_code(cache.kv_dtype)),
                       q.device)
    c = make_cache(cache)
    rc = L.smla_sparse_mla_fwd(ctypes.byref(c), _p(pt), max_pages, n_seqs, _p(seq_lens), prefix_len,
                               q_per_seq, _p(q), H, _p(idx), topk, float(sm_scale), _p(out), _p(lse),
                               _p(ws), ws.numel(), _stream(stream))
    _check(rc, "smla_sparse_mla_fwd")
    return out, lse, ws


def prefill_workspace_bytes(prefix_len, n_tokens, n_heads, h_idx, topk, kv_dtype="bf16") -> int:
    return lib().smla_sparse_mla_prefill_workspace_size(prefix_len, n_tokens, n_heads, h_idx, topk,
                                                        _dtype_code(kv_dtype))


def sparse_mla_prefill(cache, page_table, prefix_len, q, q_idx, w, topk, sm_scale, *, out=None, lse=None,
                       out_idx=None, ws=None, stream=None):
    """Steps 1-3 for the new tokens of one sequence (see smla_sparse_mla_prefill)."""
    L = lib()
    T, H, _ = q.shape
    h_idx = q_idx.shape[1]
    if out is None:
        out = torch.empty((T, H, D_V), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(prefill_workspace_bytes(prefix_len, T, H, h_idx, topk, cache.kv_dtype), q.device)
    c = make_cache(cache)
    rc = L.smla_sparse_mla_prefill(ctypes.byref(c), _p(page_table), prefix_len, T, _p(q), H, _p(q_idx), _p(w),
                                   h_idx, topk, float(sm_scale), _p(out), _p(lse), _p(out_idx), _p(ws),
                                   ws.numel(), _stream(stream))
    _check(rc, "smla_sparse_mla_prefill")
    return out, lse, out_idx, ws


def chunk_bounds(n_tokens: int, chunk) -> list:
    """[(start, end)] of the query-token chunks of HostPrefill: `chunk` is a size
    (the last chunk takes the rest) or a list of sizes that sum to n_tokens."""
    if isinstance(chunk, int):
        if chunk <= 0:
            raise ValueError("chunk size must be positive")
        return [(a, min(n_tokens, a + chunk)) for a in range(0, n_tokens, chunk)]
    sizes = [int(c) for c in chunk]
    if any(c <= 0 for c in sizes) or sum(sizes) != n_tokens:
        raise ValueError("chunk sizes must be positive and sum to n_tokens")
    bounds = [0]
    for c in sizes:
        bounds.append(bounds[-1] + c)
    return list(zip(bounds[:-1], bounds[1:]))


class HostPrefill:
    """Prefill from pinned HOST buffers: q, q_idx and w are copied in and out /
    lse copied back chunk by chunk, on two copy streams, so the copies of one
    chunk overlap the kernels of its neighbours. The kernels run on a stream
    of the object's own, joined to the caller's stream by one event at each
    end: work on the legacy default stream waits for every other blocking
    stream, so running the kernels there would hold each chunk's copies back
    until the kernels before them end. Each chunk of query tokens is
    one smla_sparse_mla_prefill call with the earlier tokens as its prefix (the
    cache already holds every token's rows), which gives the same rows the
    single call would. `chunk` is a chunk size, or a list of chunk sizes that
    sum to n_tokens (small first and last chunks shorten the copy-in before
    the first kernel and the copy-out after the last). Device buffers,
    workspace, streams and events are made once here; run() may be called
    repeatedly (each call waits for the previous call's use of a chunk's
    device buffers before reusing them).

    Chunk c is given the workspace from byte 256 * c on, so its status word
    (the first 256 bytes of what it is given) is its own: the scratch of chunk c
    covers only the status words of later chunks, which clear theirs when they
    start, so after run() every chunk's word is intact and read_status() reports
    the device errors of all of them.
    """

    def __init__(self, cache, page_table, prefix_len, n_tokens, n_heads, h_idx, d_idx, idx_dtype, topk,
                 sm_scale, chunk=2048, device="cuda"):
        self.cache, self.page_table, self.prefix_len = cache, page_table, prefix_len
        self.T, self.topk, self.sm_scale = n_tokens, topk, sm_scale
        self.chunks = chunk_bounds(n_tokens, chunk)
        idx_t = torch.bfloat16 if idx_dtype == "bf16" else torch.uint8
        self.q = torch.empty((n_tokens, n_heads, D_QK), dtype=torch.bfloat16, device=device)
        self.q_idx = torch.empty((n_tokens, h_idx, d_idx), dtype=idx_t, device=device)
        self.w = torch.empty((n_tokens, h_idx), dtype=torch.float32, device=device)
        self.out = torch.empty((n_tokens, n_heads, D_V), dtype=torch.bfloat16, device=device)
        self.lse = torch.empty((n_tokens, n_heads), dtype=torch.float32, device=device)
        need = max(prefill_workspace_bytes(prefix_len + a, b - a, n_heads, h_idx, topk, cache.kv_dtype)
                   for a, b in self.chunks)
        self.ws = workspace(need + STATUS_BYTES * len(self.chunks), device)
        self.s_in, self.s_out = torch.cuda.Stream(device), torch.cuda.Stream(device)
        self.s_comp = torch.cuda.Stream(device)
        n = len(self.chunks)
        self.ev_in = [torch.cuda.Event() for _ in range(n)]
        self.ev_comp = [torch.cuda.Event() for _ in range(n)]
        self.ev_out = [torch.cuda.Event() for _ in range(n)]

    def run(self, q_h, q_idx_h, w_h, out_h, lse_h, stream=None):
        caller = torch.cuda.current_stream() if stream is None else stream
        comp = self.s_comp
        start = torch.cuda.Event()
        start.record(caller)
        comp.wait_event(start)
        self.s_in.wait_event(start)
        self.s_out.wait_event(start)
        for c, (a, b) in enumerate(self.chunks):
            with torch.cuda.stream(self.s_in):
                self.s_in.wait_event(self.ev_comp[c])  # the previous run's kernels read these inputs
                self.q[a:b].copy_(q_h[a:b], non_blocking=True)
                self.q_idx[a:b].copy_(q_idx_h[a:b], non_blocking=True)
                self.w[a:b].copy_(w_h[a:b], non_blocking=True)
                self.ev_in[c].record(self.s_in)
            comp.wait_event(self.ev_in[c])
            comp.wait_event(self.ev_out[c])  # the previous run's copy-out of these outputs
            sparse_mla_prefill(self.cache, self.page_table, self.prefix_len + a, self.q[a:b], self.q_idx[a:b],
                               self.w[a:b], self.topk, self.sm_scale, out=self.out[a:b], lse=self.lse[a:b],
                               ws=self.ws[STATUS_BYTES * c:], stream=comp)
            self.ev_comp[c].record(comp)
            with torch.cuda.stream(self.s_out):
                self.s_out.wait_event(self.ev_comp[c])
                out_h[a:b].copy_(self.out[a:b], non_blocking=True)
                lse_h[a:b].copy_(self.lse[a:b], non_blocking=True)
                self.ev_out[c].record(self.s_out)
        for c in range(len(self.chunks)):
            caller.wait_event(self.ev_out[c])  # the call ends on `stream` once every result is on the host
        done = torch.cuda.Event()
        done.record(comp)
        caller.wait_event(done)

    def read_status(self, stream=None):
        """(status code, raw bits) over every chunk of the last run() (waits on
        the stream)."""
        return read_status_chunks(self.ws, len(self.chunks), stream)


# precedence of the device status codes (as smla_read_status orders them)
_STATUS_RANK = {0: 0, 2: 1, 5: 2, 6: 3}


def read_status_chunks(ws: torch.Tensor, n_chunks: int, stream=None):
    """Status of n_chunks calls whose workspaces start at ws + 256 * c: the most
    severe code and the union of the raw bits."""
    code, bits = 0, 0
    for c in range(n_chunks):
        rc, b = read_status(ws[STATUS_BYTES * c:], stream)
        bits |= b
        if _STATUS_RANK.get(rc, 4) > _STATUS_RANK.get(code, 4):
            code = rc
    return code, bits


def decode_workspace_bytes(n_seqs, max_seq_len, q_per_seq, n_heads, h_idx, topk) -> int:
    return lib().smla_sparse_mla_decode_workspace_size(n_seqs, max_seq_len, q_per_seq, n_heads, h_idx, topk)


def sparse_mla_decode(cache, page_tables, seq_lens, max_seq_len, q_per_seq, q, q_idx, w, topk, sm_scale, *,
                      out=None, lse=None, out_idx=None, ws=None, stream=None):
    """Steps 1-3 for a decode batch (see smla_sparse_mla_decode)."""
    L = lib()
    n_seqs, max_pages = page_tables.shape
    rows, H, _ = q.shape
    h_idx = q_idx.shape[1]
    if out is None:
        out = torch.empty((rows, H, D_V), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((rows, H), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(decode_workspace_bytes(n_seqs, max_seq_len, q_per_seq, H, h_idx, topk), q.device)
    c = make_cache(cache)
    rc = L.smla_sparse_mla_decode(ctypes.byref(c), _p(page_tables), max_pages, n_seqs, _p(seq_lens),
                                  max_seq_len, q_per_seq, _p(q), H, _p(q_idx), _p(w), h_idx, topk,
                                  float(sm_scale), _p(out), _p(lse), _p(out_idx), _p(ws), ws.numel(),
                                  _stream(stream))
    _check(rc, "smla_sparse_mla_decode")
    return out, lse, out_idx, ws


# ---------------------------------------------------------------------------- serving steps
# The checks here are plain ifs on attributes: at decode sizes a call costs the host
# about as much as the GPU.
_I32, _F32, _BF16 = torch.int32, torch.float32, torch.bfloat16


def _int32(*tensors):
    for t in tensors:
        if t is not None and (t.dtype is not _I32 or not t.is_contiguous()):
            raise ValueError("lengths, tables, positions and maps are contiguous int32 tensors")


def _fp32(t, n, what):
    if t is not None and (t.dtype is not _F32 or t.numel() != n or not t.is_contiguous()):
        raise ValueError(f"{what} is a contiguous fp32 tensor of {n} values")


def build_tables(ctx_lens, new_lens, page_tables, free_pages, max_new, *, seq_lens=None, cu_new=None,
                 positions=None, slots=None, row_seq=None, pages_used=None, ws=None, stream=None):
    """Pages and slots of every request's next tokens (see smla_build_tables);
    page_tables is updated in place. Returns (seq_lens, cu_new, positions, slots,
    row_seq, pages_used, ws)."""
    L = lib()
    _int32(ctx_lens, new_lens, page_tables, free_pages, seq_lens, cu_new, positions, slots, row_seq, pages_used)
    n, max_pages = page_tables.shape
    if ctx_lens.numel() != n or new_lens.numel() != n:
        raise ValueError("ctx_lens and new_lens have one length per row of page_tables")
    dev = page_tables.device

    def out(t, k):
        if t is None:
            return torch.empty(k, dtype=_I32, device=dev)
        if t.numel() < k:
            raise ValueError("an output is too small")
        return t

    seq_lens, cu_new, pages_used = out(seq_lens, n), out(cu_new, n + 1), out(pages_used, 1)
    positions, slots, row_seq = out(positions, max_new), out(slots, max_new), out(row_seq, max_new)
    if ws is None:
        ws = workspace(STATUS_BYTES, dev)
    rc = L.smla_build_tables(ctx_lens.data_ptr(), new_lens.data_ptr(), n, page_tables.data_ptr(), max_pages,
                             _p(free_pages), 0 if free_pages is None else free_pages.numel(), max_new,
                             seq_lens.data_ptr(), cu_new.data_ptr(), positions.data_ptr(), slots.data_ptr(),
                             row_seq.data_ptr(), pages_used.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream))
    _check(rc, "smla_build_tables")
    return seq_lens, cu_new, positions, slots, row_seq, pages_used, ws


def _rope(table, kv_interleaved, idx_interleaved) -> RopeTable:
    if table.dtype is not _F32 or table.dim() != 2 or table.shape[1] != 64 or not table.is_contiguous():
        raise ValueError("rope is a contiguous fp32 [max_pos, 64] table")
    return RopeTable(table.data_ptr(), table.shape[0], int(kv_interleaved), int(idx_interleaved))


def _bf16_rows(t, rows, width):
    """Row stride of a [rows, width] bf16 matrix whose rows are dense."""
    if t is None:
        return 0
    if t.dtype is not _BF16 or t.dim() != 2 or t.shape[0] != rows or t.shape[1] != width or t.stride(1) != 1:
        raise ValueError(f"rows are bf16 [{rows}, {width}] with a row's values next to each other")
    return t.stride(0) if rows > 1 else -(-width // 8) * 8


def cache_append(cache, slots, positions, rope, *, ckv=None, kv_norm=None, k_idx=None, idx_norm=None, idx_bias=None,
                 eps=1e-6, kv_interleaved=True, idx_interleaved=False, ws=None, stream=None):
    """Norm, rotation, quantisation and paged write of new latent rows (ckv
    [rows, 576] bf16) and indexer keys (k_idx [rows, d_idx] bf16) into `cache`
    (see smla_cache_append). Rows may be strided. Returns ws."""
    L = lib()
    rows = slots.numel()
    _int32(slots, positions)
    if positions.numel() != rows:
        raise ValueError("positions and slots have one entry per row")
    d = cache.k_idx.shape[-1]
    kv_stride, k_stride = _bf16_rows(ckv, rows, D_QK), _bf16_rows(k_idx, rows, d)
    _fp32(kv_norm, D_V, "kv_norm")
    _fp32(idx_norm, d, "idx_norm")
    _fp32(idx_bias, d, "idx_bias")
    if ws is None:
        ws = workspace(STATUS_BYTES, slots.device)
    c, r = make_cache(cache), _rope(rope, kv_interleaved, idx_interleaved)
    rc = L.smla_cache_append(ctypes.byref(c), ctypes.byref(r), rows, slots.data_ptr(), positions.data_ptr(), _p(ckv),
                             kv_stride, _p(kv_norm), _p(k_idx), k_stride, _p(idx_norm), _p(idx_bias), eps,
                             ws.data_ptr(), ws.numel(), _stream(stream))
    _check(rc, "smla_cache_append")
    return ws


def query_prep(positions, rope, *, q_pe=None, q=None, q_idx_raw=None, w=None, idx_dtype="fp8", idx_norm=None,
               eps=1e-6, w_scale=1.0, kv_interleaved=True, idx_interleaved=False, q_idx=None, w_out=None, ws=None,
               stream=None):
    """Rotation of the attention queries' 64 rope values (q_pe [rows, H, 64],
    strided) into the last 64 values of q [rows, H, 576], and norm, rotation and
    quantisation of the indexer queries q_idx_raw [rows, h_idx, d_idx] with the
    scale folded into the head weights (see smla_query_prep). Returns (q, q_idx,
    w_out, ws)."""
    L = lib()
    rows = positions.numel()
    _int32(positions)
    n_heads = h_idx = d_idx = pe_row = pe_head = raw_row = 0
    if q_pe is not None:
        n, n_heads, d = q_pe.shape
        pe_row, pe_head, unit = q_pe.stride()
        if q_pe.dtype is not _BF16 or n != rows or d != D_QK - D_V or unit != 1:
            raise ValueError("q_pe is bf16 [rows, heads, 64] with a head's values next to each other")
        if rows == 1:
            pe_row = 0
        if q is None:
            q = torch.empty((rows, n_heads, D_QK), dtype=_BF16, device=q_pe.device)
        elif q.dtype is not _BF16 or q.numel() != rows * n_heads * D_QK or not q.is_contiguous():
            raise ValueError("q is contiguous bf16 [rows, heads, 576]")
    if q_idx_raw is not None:
        n, h_idx, d_idx = q_idx_raw.shape
        raw_row, head, unit = q_idx_raw.stride()
        values = rows * h_idx * d_idx
        if q_idx_raw.dtype is not _BF16 or n != rows or unit != 1 or (head != d_idx and h_idx > 1):
            raise ValueError("q_idx_raw is bf16 [rows, h_idx, d_idx], each row dense")
        if rows == 1:
            raw_row = h_idx * d_idx
        if w is None:
            raise ValueError("indexer queries need their head weights w")
        _fp32(w, rows * h_idx, "w")
        _fp32(w_out, rows * h_idx, "w_out")
        _fp32(idx_norm, d_idx, "idx_norm")
        if q_idx is None:
            q_idx = torch.empty((rows, h_idx, d_idx), device=w.device, dtype=_BF16 if idx_dtype == "bf16" else torch.uint8)
        elif q_idx.numel() != values or q_idx.element_size() != (2 if idx_dtype == "bf16" else 1) or not q_idx.is_contiguous():
            raise ValueError("q_idx is contiguous [rows, h_idx, d_idx] of idx_dtype")
        if w_out is None:
            w_out = torch.empty_like(w)
    if ws is None:
        ws = workspace(STATUS_BYTES, positions.device)
    r = _rope(rope, kv_interleaved, idx_interleaved)
    rc = L.smla_query_prep(ctypes.byref(r), rows, positions.data_ptr(), _p(q_pe), pe_row, pe_head, n_heads, _p(q),
                           _p(q_idx_raw), raw_row, h_idx, d_idx, _dtype_code(idx_dtype), _p(idx_norm), eps, _p(w),
                           w_scale, _p(q_idx), _p(w_out), ws.data_ptr(), ws.numel(), _stream(stream))
    _check(rc, "smla_query_prep")
    return q, q_idx, w_out, ws


def shared_prefix_workspace_bytes(n_seqs, max_seq_len, shared_len, q_per_seq, n_heads, kv_dtype="bf16") -> int:
    return lib().smla_shared_prefix_fwd_workspace_size(n_seqs, max_seq_len, shared_len, q_per_seq, n_heads,
                                                       _dtype_code(kv_dtype))


def shared_prefix_fwd(cache, page_tables, seq_lens, max_seq_len, shared_len, q_per_seq, q, sm_scale, *, out=None,
                      lse=None, ws=None, stream=None):
    """Attention of a batch whose requests share their first shared_len tokens:
    the shared part is read once for all query rows (see smla_shared_prefix_fwd).
    Returns (out, lse, ws)."""
    L = lib()
    n_seqs, max_pages = page_tables.shape
    rows, H, _ = q.shape
    _int32(page_tables, seq_lens)
    if q.dtype is not _BF16 or not q.is_contiguous() or q.shape[2] != D_QK or rows != n_seqs * q_per_seq:
        raise ValueError("q is contiguous bf16 [n_seqs * q_per_seq, heads, 576]")
    if seq_lens.numel() != n_seqs:
        raise ValueError("seq_lens has one length per row of page_tables")
    if out is None:
        out = torch.empty((rows, H, D_V), dtype=_BF16, device=q.device)
    elif out.dtype is not _BF16 or out.numel() != rows * H * D_V or not out.is_contiguous():
        raise ValueError("out is contiguous bf16 [rows, heads, 512]")
    if lse is None:
        lse = torch.empty((rows, H), dtype=_F32, device=q.device)
    else:
        _fp32(lse, rows * H, "lse")
    if ws is None:
        ws = workspace(shared_prefix_workspace_bytes(n_seqs, max_seq_len, shared_len, q_per_seq, H, cache.kv_dtype),
                       q.device)
    c = make_cache(cache)
    rc = L.smla_shared_prefix_fwd(ctypes.byref(c), page_tables.data_ptr(), max_pages, n_seqs, seq_lens.data_ptr(),
                                  max_seq_len, shared_len, q_per_seq, q.data_ptr(), H, sm_scale, out.data_ptr(),
                                  lse.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream))
    _check(rc, "smla_shared_prefix_fwd")
    return out, lse, ws


def read_status(ws: torch.Tensor, stream=None):
    """(status code, raw bits) of the device status word in `ws` (waits on the stream)."""
    bits = ctypes.c_uint32(0)
    rc = lib().smla_read_status(_p(ws), _stream(stream), ctypes.byref(bits))
    return rc, bits.value
