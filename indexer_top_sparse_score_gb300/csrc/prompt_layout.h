// The workspace of smla_prompt_fwd: its parts and where they lie. Plain C++, so that the addresses can be
// checked without a GPU.
#pragma once
#include <cstddef>
#include <cstdint>

namespace smla {

constexpr int kPromptRows = 512;  // rows of a block
constexpr int kPromptVal = 128;   // values of a head's v

struct Block {      // of the plan
  int32_t tok0, n_tok;    // rows of q
  int32_t key0, lim0;     // first key's row; keys that its first token sees (causal: may be <= 0)
  int32_t n_keys, tiles;  // keys that its last token sees; tiles of them, at least one
  int32_t pad[2];
};
struct Cut {              // a block and head group whose pieces lie with the pairs from this one on (pieces 0: none)
  int32_t tok0, n_tok, unit, pieces;
};
struct Plan {
  unsigned long long next;  // item to be taken
  long long line;           // length of the line of work
  int32_t n_blocks, even;   // even: the line is cut evenly
  int32_t pairs;            // stretches of the line
};

// Bytes from the workspace's start.
struct PromptParts {
  size_t plan, cuts, blocks, line_at, sorted, block_at;
  size_t part_ml, part_o;  // partial results; 0: none
  size_t bytes;            // of all of it
};

// `base` is the workspace's address, on a 16-byte boundary. Partial values are written 32 bytes at a time and
// start on a boundary of those; bytes has the room for that whatever the base.
inline PromptParts prompt_parts(uintptr_t base, size_t head, int32_t max_blocks, int32_t pairs, int32_t n_seqs, bool can_cut) {
  auto up = [](size_t b, size_t to) { return (b + to - 1) / to * to; };
  PromptParts w{};
  size_t at = head;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += up(n, 256);
    return here;
  };
  w.plan = take(sizeof(Plan));
  w.cuts = take(static_cast<size_t>(pairs) * sizeof(Cut));
  w.blocks = take(static_cast<size_t>(max_blocks) * sizeof(Block));
  w.line_at = take(static_cast<size_t>(max_blocks) * 8);
  w.sorted = take(static_cast<size_t>(max_blocks) * sizeof(Block));
  w.block_at = take((static_cast<size_t>(n_seqs) + 1) * 4);
  if (can_cut) {
    const size_t rows = static_cast<size_t>(pairs) * 2 * kPromptRows;
    w.part_ml = take(rows * 8);
    w.part_o = static_cast<size_t>(up(base + at, 32) - base);
    at += rows * kPromptVal * 4 + 16;
  }
  w.bytes = at;
  return w;
}

}  // namespace smla
