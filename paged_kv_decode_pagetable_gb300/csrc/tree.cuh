// Drafted trees of a speculative step, as every tree call reads them: row b's nodes are the
// packed tokens row_start[b] .. row_start[b + 1], node i of a row stands at cache position
// ctx + i and at rotation position ctx + depth(i); parents[n] is the index of a node's parent
// inside its row (before it), -1 for a root.
#pragma once

#include <cstdint>

#include "pkv_internal.h"

namespace {

constexpr int kTreeMax = PKV_TREE_MAX;   // nodes of a row: one bit each of a 64-bit set
constexpr int kTreeRows = 512;           // rows of a call

struct TreeRow {
  int n0, n;        // first node, nodes (0 where something is wrong)
  int slot, ctx;
  int bits;         // PKV_ERR_* of the row
};

// Row b, checked: its nodes lie inside the N packed ones, its slot inside the table and its
// tokens inside a table row.
__device__ __forceinline__ TreeRow tree_row(int b, int N, const int32_t *row_start,
                                            const int32_t *batch_idx, const int32_t *ctx_lens,
                                            int n_slots, int max_pages, int page_size) {
  TreeRow r;
  const int n0 = row_start[b], n1 = row_start[b + 1];
  r.slot = batch_idx ? batch_idx[b] : b;
  r.ctx = ctx_lens[b];
  r.bits = 0;
  r.n0 = n0;
  r.n = n1 - n0;
  if (n0 < 0 || n1 < n0 || n1 > N || n1 - n0 > kTreeMax) {
    r.bits = PKV_ERR_TREE;
    r.n = 0;
    return r;
  }
  if (r.n == 0) return r;   // an empty row names nothing else
  if (r.slot < 0 || r.slot >= n_slots) r.bits |= PKV_ERR_SLOT;
  // (positions are 32-bit numbers, also where a table row has room for more)
  if (r.ctx < 0 || static_cast<long long>(r.ctx) + (n1 - n0) >
                       min(static_cast<long long>(max_pages) * page_size, 0x7fffffffLL))
    r.bits |= PKV_ERR_POS;
  if (r.bits) r.n = 0;
  return r;
}

__device__ __forceinline__ void tree_report(int32_t *err, int bits) {
  if (err && bits) atomicOr(err, bits);
}

// Parent of node i; one that does not lie before it counts as none.
__device__ __forceinline__ int tree_parent(const int32_t *parents, int n0, int i, int &bits) {
  const int p = parents[n0 + i];
  if (p < -1 || p >= i) {
    bits |= PKV_ERR_TREE;
    return -1;
  }
  return p;
}

}  // namespace
