// kv_keep_path: after verification, the accepted nodes' keys and values go from where the tree
// put them to the positions behind the context, in every cache of the model at once:
//   cache token ctx + path[t] -> ctx + t,  t = 1 .. accepted.
//
// A pure copy of few bytes, bound by latency: the row's path, its pages, a load and a store
// behind one another. Paths ascend, so path[t] >= t and a destination never lies behind a later
// source: a thread that owns a column of a (cache, head) and goes through the path in order
// needs no other thread's word. What the copy needs of the path (source and destination rows)
// is looked up once a CTA; tokens that stay where they are cost nothing. Measured: 64 rows in 48
// caches of 8 heads of 128, one launch, 6.6 us (floor 1.9 us of bytes), 8 rows in two 2.9.
#include <cuda_runtime.h>

#include <algorithm>
#include <functional>
#include <memory>
#include <new>
#include <numeric>

#include "pkv_internal.h"
#include "tree.cuh"

namespace {

constexpr int kThreads = 128;
constexpr int kEach = 8;          // tokens in flight
constexpr int kMaxCaches = 64;    // caches of a launch

struct Cache {
  unsigned char *base;
  pkv::Divisor words;   // words of `vec` bytes in a token
  int vec;              // 16, 4 or 1
  int heads;
  uint32_t block0;      // CTAs (of a row) of the caches before this one
};
struct KeepArgs {
  Cache cache[kMaxCaches];
  const int32_t *table, *batch_idx, *ctx_lens, *accepted, *path;
  int32_t *err;
  int n_caches, n_slots, max_pages, page_size, n_pages, path_cols, report;
};

template <typename T>
__device__ __forceinline__ void move(const Cache &k, long long head_rows, const int2 *rows, int n) {
  const uint32_t w = (blockIdx.x - k.block0) * kThreads + threadIdx.x;
  const uint32_t words = k.words.d;
  const uint32_t head = k.words.quotient(w);
  if (head >= static_cast<uint32_t>(k.heads)) return;
  T *col = reinterpret_cast<T *>(k.base) + head * head_rows * words + (w - head * words);
  for (int t0 = 0; t0 < n; t0 += kEach) {
    T v[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (t0 + e < n) v[e] = col[static_cast<long long>(rows[t0 + e].x) * words];
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (t0 + e < n) col[static_cast<long long>(rows[t0 + e].y) * words] = v[e];
  }
}

__global__ void __launch_bounds__(kThreads) keep_path_kernel(const __grid_constant__ KeepArgs a) {
  __shared__ int2 s_rows[kTreeMax];
  __shared__ int s_n;
  pkv_wait_prior_grid();
  pkv_allow_next_grid();
  const int b = blockIdx.y;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const int acc = a.accepted[b], slot = a.batch_idx ? a.batch_idx[b] : b, ctx = a.ctx_lens[b];
    const int32_t *path = a.path + static_cast<long long>(b) * a.path_cols;
    int bits = 0, n = 0;
    if (acc < 0 || acc >= kTreeMax || acc >= a.path_cols) bits = PKV_ERR_TREE;
    else if (acc > 0 && (slot < 0 || slot >= a.n_slots)) bits = PKV_ERR_SLOT;
    else if (acc > 0 && slot != 0) {
      // lanes take nodes 1 + lane and 33 + lane
      int from[2] = {0, 0}, prev[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = 1 + lane + 32 * j;
        if (t <= acc) {
          from[j] = path[t];
          prev[j] = path[t - 1];
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = 1 + lane + 32 * j;
        if (t <= acc && (from[j] <= prev[j] || from[j] < t || from[j] >= kTreeMax))
          bits |= PKV_ERR_TREE;
      }
      const long long room = static_cast<long long>(a.max_pages) * a.page_size;
      if (ctx < 0 || static_cast<long long>(ctx) + kTreeMax > 0x7fffffffLL) bits |= PKV_ERR_POS;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (1 + lane + 32 * j <= acc && static_cast<long long>(ctx) + from[j] >= room)
          bits |= PKV_ERR_POS;
      bits = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(bits));
      if (!bits) {
        const int32_t *pages = a.table + static_cast<long long>(slot) * a.max_pages;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int t = 1 + lane + 32 * j;
          const bool go = t <= acc && from[j] != t;
          int2 r = make_int2(0, 0);
          if (go) {
            const int p = ctx + from[j], d = ctx + t;
            const int pp = pages[p / a.page_size], pd = pages[d / a.page_size];
            if (pp < 0 || pd < 0) bits |= PKV_ERR_PAGE_NEG;
            if (pp >= a.n_pages || pd >= a.n_pages) bits |= PKV_ERR_PAGE_RANGE;
            r = make_int2(pp * a.page_size + p % a.page_size, pd * a.page_size + d % a.page_size);
          }
          const unsigned who = __ballot_sync(0xffffffffu, go);
          if (go) s_rows[n + __popc(who & ((1u << lane) - 1))] = r;
          n += __popc(who);
        }
        bits = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(bits));
      }
    }
    if (bits) n = 0;   // the row is left as it is
    if (lane == 0) {
      s_n = n;
      if (a.report && blockIdx.x == 0) tree_report(a.err, bits);
    }
  }
  __syncthreads();
  const int n = s_n;
  if (n == 0) return;
  int c = 0;   // the last cache that begins at or before this CTA
  for (int step = kMaxCaches / 2; step > 0; step /= 2)
    if (c + step < a.n_caches && a.cache[c + step].block0 <= blockIdx.x) c += step;
  const Cache &k = a.cache[c];
  const long long head_rows = static_cast<long long>(a.n_pages) * a.page_size;
  if (k.vec == 16) move<uint4>(k, head_rows, s_rows, n);
  else if (k.vec == 4) move<uint32_t>(k, head_rows, s_rows, n);
  else move<unsigned char>(k, head_rows, s_rows, n);
}

}  // namespace

extern "C" int kv_keep_path(void *const *caches, const int *heads, const int64_t *token_bytes,
                            int n_caches, const int32_t *dev_table, int n_slots,
                            int max_pages_per_seq, int page_size, int n_pages,
                            const int32_t *batch_idx, const int32_t *ctx_lens,
                            const int32_t *accepted, const int32_t *path, int path_cols, int B,
                            int32_t *err_word, void *stream) {
  static const char *fn = "kv_keep_path";
  if (n_caches < 0 || B < 0 || B > 65535 || path_cols < 1)
    return pkv::fail(PKV_E_BAD_ARG, "%s: bad size argument", fn);
  if (page_size < 1 || n_pages < 1 || n_slots < 1 || max_pages_per_seq < 1 ||
      static_cast<long long>(page_size) * n_pages > 0x7fffffffLL)
    return pkv::fail(PKV_E_BAD_ARG, "%s: bad table geometry", fn);
  if (n_caches == 0 || B == 0) return pkv::ok();
  if (!caches || !heads || !token_bytes || !dev_table || !ctx_lens || !accepted || !path)
    return pkv::fail(PKV_E_BAD_ARG, "%s: NULL pointer", fn);
  const long long rows = static_cast<long long>(page_size) * n_pages;
  bool ascending = true;   // each behind the one before, as a program mostly has them
  uintptr_t end = 0;
  for (int c = 0; c < n_caches; ++c) {
    if (!caches[c]) return pkv::fail(PKV_E_BAD_ARG, "%s: NULL cache", fn);
    if (heads[c] < 1 || heads[c] > 65535 || token_bytes[c] < 1 || token_bytes[c] > (1 << 20) ||
        heads[c] * token_bytes[c] > (1LL << 30) ||
        heads[c] * token_bytes[c] >= (1LL << 46) / rows)
      return pkv::fail(PKV_E_BAD_ARG, "%s: cache %d: bad heads or token_bytes", fn, c);
    const uintptr_t base = reinterpret_cast<uintptr_t>(caches[c]);
    ascending = ascending && base >= end;
    end = base + static_cast<uintptr_t>(heads[c] * token_bytes[c] * rows);
  }
  // The move is in place and each cache's CTAs know nothing of another's: one that is named again
  // (layers may share one) is left to the first, what overlaps otherwise is refused.
  std::unique_ptr<int[]> order;
  int n_all = n_caches;
  if (!ascending) {
    order.reset(new (std::nothrow) int[n_caches]);
    if (!order) return pkv::fail(PKV_E_BAD_ARG, "%s: no memory for %d caches", fn, n_caches);
    std::iota(order.get(), order.get() + n_caches, 0);
    const std::less<const void *> before;
    std::sort(order.get(), order.get() + n_caches, [&](int x, int y) {
      return caches[x] == caches[y] ? x < y : before(caches[x], caches[y]);
    });
    n_all = 1;
    for (int i = 1; i < n_caches; ++i) {
      const int x = order[n_all - 1], y = order[i];   // x: the last that is kept
      if (caches[x] == caches[y] && heads[x] == heads[y] && token_bytes[x] == token_bytes[y])
        continue;
      if (reinterpret_cast<uintptr_t>(caches[y]) - reinterpret_cast<uintptr_t>(caches[x]) <
          static_cast<uintptr_t>(heads[x] * token_bytes[x] * rows))
        return pkv::fail(PKV_E_BAD_ARG, "%s: caches %d and %d overlap", fn, x, y);
      order[n_all++] = y;
    }
  }
  KeepArgs a;
  a.table = dev_table;
  a.batch_idx = batch_idx;
  a.ctx_lens = ctx_lens;
  a.accepted = accepted;
  a.path = path;
  a.err = err_word;
  a.n_slots = n_slots;
  a.max_pages = max_pages_per_seq;
  a.page_size = page_size;
  a.n_pages = n_pages;
  a.path_cols = path_cols;
  for (int c0 = 0; c0 < n_all; c0 += kMaxCaches) {
    long long blocks = 0;
    const int n = n_all - c0 < kMaxCaches ? n_all - c0 : kMaxCaches;
    for (int i = 0; i < n; ++i) {
      Cache &k = a.cache[i];
      const int c = order ? order[c0 + i] : c0 + i;
      k.base = static_cast<unsigned char *>(caches[c]);
      const int64_t bytes = token_bytes[c];
      const uintptr_t both = reinterpret_cast<uintptr_t>(k.base) | bytes;
      k.vec = both % 16 == 0 ? 16 : both % 4 == 0 ? 4 : 1;
      k.words.set(static_cast<uint32_t>(bytes / k.vec));
      k.heads = heads[c];
      k.block0 = static_cast<uint32_t>(blocks);
      blocks += (k.heads * static_cast<long long>(k.words.d) + kThreads - 1) / kThreads;
    }
    if (blocks > 0x7fffffffLL) return pkv::fail(PKV_E_BAD_ARG, "%s: too large", fn);
    a.n_caches = n;
    a.report = c0 == 0;
    PKV_CUDA_CHECK(pkv::launch_pdl(keep_path_kernel, dim3(static_cast<unsigned>(blocks), B),
                                   dim3(kThreads), 0, static_cast<cudaStream_t>(stream), a));
  }
  return pkv::ok();
}
