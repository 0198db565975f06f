// kv_copy_pages: copies of pages inside caches (forked, rewound and compacted
// sequences).
//
// A pure copy: bound by reading and writing the pages once. The pairs and the caches'
// descriptions travel as kernel parameters, so a call uploads nothing and can be
// captured. A cache's pages to copy, head by head, are laid end to end and cut into
// equal tiles of 16-byte vectors (smaller words where a cache is not so aligned), one a
// CTA, whatever the page size; a thread has four loads in flight before it stores. CTAs of
// 128 threads, four words each: 43.7 us where the sources repeat and 2.2 for one page; 256
// threads 45.0 and 2.5, 512 47.7 and 2.9; 256 with two words 48.5 and 2.0, with eight 47.7
// and 3.4; larger copies alike to 1%.
// Measured against a copy at 6789 GB/s: 1311 pages of two bf16 layers moved together 197 us
// (1.03 of it), 448 pages of 64 forked prompts on four 8-bit layers 43.7 us (1.58: each
// source is read from memory once; 0.91 by the bytes that move; bound by issuing its
// instructions, 54.7 us, when it divided by numbers only known at run time), 2000 pages of 1 KB x 8
// heads x 8 caches 40.4 us (0.96); one page 2.2 us, the latency of a launch and of a load
// behind another.
#include <cuda_runtime.h>

#include <vector>

#include "pkv_internal.h"

namespace {

constexpr int kThreads = 128;
constexpr int kEach = 4;                      // words a thread copies
constexpr int kTile = kThreads * kEach;

struct Cache {
  unsigned char *base;
  long long head_bytes;   // from one head to the next
  pkv::Divisor page_words;     // words of `vec` bytes in a page
  int vec;                // 16, 4 or 1
  uint32_t block0;        // CTAs of the caches before this one
  uint32_t rows;          // pages to copy: pairs x heads
};

// Kernel parameters may hold 32,764 bytes. A call of few pairs (a fork) passes 4 KB of them
// instead of 31: 9.3 to 10.2 us of host time with four caches against 10.6 to 11.1.
constexpr int kMaxCaches = 64;
constexpr int kMaxPairs = 3500;
template <int NP>
struct CopyArgs {
  Cache cache[kMaxCaches];
  int n_caches;
  pkv::Divisor n_pairs;
  int2 pair[NP];
};
static_assert(sizeof(CopyArgs<kMaxPairs>) <= 32000, "kernel parameters");

template <typename T, int NP>
__device__ __forceinline__ void copy_tile(const CopyArgs<NP> &a, const Cache &k) {
  const uint64_t first = static_cast<uint64_t>(blockIdx.x - k.block0) * kTile + threadIdx.x;
  const uint32_t page_words = k.page_words.d;
  const uint64_t words = static_cast<uint64_t>(k.rows) * page_words;
  T v[kEach];
  T *to[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const uint64_t w = first + i * kThreads;
    to[i] = nullptr;
    if (w < words) {
      // (2^31 words are 32 GB of vectors)
      const uint32_t row = words >> 31 ? static_cast<uint32_t>(w / page_words)
                                       : k.page_words.quotient(static_cast<uint32_t>(w));
      const uint32_t in = static_cast<uint32_t>(w) - row * page_words;
      const uint32_t head = a.n_pairs.quotient(row);
      const int2 pr = a.pair[row - head * a.n_pairs.d];
      T *page0 = reinterpret_cast<T *>(k.base + head * k.head_bytes) + in;
      v[i] = page0[static_cast<uint64_t>(static_cast<uint32_t>(pr.x)) * page_words];
      to[i] = page0 + static_cast<uint64_t>(static_cast<uint32_t>(pr.y)) * page_words;
    }
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (to[i]) *to[i] = v[i];
}

template <int NP>
__global__ void __launch_bounds__(kThreads)
    copy_pages_kernel(const __grid_constant__ CopyArgs<NP> a) {
  pkv_wait_prior_grid();
  int c = 0;   // the last cache that begins at or before this CTA
  for (int step = kMaxCaches / 2; step > 0; step /= 2)
    if (c + step < a.n_caches && a.cache[c + step].block0 <= blockIdx.x) c += step;
  const Cache &k = a.cache[c];
  if (k.vec == 16) copy_tile<uint4>(a, k);
  else if (k.vec == 4) copy_tile<uint32_t>(a, k);
  else copy_tile<unsigned char>(a, k);
}

template <int NP>
int launch_copy(void *const *caches, const int *heads, const int64_t *page_bytes, int n_caches,
                int n_pages, const int32_t *pairs, int n_pairs, cudaStream_t stream) {
  CopyArgs<NP> a;
  for (int p0 = 0; p0 < n_pairs; p0 += NP) {
    const int here = n_pairs - p0 < NP ? n_pairs - p0 : NP;
    a.n_pairs.set(here);
    for (int i = 0; i < here; ++i)
      a.pair[i] = make_int2(pairs[2 * (p0 + i)], pairs[2 * (p0 + i) + 1]);
    for (int c0 = 0; c0 < n_caches;) {
      long long blocks = 0;
      int n = 0;
      for (; c0 + n < n_caches && n < kMaxCaches; ++n) {
        Cache k;
        k.base = static_cast<unsigned char *>(caches[c0 + n]);
        const int64_t bytes = page_bytes[c0 + n];
        const uintptr_t both = reinterpret_cast<uintptr_t>(k.base) | bytes;
        k.vec = both % 16 == 0 ? 16 : both % 4 == 0 ? 4 : 1;
        k.page_words.set(static_cast<uint32_t>(bytes / k.vec));
        k.head_bytes = bytes * n_pages;
        k.rows = static_cast<uint32_t>(heads[c0 + n]) * here;
        k.block0 = static_cast<uint32_t>(blocks);
        const uint64_t words = static_cast<uint64_t>(k.rows) * k.page_words.d;
        const long long more = static_cast<long long>((words + kTile - 1) / kTile);
        if (n > 0 && blocks + more > 0x7fffffffLL) break;
        if (more > 0x7fffffffLL)
          return pkv::fail(PKV_E_BAD_ARG, "kv_copy_pages: cache %d too large", c0);
        a.cache[n] = k;
        blocks += more;
      }
      a.n_caches = n;
      copy_pages_kernel<NP><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a);
      PKV_CUDA_CHECK(cudaGetLastError());
      c0 += n;
    }
  }
  return pkv::ok();
}

}  // namespace

extern "C" int kv_copy_pages(void *const *caches, const int *heads, const int64_t *page_bytes,
                             int n_caches, int n_pages, const int32_t *pairs, int n_pairs,
                             void *stream) {
  if (n_caches < 0 || n_pairs < 0 || n_pages < 1)
    return pkv::fail(PKV_E_BAD_ARG, "kv_copy_pages: bad size argument");
  if (n_caches == 0) return pkv::ok();
  if (!caches || !heads || !page_bytes || (n_pairs > 0 && !pairs))
    return pkv::fail(PKV_E_BAD_ARG, "kv_copy_pages: NULL pointer");
  for (int c = 0; c < n_caches; ++c) {
    if (!caches[c]) return pkv::fail(PKV_E_BAD_ARG, "kv_copy_pages: NULL cache");
    if (heads[c] < 1 || heads[c] > 65535 || page_bytes[c] < 1 ||
        page_bytes[c] > (1LL << 31) || page_bytes[c] >= (1LL << 46) / n_pages / heads[c])
      return pkv::fail(PKV_E_BAD_ARG, "kv_copy_pages: cache %d: bad heads or page_bytes", c);
  }
  if (n_pairs == 0) return pkv::ok();
  std::vector<unsigned char> role;   // 1: a source, 2: a destination
  try {
    role.assign(n_pages, 0);
  } catch (...) {
    return pkv::fail(PKV_E_BAD_ARG, "kv_copy_pages: out of host memory");
  }
  for (int i = 0; i < n_pairs; ++i) {
    const int s = pairs[2 * i], d = pairs[2 * i + 1];
    if (s < 0 || s >= n_pages || d < 0 || d >= n_pages)
      return pkv::fail(PKV_E_BAD_ARG, "kv_copy_pages: pair %d (%d, %d) outside [0, %d)", i, s, d,
                       n_pages);
    if (role[d] || role[s] == 2 || s == d)
      return pkv::fail(PKV_E_BAD_ARG,
                       "kv_copy_pages: pair %d (%d, %d): a destination is named twice or is "
                       "also a source", i, s, d);
    role[s] = 1;
    role[d] = 2;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return n_pairs <= 64 ? launch_copy<64>(caches, heads, page_bytes, n_caches, n_pages, pairs,
                                         n_pairs, s)
                       : launch_copy<kMaxPairs>(caches, heads, page_bytes, n_caches, n_pages,
                                                pairs, n_pairs, s);
}
