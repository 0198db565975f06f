// kv_copy_pages: copies of pages inside caches (forked, rewound and compacted
// sequences).
//
// A pure copy: bound by reading and writing the pages once. The pairs and
// the caches' descriptions travel as kernel parameters, so a call uploads
// nothing and can be captured.
#include <cuda_runtime.h>

#include <vector>

#include "pkv_internal.h"

namespace {

struct Cache {
  unsigned char *base;
  long long page_bytes;
  int head0;     // heads of the caches before this one
  int vec;       // bytes moved per access: 16, 4 or 1
};

// Kernel parameters may hold 32,764 bytes.
constexpr int kMaxCaches = 64;
constexpr int kMaxPairs = 3500;
template <int NP>
struct CopyArgs {
  Cache cache[kMaxCaches];
  int n_caches, n_pages, n_pairs;
  int2 pair[NP];
};
static_assert(sizeof(CopyArgs<kMaxPairs>) <= 32000, "kernel parameters");

template <typename T>
__device__ __forceinline__ void copy_page(unsigned char *base, long long src, long long dst,
                                          long long bytes) {
  const T *s = reinterpret_cast<const T *>(base + src);
  T *d = reinterpret_cast<T *>(base + dst);
  const long long n = bytes / static_cast<long long>(sizeof(T));
  for (long long i = threadIdx.x; i < n; i += blockDim.x) d[i] = s[i];
}

// One CTA per (pair, head of a cache).
template <int NP>
__global__ void copy_pages_kernel(const __grid_constant__ CopyArgs<NP> a) {
  pkv_wait_prior_grid();
  const int2 pr = a.pair[blockIdx.x];
  const int row = blockIdx.y;
  int c = 0;
  while (c + 1 < a.n_caches && a.cache[c + 1].head0 <= row) ++c;
  const Cache &k = a.cache[c];
  const long long head = static_cast<long long>(row - k.head0) * a.n_pages;
  const long long src = (head + pr.x) * k.page_bytes, dst = (head + pr.y) * k.page_bytes;
  if (k.vec == 16) copy_page<uint4>(k.base, src, dst, k.page_bytes);
  else if (k.vec == 4) copy_page<uint32_t>(k.base, src, dst, k.page_bytes);
  else copy_page<unsigned char>(k.base, src, dst, k.page_bytes);
}

template <int NP>
int launch_copy(void *const *caches, const int *heads, const int64_t *page_bytes, int n_caches,
                int n_pages, const int32_t *pairs, int n_pairs, cudaStream_t stream) {
  CopyArgs<NP> a;
  a.n_pages = n_pages;
  for (int c0 = 0; c0 < n_caches;) {
    int n = 0, rows = 0;
    for (; c0 + n < n_caches && n < kMaxCaches && rows + heads[c0 + n] <= 65535; ++n) {
      Cache &k = a.cache[n];
      k.base = static_cast<unsigned char *>(caches[c0 + n]);
      k.page_bytes = page_bytes[c0 + n];
      k.head0 = rows;
      const uintptr_t both = reinterpret_cast<uintptr_t>(k.base) | k.page_bytes;
      k.vec = both % 16 == 0 ? 16 : both % 4 == 0 ? 4 : 1;
      rows += heads[c0 + n];
    }
    a.n_caches = n;
    for (int p0 = 0; p0 < n_pairs; p0 += NP) {
      a.n_pairs = n_pairs - p0 < NP ? n_pairs - p0 : NP;
      for (int i = 0; i < a.n_pairs; ++i)
        a.pair[i] = make_int2(pairs[2 * (p0 + i)], pairs[2 * (p0 + i) + 1]);
      copy_pages_kernel<NP><<<dim3(a.n_pairs, rows), 256, 0, stream>>>(a);
      PKV_CUDA_CHECK(cudaGetLastError());
    }
    c0 += n;
  }
  return pkv::ok();
}

}  // namespace

extern "C" int kv_copy_pages(void *const *caches, const int *heads, const int64_t *page_bytes,
                             int n_caches, int n_pages, const int32_t *pairs, int n_pairs,
                             void *stream) {
  if (n_caches < 0 || n_pairs < 0 || n_pages < 1)
    return pkv::fail(PKV_E_BAD_ARG, "kv_copy_pages: bad size argument");
  if (n_caches == 0 || n_pairs == 0) return pkv::ok();
  if (!caches || !heads || !page_bytes || !pairs)
    return pkv::fail(PKV_E_BAD_ARG, "kv_copy_pages: NULL pointer");
  for (int c = 0; c < n_caches; ++c) {
    if (!caches[c]) return pkv::fail(PKV_E_BAD_ARG, "kv_copy_pages: NULL cache");
    if (heads[c] < 1 || heads[c] > 65535 || page_bytes[c] < 1 ||
        page_bytes[c] >= (1LL << 46) / n_pages / heads[c])
      return pkv::fail(PKV_E_BAD_ARG, "kv_copy_pages: cache %d: bad heads or page_bytes", c);
  }
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
