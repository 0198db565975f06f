// paged_tree_attn: attention of every row's tree of drafted tokens over the paged cache.
//
//   out[t][h] = sum_j softmax_j(scale q[t][h] . k_j) v_j
// over the keys j < ctx of the context and, among the row's own nodes (at cache positions ctx ..),
// those on t's path to its root, t included; with a window W only keys less than W positions
// behind t (a node's position is ctx + its depth).
//
// A simple form: one CTA of four warps a (node, head), each warp its own keys with a running
// maximum and sum, joined at the end.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "pkv_internal.h"
#include "tree.cuh"

namespace {

constexpr int kWarps = 4;

template <int D>
__global__ void __launch_bounds__(kWarps * 32)
    tree_attn_kernel(const __nv_bfloat16 *q, const __nv_bfloat16 *kc, const __nv_bfloat16 *vc,
                     const int32_t *table, int n_slots, int max_pages, int page_size, int n_pages,
                     const int32_t *batch_idx, const int32_t *ctx_lens, const int32_t *row_start,
                     const int32_t *parents, int window, float scale, int B, int N, int Hq, int G,
                     __nv_bfloat16 *out, int32_t *err) {
  constexpr int E = D / 32;
  __shared__ int s_par[kTreeMax], s_depth[kTreeMax];
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  pkv_wait_prior_grid();
  pkv_allow_next_grid();
  const int node = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  int before = 0;
  for (int i0 = 0; i0 <= B; i0 += blockDim.x)
    before += __syncthreads_count(i0 + tid <= B && row_start[i0 + tid] <= node);
  const int b = before - 1;
  if (b < 0 || b >= B) return;
  const TreeRow r = tree_row(b, N, row_start, batch_idx, ctx_lens, n_slots, max_pages, page_size);
  const int t = node - r.n0;
  if (r.bits || t < 0 || t >= r.n) {
    if (tid == 0) tree_report(err, r.bits);
    return;
  }
  int bits = 0;
  if (tid < r.n) s_par[tid] = tree_parent(parents, r.n0, tid, bits);
  __syncthreads();
  if (tid < r.n) {
    int d = 0;
    for (int i = s_par[tid]; i >= 0; i = s_par[i]) ++d;
    s_depth[tid] = d;
  }
  __syncthreads();
  unsigned long long seen = 0;
  for (int i = t; i >= 0; i = s_par[i]) seen |= 1ull << i;
  float qv[E], o[E];
  for (int e = 0; e < E; ++e) {
    qv[e] = __bfloat162float(q[(static_cast<long long>(node) * Hq + h) * D + lane + 32 * e]);
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int total = r.slot == 0 ? 0 : r.ctx + r.n;
  for (int j = warp; j < total; j += kWarps) {
    const int i = j - r.ctx;
    bool keep = i < 0 || (seen >> i & 1);
    const int pos = i < 0 ? j : r.ctx + s_depth[i];
    if (window > 0) keep = keep && r.ctx + s_depth[t] - pos < window;
    if (!keep) continue;
    const int page = table[static_cast<long long>(r.slot) * max_pages + j / page_size];
    if (page < 0 || page >= n_pages) {
      bits |= page < 0 ? PKV_ERR_PAGE_NEG : PKV_ERR_PAGE_RANGE;
      continue;
    }
    const long long row = ((static_cast<long long>(h / G) * n_pages + page) * page_size +
                           j % page_size) * D;
    float s = 0.f;
    for (int e = 0; e < E; ++e) s = fmaf(qv[e], __bfloat162float(kc[row + lane + 32 * e]), s);
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= scale;
    const float mn = fmaxf(m, s), a = expf(m - mn), p = expf(s - mn);
    m = mn;
    l = l * a + p;
    for (int e = 0; e < E; ++e) o[e] = o[e] * a + p * __bfloat162float(vc[row + lane + 32 * e]);
  }
  tree_report(err, bits);
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  for (int e = 0; e < E; ++e) s_o[warp][lane + 32 * e] = o[e];
  __syncthreads();
  float mm = -INFINITY, ll = 0.f;
  for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w]);
  for (int w = 0; w < kWarps; ++w) ll += s_l[w] > 0.f ? s_l[w] * expf(s_m[w] - mm) : 0.f;
  for (int d = tid; d < D; d += blockDim.x) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += s_l[w] > 0.f ? s_o[w][d] * expf(s_m[w] - mm) : 0.f;
    out[(static_cast<long long>(node) * Hq + h) * D + d] =
        __float2bfloat16_rn(ll > 0.f ? x / ll : 0.f);
  }
}

template <int D>
cudaError_t launch(const pkv_bf16 *q, const pkv_bf16 *k, const pkv_bf16 *v, const int32_t *table,
                   int n_slots, int max_pages, int page_size, int n_pages, const int32_t *batch_idx,
                   const int32_t *ctx_lens, const int32_t *row_start, const int32_t *parents,
                   int window, float scale, int B, int N, int Hq, int Hkv, pkv_bf16 *out,
                   int32_t *err, cudaStream_t s) {
  return pkv::launch_pdl(tree_attn_kernel<D>, dim3(N, Hq), dim3(kWarps * 32), 0, s,
                         reinterpret_cast<const __nv_bfloat16 *>(q),
                         reinterpret_cast<const __nv_bfloat16 *>(k),
                         reinterpret_cast<const __nv_bfloat16 *>(v), table, n_slots, max_pages,
                         page_size, n_pages, batch_idx, ctx_lens, row_start, parents, window,
                         scale, B, N, Hq, Hq / Hkv, reinterpret_cast<__nv_bfloat16 *>(out), err);
}

}  // namespace

extern "C" size_t paged_tree_attn_workspace(int Hq, int Hkv, int D) {
  if ((D != 64 && D != 128 && D != 256 && D != 512) || Hkv < 1 || Hq < Hkv || Hq % Hkv ||
      Hq / Hkv > 8 || Hq > 65535)
    return 0;
  return 16;
}

extern "C" int paged_tree_attn(const pkv_bf16 *q, const pkv_bf16 *k_cache, const pkv_bf16 *v_cache,
                               const int32_t *dev_table, int n_slots, int max_pages_per_seq,
                               int page_size, int n_pages, const int32_t *batch_idx,
                               const int32_t *ctx_lens, const int32_t *row_start,
                               const int32_t *parents, int window, float scale, int B, int N,
                               int Hq, int Hkv, int D, void *workspace, size_t workspace_bytes,
                               pkv_bf16 *out, int32_t *err_word, void *stream) {
  static const char *fn = "paged_tree_attn";
  if (D != 64 && D != 128 && D != 256 && D != 512)
    return pkv::fail(PKV_E_BAD_ARG, "%s: D must be 64, 128, 256 or 512", fn);
  if (B < 0 || B > kTreeRows || N < 0)
    return pkv::fail(PKV_E_BAD_ARG, "%s: bad shape (at most %d rows)", fn, kTreeRows);
  if (Hkv < 1 || Hq < Hkv || Hq % Hkv || Hq / Hkv > 8 || Hq > 65535)
    return pkv::fail(PKV_E_BAD_ARG, "%s: Hq must be 1 to 8 times Hkv", fn);
  if (page_size < 8 || !pkv::is_pow2(page_size) || n_pages < 1 || n_slots < 1 ||
      max_pages_per_seq < 1 || static_cast<long long>(page_size) * n_pages > 0x7fffffffLL ||
      static_cast<long long>(page_size) * max_pages_per_seq > 0x7fffffffLL - 1024)
    return pkv::fail(PKV_E_BAD_ARG, "%s: bad table geometry (page_size a power of two >= 8)", fn);
  if (window < 0) return pkv::fail(PKV_E_BAD_ARG, "%s: window must be >= 0", fn);
  if (!(scale > 0.f) || std::isinf(scale))
    return pkv::fail(PKV_E_BAD_ARG, "%s: scale must be finite and > 0", fn);
  if (B == 0 || N == 0) return pkv::ok();
  if (!q || !k_cache || !v_cache || !dev_table || !ctx_lens || !row_start || !parents || !out ||
      !workspace)
    return pkv::fail(PKV_E_BAD_ARG, "%s: NULL tensor", fn);
  if (!pkv::aligned16(q) || !pkv::aligned16(k_cache) || !pkv::aligned16(v_cache) ||
      !pkv::aligned16(out) || !pkv::aligned16(workspace))
    return pkv::fail(PKV_E_BAD_ARG, "%s: tensors must be 16-byte aligned", fn);
  if (workspace_bytes < paged_tree_attn_workspace(Hq, Hkv, D))
    return pkv::fail(PKV_E_BAD_ARG, "%s: workspace too small", fn);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
#define PKV_TREE_LAUNCH(DIM)                                                                      \
  PKV_CUDA_CHECK(launch<DIM>(q, k_cache, v_cache, dev_table, n_slots, max_pages_per_seq,          \
                             page_size, n_pages, batch_idx, ctx_lens, row_start, parents, window, \
                             scale, B, N, Hq, Hkv, out, err_word, s))
  if (D == 64) PKV_TREE_LAUNCH(64);
  else if (D == 128) PKV_TREE_LAUNCH(128);
  else if (D == 256) PKV_TREE_LAUNCH(256);
  else PKV_TREE_LAUNCH(512);
#undef PKV_TREE_LAUNCH
  return pkv::ok();
}
