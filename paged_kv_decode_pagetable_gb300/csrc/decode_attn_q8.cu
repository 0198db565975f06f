// paged_decode_attn_q8: GQA single-token decode attention over the paged 8-bit
// cache (e4m3 codes, one scale per kv head and block of tokens).
//
// One CTA per (row, query head): its warps take every fourth key, each with
// an online softmax of its own (running maximum, sum and output in fp32), and
// join at the end.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>

#include "pkv_internal.h"

namespace {

constexpr int kMaxG = 8;         // query heads per kv head
constexpr int kMaxRows = 512;
constexpr int kMaxCtas = 1024;   // CTAs the workspace has room for

struct Problem {
  const __nv_bfloat16 *q;
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int32_t *table, *batch_idx, *seq_lens;
  int n_slots, max_pages, log2_ps, n_pages, log2_block, window, B, Hq, Hkv, G;
  float scale_log2;
  __nv_bfloat16 *out;
  int32_t *err;
};

template <int D>
__global__ void __launch_bounds__(128) decode_q8_kernel(const Problem p) {
  constexpr int E = D / 32;   // elements a lane holds
  pkv_wait_prior_grid();
  pkv_allow_next_grid();
  const int b = blockIdx.x / p.Hq, hq = blockIdx.x % p.Hq, g = hq / p.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ float sm_m[4], sm_l[4], sm_o[4][D];
  const int slot = p.batch_idx ? p.batch_idx[b] : b;
  int L = p.seq_lens[b];
  const int Lmax = p.max_pages << p.log2_ps;
  int bits = 0;
  if (slot < 0 || slot >= p.n_slots) bits |= PKV_ERR_SLOT;
  if (L > Lmax || L < 0) bits |= PKV_ERR_POS;
  if (bits && hq == 0 && threadIdx.x == 0 && p.err) atomicOr(p.err, bits);
  L = min(L, Lmax);
  if (slot <= 0 || slot >= p.n_slots) L = 0;
  const int lo = p.window > 0 ? max(0, L - p.window) : 0;
  const __nv_bfloat16 *q = p.q + (static_cast<long long>(b) * p.Hq + hq) * D + lane * E;
  float qf[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    qf[i] = __bfloat162float(q[i]);
    o[i] = 0.f;
  }
  for (int j = lo + warp; j < L; j += 4) {
    const int page = p.table[static_cast<long long>(slot) * p.max_pages + (j >> p.log2_ps)];
    if (page < 0 || page >= p.n_pages) {
      if (lane == 0 && p.err) atomicOr(p.err, page < 0 ? PKV_ERR_PAGE_NEG : PKV_ERR_PAGE_RANGE);
      continue;
    }
    const long long row = ((static_cast<long long>(g) * p.n_pages + page) << p.log2_ps) +
                          (j & ((1 << p.log2_ps) - 1));
    const uint8_t *kc = p.k_cache + row * D + lane * E, *vc = p.v_cache + row * D + lane * E;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      __nv_fp8_e4m3 c;
      c.__x = kc[i];
      s = fmaf(qf[i], static_cast<float>(c), s);
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    s *= p.scale_log2 * p.k_scale[row >> p.log2_block];
    const float mn = fmaxf(m, s), al = exp2f(m - mn), pr = exp2f(s - mn);
    const float wv = pr * p.v_scale[row >> p.log2_block];
    l = l * al + pr;
    m = mn;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      __nv_fp8_e4m3 c;
      c.__x = vc[i];
      o[i] = fmaf(wv, static_cast<float>(c), o[i] * al);
    }
  }
  if (lane == 0) {
    sm_m[warp] = m;
    sm_l[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < E; ++i) sm_o[warp][lane * E + i] = o[i];
  __syncthreads();
  const float mt = fmaxf(fmaxf(sm_m[0], sm_m[1]), fmaxf(sm_m[2], sm_m[3]));
  for (int d = threadIdx.x; d < D; d += 128) {
    float sum = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = sm_m[w] == -INFINITY ? 0.f : exp2f(sm_m[w] - mt);
      sum += sm_l[w] * f;
      acc += sm_o[w][d] * f;
    }
    p.out[(static_cast<long long>(b) * p.Hq + hq) * D + d] =
        __float2bfloat16_rn(sum != 0.f ? acc / sum : 0.f);
  }
}

bool good_heads(int Hq, int Hkv, int D) {
  return (D == 64 || D == 128 || D == 256 || D == 512) && Hkv >= 1 && Hq >= Hkv &&
         Hq % Hkv == 0 && Hq / Hkv <= kMaxG;
}

}  // namespace

extern "C" {

size_t paged_decode_attn_q8_workspace(int Hq, int Hkv, int D) {
  if (!good_heads(Hq, Hkv, D)) return 0;
  const size_t G = Hq / Hkv;
  return kMaxCtas * (sizeof(int) + 2 * G * (D + 3) * sizeof(float));
}

int paged_decode_attn_q8(const pkv_bf16 *q, const pkv_e4m3 *k_cache, const pkv_e4m3 *v_cache,
                         const float *k_scale, const float *v_scale, const int32_t *dev_table,
                         int n_slots, int max_pages_per_seq, int page_size, int n_pages,
                         int scale_block, const int32_t *batch_idx, const int32_t *seq_lens,
                         int window, float scale, int B, int Hq, int Hkv, int D,
                         void *workspace, size_t workspace_bytes, pkv_bf16 *out,
                         int32_t *err_word, void *stream) {
  const char *fn = "paged_decode_attn_q8";
  if (D != 64 && D != 128 && D != 256 && D != 512)
    return pkv::fail(PKV_E_BAD_ARG, "%s: D must be 64, 128, 256 or 512", fn);
  if (!good_heads(Hq, Hkv, D))
    return pkv::fail(PKV_E_BAD_ARG, "%s: need Hq %% Hkv == 0 and Hq/Hkv <= %d", fn, kMaxG);
  if (!pkv::is_pow2(page_size) || page_size < 8)
    return pkv::fail(PKV_E_BAD_ARG, "%s: page_size must be a power of two >= 8", fn);
  if (!pkv::is_pow2(scale_block) || scale_block > page_size)
    return pkv::fail(PKV_E_BAD_ARG,
                     "%s: scale_block must be a power of two that divides page_size", fn);
  if (B < 0 || n_slots < 1 || max_pages_per_seq < 1 || n_pages < 1)
    return pkv::fail(PKV_E_BAD_ARG, "%s: bad size argument", fn);
  if (B > kMaxRows) return pkv::fail(PKV_E_BAD_ARG, "%s: B must be <= %d", fn, kMaxRows);
  if (1LL * max_pages_per_seq * page_size > (1LL << 30))
    return pkv::fail(PKV_E_BAD_ARG, "%s: table row too long", fn);
  if (1LL * Hkv * n_pages * page_size >= (1LL << 31))
    return pkv::fail(PKV_E_BAD_ARG, "%s: cache has too many rows", fn);
  if (!(scale > 0.f) || !std::isfinite(scale))
    return pkv::fail(PKV_E_BAD_ARG, "%s: scale must be finite and > 0", fn);
  if (B == 0) return pkv::ok();
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !dev_table || !seq_lens || !out)
    return pkv::fail(PKV_E_BAD_ARG, "%s: NULL tensor", fn);
  if (!pkv::aligned16(q) || !pkv::aligned16(out) || !pkv::aligned16(k_cache) ||
      !pkv::aligned16(v_cache))
    return pkv::fail(PKV_E_BAD_ARG, "%s: tensors must be 16-byte aligned", fn);
  const size_t need = paged_decode_attn_q8_workspace(Hq, Hkv, D);
  if (!workspace || workspace_bytes < need)
    return pkv::fail(PKV_E_BAD_ARG, "%s: workspace needs %zu bytes", fn, need);
  if (!pkv::aligned16(workspace))
    return pkv::fail(PKV_E_BAD_ARG, "%s: workspace must be 16-byte aligned", fn);
  auto log2i = [](int x) {
    int l = 0;
    while ((1 << l) < x) ++l;
    return l;
  };
  Problem p;
  p.q = reinterpret_cast<const __nv_bfloat16 *>(q);
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.table = dev_table;
  p.batch_idx = batch_idx;
  p.seq_lens = seq_lens;
  p.n_slots = n_slots;
  p.max_pages = max_pages_per_seq;
  p.log2_ps = log2i(page_size);
  p.n_pages = n_pages;
  p.log2_block = log2i(scale_block);
  p.window = window;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.out = reinterpret_cast<__nv_bfloat16 *>(out);
  p.err = err_word;
  auto *kern = D == 64    ? decode_q8_kernel<64>
               : D == 128 ? decode_q8_kernel<128>
               : D == 256 ? decode_q8_kernel<256>
                          : decode_q8_kernel<512>;
  PKV_CUDA_CHECK(pkv::launch_pdl(kern, dim3(static_cast<unsigned>(B * Hq)), dim3(128), 0,
                                 static_cast<cudaStream_t>(stream), p));
  return pkv::ok();
}

}  // extern "C"
