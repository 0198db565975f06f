// kv_append_q8, kv_append_prefill_q8: the paged write of new K/V tokens into
// the 8-bit cache (e4m3 codes, one power-of-two scale per kv head and block of
// tokens).
//
// A power of two as scale costs e4m3 none of its precision (the codes are
// floating point) and makes x / s and the rescaling of codes already held
// plain exponent shifts, so a block filled token by token holds what one call
// would have written, but for values below the codes' normal range.
//
// Work: the tokens of one block that the call brings stand next to each
// other (a run); the warp that meets a run's first token in a block handles
// the whole run there, for one head of K or V: the run's largest magnitude,
// the block's scale, the rescaling of older codes if the scale grew, the new
// codes. Bound by reading k and v and writing half their bytes.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "pkv_internal.h"

namespace {

constexpr int kWarps = 4;
constexpr int kKeep = 8;   // 16-byte vectors of a run a lane keeps between the two passes

struct Args {
  const __nv_bfloat16 *k, *v;
  const int32_t *batch_idx, *input_pos, *table;
  int N, n_slots, max_pages, page_size, n_pages, block;
  uint8_t *k_cache, *v_cache;
  float *k_scale, *v_scale;
  int Hkv, D;
  long long token_stride, head_stride;   // of k and v, in elements
  int window;                            // tokens a warp looks at (1 .. 31)
  int32_t *err;
};

// Largest finite magnitude of 8 bf16, as the bits of the two halves' maxima.
__device__ __forceinline__ uint32_t max_finite(uint32_t m, uint4 x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i] & 0x7fff7fffu;
    m = __vmaxu2(m, a & __vcmpltu2(a, 0x7f807f80u));
  }
  return m;
}

__device__ __forceinline__ uint32_t quantise2(uint32_t x, float inv) {
  const float lo = __uint_as_float(x << 16) * inv, hi = __uint_as_float(x & 0xffff0000u) * inv;
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint2 quantise8(uint4 x, float inv) {
  return make_uint2(quantise2(x.x, inv) | quantise2(x.y, inv) << 16,
                    quantise2(x.z, inv) | quantise2(x.w, inv) << 16);
}
__device__ __forceinline__ uint32_t rescale2(uint32_t c, float ratio) {
  const __half2 h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c), __NV_E4M3);
  const float2 f = __half22float2(h);
  return __nv_cvt_float2_to_fp8x2(make_float2(f.x * ratio, f.y * ratio), __NV_SATFINITE,
                                  __NV_E4M3);
}
__device__ __forceinline__ uint32_t rescale4(uint32_t c, float ratio) {
  return rescale2(c & 0xffffu, ratio) | rescale2(c >> 16, ratio) << 16;
}

// Exponent of the smallest power of two s >= 2^-126 with a / s <= 448 for a
// finite bf16 a >= 0 given by its bits: 448 = 1.75 * 2^8.
__device__ __forceinline__ int need_exponent(uint32_t bits) {
  const int k = static_cast<int>(bits >> 7) - 127 - 8 + ((bits & 0x7fu) > 0x60u ? 1 : 0);
  return k > -126 ? k : -126;
}
__device__ __forceinline__ float exp2i(int k) {   // 2^k, -126 <= k <= 127
  return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

__global__ void __launch_bounds__(kWarps * 32) append_q8_kernel(const Args a) {
  pkv_wait_prior_grid();
  pkv_allow_next_grid();
  const int lane = threadIdx.x & 31;
  const long long task = blockIdx.x * static_cast<long long>(kWarps) + (threadIdx.x >> 5);
  const int per_window = 2 * a.Hkv;
  const long long i0 = task / per_window * a.window;
  if (i0 >= a.N) return;
  const int which = static_cast<int>(task % per_window);
  const bool is_v = which >= a.Hkv;
  const int h = is_v ? which - a.Hkv : which;
  const bool reporter = which == 0;
  const int bmask = a.block - 1;

  // lane l looks at token i0 + l - 1: the window's tokens and the one before
  const long long mine = i0 + lane - 1;
  const bool there = mine >= 0 && mine < a.N && lane <= a.window;
  const int my_slot = there ? (a.batch_idx ? a.batch_idx[mine] : static_cast<int>(mine)) : -1;
  const int my_pos = there ? a.input_pos[mine] : -1;
  const int prev_slot = __shfl_up_sync(0xffffffffu, my_slot, 1);
  const int prev_pos = __shfl_up_sync(0xffffffffu, my_pos, 1);
  const bool follows = mine > 0 && prev_slot == my_slot && prev_pos >= 0 &&
                       my_pos - 1 == prev_pos;
  uint32_t leaders = __ballot_sync(
      0xffffffffu, there && lane > 0 && (!follows || my_pos < 0 || (my_pos & bmask) == 0));
  const uint32_t starts = __ballot_sync(0xffffffffu, !follows);

  while (leaders) {
    const int l = __ffs(leaders) - 1;
    leaders &= leaders - 1;
    const long long i = i0 + l - 1;
    const int slot = __shfl_sync(0xffffffffu, my_slot, l);
    const int pos = __shfl_sync(0xffffffffu, my_pos, l);
    int bits = 0, page = 0;
    if (slot < 0 || slot >= a.n_slots) {
      bits = PKV_ERR_SLOT;
    } else if (slot == 0) {
      continue;                      // padding
    } else if (pos < 0 || pos / a.page_size >= a.max_pages) {
      bits = PKV_ERR_POS;
    } else {
      page = a.table[static_cast<long long>(slot) * a.max_pages + pos / a.page_size];
      if (page < 0) bits = PKV_ERR_PAGE_NEG;
      else if (page >= a.n_pages) bits = PKV_ERR_PAGE_RANGE;
    }
    if (bits) {
      if (reporter && lane == 0 && a.err) atomicOr(a.err, bits);
      continue;
    }
    // the run in this block: tokens i .. i + n - 1
    const int first = pos & bmask, room = a.block - first;
    int n = 1;
    while (n < room) {
      const long long j = i + n + lane;
      const bool in = n + lane < room && j < a.N &&
                      (a.batch_idx ? a.batch_idx[j] : static_cast<int>(j)) == slot &&
                      a.input_pos[j] == pos + n + lane;
      const uint32_t m = __ballot_sync(0xffffffffu, in);
      const int more = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
      n += more;
      if (more < 32) break;
    }
    // A run's start also looks for tokens of its block elsewhere in the call (of two
    // runs that meet in a block, one starts in a block of the other); the warps of all
    // heads share the tokens to look at.
    if (starts >> l & 1) {
      bool clash = false;
#pragma unroll 8
      for (long long j = which * 32 + lane; j < a.N; j += per_window * 32) {
        const int s = a.batch_idx ? a.batch_idx[j] : static_cast<int>(j);
        clash |= s == slot && (a.input_pos[j] & ~bmask) == (pos & ~bmask) && (j < i || j >= i + n);
      }
      if (__any_sync(0xffffffffu, clash) && lane == 0 && a.err) atomicOr(a.err, PKV_ERR_ORDER);
    }

    const __nv_bfloat16 *x = (is_v ? a.v : a.k) + i * a.token_stride + h * a.head_stride;
    const int chunks = a.D / 8;                 // 16-byte vectors a token
    const long long row0 = static_cast<long long>(h) * a.n_pages * a.page_size +
                           static_cast<long long>(page) * a.page_size + pos % a.page_size;
    uint8_t *codes = (is_v ? a.v_cache : a.k_cache) + row0 * a.D;
    float *scale = (is_v ? a.v_scale : a.k_scale) + row0 / a.block;
    const float held_raw = first ? *scale : 0.f;
    // pass 1: the largest magnitude; a lane's first kKeep vectors stay
    uint4 keep[kKeep];
    uint32_t m2 = 0;
    const int total = n * chunks;
    {
      int tok = lane / chunks, c = lane % chunks;
#pragma unroll
      for (int j = 0; j < kKeep; ++j) {
        const int u = lane + 32 * j;
        keep[j] = u < total ? *reinterpret_cast<const uint4 *>(x + tok * a.token_stride + 8 * c)
                            : make_uint4(0u, 0u, 0u, 0u);
        for (c += 32; c >= chunks; c -= chunks) ++tok;
      }
#pragma unroll
      for (int j = 0; j < kKeep; ++j) m2 = max_finite(m2, keep[j]);
      for (int u = lane + 32 * kKeep; u < total; u += 32) {
        m2 = max_finite(m2, *reinterpret_cast<const uint4 *>(x + tok * a.token_stride + 8 * c));
        for (c += 32; c >= chunks; c -= chunks) ++tok;
      }
    }
    const uint32_t amax = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
    const float held = held_raw > 0.f && held_raw < INFINITY ? held_raw : 0.f;
    int e = need_exponent(amax);
    if (held > 0.f) {   // the held scale, rounded up to a power of two
      const uint32_t hb = __float_as_uint(held);
      int he = static_cast<int>(hb >> 23) - 127 + ((hb & 0x7fffffu) ? 1 : 0);
      he = min(max(he, -126), 126);
      e = max(e, he);
    }
    const float s = exp2i(e), inv = exp2i(-e);
    if (first && s != held_raw) {
      const float ratio = held * inv;
      uint2 *old = reinterpret_cast<uint2 *>(codes - static_cast<long long>(first) * a.D);
      for (int u = lane; u < first * chunks; u += 32) {
        const uint2 c = old[u];
        old[u] = make_uint2(rescale4(c.x, ratio), rescale4(c.y, ratio));
      }
    }
    if (lane == 0) *scale = s;
    // pass 2: the codes
    uint2 *dst = reinterpret_cast<uint2 *>(codes);
    int tok = lane / chunks, c = lane % chunks;
#pragma unroll
    for (int j = 0; j < kKeep; ++j) {
      const int u = lane + 32 * j;
      if (u < total) dst[u] = quantise8(keep[j], inv);
      for (c += 32; c >= chunks; c -= chunks) ++tok;
    }
    for (int u = lane + 32 * kKeep; u < total; u += 32) {
      dst[u] = quantise8(*reinterpret_cast<const uint4 *>(x + tok * a.token_stride + 8 * c), inv);
      for (c += 32; c >= chunks; c -= chunks) ++tok;
    }
  }
}

int launch_append_q8(const char *fn, const pkv_bf16 *k, const pkv_bf16 *v,
                     const int32_t *batch_idx, const int32_t *input_pos, int N,
                     const int32_t *dev_table, int n_slots, int max_pages_per_seq,
                     int page_size, int n_pages, int scale_block, pkv_e4m3 *k_cache,
                     pkv_e4m3 *v_cache, float *k_scale, float *v_scale, int Hkv, int D,
                     bool head_major, int32_t *err_word, void *stream) {
  if (N < 0 || Hkv < 1 || D < 16 || D % 16 || page_size < 1 || n_pages < 1 || n_slots < 1 ||
      max_pages_per_seq < 1)
    return pkv::fail(PKV_E_BAD_ARG, "%s: bad shape (D must be a multiple of 16)", fn);
  if (!pkv::is_pow2(scale_block) || page_size % scale_block)
    return pkv::fail(PKV_E_BAD_ARG,
                     "%s: scale_block must be a power of two that divides page_size", fn);
  if (1LL * D * scale_block > (1 << 30))
    return pkv::fail(PKV_E_BAD_ARG, "%s: scale block too large", fn);
  if (N == 0) return pkv::ok();
  if (!k || !v || !input_pos || !dev_table || !k_cache || !v_cache || !k_scale || !v_scale)
    return pkv::fail(PKV_E_BAD_ARG, "%s: NULL tensor", fn);
  if (!pkv::aligned16(k) || !pkv::aligned16(v) || !pkv::aligned16(k_cache) ||
      !pkv::aligned16(v_cache))
    return pkv::fail(PKV_E_BAD_ARG, "%s: tensors must be 16-byte aligned", fn);
  const int sms = pkv::sm_count();
  if (sms <= 0) return pkv::fail(PKV_E_CUDA, "%s: no SM count", fn);
  Args a;
  a.k = reinterpret_cast<const __nv_bfloat16 *>(k);
  a.v = reinterpret_cast<const __nv_bfloat16 *>(v);
  a.batch_idx = batch_idx;
  a.input_pos = input_pos;
  a.table = dev_table;
  a.N = N;
  a.n_slots = n_slots;
  a.max_pages = max_pages_per_seq;
  a.page_size = page_size;
  a.n_pages = n_pages;
  a.block = scale_block;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.Hkv = Hkv;
  a.D = D;
  a.token_stride = head_major ? D : 1LL * Hkv * D;
  a.head_stride = head_major ? 1LL * N * D : D;
  a.err = err_word;
  // one token a warp while those warps fit the GPU at once (a decode step),
  // else 16 (a packed prompt, where few tokens lead a run)
  const long long pairs = 2LL * Hkv;
  a.window = N * pairs <= 32LL * sms ? 1 : 16;
  const long long tasks = (N + a.window - 1LL) / a.window * pairs;
  const long long blocks = (tasks + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return pkv::fail(PKV_E_BAD_ARG, "%s: too large", fn);
  PKV_CUDA_CHECK(pkv::launch_pdl(append_q8_kernel, dim3(static_cast<unsigned>(blocks)),
                                 dim3(kWarps * 32), 0, static_cast<cudaStream_t>(stream), a));
  return pkv::ok();
}

}  // namespace

extern "C" int kv_append_q8(const pkv_bf16 *k, const pkv_bf16 *v, const int32_t *batch_idx,
                            const int32_t *input_pos, int B, const int32_t *dev_table,
                            int n_slots, int max_pages_per_seq, int page_size, int n_pages,
                            int scale_block, pkv_e4m3 *k_cache, pkv_e4m3 *v_cache,
                            float *k_scale, float *v_scale, int Hkv, int D, int32_t *err_word,
                            void *stream) {
  return launch_append_q8("kv_append_q8", k, v, batch_idx, input_pos, B, dev_table, n_slots,
                          max_pages_per_seq, page_size, n_pages, scale_block, k_cache, v_cache,
                          k_scale, v_scale, Hkv, D, false, err_word, stream);
}

extern "C" int kv_append_prefill_q8(const pkv_bf16 *k, const pkv_bf16 *v,
                                    const int32_t *batch_idx, const int32_t *input_pos, int L,
                                    const int32_t *dev_table, int n_slots,
                                    int max_pages_per_seq, int page_size, int n_pages,
                                    int scale_block, pkv_e4m3 *k_cache, pkv_e4m3 *v_cache,
                                    float *k_scale, float *v_scale, int Hkv, int D,
                                    int32_t *err_word, void *stream) {
  return launch_append_q8("kv_append_prefill_q8", k, v, batch_idx, input_pos, L, dev_table,
                          n_slots, max_pages_per_seq, page_size, n_pages, scale_block, k_cache,
                          v_cache, k_scale, v_scale, Hkv, D, true, err_word, stream);
}
