// tree_qkv_norm_rope_append: a speculative step's prologue in one pass over q, k and v:
// per-head RMSNorm, rotate-half RoPE at ctx + depth, and the scatter of K and V to the cache
// positions ctx + index (siblings share a rotation position, not a cache row).
//
//   r = x / sqrt(mean(x^2) + eps) * gamma
//   y_i = r_i cos phi_i - r_{i+D/2} sin phi_i,  y_{i+D/2} = r_{i+D/2} cos phi_i + r_i sin phi_i
//   phi_i = (ctx + depth) theta^(-2i/D)
//
// The order of "unsloth: compare main...flex-moe-qwen3" · flex_gemma4_moe.py · attention
// forward (norm, rotary, then the paged write), as qkv_norm_rope and kv_append have it.
//
// The angle is kept as a fraction of a turn in 64-bit fixed point: with F_i = 2^64
// theta^(-2i/D) / (2 pi) modulo 2^64, computed once on the host (turns.h), position * F_i modulo
// 2^64 is the fraction to 2^-29 of a turn however far the position, and its nearest fp32 the angle
// to 2^-24 of a half turn (in fp32 throughout the angle of position 30000 is off by 10^-3 radians
// already, more than the output's rounding).
//
// Bound by its bytes where there are many nodes, else by latency: row_start, the row's entries,
// the table and parents behind one another, with q, k and v on their way meanwhile. Measured:
// 1152 nodes of 32 + 8 + 8 heads of 128, 28 MB, 9.1 us (0.45 of 6769 GB/s); 18.5 with a CTA a
// node, whose 1152 looked their rows up in three waves; 40 nodes 3.8 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "pkv_internal.h"
#include "tree.cuh"
#include "turns.h"

namespace {

constexpr int kMaxThreads = 384;
constexpr int kEach = 4;      // nodes of a CTA where there are more than a few an SM
constexpr int kAlone = 2;     // up to so many nodes an SM are CTAs of their own

template <int D>
struct Turns {
  uint64_t f[D / 2];
};

struct AppendArgs {
  const __nv_bfloat16 *q, *k, *v, *gq, *gk;
  long long sq, sk, sv;   // elements from one token to the next
  const int32_t *batch_idx, *ctx_lens, *row_start, *parents, *table;
  __nv_bfloat16 *k_cache, *v_cache, *q_out;
  int32_t *err;
  float eps;
  int v_norm, B, N, Hq, Hkv, n_slots, max_pages, page_size, n_pages;
};

__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// EACH nodes a CTA; D / 16 lanes a head, each with 8 rotation pairs (two 16-byte words) of every
// node. A warp a node finds its row, pages and depth while the nodes' q, k and v are on their way.
template <int D, int EACH>
__global__ void __launch_bounds__(kMaxThreads, 2)
    tree_append_kernel(const __grid_constant__ AppendArgs a,
                       const __grid_constant__ Turns<D> turns) {
  constexpr int LANES = D / 16;
  __shared__ int s_par[EACH][kTreeMax];
  __shared__ float2 s_rot[EACH][D / 2];
  __shared__ int s_pos[EACH];           // rotation position, -1: no node of a row
  __shared__ long long s_row[EACH];     // cache row, -1: none
  pkv_wait_prior_grid();
  pkv_allow_next_grid();
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int node0 = blockIdx.x * EACH;
  const int heads = a.Hq + 2 * a.Hkv;
  const int part = tid % LANES;
  auto load = [&](int n, int h, uint4 &lo, uint4 &hi) {
    const __nv_bfloat16 *x = h < a.Hq             ? a.q + n * a.sq + h * D
                             : h < a.Hq + a.Hkv ? a.k + n * a.sk + (h - a.Hq) * D
                                                : a.v + n * a.sv + (h - a.Hq - a.Hkv) * D;
    lo = *reinterpret_cast<const uint4 *>(x + 8 * part);
    hi = *reinterpret_cast<const uint4 *>(x + D / 2 + 8 * part);
  };
  int h = tid / LANES;
  uint4 lo4[EACH], hi4[EACH];
#pragma unroll
  for (int j = 0; j < EACH; ++j) {
    lo4[j] = hi4[j] = make_uint4(0, 0, 0, 0);
    if (h < heads && node0 + j < a.N) load(node0 + j, h, lo4[j], hi4[j]);
  }
  if (blockIdx.x == 0 && warp == blockDim.x / 32 - 1) {
    // rows outside the packed nodes are reported here: no node finds them
    int bits = 0;
    for (int i = lane; i < a.B; i += 32) {
      const int n0 = a.row_start[i], n1 = a.row_start[i + 1];
      if (n0 < 0 || n1 < n0 || n1 > a.N) bits = PKV_ERR_TREE;
    }
    tree_report(a.err, bits);
  }
  for (int j = warp; j < EACH; j += blockDim.x / 32) {
    const int node = node0 + j;
    int before = 0;   // the node's row: the last that starts at or before it
    for (int i = lane; i <= a.B; i += 32) before += a.row_start[i] <= node;
    const int b = __reduce_add_sync(0xffffffffu, before) - 1;
    int bits = 0, pos = -1;
    long long to = -1;
    if (node < a.N && b >= 0 && b < a.B) {   // (others are nodes of no row)
      const TreeRow r = tree_row(b, a.N, a.row_start, a.batch_idx, a.ctx_lens, a.n_slots,
                                 a.max_pages, a.page_size);
      const int i = node - r.n0;
      bits = r.bits;
      if (!r.bits && i >= 0 && i < r.n) {
        const int at = r.ctx + i;
        const int page = a.table[static_cast<long long>(r.slot) * a.max_pages + at / a.page_size];
        for (int t = lane; t <= i; t += 32) s_par[j][t] = tree_parent(a.parents, r.n0, t, bits);
        __syncwarp();
        pos = r.ctx;
        for (int t = s_par[j][i]; t >= 0; t = s_par[j][t]) ++pos;
        if (page < 0) bits |= PKV_ERR_PAGE_NEG;
        else if (page >= a.n_pages) bits |= PKV_ERR_PAGE_RANGE;
        else to = static_cast<long long>(page) * a.page_size + at % a.page_size;
      }
    }
    tree_report(a.err, bits);
    if (lane == 0) {
      s_pos[j] = pos;
      s_row[j] = to;
    }
  }
  __syncthreads();
  for (int t = tid; t < EACH * (D / 2); t += blockDim.x) {
    const int j = t / (D / 2), i = t % (D / 2);
    // the nearest half turn's fraction, in units of half a turn
    const int32_t frac =
        static_cast<int32_t>((static_cast<uint64_t>(s_pos[j]) * turns.f[i]) >> 32);
    float sn, cs;
    sincospif(static_cast<float>(frac) * 0x1p-31f, &sn, &cs);
    s_rot[j][i] = make_float2(cs, sn);
  }
  __syncthreads();
  const long long head_rows = static_cast<long long>(a.n_pages) * a.page_size;
  // (whole warps go round together: the lanes of a head reduce with shuffles)
  for (int h0 = 0; h0 < heads; h0 += blockDim.x / LANES, h += blockDim.x / LANES) {
    const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
    const __nv_bfloat16 *g = is_q ? a.gq : is_v ? nullptr : a.gk;
    const bool norm = is_v ? a.v_norm != 0 : g != nullptr;
    uint4 gl4 = make_uint4(0, 0, 0, 0), gh4 = gl4;
    if (g) {
      gl4 = *reinterpret_cast<const uint4 *>(g + 8 * part);
      gh4 = *reinterpret_cast<const uint4 *>(g + D / 2 + 8 * part);
    }
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
      const int pos = s_pos[j];
      if (pos < 0) continue;
      if (h0 > 0 && h < heads) load(node0 + j, h, lo4[j], hi4[j]);
      float lo[8], hi[8];
      unpack8(lo4[j], lo);
      unpack8(hi4[j], hi);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(lo[e], lo[e], fmaf(hi[e], hi[e], ss));
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (h >= heads) continue;
      if (norm) {
        const float inv = rsqrtf(ss / D + a.eps);
        float gl[8], gh[8];
        unpack8(gl4, gl);
        unpack8(gh4, gh);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          lo[e] *= g ? inv * gl[e] : inv;
          hi[e] *= g ? inv * gh[e] : inv;
        }
      }
      if (!is_v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 w = s_rot[j][8 * part + e];
          const float x1 = lo[e], x2 = hi[e];
          lo[e] = x1 * w.x - x2 * w.y;
          hi[e] = x2 * w.x + x1 * w.y;
        }
      }
      __nv_bfloat16 *to;
      if (is_q) {
        to = a.q_out + (static_cast<long long>(node0 + j) * a.Hq + h) * D;
      } else {
        if (s_row[j] < 0) continue;
        const int hk = is_v ? h - a.Hq - a.Hkv : h - a.Hq;
        to = (is_v ? a.v_cache : a.k_cache) + (hk * head_rows + s_row[j]) * D;
      }
      *reinterpret_cast<uint4 *>(to + 8 * part) = pack8(lo);
      *reinterpret_cast<uint4 *>(to + D / 2 + 8 * part) = pack8(hi);
    }
  }
}

template <int D>
cudaError_t launch(const AppendArgs &a, float theta, int rotary_dims, cudaStream_t s) {
  // the table of the thread's last theta and rotary_dims (1 to 3 us of products; a model's
  // layers have one or two of them)
  static thread_local Turns<D> t;
  static thread_local float t_theta = 0.f;
  static thread_local int t_rotary = -1;
  if (theta != t_theta || rotary_dims != t_rotary) {
    pkv::rotation_turns(theta, rotary_dims / 2, D, t.f);
    for (int i = rotary_dims / 2; i < D / 2; ++i) t.f[i] = 0;
    t_theta = theta, t_rotary = rotary_dims;
  }
  const int want = (a.Hq + 2 * a.Hkv) * (D / 16);
  const int threads = want >= kMaxThreads ? kMaxThreads : (want + 31) / 32 * 32;
  if (a.N <= kAlone * pkv::sm_count())
    return pkv::launch_pdl(tree_append_kernel<D, 1>, dim3(a.N), dim3(threads), 0, s, a, t);
  return pkv::launch_pdl(tree_append_kernel<D, kEach>, dim3((a.N + kEach - 1) / kEach),
                         dim3(threads), 0, s, a, t);
}

}  // namespace

extern "C" int tree_qkv_norm_rope_append(
    const pkv_bf16 *q, const pkv_bf16 *k, const pkv_bf16 *v, int64_t q_stride, int64_t k_stride,
    int64_t v_stride, const pkv_bf16 *gamma_q, const pkv_bf16 *gamma_k, const int32_t *batch_idx,
    const int32_t *ctx_lens, const int32_t *row_start, const int32_t *parents, float theta,
    float eps, int rotary_dims, int v_norm, int B, int N, int Hq, int Hkv, int D,
    const int32_t *dev_table, int n_slots, int max_pages_per_seq, int page_size, int n_pages,
    pkv_bf16 *k_cache, pkv_bf16 *v_cache, pkv_bf16 *q_out, int32_t *err_word, void *stream) {
  static const char *fn = "tree_qkv_norm_rope_append";
  if (D != 64 && D != 128 && D != 256 && D != 512)
    return pkv::fail(PKV_E_BAD_ARG, "%s: D must be 64, 128, 256 or 512", fn);
  if (B < 0 || B > kTreeRows || N < 0 || Hq < 1 || Hq > 65535 || Hkv < 1 || Hkv > 65535)
    return pkv::fail(PKV_E_BAD_ARG, "%s: bad shape (at most %d rows)", fn, kTreeRows);
  if (page_size < 1 || n_pages < 1 || n_slots < 1 || max_pages_per_seq < 1)
    return pkv::fail(PKV_E_BAD_ARG, "%s: bad table geometry", fn);
  if (rotary_dims < 0 || rotary_dims > D || rotary_dims % 2)
    return pkv::fail(PKV_E_BAD_ARG, "%s: rotary_dims must be even and in [0, D]", fn);
  if (!(theta >= pkv::kLeastTheta) || std::isinf(theta))
    return pkv::fail(PKV_E_BAD_ARG, "%s: theta must be finite and at least 2^-56", fn);
  if (!(eps >= 0.f)) return pkv::fail(PKV_E_BAD_ARG, "%s: eps must be >= 0", fn);
  if ((gamma_q == nullptr) != (gamma_k == nullptr))
    return pkv::fail(PKV_E_BAD_ARG, "%s: give both gains or neither", fn);
  if (B == 0 || N == 0) return pkv::ok();
  if (!q || !k || !ctx_lens || !row_start || !parents || !dev_table || !k_cache || !v_cache ||
      !q_out)
    return pkv::fail(PKV_E_BAD_ARG, "%s: NULL tensor", fn);
  if (!v) {   // the value is the raw key
    v = k;
    v_stride = k_stride;
  }
  if (!pkv::aligned16(q) || !pkv::aligned16(k) || !pkv::aligned16(v) || !pkv::aligned16(k_cache) ||
      !pkv::aligned16(v_cache) || !pkv::aligned16(q_out) || !pkv::aligned16(gamma_q) ||
      !pkv::aligned16(gamma_k))
    return pkv::fail(PKV_E_BAD_ARG, "%s: tensors must be 16-byte aligned", fn);
  const int64_t most = int64_t(1) << 40;
  if (q_stride % 8 || k_stride % 8 || v_stride % 8 || q_stride < 0 || k_stride < 0 ||
      v_stride < 0 || q_stride > most || k_stride > most || v_stride > most)
    return pkv::fail(PKV_E_BAD_ARG, "%s: token strides must be multiples of 8 elements", fn);
  const AppendArgs a = {reinterpret_cast<const __nv_bfloat16 *>(q),
                        reinterpret_cast<const __nv_bfloat16 *>(k),
                        reinterpret_cast<const __nv_bfloat16 *>(v),
                        reinterpret_cast<const __nv_bfloat16 *>(gamma_q),
                        reinterpret_cast<const __nv_bfloat16 *>(gamma_k),
                        q_stride, k_stride, v_stride, batch_idx, ctx_lens, row_start, parents,
                        dev_table, reinterpret_cast<__nv_bfloat16 *>(k_cache),
                        reinterpret_cast<__nv_bfloat16 *>(v_cache),
                        reinterpret_cast<__nv_bfloat16 *>(q_out), err_word, eps, v_norm, B, N, Hq,
                        Hkv, n_slots, max_pages_per_seq, page_size, n_pages};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  PKV_CUDA_CHECK(D == 64    ? launch<64>(a, theta, rotary_dims, s)
                 : D == 128 ? launch<128>(a, theta, rotary_dims, s)
                 : D == 256 ? launch<256>(a, theta, rotary_dims, s)
                            : launch<512>(a, theta, rotary_dims, s));
  return pkv::ok();
}
