// kv_append_q8, kv_append_prefill_q8: the paged write of new K/V tokens into
// the 8-bit cache (e4m3 codes, one power-of-two scale per kv head and block of
// tokens).
//
// A power of two as scale costs e4m3 none of its precision (the codes are
// floating point) and makes x / s and the rescaling of codes already held
// plain exponent shifts, so a block filled token by token holds what one call
// would have written, but for values below the codes' normal range.
//
// Work: the tokens of one block that the call brings stand next to each other (a run).
// A warp looks at a window of tokens for one head of K or V or both; the first token of
// each run there is taken by a group of lanes (4 to 32, or the CTA's 128 threads, by the
// size of a run), which finds the run's largest magnitude and the block's scale,
// rescales older codes if the scale grew and writes the new ones. Extra CTAs look for
// tokens of one block that stand apart. Bound by reading k and v and writing half their
// bytes: 16411 tokens of 16 prompts (8 heads of 128, blocks of 16; 101 MB) take 21.4 us,
// 0.69 of the measured 6789 GB/s (an elementwise copy of as many bytes: 16.1 us; the warps
// issue in 43% of the cycles and wait for loads in most others), a decode step of 8 rows
// 2.7 us, one of 512 rows 4.4 us, both the latency of index, table, token and store.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "pkv_internal.h"

namespace {

constexpr int kWarps = 4;
constexpr int kChecked = 4096; // tokens of a call that are looked at for their order
constexpr int kTable = 2048;   // places of a checking CTA's table, for about 1024 blocks

struct Args {
  const __nv_bfloat16 *k, *v;
  const int32_t *batch_idx, *input_pos, *table;
  int N, n_slots, max_pages, page_size, n_pages, block, log2_block;
  pkv::Divisor page;   // by page_size
  uint8_t *k_cache, *v_cache;
  float *k_scale, *v_scale;
  int Hkv, D;
  long long token_stride, head_stride;   // of k and v, in elements
  int window;                            // tokens a task covers, looked at 31 at a time
  int tensors;                           // 2: a warp does K and V of its head, 1: one of them
  int group;                             // lanes a run: 4 .. 32 (unused when a CTA takes one)
  int checkers;                          // CTAs that look for tokens of a block apart
  int32_t *err;
};

struct Unit {   // 16 bf16 values
  uint4 lo, hi;
};
__device__ __forceinline__ Unit load_unit(const __nv_bfloat16 *x) {
  const uint4 *a = reinterpret_cast<const uint4 *>(x);
  return {a[0], a[1]};
}
__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t x) {
  return *reinterpret_cast<const __nv_bfloat162 *>(&x);
}
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 x) {
  return *reinterpret_cast<const uint32_t *>(&x);
}
// Running maxima of |x| (a NaN counts nothing, an infinity does).
__device__ __forceinline__ __nv_bfloat162 max_abs(__nv_bfloat162 m, const uint4 &x) {
  m = __hmax2(m, __habs2(as_bf162(x.x)));
  m = __hmax2(m, __habs2(as_bf162(x.y)));
  m = __hmax2(m, __habs2(as_bf162(x.z)));
  return __hmax2(m, __habs2(as_bf162(x.w)));
}
// The same over finite values alone.
__device__ __forceinline__ uint32_t finite(uint32_t x) {
  const uint32_t a = x & 0x7fff7fffu;
  return a & __vcmpltu2(a, 0x7f807f80u);
}
__device__ __forceinline__ __nv_bfloat162 max_finite(__nv_bfloat162 m, const uint4 &x) {
  return max_abs(m, make_uint4(finite(x.x), finite(x.y), finite(x.z), finite(x.w)));
}

// Two values times a power of two (exact in bf16 but below 2^-126, which rounds to 0
// in e4m3 all the same), to e4m3.
__device__ __forceinline__ uint32_t quantise2(uint32_t x, __nv_bfloat162 inv) {
  const uint32_t y = as_u32(__hmul2(as_bf162(x), inv));
  return __nv_cvt_float2_to_fp8x2(
      make_float2(__uint_as_float(y << 16), __uint_as_float(y & 0xffff0000u)), __NV_SATFINITE,
      __NV_E4M3);
}
__device__ __forceinline__ uint32_t quantise4(uint32_t a, uint32_t b, __nv_bfloat162 inv) {
  return __byte_perm(quantise2(a, inv), quantise2(b, inv), 0x5410);
}
__device__ __forceinline__ uint4 quantise(const Unit &x, __nv_bfloat162 inv) {
  return make_uint4(quantise4(x.lo.x, x.lo.y, inv), quantise4(x.lo.z, x.lo.w, inv),
                    quantise4(x.hi.x, x.hi.y, inv), quantise4(x.hi.z, x.hi.w, inv));
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

__device__ __forceinline__ int slot_of(const Args &a, long long i) {
  return a.batch_idx ? a.batch_idx[i] : static_cast<int>(i);
}
// Tokens of one block apart: then the block has two leading tokens, tokens that start a
// run or are their block's first. So every leading token's (slot, block) must be new.
// Each checking CTA looks at the first kChecked tokens and keeps the leading ones whose
// hash is its share in a table in shared memory. (All tokens, by every checking CTA,
// would take longer than the append itself: 256k tokens of one 64-wide head are 15 us.)
__device__ __forceinline__ void check_order(const Args &a) {
  __shared__ unsigned long long table[kTable];
  const int bmask = a.block - 1, n = min(a.N, kChecked), lane = threadIdx.x & 31;
  bool clash = false;
  for (int i = threadIdx.x; i < kTable; i += blockDim.x) table[i] = 0;
  __syncthreads();
  constexpr int U = 8;   // tokens a thread has in flight
#pragma unroll 1
  for (int i0 = threadIdx.x; i0 - static_cast<int>(threadIdx.x) < n; i0 += U * kWarps * 32) {
    int slots[U], poss[U], before_slot[U], before_pos[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kWarps * 32;
      slots[u] = i < n ? slot_of(a, i) : -1;
      poss[u] = i < n ? a.input_pos[i] : -1;
      before_slot[u] = lane == 0 && i > 0 && i < n ? slot_of(a, i - 1) : -1;
      before_pos[u] = lane == 0 && i > 0 && i < n ? a.input_pos[i - 1] : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int slot = slots[u], pos = poss[u];
      int prev_slot = __shfl_up_sync(0xffffffffu, slot, 1);
      int prev_pos = __shfl_up_sync(0xffffffffu, pos, 1);
      if (lane == 0) {
        prev_slot = before_slot[u];
        prev_pos = before_pos[u];
      }
      if (slot > 0 && slot < a.n_slots && pos >= 0 &&
          ((pos & bmask) == 0 || prev_slot != slot || prev_pos != pos - 1)) {
        const unsigned long long key =
            static_cast<unsigned long long>(slot) << 32 | static_cast<uint32_t>(pos & ~bmask);
        uint32_t h = static_cast<uint32_t>(pos & ~bmask) * 0x9e3779b1u + slot * 0x85ebca77u;
        h = (h ^ h >> 15) * 0x2c1b3c6du;
        h ^= h >> 13;
        if (__umulhi(h, a.checkers) == blockIdx.x) {
          uint32_t at = h * 0x297a2d39u >> 16;
          for (int k = 0; k < kTable; ++k, ++at) {
            const unsigned long long old = atomicCAS(table + at % kTable, 0ull, key);
            clash |= old == key;
            if (old == 0ull || old == key) break;
          }
        }
      }
      __syncwarp();
    }
  }
  if (__any_sync(0xffffffffu, clash) && lane == 0 && a.err) atomicOr(a.err, PKV_ERR_ORDER);
}

// CTA: one run at a time for the whole CTA, else for a group of lanes. KEEP: 16-value
// units of a run that a lane keeps between the two passes. CTAs an SM, by the registers
// left to them (us for the cases named at the launch): KEEP 2: 5 28.9 (blocks of 1), 21.5
// (one head); 7 24.3, 19.1; 8 23.9, 18.7; 9 24.9, 19.4. KEEP 4: 4 23.3; 5 21.6; 6 21.4;
// 7 21.6. A CTA a run: 5 29.3; 8 24.1.
template <bool CTA, int KEEP>
__global__ void __launch_bounds__(kWarps * 32, CTA || KEEP == 2 ? 8 : 6)
    append_q8_kernel(const Args a) {
  pkv_wait_prior_grid();
  pkv_allow_next_grid();
  if (static_cast<int>(blockIdx.x) < a.checkers) {
    check_order(a);
    return;
  }
  const int lane = threadIdx.x & 31;
  const uint32_t block = blockIdx.x - a.checkers;
  const uint32_t task = CTA ? block : block * kWarps + (threadIdx.x >> 5);
  const uint32_t per_window = a.tensors == 2 ? a.Hkv : 2 * a.Hkv;
  const uint32_t window = task / per_window;
  const long long i0 = static_cast<long long>(window) * a.window;
  if (i0 >= a.N) return;
  const int which = static_cast<int>(task - window * per_window);
  const int kv0 = which >= a.Hkv ? 1 : 0;   // 0: K, 1: V
  const int h = which - kv0 * a.Hkv;
  const bool reporter = which == 0;
  const int bmask = a.block - 1;
  const int units = a.D / 16;   // of a token
  // this lane's place in its group
  const int gs = CTA ? kWarps * 32 : a.group;
  const int gw = CTA ? 32 : gs;                  // lanes of the group in this warp
  const int g0 = lane & ~(gw - 1);               // the group's first lane here
  const int gl = CTA ? threadIdx.x : lane - g0;
  const uint32_t gmask = (gw == 32 ? 0xffffffffu : (1u << gw) - 1u) << g0;
  __shared__ uint32_t part[2][kWarps];
  int turn = 0;
  auto group_max = [&](uint32_t v) -> uint32_t {
    v = __reduce_max_sync(gmask, v);
    if constexpr (CTA) {
      turn ^= 1;
      if (lane == 0) part[turn][threadIdx.x >> 5] = v;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kWarps; ++i) v = max(v, part[turn][i]);
    }
    return v;
  };

  const long long i1 = min(static_cast<long long>(a.N), i0 + a.window);
  for (long long w0 = i0; w0 < i1; w0 += 31) {
    const long long w1 = min(i1, w0 + 31);
    // lane l looks at token w0 + l - 1: the one before the window, the window, and
    // what a run that begins there goes on to
    const long long mine = w0 + lane - 1;
    const bool there = mine >= 0 && mine < a.N;
    const int my_slot = there ? slot_of(a, mine) : -1;
    const int my_pos = there ? a.input_pos[mine] : -1;
    const int prev_slot = __shfl_up_sync(0xffffffffu, my_slot, 1);
    const int prev_pos = __shfl_up_sync(0xffffffffu, my_pos, 1);
    const uint32_t goes_on = __ballot_sync(
        0xffffffffu, there && lane > 0 && mine > 0 && my_pos > 0 && prev_slot == my_slot &&
                         prev_pos == my_pos - 1 && (my_pos & bmask) != 0);
    // tokens of the window that lead a run of their block
    uint32_t leaders = ~goes_on & __ballot_sync(0xffffffffu, there && lane > 0 && lane <= w1 - w0);

    while (leaders) {
      int l = 0;   // this group's: the groups take the next ones in turn
      for (int q = 0; q < 32; q += gw) {
        if (q == g0 && leaders) l = __ffs(leaders) - 1;
        leaders &= leaders - 1;   // (0 stays 0)
      }
      const int slot = __shfl_sync(0xffffffffu, my_slot, l);
      const int pos = __shfl_sync(0xffffffffu, my_pos, l);
      const long long i = w0 + l - 1;
      if (l > 0 && slot != 0) {   // a leader, and not padding
        int bits = 0;
        if (slot < 0 || slot >= a.n_slots) bits = PKV_ERR_SLOT;
        else if (pos < 0 || a.page.quotient(pos) >= a.max_pages) bits = PKV_ERR_POS;
        int page = 0, in_page = 0;
        if (!bits) {
          const int pb = a.page.quotient(pos);
          in_page = pos - pb * a.page_size;
          page = a.table[static_cast<long long>(slot) * a.max_pages + pb];
        }
        // the run in this block: tokens i .. i + n - 1
        const int first = pos & bmask, room = a.block - first;
        int n = 32 - l;   // tokens in sight
        if (l < 31) {
          const uint32_t after = ~goes_on >> (l + 1);   // a zero bit: that token goes on
          if (after & (0x7fffffffu >> l)) n = __ffs(after);
        }
        if (n == 32 - l) {   // it may go on out of sight
          while (n < room) {
            const long long j = i + n + (lane - g0);
            const bool in = n + (lane - g0) < room && j < a.N && slot_of(a, j) == slot &&
                            a.input_pos[j] == pos + n + (lane - g0);
            const uint32_t m = __ballot_sync(gmask, in) >> g0;
            const int more = min(__ffs(~m) == 0 ? 32 : __ffs(~m) - 1, gw);
            n += more;
            if (more < gw) break;
          }
        }
        const int total = n * units;
        const bool flat = a.token_stride == a.D || n == 1;
        for (int kv = kv0; kv < kv0 + a.tensors; ++kv) {
          const __nv_bfloat16 *x = (kv ? a.v : a.k) + i * a.token_stride + h * a.head_stride;
          auto unit = [&](int u) -> const __nv_bfloat16 * {
            if (flat) return x + 16 * u;
            const int t = u / units;
            return x + t * a.token_stride + 16 * (u - t * units);
          };
          // pass 1: the largest magnitude; a lane's first KEEP units stay (their loads
          // go out beside the table's)
          Unit keep[KEEP];
#pragma unroll
          for (int j = 0; j < KEEP; ++j) {
            const int u = gl + gs * j;
            if (u < total) keep[j] = load_unit(unit(u));
            else keep[j].lo = keep[j].hi = make_uint4(0u, 0u, 0u, 0u);
          }
          if (!bits) {
            if (page < 0) bits = PKV_ERR_PAGE_NEG;
            else if (page >= a.n_pages) bits = PKV_ERR_PAGE_RANGE;
          }
          if (bits) break;
          const long long row0 = static_cast<long long>(h) * a.n_pages * a.page_size +
                                 static_cast<long long>(page) * a.page_size + in_page;
          uint8_t *codes = (kv ? a.v_cache : a.k_cache) + row0 * a.D;
          float *scale = (kv ? a.v_scale : a.k_scale) + (row0 >> a.log2_block);
          // read by the lane that replaces it (the maximum's exchange orders no memory
          // between lanes), or by all threads of a CTA, whose barrier does
          float held_raw = first && (CTA || gl == 0) ? *scale : 0.f;
          __nv_bfloat162 m2 = __float2bfloat162_rn(0.f);
#pragma unroll
          for (int j = 0; j < KEEP; ++j) m2 = max_abs(max_abs(m2, keep[j].lo), keep[j].hi);
#pragma unroll 2
          for (int u = gl + gs * KEEP; u < total; u += gs) {
            const Unit y = load_unit(unit(u));
            m2 = max_abs(max_abs(m2, y.lo), y.hi);
          }
          uint32_t amax = group_max(max(as_u32(m2) & 0xffffu, as_u32(m2) >> 16));
          if (amax >= 0x7f80u) {   // an infinity among them: the finite ones again
            m2 = __float2bfloat162_rn(0.f);
            for (int u = gl; u < total; u += gs) {
              const Unit y = load_unit(unit(u));
              m2 = max_finite(max_finite(m2, y.lo), y.hi);
            }
            amax = group_max(max(as_u32(m2) & 0xffffu, as_u32(m2) >> 16));
          }
          if constexpr (!CTA)
            if (first) held_raw = __shfl_sync(gmask, held_raw, g0);
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
            uint4 *old = reinterpret_cast<uint4 *>(codes - static_cast<long long>(first) * a.D);
            for (int u = gl; u < first * units; u += gs) {
              const uint4 c = old[u];
              old[u] = make_uint4(rescale4(c.x, ratio), rescale4(c.y, ratio), rescale4(c.z, ratio),
                                  rescale4(c.w, ratio));
            }
          }
          if (gl == 0) *scale = s;
          // pass 2: the codes
          const __nv_bfloat162 inv2 = __float2bfloat162_rn(inv);
          uint4 *dst = reinterpret_cast<uint4 *>(codes);
#pragma unroll
          for (int j = 0; j < KEEP; ++j) {
            const int u = gl + gs * j;
            if (u < total) dst[u] = quantise(keep[j], inv2);
          }
#pragma unroll 1
          for (int u = gl + gs * KEEP; u < total; u += gs)
            dst[u] = quantise(load_unit(unit(u)), inv2);
        }
        if (bits && reporter && gl == 0 && a.err) atomicOr(a.err, bits);
      }
      __syncwarp();
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
  a.page.set(page_size);
  a.n_pages = n_pages;
  a.block = scale_block;
  a.log2_block = 0;
  while ((1 << a.log2_block) < scale_block) ++a.log2_block;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.Hkv = Hkv;
  a.D = D;
  a.token_stride = head_major ? D : 1LL * Hkv * D;
  a.head_stride = head_major ? 1LL * N * D : D;
  a.err = err_word;
  // A run's expected units of 16 values: a block's tokens in a prompt, one token else.
  const long long run = 1LL * (head_major ? scale_block : 1) * D / 16;
  // Measured, in us (16411 tokens of 8 heads of 128 in blocks of 16 / 64 / 1; 200003 tokens
  // of one head of 64 in blocks of 16; 8200 tokens of 2 heads of 512 in blocks of 16):
  // - few: one token of K or V a warp, for the shortest latency, up to 64 warps an SM (24
  //   to 32 of them resident at a time). 8 and 512 rows: 2.8 and 4.5, without it 4.7 and 13.0;
  //   steps of 300, 512, 700 and 1200 rows of 8 heads of 128: 4.2, 6.2, 7.8 and 12.1, without
  //   it 8.2, 8.2, 8.3 and 8.4; packed tokens, 300, 580, 700 and 1200: 3.6, 4.6, 5.1 and 7.1,
  //   without it 5.3, 5.2, 5.7 and 5.4; used for all calls 78 / 92 / 147, 104, 27.
  // - whole_cta: a CTA a run of 8 units a lane of a warp and more. 24.1 (blocks of 64) and
  //   12.1 (512 wide); never: 34.2 and 33.0; from half that size on: 42 instead of 21.4
  //   for the first.
  // - window: 16 tokens 21.4 / - / 23.9, 18.7; 8: 21.5 / - / 24.5, 24.1; 31: 23.1 / - /
  //   24.6, 20.5. A CTA takes a block's tokens: 24.1 for 64; 16 of them: 29.1.
  // - tensors: K and V one after the other, which share what is looked up: 21.4 / - / 23.9,
  //   18.7; a warp each: 22.2 / - / 27.2, 20.8. (A CTA or a lone token: one, for more warps.)
  // - group: two units of a run a lane, four lanes at least: 23.9 (blocks of 1); one unit
  //   a lane 33.5; always a whole warp 102.
  // - KEEP: room for two units where a run fits that: 23.9 and 18.7, for four 30.6 and 21.9;
  //   for two only, with the others read again: 26.9 instead of 21.4.
  const bool few = 2LL * N * Hkv <= 64LL * sms;
  const bool whole_cta = !few && run >= 256;
  a.window = few ? 1 : whole_cta && scale_block > 16 ? scale_block : 16;
  a.tensors = few || whole_cta ? 1 : 2;
  a.group = 32;
  if (!few)
    while (a.group > 4 && a.group >= run) a.group /= 2;
  a.checkers = ((N < kChecked ? N : kChecked) + 1023) / 1024;
  const long long tasks = (N + a.window - 1LL) / a.window * Hkv * (3 - a.tensors);
  const long long blocks = a.checkers + (whole_cta ? tasks : (tasks + kWarps - 1) / kWarps);
  if (blocks > 0x7fffffffLL || tasks > 0xfffffff0LL) return pkv::fail(PKV_E_BAD_ARG, "%s: too large", fn);
  auto *kern = whole_cta               ? append_q8_kernel<true, 4>
               : run <= 2 * a.group ? append_q8_kernel<false, 2>
                                    : append_q8_kernel<false, 4>;
  PKV_CUDA_CHECK(pkv::launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(kWarps * 32), 0,
                                 static_cast<cudaStream_t>(stream), a));
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
