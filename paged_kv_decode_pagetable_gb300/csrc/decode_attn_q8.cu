// paged_decode_attn_q8: split-KV GQA decode attention over the paged 8-bit cache
// (e4m3 codes, one fp32 scale per kv head and block of tokens).
//
//   s_j = scale * sk_j * (q . ck_j),  out = sum_j softmax(s)_j sv_j cv_j
//
// Bound by reading the codes and scales of every key once. Measured against the measured
// 6789 GB/s: 16 rows of 16k to 32k tokens (8 heads of 128, blocks of 32) 123.3 us, 0.96;
// 256 rows of 500 to 1500 tokens 88.9 us, 0.88; 64 rows of 100 to 1024 tokens 19.2 us, 0.57;
// 64 rows of 256 to 2048 tokens with one 512-wide head 23.4 us, 0.48; one row of 32k
// tokens 19.0 us, 0.52; 64-wide heads, 16 rows of 8k to 16k tokens 51.5 us, 0.58. Without
// its arithmetic (an earlier state, of 19.0 and 50.6) the kernel took 16.5 and 40 us for the
// 64 rows and the 64-wide ones: what small calls cost beyond their bytes is the start (launch,
// row set-up, page lookups, the first tiles' latency: about 5 us) and the joins (2 to 5 us);
// at D = 64 the fixed work of a tile of 4 KB.
// Design (GB300):
//   * work: the 64-key tiles of every (row, kv head), plus START positions for each
//     start of a (row, head), laid on one line from the actual lengths; every
//     persistent CTA takes an equal share of it. A (row, head) that straddles
//     CTAs is cut into parts; a CTA has at most one part that is not its (row,
//     head)'s first, and that part is its first work, so the workspace is one fp32
//     record a CTA. Each word of a record is the complement of the value's bits, so
//     a zero word is one not yet written: who takes a part in polls the words
//     themselves (no flag, no fence) and clears them. Parts are joined in a tree of
//     eights (part j takes in j + 1 .. j + 7, then j + 8 ..; a tree of sixteens: one
//     row of 32k tokens 19.9 -> 22.9 us) in a fixed order: results do not depend on
//     timing. A first part is its CTA's last work, and a part that takes in others
//     but is not first its CTA's only work, so they find the others written, or
//     wait for CTAs that began with that very work. The shares are given out from the
//     line's end: a part's takers lie before it on the line, so a CTA waits only for CTAs
//     with lower block numbers, which are started before it, and a call ends however few
//     CTAs can be resident beside other work (given out from the front, three or four CTAs
//     that each wait for one not started could hold all there is);
//   * one producer warp streams query rows (cp.async.bulk), K and V tiles
//     (cp.async.bulk.tensor into a swizzled ring, K and V entries of their own) and
//     the scales of up to 32 tiles at a time (cp.async) ahead of four consumer warps,
//     looking up the next unit's pages while the current one moves;
//   * a consumer warp owns 16 keys of every tile (D >= 256) or 32 keys of every
//     other tile (two teams of two warps: twice the independent work between two
//     steps of the softmax) and keeps its own online softmax over the whole unit, so
//     no tile needs a barrier between warps. At a unit's end it leaves its state in
//     shared memory and goes on; a joining warp adds the four states and writes the
//     output or the partial. A part that is its CTA's last work, as every part that takes
//     others in is, is added up by the consumer warps themselves, the loads of several
//     parts in flight at once (last parts that take none in, too: sliding 11.8 -> 11.2 us,
//     B = 8 9.5 -> 9.2; whole rows stay with the joining warp: one short row 3.5, not 4.0).
//     At D = 512 the consumer warps join every unit;
//   * keys are the M rows of S^T = K q^T and head-dim is the M rows of O^T = V^T P^T
//     (mma.sync m16n8k16, fp16 in, fp32 out), the <= 8 query heads of the group are N;
//     P goes from one product to the other through movmatrix. The products are 4 G
//     FLOP a code byte and busy the tensor pipe about a tenth of the time, so
//     tcgen05.mma has no rate to add: its operands come from shared memory, where the
//     codes would have to be written back as fp16 first (with q and P in e4m3 instead,
//     the result would lose most of q's and P's bits);
//   * codes become fp16 in registers (exact). q is scaled by a power of two that
//     brings its row's largest magnitude to 2^15 .. 2^16, so it is exact in fp16 too (elements
//     below 2^-29 of the largest lose at most 2^-40 of it). The scale of v is part of
//     the softmax weight: w_j = 2^(s_j + log2 sv_j - M) with M the running
//     maximum of that sum, so w is at most 1 however far the scales lie apart; the
//     denominator keeps a running maximum of its own, per lane. w enters the product as
//     fp16 times 2^15, so that weights down to 2^-29 keep 11 bits and none above 2^-40 is
//     lost (times 1, a key 2^-25 as heavy as its warp's heaviest would add nothing); the
//     factor goes where the warps' states are joined. The sum is rounded up for M alone and
//     w taken as 2^((s_j - M) + log2 sv_j), whose difference is exact where w counts: added
//     to a score of 10^5 the logarithm would keep 7 bits behind the point;
//   * every wait is bounded; one that gives up sets PKV_ERR_TIMEOUT,
//     the CTA drains its copies and exits. Invalid table entries are reported
//     and never dereferenced.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <mutex>

#include "pkv_internal.h"

namespace {

constexpr int kT = 64;               // keys per tile
constexpr int kCWarps = 4;           // consumer warps
constexpr int kScaleWords = 512;     // scales of K (and of V) handed over at once
constexpr int kCThreads = kCWarps * 32;
constexpr int kThreads = kCThreads + 64;   // + producer warp and joining warp
constexpr int kMaxG = 8;             // query heads per kv head (MMA N)
constexpr float kLift = 15.f;        // log2 of the weights' factor in the product with V
constexpr float kUnlift = 1.f / 32768.f;
constexpr int kMaxRows = 512;        // rows per call (row cache kept in smem)
constexpr int kMaxCtas = 512;        // CTAs the workspace has room for
constexpr int kSpinLimit = 1 << 22;
constexpr int kPollLimit = 1 << 20;
constexpr int kFan = 8;              // fan-in of the tree that joins a cut row's parts
constexpr int kMaxSources = 24;      // parts one part takes in, 7 a level, rounded up to 4
constexpr int kMergeCols = 128;      // columns handed to the joining warp at once
constexpr int kMergeRow = kMergeCols + 4;   // padded: conflict-free 8-byte stores

template <int D>
struct Cfg {
  // One CTA per SM: D = 128 rollout batch 19.3 -> 24.9 us, 16 long rows 123 -> 169; D = 256
  // mixed (16 rows of 8k to 16k tokens 39.7 -> 43.1, 64 rows of 256 to 2048 16.2 -> 14.9,
  // sliding 11.2 -> 11.5); D = 512 has room for one. Three at D = 64, with half the ring: 16
  // rows of 8k to 16k tokens 51.5 -> 48.0, one short row 3.6 -> 4.1.
  static constexpr int CTAS_PER_SM = D <= 256 ? 2 : 1;
  // What starting a (row, head) costs, in tiles (a unit's state, its query and the part
  // of its last tile not used). 1, 2, 3, 4: rollout batch at D = 128 20.2, 18.8, 19.3, 19.7
  // us; 64 rows at D = 256 17.4, 16.4, 16.2, 15.9, at D = 512 24.4, 23.8, 23.4, 23.9.
  static constexpr int START = 3;
  // 16-key blocks of a tile a warp owns. D = 128: 1 rollout batch 20.9 us, 256 rows 98.8;
  // 2 19.3, 88.9 (4, in an earlier state: 22.2 and 94.9 against 18.8 and 89.1). D = 256: 1 and
  // 2 alike (sliding 11.2, 11.5).
  static constexpr int MB = D <= 128 ? 2 : 1;
  static constexpr int TEAM = kT / 16 / MB;        // warps that share a tile
  static constexpr int TEAMS = kCWarps / TEAM;
  // Ring entries, one K or V tile each. An entry always belongs to the same team: a
  // wait for a phase of an entry is told from the phase before by parity alone, which
  // holds only for who has waited for that one too.
  static constexpr int NS = D == 64 ? 16 : D == 128 ? 8 : D == 256 ? 4 : 5;
  static_assert(TEAMS == 1 || NS % (2 * TEAMS) == 0, "entries keep their team");
  static constexpr int COLS = D < 128 ? D : 128;   // bytes of a token in one box
  static constexpr int TOKENS = D < 128 ? 2 : 1;   // tokens in a 128-byte row of the copy
  static constexpr int CHUNKS = D / COLS;
  static constexpr int CHUNK_BYTES = kT * COLS;
  static constexpr int TILE_BYTES = kT * D;
  static constexpr int Q_ROW = D * 2 + 32;   // padded: conflict-free 8-byte loads
  static constexpr int Q_STAGE = kMaxG * Q_ROW;
  static constexpr int OFF_Q = NS * TILE_BYTES;
  static constexpr int OFF_SCALE = OFF_Q + 2 * Q_STAGE;      // [2][2][kScaleWords] f32
  // states handed over: [4 warps][8 heads] rows, then M [4][8], then m and l of every
  // lane, [4 warps][8 lanes][8 heads] each
  static constexpr int MERGE_BYTES = (kCWarps * kMaxG * kMergeRow + 17 * kCWarps * kMaxG) * 4;
  static constexpr int OFF_MERGE = OFF_SCALE + 4 * kScaleWords * 4;
  static constexpr int OFF_QS = OFF_MERGE + MERGE_BYTES;   // [2][8] f32
  // weights of the states added up: the warps' and the parts' taken in
  static constexpr int OFF_SRC = OFF_QS + 2 * kMaxG * 4;   // [4 + kMaxSources][8] f32
  static constexpr int OFF_BAR = OFF_SRC + (4 + kMaxSources) * kMaxG * 4;
  // the warps' states of a part that is the CTA's last work, where the ring was:
  // [4][8][DUMP_ROW] f32, then m, l, M [4][8] each
  // Whether the consumer warps join whole units and first works too, round by round. At
  // D = 512 they would wait for four rounds of the joining warp, 1.2 us each: 64 rows 24.8 ->
  // 23.4 us, 226 rows of 58 to 227 tokens 22.9 -> 19.5. At D = 256 no difference.
  static constexpr bool SELF = D == 512;
  static constexpr int DUMP_ROW = D + 4;
  static constexpr int DUMP_STATS = kCWarps * kMaxG * DUMP_ROW;
  static_assert((DUMP_STATS + 3 * kCWarps * kMaxG) * 4 <= NS * TILE_BYTES, "states fit the ring");
  static constexpr int N_BARS = 2 * NS + 12;
  static constexpr int OFF_TILE = OFF_BAR + N_BARS * 8;   // [NS] u32: box mask, row offset
  static constexpr int OFF_MISC = OFF_TILE + NS * 4;      // abort flag, admitted units [2]
  static constexpr int OFF_DESC = (OFF_MISC + 12 + 15) & ~15;      // Unit [2]
  static constexpr int OFF_LEN = OFF_DESC + 2 * 48;                // int [kMaxRows]
  static constexpr int OFF_SLOT = OFF_LEN + kMaxRows * 4;          // int [kMaxRows]
  static constexpr int OFF_PRE = OFF_SLOT + kMaxRows * 4;          // int [kMaxRows + 1]
  static constexpr int SMEM = OFF_PRE + (kMaxRows + 1) * 4 + 1024;  // + alignment
};
// shared memory per SM on sm_103a: 228 KB, of which 1 KB is reserved per CTA
static_assert(Cfg<64>::CTAS_PER_SM * (Cfg<64>::SMEM + 1024) <= 228 * 1024, "D=64 residency");
static_assert(Cfg<128>::CTAS_PER_SM * (Cfg<128>::SMEM + 1024) <= 228 * 1024, "D=128 residency");
static_assert(Cfg<256>::CTAS_PER_SM * (Cfg<256>::SMEM + 1024) <= 228 * 1024, "D=256 residency");
static_assert(Cfg<512>::SMEM <= 227 * 1024, "D=512 smem per CTA");

// ---------------------------------------------------------------- PTX ----
__device__ __forceinline__ uint32_t smem_u32(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait: gives up after kSpinLimit polls (each may suspend the thread for
// a hardware-defined time) or as soon as the CTA aborts.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity,
                                          volatile int *abort_flag) {
  for (int i = 0; i < kSpinLimit; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) == 63 && *abort_flag) return false;
  }
  return false;
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *tm, int x, int y,
                                            int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void copy_word(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src))
               : "memory");
}
__device__ __forceinline__ void copy_words(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src))
               : "memory");
}
// Arrives on the barrier once this thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap *tm) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tm)) : "memory");
}
// The consumer warps' wait for the joining warp's word on their next unit, which comes
// within a few of its own bounded waits: the limit lies beyond them, so that all consumer
// warps get the same word.
__device__ __forceinline__ bool mbar_wait_word(uint32_t bar, uint32_t parity) {
  for (int i = 0; i < 16 * kSpinLimit; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return false;
}
// All warps meet once the mbarriers are set up.
__device__ __forceinline__ void setup_sync() {
  asm volatile("bar.sync 2, %0;" ::"n"(kThreads) : "memory");
}
// A barrier of the consumer threads that returns the OR of `v` over them. All their warps
// pass the same ones: they work through the units that the joining warp admits.
__device__ __forceinline__ bool consumer_sync_or(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "bar.red.or.pred p, 1, %2, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "n"(kCThreads)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The e4m3 codes in the low and the high half of a word as fp16 pairs (exact).
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float ex2(float x) {   // 2^x to 2 ulp; below 2^-126: 0
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float exp2i(int k) {   // 2^k, -126 <= k <= 127
  return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

// Where 16-byte unit u of tile row r lies in a tile written by the swizzled copy:
// row_base(r) ^ unit_bits(u). The copy's rows are 128 bytes (D = 64: two tokens; above
// 128: one of the 128-byte chunks, each a [kT][128 B] block), whose units are XORed with
// the row mod 8.
template <int D>
__device__ __forceinline__ uint32_t row_base(int r) {
  if (D == 64) return (r >> 1) * 128 + ((((r & 1) << 2) ^ ((r >> 1) & 7)) << 4);
  return r * 128 + ((r & 7) << 4);
}
template <int D>
__device__ __forceinline__ uint32_t unit_addr(uint32_t tile, uint32_t base, int u) {
  return D == 64 ? tile + (base ^ (u << 4))
                 : tile + (u >> 3) * Cfg<D>::CHUNK_BYTES + (base ^ ((u & 7) << 4));
}

// ------------------------------------------------------- row geometry ----
struct Problem {
  const __nv_bfloat16 *q;
  const float *k_scale, *v_scale;
  const int32_t *table, *batch_idx, *seq_lens;
  int n_slots, max_pages, log2_ps, n_pages, log2_block, window, B, Hq, Hkv, G;
  float scale_log2;
  int scale_vec;           // scale words copied at once: 4 or 1
  uint32_t *o_part, *st_part;   // [kMaxCtas] records of G * D and G * 3 words, zero between calls
  __nv_bfloat16 *out;
  int32_t *err;
};

struct RowInfo {
  int slot, L, lo, t_first, n_tiles;
};
__device__ __forceinline__ RowInfo row_keys(const Problem &p, int slot, int L) {
  RowInfo r;
  r.slot = slot;
  r.L = L;
  r.lo = p.window > 0 ? max(0, L - p.window) : 0;
  r.t_first = r.lo / kT;
  r.n_tiles = (slot <= 0 || L <= 0) ? 0 : (L + kT - 1) / kT - r.t_first;
  return r;
}
// Row b's slot (0 when invalid) and clamped length; `bits` gets its errors.
__device__ __forceinline__ int2 row_read(const Problem &p, int b, int &bits) {
  int slot = p.batch_idx ? p.batch_idx[b] : b;
  int L = p.seq_lens[b];
  bits = 0;
  if (slot < 0 || slot >= p.n_slots) {
    bits |= PKV_ERR_SLOT;
    slot = 0;
  }
  const int most = p.max_pages << p.log2_ps;
  if (L < 0 || L > most) {
    bits |= PKV_ERR_POS;
    L = L < 0 ? 0 : most;
  }
  return make_int2(slot, L);
}

// The line of work: a (row, head) with n > 0 tiles takes START + n positions, its start
// and its tiles; pre[b] is the prefix sum of that over rows, (b, g)'s positions begin
// at Hkv * pre[b] + g * (START + n). The `total` positions are shared by
// min(CTAs, total) of them: the first `few` own `each`, the others, which are started
// earlier, each + 1 (64 rows of 100 to 1024 tokens 19.3 us; the larger shares first on the
// line 19.8), so every share has a position and every CTA between a (row, head)'s first and
// last has tiles of it.
// x / d for a quotient below 2^20: the approximate one is at most one off.
__device__ __forceinline__ uint32_t small_quotient(uint32_t x, uint32_t d) {
  const uint32_t q = static_cast<uint32_t>(__fdividef(__uint2float_rz(x), __uint2float_rz(d)));
  const int r = static_cast<int>(x - q * d);
  return r < 0 ? q - 1 : r >= static_cast<int>(d) ? q + 1 : q;
}
struct Line {
  uint32_t each, few;
  __device__ __forceinline__ int bound(uint32_t c) const {
    return static_cast<int>(c * each + max(c, few) - few);
  }
  __device__ __forceinline__ int owner(uint32_t x) const {
    const uint32_t narrow = few * each;
    return static_cast<int>(x < narrow ? small_quotient(x, each)
                                       : few + small_quotient(x - narrow, each + 1));
  }
};

// A run of tiles [ta, tb) of one (row, kv head), keys [k0, k1), the part-th of
// `parts`; b < 0: no more work.
struct alignas(16) Unit {
  int b, g, slot, ta, tb, k0, k1, part, parts, first_cta;
  int last;   // the CTA's last work
};
static_assert(sizeof(Unit) <= 48, "unit descriptor slot");

// The next unit from position x on (advanced past it), in row w.b at the earliest (searched
// from there: 217 short rows 18.1 -> 17.1 us); false at the share's end. Which
// part of its (row, head) it is comes later (which_part): `first_cta` and `parts` hold
// the (row, head)'s first position and width until then, `part` whether its first
// (bit 0) and last tile (bit 1) are this unit's.
// The whole converged producer warp calls it with uniform arguments.
template <int START>
__device__ __forceinline__ bool next_unit(const Problem &p, const int *slots, const int *lens,
                                          const int *pre, int end, int &x, Unit &w, int lane) {
  while (x < end) {
    int b = (w.b & ~31) - 1;   // the last row whose positions begin at or before x
    for (int base = w.b & ~31; base < p.B; base += 32) {
      const int i = base + lane;
      const unsigned le = __ballot_sync(0xffffffffu, i < p.B && p.Hkv * pre[i] <= x);
      b += __popc(le);
      if (le != 0xffffffffu) break;
    }
    const int width = pre[b + 1] - pre[b];
    const int within = x - p.Hkv * pre[b];
    const int g = static_cast<int>(small_quotient(within, width));
    const int r = within - g * width;
    const int n = min(end - x, width - r);
    x += n;
    const int t0 = max(r, START) - START, t1 = r + n - START;   // tiles of the row: [t0, t1)
    if (t1 <= t0) continue;                          // only positions of the start
    const RowInfo ri = row_keys(p, slots[b], lens[b]);
    w.b = b;
    w.g = g;
    w.slot = ri.slot;
    w.ta = ri.t_first + t0;
    w.tb = ri.t_first + t1;
    w.k0 = max(ri.lo, w.ta * kT);
    w.k1 = min(ri.L, w.tb * kT);
    w.first_cta = p.Hkv * pre[b] + g * width;
    w.parts = width;
    w.part = (r <= START ? 1 : 0) | (r + n == width ? 2 : 0);
    w.last = end - x <= START;   // no room for a tile of another (row, head)
    return true;
  }
  return false;
}
// `me` is the share's number on the line.
template <int START>
__device__ __forceinline__ void which_part(const Line &line, int me, Unit &w) {
  const int start = w.first_cta, last = start + w.parts - 1;
  w.first_cta = w.part & 1 ? me : line.owner(start + START);
  w.parts = (w.part & 2 ? me : line.owner(last)) - w.first_cta + 1;
  w.part = me - w.first_cta;
}

// The record of a part that is not first: its share's.
__device__ __forceinline__ size_t own_record(const Unit &w) { return w.first_cta + w.part; }

// A sum l held relative to maximum m, relative to n >= m instead (a NaN stays one).
__device__ __forceinline__ float sum_at(float l, float m, float n) {
  return m == -INFINITY ? (l != l ? l : 0.f) : l * ex2(m - n);
}

// ---------------------------------------------------------- joining ----
__device__ __forceinline__ void fma4(float4 &a, float f, const float4 &v) {
  a.x = fmaf(f, v.x, a.x);
  a.y = fmaf(f, v.y, a.y);
  a.z = fmaf(f, v.z, a.z);
  a.w = fmaf(f, v.w, a.w);
}
// Words of a partial: the complement of the value's bits, never 0 (the one float
// whose complement is 0 is a NaN, stored as the canonical one).
__device__ __forceinline__ uint32_t part_word(float v) {
  const uint32_t u = __float_as_uint(v);
  return ~(u == 0xffffffffu ? 0x7fffffffu : u);
}
__device__ __forceinline__ float part_value(uint32_t w) { return __uint_as_float(~w); }
__device__ __forceinline__ uint32_t ld_word(const uint32_t *a) {
  uint32_t v;
  asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(a) : "memory");
  return v;
}
__device__ __forceinline__ void st_word(uint32_t *a, uint32_t v) {
  asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" ::"l"(a), "r"(v) : "memory");
}
__device__ __forceinline__ uint4 ld_words(const uint32_t *a) {
  uint4 v;
  asm volatile("ld.relaxed.gpu.global.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_words(uint32_t *a, uint4 v) {
  asm volatile("st.relaxed.gpu.global.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(a), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ bool written(const uint4 &v) {
  return v.x != 0u && v.y != 0u && v.z != 0u && v.w != 0u;
}

// The parts a part takes in: at level s = 1, 8, 64 the parts part + s .. part + 7 s, if
// part is a multiple of 8 s and there are as many. Bit q of the mask: source q =
// 7 level + k - 1; lane q gets its CTA.
__device__ __forceinline__ uint32_t sources(const Unit &w, int lane, int &cta) {
  const int level = lane / 7, s = 1 << (3 * min(level, 3)), j = w.part + (lane % 7 + 1) * s;
  const bool t = level < 3 && w.part % (kFan * s) == 0 && j < w.parts;
  cta = w.first_cta + (t ? j : 0);
  return __ballot_sync(0xffffffffu, t);
}
// Whether the consumer warps join a unit themselves. (A part that takes others in goes on
// in the next CTA, so it is the last.)
__device__ __forceinline__ bool joined_by_all(const Unit &w) { return w.last && w.parts > 1; }
// What a sum of outputs relative to M is multiplied by: 1 for a partial, else
// 2^(M - m) / l (no key of weight, or no key: 0; a NaN stays one).
__device__ __forceinline__ float last_factor(bool partial, float m, float l, float M) {
  return partial ? 1.f : l != l ? l : M == -INFINITY || l == 0.f ? 0.f : ex2(M - m) / l;
}
__device__ __forceinline__ uint2 pack4_bf16(const float4 &v, float f) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * f, v.y * f);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(v.z * f, v.w * f);
  return make_uint2(*reinterpret_cast<const uint32_t *>(&lo),
                    *reinterpret_cast<const uint32_t *>(&hi));
}

// The joining warp: adds up the states of the four consumer warps at the end of every
// unit that they do not join themselves. Lanes are (warp, head) for the statistics and (head,
// four columns) for the outputs. Rolled loops: what runs once or twice a CTA takes the
// time of fetching its instructions.
template <int D>
__device__ __forceinline__ void join_units(const Problem &p, uint8_t *sm, uint32_t fullQ,
                                           uint32_t readyQ, uint32_t emptyQ, uint32_t fullM,
                                           uint32_t emptyM, const Unit *udesc,
                                           volatile int *abort_flag, int lane) {
  using Cf = Cfg<D>;
  constexpr int COLS = D < kMergeCols ? D : kMergeCols;
  constexpr int ROUNDS = D / COLS;
  constexpr int LPH = COLS / 4;            // lanes a head
  constexpr int HPS = 32 / LPH;            // heads a step
  const int hs = lane / LPH, col = lane % LPH * 4;
  int it_q = 0, it_m = 0;
  volatile int *admitted = abort_flag + 1;
  pkv_wait_prior_grid();
  // The next unit: its query rows become fp16 in place, each scaled by a power of two
  // that brings its largest magnitude to 2^15 .. 2^16 (65280 at most, below fp16's largest),
  // before the consumer warps need them.
  auto receive = [&](Unit &w) {
    const int qs = it_q & 1;
    const bool q_ok = mbar_wait(fullQ + 8 * qs, (it_q >> 1) & 1, abort_flag);
    w.b = -1;
    if (q_ok) w = udesc[qs];
    __syncwarp();
    if (__any_sync(0xffffffffu, w.b < 0)) w.b = -1;
    if (w.b >= 0) {
#pragma unroll 1
      for (int h = 0; h < p.G; ++h) {
        uint32_t *row = reinterpret_cast<uint32_t *>(sm + Cf::OFF_Q + qs * Cf::Q_STAGE +
                                                     h * Cf::Q_ROW);
        uint32_t v[D / 64], m = 0;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          v[j] = row[lane + 32 * j];
          m = __vmaxu2(m, v[j] & 0x7fff7fffu);
        }
        m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
        const int e = max(static_cast<int>(m >> 7) - 127 - 15, -126);
        const float f = exp2i(-e);
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
          row[lane + 32 * j] = pack_f16(__uint_as_float(v[j] << 16) * f,
                                        __uint_as_float(v[j] & 0xffff0000u) * f);
        if (lane == 0)
          reinterpret_cast<float *>(sm + Cf::OFF_QS)[qs * kMaxG + h] = p.scale_log2 * exp2i(e);
      }
      fence_proxy_async();   // the next copy into the stage comes after these accesses
    }
    __syncwarp();
    if (lane == 0) {
      if (!q_ok) {
        *abort_flag = 1;
        if (p.err) atomicOr(p.err, PKV_ERR_TIMEOUT);
      }
      admitted[qs] = w.b >= 0;
      mbar_arrive(readyQ + 8 * qs);   // whatever came, for the consumer warps wait for it
      if (w.b >= 0) mbar_arrive(emptyQ + 8 * qs);
    }
    ++it_q;
  };
  Unit w, next;
  receive(next);
  while (true) {
    w = next;
    if (w.b < 0) return;
    receive(next);
    if (Cf::SELF || joined_by_all(w)) continue;
    const bool partial = w.part > 0;
    float f = 0.f, last = 0.f, m = 0.f, l = 0.f, M = 0.f;
#pragma unroll 1
    for (int r = 0; r < ROUNDS; ++r, ++it_m) {
      bool ok = mbar_wait(fullM, it_m & 1, abort_flag);
      ok = __all_sync(0xffffffffu, ok && !*abort_flag);
      const float *merge = reinterpret_cast<const float *>(sm + Cf::OFF_MERGE);
      if (r == 0) {
        const float *a = merge + kCWarps * kMaxG * kMergeRow;
        const float own_M = a[lane];
        a += 32 + (lane >> 3) * 64 + (lane & 7);   // the warp's lanes, for this head
        float own_m = -INFINITY, own_l = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) own_m = fmaxf(own_m, a[8 * i]);
#pragma unroll
        for (int i = 0; i < 8; ++i) own_l += sum_at(a[256 + 8 * i], a[8 * i], own_m);
        m = own_m;
        M = own_M;
#pragma unroll
        for (int i = 8; i < 32; i <<= 1) {
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
          M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, i));
        }
        l = sum_at(own_l, own_m, m);
#pragma unroll
        for (int i = 8; i < 32; i <<= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
        f = own_M == -INFINITY ? 0.f : kUnlift * ex2(own_M - M);
        last = last_factor(partial, m, l, M);
      }
#pragma unroll 1
      for (int i0 = 0; i0 < p.G; i0 += HPS) {
        const int h = (i0 + hs) & 7;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < kCWarps; ++j)
          fma4(acc, __shfl_sync(0xffffffffu, f, 8 * j + h),
               *reinterpret_cast<const float4 *>(merge + (j * kMaxG + h) * kMergeRow + col));
        const float fl = __shfl_sync(0xffffffffu, last, h);
        if (i0 + hs >= p.G || !ok) continue;
        const int at = r * COLS + col;
        if (partial)
          st_words(p.o_part + (own_record(w) * p.G + h) * D + at,
                   make_uint4(part_word(acc.x), part_word(acc.y), part_word(acc.z),
                              part_word(acc.w)));
        else
          *reinterpret_cast<uint2 *>(
              p.out + (static_cast<size_t>(w.b) * p.Hq + w.g * p.G + h) * D + at) =
              pack4_bf16(acc, fl);
      }
      if (partial && r == 0 && ok && lane < p.G) {
        uint32_t *a = p.st_part + (own_record(w) * p.G + lane) * 3;
        st_word(a, part_word(m));
        st_word(a + 1, part_word(l));
        st_word(a + 2, part_word(M));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(emptyM);
    }
  }
}

// The end of a part that is the CTA's last work, by the consumer warps, whose states lie where
// the ring was: warp 0 gathers the statistics and weighs the states, then every thread
// adds up IB places (four columns of a head) at once, of SRC parts.
template <int D, int IB, int SRC>
__device__ __forceinline__ void join_parts(const Problem &p, uint8_t *sm, const Unit &w,
                                           volatile int *abort_flag, int warp, int lane) {
  using Cf = Cfg<D>;
  const int tid = warp * 32 + lane;
  const float *dump = reinterpret_cast<const float *>(sm);
  float *weight = reinterpret_cast<float *>(sm + Cf::OFF_SRC);   // [4 + kMaxSources][8]
  int my_cta;
  const uint32_t takes = sources(w, lane, my_cta);
  const int n_src = 32 - __clz(takes);
  const bool partial = w.part > 0;
  bool bad = false;
  const int places = p.G * D / 4;
  uint32_t *a[SRC];
  uint4 v[SRC][IB];
  // sources k0 .. k0 + SRC - 1 at places i0 + i * kCThreads: what there is to wait for
  auto start_loads = [&](int i0, int k0) {
#pragma unroll
    for (int j = 0; j < SRC; ++j) {
      const int cta = __shfl_sync(0xffffffffu, my_cta, k0 + j);
      a[j] = p.o_part + static_cast<size_t>(cta) * p.G * D + 4 * i0;
#pragma unroll
      for (int i = 0; i < IB; ++i)
        v[j][i] = (takes >> (k0 + j) & 1u) && i0 + i * kCThreads < places
                      ? ld_words(a[j] + 4 * i * kCThreads)
                      : make_uint4(~0u, ~0u, ~0u, ~0u);
    }
  };
  start_loads(tid, 0);   // on their way while the statistics come in
  if (warp == 0) {
    const int sh = lane & 7, sk = lane >> 3;
    const float *own = dump + Cf::DUMP_STATS + lane;
    const float own_M = own[64];
    float m = own[0], l = own[32], M = own_M;   // of this lane's states
#pragma unroll 1
    for (int k0 = 0; k0 < n_src; k0 += 4) {
      const int k = k0 + sk;
      const int cta = __shfl_sync(0xffffffffu, my_cta, k);
      const bool mine = (takes >> k & 1u) && sh < p.G;
      uint32_t *s = p.st_part + (static_cast<size_t>(cta) * p.G + sh) * 3;
      uint32_t x0 = 0, x1 = 0, x2 = 0;
      for (int i = 0; mine; ++i) {
        x0 = ld_word(s);
        x1 = ld_word(s + 1);
        x2 = ld_word(s + 2);
        if (x0 != 0u && x1 != 0u && x2 != 0u) break;
        if (i >= kPollLimit || *abort_flag) {
          bad = true;
          break;
        }
      }
      if (mine) {
        st_word(s, 0u);
        st_word(s + 1, 0u);
        st_word(s + 2, 0u);
      }
      const float xm = mine ? part_value(x0) : -INFINITY, xM = mine ? part_value(x2) : -INFINITY;
      weight[(4 + k) * kMaxG + sh] = xM;
      const float mn = fmaxf(m, xm);
      l = sum_at(l, m, mn) + sum_at(mine ? part_value(x1) : 0.f, xm, mn);
      m = mn;
      M = fmaxf(M, xM);
    }
    const float lane_m = m;
#pragma unroll
    for (int i = 8; i < 32; i <<= 1) {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, i));
    }
    l = sum_at(l, lane_m, m);
#pragma unroll
    for (int i = 8; i < 32; i <<= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
    const float last = last_factor(partial, m, l, M);
    weight[lane] = own_M == -INFINITY ? 0.f : last * ex2(own_M - M);
#pragma unroll 1
    for (int k = 4 + sk; k < 4 + n_src; k += 4) {   // each lane the words it wrote
      const float x = weight[k * kMaxG + sh];
      weight[k * kMaxG + sh] = x == -INFINITY ? 0.f : last * ex2(x - M);
    }
    if (partial && !bad && lane < p.G) {
      uint32_t *s = p.st_part + (own_record(w) * p.G + lane) * 3;
      st_word(s, part_word(m));
      st_word(s + 1, part_word(l));
      st_word(s + 2, part_word(M));
    }
  }
  bad = consumer_sync_or(bad || *abort_flag);
  __nv_bfloat16 *out = p.out + (static_cast<size_t>(w.b) * p.Hq + w.g * p.G) * D;
#pragma unroll 1
  for (int i0 = tid; i0 - tid < places && !bad; i0 += kCThreads * IB) {
    float4 acc[IB];
    int h[IB];
#pragma unroll
    for (int i = 0; i < IB; ++i) {
      const int at = min(i0 + i * kCThreads, places - 1);
      h[i] = at / (D / 4);
      acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < kCWarps; ++j)
        fma4(acc[i], weight[j * kMaxG + h[i]],
             *reinterpret_cast<const float4 *>(dump + (j * kMaxG + h[i]) * Cf::DUMP_ROW +
                                               at % (D / 4) * 4));
    }
#pragma unroll 1
    for (int k0 = 0; k0 < n_src; k0 += SRC) {
      if (i0 != tid || k0 != 0) start_loads(i0, k0);
      for (int n = 0;; ++n) {
        bool there = true;
#pragma unroll
        for (int j = 0; j < SRC; ++j)
#pragma unroll
          for (int i = 0; i < IB; ++i) there = there && written(v[j][i]);
        if (there) break;
        if (n >= kPollLimit || *abort_flag) {
          bad = true;
          break;
        }
#pragma unroll
        for (int j = 0; j < SRC; ++j)
#pragma unroll
          for (int i = 0; i < IB; ++i)
            if (!written(v[j][i])) v[j][i] = ld_words(a[j] + 4 * i * kCThreads);
      }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < SRC; ++j)
#pragma unroll
        for (int i = 0; i < IB; ++i)
          if ((takes >> (k0 + j) & 1u) && i0 + i * kCThreads < places) {
            st_words(a[j] + 4 * i * kCThreads, make_uint4(0u, 0u, 0u, 0u));
            fma4(acc[i], weight[(4 + k0 + j) * kMaxG + h[i]],
                 make_float4(part_value(v[j][i].x), part_value(v[j][i].y),
                             part_value(v[j][i].z), part_value(v[j][i].w)));
          }
    }
    bad = __any_sync(0xffffffffu, bad);
#pragma unroll
    for (int i = 0; i < IB; ++i) {
      const int at = i0 + i * kCThreads;
      if (at >= places || bad) continue;
      const float4 &o = acc[i];
      if (partial)
        st_words(p.o_part + own_record(w) * p.G * D + 4 * at,
                 make_uint4(part_word(o.x), part_word(o.y), part_word(o.z), part_word(o.w)));
      else
        *reinterpret_cast<uint2 *>(out + 4 * at) = pack4_bf16(o, 1.f);
    }
  }
  if (bad && lane == 0 && p.err) atomicOr(p.err, PKV_ERR_TIMEOUT);
}

// ------------------------------------------------------------- kernel ----
template <int D>
__global__ void __launch_bounds__(kThreads, Cfg<D>::CTAS_PER_SM)
    decode_q8_kernel(const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const Problem p) {
  using Cf = Cfg<D>;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t s0 = smem_u32(sm);
  const uint32_t full = s0 + Cf::OFF_BAR, empty = full + 8 * Cf::NS,
                 fullQ = empty + 8 * Cf::NS, emptyQ = fullQ + 16, fullM = emptyQ + 16,
                 emptyM = fullM + 8, fullS = emptyM + 8, emptyS = fullS + 16,
                 readyQ = emptyS + 16;
  uint32_t *tile_word = reinterpret_cast<uint32_t *>(sm + Cf::OFF_TILE);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + Cf::OFF_MISC);
  Unit *udesc = reinterpret_cast<Unit *>(sm + Cf::OFF_DESC);
  int *lens = reinterpret_cast<int *>(sm + Cf::OFF_LEN);
  int *slots = reinterpret_cast<int *>(sm + Cf::OFF_SLOT);
  int *pre = reinterpret_cast<int *>(sm + Cf::OFF_PRE);

  const int ps = 1 << p.log2_ps;
  const int log2_box = min(p.log2_ps, 6);
  const int box_rows = 1 << log2_box;          // rows of one copy
  const int boxes = kT >> log2_box;            // copies a tile
  const int log2_sc = min(p.log2_block, 6);    // keys of a tile that share a scale word
  const int scales = kT >> log2_sc;            // scale words of a tile, for K and for V
  const int batch = min(32 / boxes, kScaleWords / scales);   // tiles looked up at once

  if (warp == kCWarps) {
    // ======================== producer (one warp) ========================
    // Set-up, before the dependency wait: row cache, prefix sums, the first unit and
    // its pages. It reads only seq_lens, batch_idx and the table, which no kernel that
    // may still run writes (the header's rule).
    int row_bits = 0, carry = 0;
#pragma unroll 1
    for (int base = 0; base < p.B; base += 64) {
      int2 rc[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int b = base + 32 * i + lane;
        int bits = 0;
        rc[i] = b < p.B ? row_read(p, b, bits) : make_int2(0, 0);
        row_bits |= bits;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int b = base + 32 * i + lane;
        const int n = row_keys(p, rc[i].x, rc[i].y).n_tiles;
        int v = n > 0 ? Cf::START + n : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += t;
        }
        if (b < p.B) {
          slots[b] = rc[i].x;
          lens[b] = rc[i].y;
          pre[b + 1] = carry + v;
        }
        carry += __shfl_sync(0xffffffffu, v, 31);
      }
    }
    if (lane == 0) pre[0] = 0;
    __syncwarp();
    const uint32_t total = p.Hkv * carry, ctas = min(gridDim.x, max(total, 1u));
    const Line line = {total / ctas, ctas - total % ctas};
    // Lane j looks up box j of a unit (a page's segment of one tile). box_page only
    // issues the table load; box_row checks the entry when it is used, so a
    // look-ahead load never stalls the warp.
    auto box_key = [&](const Unit &u, int j) -> int {   // first key of box j, -1 if unused
      if (j >= (u.tb - u.ta) * boxes) return -1;
      const int key = u.ta * kT + j * box_rows;
      return key + box_rows <= u.k0 || key >= u.k1 ? -1 : key;
    };
    auto box_page = [&](const Unit &u, int j) -> int {
      const int key = box_key(u, j);
      return key < 0 ? -1
                     : __ldg(p.table + static_cast<size_t>(u.slot) * p.max_pages +
                             (key >> p.log2_ps));
    };
    auto box_row = [&](const Unit &u, int j, int page) -> int {   // the box's first cache row
      const int key = box_key(u, j);
      if (key < 0) return -1;
      if (page < 0 || page >= p.n_pages) {
        if (p.err) atomicOr(p.err, page < 0 ? PKV_ERR_PAGE_NEG : PKV_ERR_PAGE_RANGE);
        return -1;
      }
      return ((u.g * p.n_pages + page) << p.log2_ps) + (key & (ps - 1));
    };
    int x = 0, end = 0;
    const int me = static_cast<int>(ctas - 1 - blockIdx.x);   // this CTA's share of the line
    if (blockIdx.x < ctas) {
      x = line.bound(me);
      end = line.bound(me + 1);
    }
    Unit w, wn;
    w.b = 0;
    int it = 0, it_q = 0, it_s = 0;
    bool ok = true;
    bool have = next_unit<Cf::START>(p, slots, lens, pre, end, x, w, lane);
    int page_first = have ? box_page(w, lane) : -1;
    if (have) which_part<Cf::START>(line, me, w);
    setup_sync();
    pkv_wait_prior_grid();
    if (blockIdx.x == 0 && row_bits && p.err) atomicOr(p.err, row_bits);
    while (ok && have) {
      bool have_next = false, looked_ahead = false;
      int page_next = -1;
      {   // the query rows of the group, and the unit itself
        const int qs = it_q & 1;
        if (lane == 0) {
          ok = mbar_wait(emptyQ + 8 * qs, ((it_q >> 1) & 1) ^ 1, abort_flag);
          if (ok) {
            udesc[qs] = w;   // published by the arrive
            mbar_expect_tx(fullQ + 8 * qs, static_cast<uint32_t>(p.G * D * 2));
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (lane < p.G)
          bulk_load(s0 + Cf::OFF_Q + qs * Cf::Q_STAGE + lane * Cf::Q_ROW,
                    p.q + (static_cast<size_t>(w.b) * p.Hq + w.g * p.G + lane) * D,
                    static_cast<uint32_t>(D * 2), fullQ + 8 * qs);
        ++it_q;
      }
      const int n_tiles = w.tb - w.ta;
      for (int base = 0; base < n_tiles && ok; base += batch) {
        const int j0 = base * boxes;
        const int row = box_row(w, j0 + lane, base == 0 ? page_first : box_page(w, j0 + lane));
        const int tiles_here = min(batch, n_tiles - base);
        for (int tt = 0; tt < tiles_here; ++tt) {
          const int t = w.ta + base + tt;
          const uint32_t mask =
              (__ballot_sync(0xffffffffu, row >= 0) >> (tt * boxes)) & ((1u << boxes) - 1u);
          // One box per tile (pages of >= 64 keys): a tile whose keys end or start
          // inside it is loaded as the 64 rows that end at its last key or start
          // at its first; rows outside the page are zero-filled by the copy and
          // never read from memory. Tile row r then holds key t * 64 + r + off.
          int off = 0;
          if (boxes == 1) {
            const int lo_r = max(w.k0 - t * kT, 0), hi_r = min(w.k1 - t * kT, kT);
            if (hi_r < kT && (lo_r == 0 || hi_r <= kT - lo_r)) off = hi_r - kT;
            else if (lo_r > 0) off = lo_r;
            off = off / Cf::TOKENS * Cf::TOKENS;   // whole rows of the copy, towards the tile's
          }
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const int st = it % Cf::NS;
            ok = ok && mbar_wait(empty + 8 * st, ((it / Cf::NS) & 1) ^ 1, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint32_t bar = full + 8 * st;
            const uint32_t dst = s0 + st * Cf::TILE_BYTES;
            if (lane == 0) {
              tile_word[st] = mask | (static_cast<uint32_t>(off & 0xff) << 8);
              mbar_expect_tx(bar, __popc(mask) * box_rows * D);
            }
            __syncwarp();
            if (lane >= tt * boxes && lane < (tt + 1) * boxes && row >= 0) {
              const int i = lane - tt * boxes;
              const int y = ((row & (ps - 1)) + off) / Cf::TOKENS, z = row >> p.log2_ps;
#pragma unroll
              for (int cc = 0; cc < Cf::CHUNKS; ++cc)
                tma_load_3d(dst + cc * Cf::CHUNK_BYTES + i * box_rows * Cf::COLS,
                            kv ? &tmV : &tmK, cc * Cf::COLS, y, z, bar);
            }
            ++it;
          }
          if (!ok) break;
          if (tt == 0) {   // the scales of all tiles here
            const int ss = it_s & 1;
            ok = mbar_wait(emptyS + 8 * ss, ((it_s >> 1) & 1) ^ 1, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const int log2_items = 31 - __clz(scales / p.scale_vec);   // a tile's copies
            const int items = tiles_here << log2_items;
            for (int e0 = 0; e0 < 2 * items; e0 += 32) {
              const int e = e0 + lane, kv = e >= items, ee = kv ? e - items : e;
              const int tile = ee >> log2_items;
              const int word = (ee & ((1 << log2_items) - 1)) * p.scale_vec;
              const int key = word << log2_sc;   // within the tile
              const int r =
                  __shfl_sync(0xffffffffu, row, (tile * boxes + (key >> log2_box)) & 31);
              if (e < 2 * items && r >= 0) {
                const uint32_t dst = s0 + Cf::OFF_SCALE +
                                     ((ss * 2 + kv) * kScaleWords + tile * scales + word) * 4;
                const float *src = (kv ? p.v_scale : p.k_scale) +
                                   ((r + (key & (box_rows - 1))) >> p.log2_block);
                if (p.scale_vec == 4) copy_words(dst, src);
                else copy_word(dst, src);
              }
            }
            copies_arrive(fullS + 8 * ss);
            ++it_s;
          }
          if (!looked_ahead) {   // the next unit's lookups, once this one is moving
            looked_ahead = true;
            wn.b = w.b;
            have_next = next_unit<Cf::START>(p, slots, lens, pre, end, x, wn, lane);
            page_next = have_next ? box_page(wn, lane) : -1;
            if (have_next) which_part<Cf::START>(line, me, wn);
          }
        }
      }
      w = wn;
      page_first = page_next;
      have = have_next;
    }
    if (ok && lane == 0) {   // end of work, in the next Q stage
      const int qs = it_q & 1;
      ok = mbar_wait(emptyQ + 8 * qs, ((it_q >> 1) & 1) ^ 1, abort_flag);
      if (ok) {
        udesc[qs].b = -1;
        mbar_arrive(fullQ + 8 * qs);
        ++it_q;
      }
    }
    copies_wait();
    __syncwarp();
    if (lane != 0) return;
    if (!ok) {
      *abort_flag = 1;
      if (p.err) atomicOr(p.err, PKV_ERR_TIMEOUT);
    }
    // drain: the last phase armed on every stage must land before exit
    volatile int no_abort = 0;
    for (int s = 0; s < Cf::NS; ++s)
      if (it > s) (void)mbar_wait(full + 8 * s, ((it - 1 - s) / Cf::NS) & 1, &no_abort);
    for (int s = 0; s < 2; ++s) {
      if (it_q > s) (void)mbar_wait(fullQ + 8 * s, ((it_q - 1 - s) / 2) & 1, &no_abort);
      if (it_s > s) (void)mbar_wait(fullS + 8 * s, ((it_s - 1 - s) / 2) & 1, &no_abort);
    }
    return;
  }

  if (warp == kCWarps + 1) {   // a lane sets up an mbarrier
    for (int i = lane; i < Cf::N_BARS; i += 32) {
      constexpr int Q0 = 2 * Cf::NS, M0 = Q0 + 4, S0 = M0 + 2;
      const int count = i < Cf::NS        ? 1              // full
                        : i < Q0          ? Cf::TEAM       // empty
                        : i < Q0 + 2      ? 1              // fullQ
                        : i < M0          ? kCWarps + 1    // emptyQ: the joining warp reads too
                        : i < M0 + 1      ? kCWarps        // fullM
                        : i < S0          ? 1              // emptyM
                        : i < S0 + 2      ? 32             // fullS
                        : i < S0 + 4      ? kCWarps        // emptyS
                                          : 1;             // readyQ
      mbar_init(full + 8 * i, count);
    }
    if (lane == 0) {
      *abort_flag = 0;
      prefetch_map(&tmK);
      prefetch_map(&tmV);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async();
    __syncwarp();
    setup_sync();
    join_units<D>(p, sm, fullQ, readyQ, emptyQ, fullM, emptyM, udesc, abort_flag, lane);
    return;
  }

  // ============================== consumers ==============================
  setup_sync();
  pkv_wait_prior_grid();
  pkv_allow_next_grid();
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {   // rows without keys: zeros
    int bits;
    const int2 rc = row_read(p, b, bits);
    if (row_keys(p, rc.x, rc.y).n_tiles > 0) continue;
    uint4 *o = reinterpret_cast<uint4 *>(p.out + static_cast<size_t>(b) * p.Hq * D);
    for (int i = tid; i < p.Hq * D / 8; i += kCThreads) o[i] = make_uint4(0u, 0u, 0u, 0u);
  }

  const int gid = lane >> 2, tig = lane & 3;
  const int h0 = 2 * tig, h1 = h0 + 1;
  constexpr int KS = D / 16;      // 16-byte units of a row = MMA steps over D = m-tiles of O^T
  constexpr bool Q_REGS = D <= 256;   // the query stays in registers
  constexpr int QK = Q_REGS ? KS : 1;
  constexpr int MB = Cf::MB;
  const int team = warp / Cf::TEAM, key0 = 16 * MB * (warp % Cf::TEAM);   // this warp's tile rows
  // 16-byte units of rows key0 .. key0 + 15 for ldmatrix (the next 16: a constant on)
  const uint32_t ldsm_base = row_base<D>(key0 + ((lane >> 3) & 1) * 8 + (lane & 7));
  constexpr uint32_t ROWS16 = 16 * Cf::COLS;
  const int ldsm_unit = lane >> 4;
  const bool hv = gid < p.G;
  int tile = 0, it_q = 0, it_m = 0, it_s = 0;   // tile: tiles of the units before
  auto give_up = [&]() {
    *abort_flag = 1;
    if (lane == 0 && p.err) atomicOr(p.err, PKV_ERR_TIMEOUT);
  };

  // Hands memory back to the producer warp. What this warp has read there with plain loads
  // comes before what the copies (another proxy) write: without the fence a load still in
  // flight could read the next tile (seen at D = 256, two CTAs an SM: one call in ten of
  // three rows of 30k tokens).
  auto release = [&](uint32_t bar) {
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  while (true) {
    const int qs = it_q & 1;
    const bool go = mbar_wait_word(readyQ + 8 * qs, (it_q >> 1) & 1) && abort_flag[1 + qs];
    if (!__all_sync(0xffffffffu, go)) break;
    const Unit w = udesc[qs];
    // lane (gid, tig) holds head gid's fragments
    const uint8_t *qrow = sm + Cf::OFF_Q + qs * Cf::Q_STAGE + gid * Cf::Q_ROW + tig * 8;
    const float *qscale = reinterpret_cast<const float *>(sm + Cf::OFF_QS) + qs * kMaxG;
    const float sc0 = h0 < p.G ? qscale[h0] : 0.f, sc1 = h1 < p.G ? qscale[h1] : 0.f;
    uint2 qb[QK];
    if constexpr (Q_REGS) {
#pragma unroll
      for (int c = 0; c < KS; ++c)
        qb[c] = hv ? *reinterpret_cast<const uint2 *>(qrow + 32 * c) : make_uint2(0u, 0u);
      release(emptyQ + 8 * qs);
    }
    ++it_q;

    float o[KS][4];
#pragma unroll
    for (int u = 0; u < KS; ++u) o[u][0] = o[u][1] = o[u][2] = o[u][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;   // this lane's keys
    float M0 = -INFINITY, M1 = -INFINITY;                       // the warp's keys

    for (int t0 = w.ta; t0 < w.tb; t0 += batch, ++it_s) {   // tiles whose scales come together
      const int t1 = min(t0 + batch, w.tb);
      const int ss = it_s & 1;
      const float *scale_words =
          reinterpret_cast<const float *>(sm + Cf::OFF_SCALE) + ss * 2 * kScaleWords;
      bool have_scales = false;
      auto wait_scales = [&]() {
        if (have_scales) return;
        have_scales = true;
        if (!mbar_wait(fullS + 8 * ss, (it_s >> 1) & 1, abort_flag)) give_up();
        __syncwarp();
      };
      const int t_team = Cf::TEAMS == 2 ? t0 + (((tile + t0 - w.ta) ^ team) & 1) : t0;
      for (int t = t_team; t < t1; t += Cf::TEAMS) {
        const int ent = 2 * (tile + t - w.ta);   // ring entries: K, then V
        int st = ent % Cf::NS;
        if (!mbar_wait(full + 8 * st, (ent / Cf::NS) & 1, abort_flag)) give_up();
        __syncwarp();
        const uint32_t tw = tile_word[st];
        const int off = static_cast<int8_t>((tw >> 8) & 0xffu);
        const int tlo = max(w.k0 - t * kT, 0) - off, thi = min(w.k1 - t * kT, kT) - off;
        // tile row r holds a key of the unit?
        auto valid = [&](int r) -> bool {
          return r >= tlo && r < thi && ((tw >> (r >> log2_box)) & 1u);
        };
        const bool whole = tlo == 0 && thi == kT && (tw & 0xffu) == (1u << boxes) - 1u;
        uint32_t base = s0 + st * Cf::TILE_BYTES;

        // ---- S^T [16 MB keys x 8 heads]: lane's keys key0 + gid + 8 i, heads h0, h1.
        // Two chains of MMAs: the two key blocks, or even and odd 16-byte units of one.
        float sa[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) sa[i][0] = sa[i][1] = sa[i][2] = sa[i][3] = 0.f;
#pragma unroll
        for (int c = 0; c < KS; c += 2) {
          uint2 q0, q1;
          if constexpr (Q_REGS) {
            q0 = qb[c];
            q1 = qb[c + 1];
          } else {
            q0 = hv ? *reinterpret_cast<const uint2 *>(qrow + 32 * c) : make_uint2(0u, 0u);
            q1 = hv ? *reinterpret_cast<const uint2 *>(qrow + 32 * c + 32) : make_uint2(0u, 0u);
          }
#pragma unroll
          for (int i = 0; i < MB; ++i) {
            uint32_t r[4], a0, a1, a2, a3;
            ldsm_x4(unit_addr<D>(base, ldsm_base, c + ldsm_unit) + i * ROWS16, r);
            codes_to_f16(r[0], a0, a2);
            codes_to_f16(r[1], a1, a3);
            mma_f16(sa[i], a0, a1, a2, a3, q0.x, q0.y);
            codes_to_f16(r[2], a0, a2);
            codes_to_f16(r[3], a1, a3);
            mma_f16(sa[MB == 2 ? i : 1], a0, a1, a2, a3, q1.x, q1.y);
          }
        }
        if constexpr (MB == 1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) sa[0][i] += sa[1][i];
        }
        release(empty + 8 * st);   // the K entry
        wait_scales();
        // ---- online softmax ----
        const float *kw = scale_words + (t - t0) * scales, *vw = kw + kScaleWords;
        float sx[2 * MB][2], lv[2 * MB];
#pragma unroll
        for (int i = 0; i < 2 * MB; ++i) {
          const int r = key0 + gid + 8 * i;
          const int w0 = ((r + off) & (kT - 1)) >> log2_sc;
          const float k = kw[w0];
          lv[i] = __log2f(vw[w0]);
          sx[i][0] = sa[i >> 1][(i & 1) * 2] * (k * sc0);
          sx[i][1] = sa[i >> 1][(i & 1) * 2 + 1] * (k * sc1);
          if (!whole && !valid(r)) {
            sx[i][0] = sx[i][1] = -INFINITY;
            lv[i] = 0.f;
          }
        }
        float n0 = m0, n1 = m1, x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < 2 * MB; ++i) {
          n0 = fmaxf(n0, sx[i][0]);
          n1 = fmaxf(n1, sx[i][1]);
          x0 = fmaxf(x0, __fadd_ru(sx[i][0], lv[i]));
          x1 = fmaxf(x1, __fadd_ru(sx[i][1], lv[i]));
        }
        const float u0 = n0 == -INFINITY ? 0.f : n0, u1 = n1 == -INFINITY ? 0.f : n1;
        l0 *= ex2(m0 - u0);
        l1 *= ex2(m1 - u1);
        m0 = n0;
        m1 = n1;
#pragma unroll
        for (int i = 0; i < 2 * MB; ++i) {
          l0 += ex2(sx[i][0] - u0);
          l1 += ex2(sx[i][1] - u1);
        }
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) {
          x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, i));
          x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, i));
        }
        if (__any_sync(0xffffffffu, x0 > M0 || x1 > M1)) {
          const float N0 = fmaxf(M0, x0), N1 = fmaxf(M1, x1);
          const float a0 = M0 == -INFINITY ? 0.f : ex2(M0 - N0);
          const float a1 = M1 == -INFINITY ? 0.f : ex2(M1 - N1);
          M0 = N0;
          M1 = N1;
#pragma unroll
          for (int u = 0; u < KS; ++u) {
            o[u][0] *= a0;
            o[u][1] *= a1;
            o[u][2] *= a0;
            o[u][3] *= a1;
          }
        }
        const float U0 = M0 == -INFINITY ? 0.f : M0, U1 = M1 == -INFINITY ? 0.f : M1;
        uint32_t pb[2 * MB];
#pragma unroll
        for (int i = 0; i < 2 * MB; ++i) {   // at most 2^15: (s - M) <= -lv
          const float lift = lv[i] + kLift;
          pb[i] = transpose8x8(pack_f16(ex2(sx[i][0] - U0 + lift), ex2(sx[i][1] - U1 + lift)));
        }
        // ---- O^T [D x 8 heads] += V^T P^T ----
        st = (ent + 1) % Cf::NS;
        if (!mbar_wait(full + 8 * st, ((ent + 1) / Cf::NS) & 1, abort_flag)) give_up();
        __syncwarp();
        base = s0 + st * Cf::TILE_BYTES;
        if (!whole) {   // codes of this warp's keys outside the unit count 0, whatever they are
#pragma unroll 1
          for (int i = lane; i < 16 * MB * KS; i += 32) {
            const int r = key0 + i / KS;
            if (!valid(r))
              *reinterpret_cast<uint4 *>(sm + unit_addr<D>(st * Cf::TILE_BYTES, row_base<D>(r),
                                                           i % KS)) = make_uint4(0u, 0u, 0u, 0u);
          }
          __syncwarp();   // (the entry's release fences these stores too)
        }
#pragma unroll
        for (int u = 0; u < KS; u += 2) {
#pragma unroll
          for (int i = 0; i < MB; ++i) {
            uint32_t r[4], a0, a1, a2, a3;
            ldsm_x4_t(unit_addr<D>(base, ldsm_base, u + ldsm_unit) + i * ROWS16, r);
            // a word holds two columns of two keys; pair the keys of each column
            codes_to_f16(__byte_perm(r[0], 0, 0x3120), a0, a1);
            codes_to_f16(__byte_perm(r[1], 0, 0x3120), a2, a3);
            mma_f16(o[u], a0, a1, a2, a3, pb[2 * i], pb[2 * i + 1]);
            codes_to_f16(__byte_perm(r[2], 0, 0x3120), a0, a1);
            codes_to_f16(__byte_perm(r[3], 0, 0x3120), a2, a3);
            mma_f16(o[u + 1], a0, a1, a2, a3, pb[2 * i], pb[2 * i + 1]);
          }
        }
        release(empty + 8 * st);
      }
      wait_scales();   // a warp without a tile here keeps step too
      __syncwarp();
      if (lane == 0) mbar_arrive(emptyS + 8 * ss);
    }
    tile += w.tb - w.ta;
    if constexpr (!Q_REGS) {
      release(emptyQ + 8 * qs);
    }

    // ---- the unit's end ----
    auto hand_over = [&](float *to, int c0) {   // kMergeCols columns of the warp's state
#pragma unroll
      for (int u = 0; u < (D < kMergeCols ? D : kMergeCols) / 16; ++u) {
        const float(&f)[4] = o[c0 / 16 + u];
        float *d = to + (warp * kMaxG + h0) * kMergeRow + 16 * u + 2 * gid;
        // (the joining warp's weights of the states take the factor back at D <= 256)
        constexpr float F = Cf::SELF ? kUnlift : 1.f;
        *reinterpret_cast<float2 *>(d) = make_float2(f[0] * F, f[2] * F);
        *reinterpret_cast<float2 *>(d + kMergeRow) = make_float2(f[1] * F, f[3] * F);
      }
    };
    auto write_stats = [&](float *to) {   // the warp's m, l and M: [3][4][8]
      float n0 = m0, n1 = m1;
#pragma unroll
      for (int i = 4; i < 32; i <<= 1) {
        n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, i));
        n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, i));
      }
      l0 = sum_at(l0, m0, n0);
      l1 = sum_at(l1, m1, n1);
#pragma unroll
      for (int i = 4; i < 32; i <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, i);
        l1 += __shfl_xor_sync(0xffffffffu, l1, i);
      }
      if (gid == 0) {
        to += warp * kMaxG + h0;
        *reinterpret_cast<float2 *>(to) = make_float2(n0, n1);
        *reinterpret_cast<float2 *>(to + 32) = make_float2(l0, l1);
        *reinterpret_cast<float2 *>(to + 64) = make_float2(M0, M1);
      }
    };
    if (joined_by_all(w)) {   // the ring is free once all are here
      (void)consumer_sync_or(false);
      float *dump = reinterpret_cast<float *>(sm);
#pragma unroll
      for (int u = 0; u < KS; ++u) {
        float *d = dump + (warp * kMaxG + h0) * Cf::DUMP_ROW + 16 * u + 2 * gid;
        *reinterpret_cast<float2 *>(d) = make_float2(o[u][0] * kUnlift, o[u][2] * kUnlift);
        *reinterpret_cast<float2 *>(d + Cf::DUMP_ROW) =
            make_float2(o[u][1] * kUnlift, o[u][3] * kUnlift);
      }
      write_stats(dump + Cf::DUMP_STATS);
      (void)consumer_sync_or(false);
      // As many places as 8 heads have (D = 512 at once instead of half of them: 17.7 ->
      // 16.0 us for 10 rows of 1000 tokens), and as many parts as registers allow. Up to
      // 4 heads have half the places: at D = 128 one place of 8 parts instead of two of 4
      // (B = 8 9.2 -> 8.5 us, one row of 32k tokens 19.6 -> 19.0); at D = 512 no gain.
      constexpr int IB = D / 64, SRC = D <= 128 ? 8 / IB : D == 256 ? 4 : 2;
      bool done = false;
      if constexpr (D == 128) {
        done = p.G <= kMaxG / 2;
        if (done) join_parts<D, 1, 8>(p, sm, w, abort_flag, warp, lane);
      }
      if (!done) join_parts<D, IB, SRC>(p, sm, w, abort_flag, warp, lane);
      continue;
    }
    constexpr int COLS = D < kMergeCols ? D : kMergeCols;
    float *merge = reinterpret_cast<float *>(sm + Cf::OFF_MERGE);
    if constexpr (Cf::SELF) {
      // round by round, a thread four columns of heads warp and warp + 4
      float f[2][kCWarps];
      const bool partial = w.part > 0;
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += COLS) {
        hand_over(merge, c0);
        if (c0 == 0) write_stats(merge + kCWarps * kMaxG * kMergeRow);
        const bool bad = consumer_sync_or(*abort_flag);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int h = warp + 4 * i;
          if (h >= p.G) break;
          if (c0 == 0) {
            const float *a = merge + kCWarps * kMaxG * kMergeRow + h;
            float m = a[0], l = 0.f, M = a[64];
#pragma unroll
            for (int j = 1; j < kCWarps; ++j) {
              m = fmaxf(m, a[8 * j]);
              M = fmaxf(M, a[64 + 8 * j]);
            }
#pragma unroll
            for (int j = 0; j < kCWarps; ++j) l += sum_at(a[32 + 8 * j], a[8 * j], m);
            const float last = last_factor(partial, m, l, M);
#pragma unroll
            for (int j = 0; j < kCWarps; ++j)
              f[i][j] = a[64 + 8 * j] == -INFINITY ? 0.f : last * ex2(a[64 + 8 * j] - M);
            if (partial && !bad && lane == 0) {
              uint32_t *st = p.st_part + (own_record(w) * p.G + h) * 3;
              st_word(st, part_word(m));
              st_word(st + 1, part_word(l));
              st_word(st + 2, part_word(M));
            }
          }
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int j = 0; j < kCWarps; ++j)
            fma4(acc, f[i][j],
                 *reinterpret_cast<const float4 *>(merge + (j * kMaxG + h) * kMergeRow + 4 * lane));
          const int at = c0 + 4 * lane;
          if (bad) continue;
          if (partial)
            st_words(p.o_part + (own_record(w) * p.G + h) * D + at,
                     make_uint4(part_word(acc.x), part_word(acc.y), part_word(acc.z),
                                part_word(acc.w)));
          else
            *reinterpret_cast<uint2 *>(
                p.out + (static_cast<size_t>(w.b) * p.Hq + w.g * p.G + h) * D + at) =
                pack4_bf16(acc, 1.f);
        }
        (void)consumer_sync_or(false);   // before the buffer is written again
      }
    } else {
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += COLS, ++it_m) {
        if (!mbar_wait(emptyM, (it_m & 1) ^ 1, abort_flag)) give_up();
        hand_over(merge, c0);
        if (c0 == 0) {
          float *st = merge + kCWarps * kMaxG * kMergeRow + h0;
          if (gid == 0) *reinterpret_cast<float2 *>(st + warp * kMaxG) = make_float2(M0, M1);
          st += 32 + (warp * 8 + gid) * kMaxG;
          *reinterpret_cast<float2 *>(st) = make_float2(m0, m1);
          *reinterpret_cast<float2 *>(st + 256) = make_float2(l0, l1);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(fullM);
      }
    }
  }
}

// ------------------------------------------------------------- host ----
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static std::once_flag once;
  static EncodeTiledFn fn = nullptr;
  std::call_once(once, [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                         cudaEnableDefault, &qr) == cudaSuccess &&
        qr == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// Map over a cache of `pages` pages (all heads') of page_size rows of D bytes:
// {column, row in page, page}, boxes of box_rows rows; rows outside the page read 0.
// D = 64: two rows of the cache make one of the map.
int make_cache_map(CUtensorMap *tm, const void *base, long long pages, int page_size, int D,
                   int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return pkv::fail(PKV_E_CUDA, "cuTensorMapEncodeTiled unavailable");
  const int width = D < 128 ? 128 : D, rows = page_size * D / width;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(pages)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(D) * page_size};
  cuuint32_t box[3] = {128u, static_cast<cuuint32_t>(box_rows * D / width), 1u};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return pkv::fail(PKV_E_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return PKV_OK;
}

template <int D>
int launch_q8(const CUtensorMap &tmK, const CUtensorMap &tmV, const Problem &p,
              cudaStream_t stream) {
  static std::mutex mu;
  static bool done[64] = {false};
  int dev = 0;
  PKV_CUDA_CHECK(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return pkv::fail(PKV_E_CUDA, "device id out of range");
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      PKV_CUDA_CHECK(cudaFuncSetAttribute(
          decode_q8_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM));
      done[dev] = true;
    }
  }
  const int sms = pkv::sm_count();
  if (sms <= 0) return pkv::fail(PKV_E_CUDA, "paged_decode_attn_q8: no SM count");
  const int most = sms * Cfg<D>::CTAS_PER_SM;
  PKV_CUDA_CHECK(pkv::launch_pdl(decode_q8_kernel<D>, dim3(most < kMaxCtas ? most : kMaxCtas),
                                 dim3(kThreads), Cfg<D>::SMEM, stream, tmK, tmV, p));
  return pkv::ok();
}

bool good_heads(int Hq, int Hkv, int D) {
  return (D == 64 || D == 128 || D == 256 || D == 512) && Hkv >= 1 && Hkv <= 65535 && Hq >= Hkv &&
         Hq % Hkv == 0 && Hq / Hkv <= kMaxG;
}

}  // namespace

extern "C" {

// Workspace: [kMaxCtas] records of G * D words (partial outputs), [kMaxCtas] records of
// G * 3 words (running maxima and sum).
size_t paged_decode_attn_q8_workspace(int Hq, int Hkv, int D) {
  if (!good_heads(Hq, Hkv, D)) return 0;
  const size_t G = Hq / Hkv;
  return kMaxCtas * G * (D + 3) * sizeof(float);
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
    return pkv::fail(PKV_E_BAD_ARG, "%s: need Hkv <= 65535, Hq %% Hkv == 0 and Hq/Hkv <= %d", fn,
                     kMaxG);
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
  {
    const long long row_tiles =
        (1LL * max_pages_per_seq * page_size + kT - 1) / kT + 1 + Cfg<64>::START;
    if (1LL * B * Hkv * row_tiles >= (1LL << 31))
      return pkv::fail(PKV_E_BAD_ARG, "%s: B * Hkv * tiles per row too large", fn);
  }
  const size_t need = paged_decode_attn_q8_workspace(Hq, Hkv, D);
  if (!workspace || workspace_bytes < need)
    return pkv::fail(PKV_E_BAD_ARG, "%s: workspace needs %zu bytes", fn, need);
  if (!pkv::aligned16(workspace))
    return pkv::fail(PKV_E_BAD_ARG, "%s: workspace must be 16-byte aligned", fn);
  const long long pages = 1LL * Hkv * n_pages;
  const int box_rows = page_size < kT ? page_size : kT;
  CUtensorMap tmK, tmV;
  int st = make_cache_map(&tmK, k_cache, pages, page_size, D, box_rows);
  if (st != PKV_OK) return st;
  st = make_cache_map(&tmV, v_cache, pages, page_size, D, box_rows);
  if (st != PKV_OK) return st;
  auto log2i = [](int x) {
    int l = 0;
    while ((1 << l) < x) ++l;
    return l;
  };
  Problem p;
  p.q = reinterpret_cast<const __nv_bfloat16 *>(q);
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
  // four scales at once where the rows of one copy have as many, 16-byte aligned (217 short
  // rows with a scale a token 17.1 us, word by word 18.9)
  p.scale_vec = box_rows / scale_block >= 4 && pkv::aligned16(k_scale) && pkv::aligned16(v_scale)
                    ? 4 : 1;
  p.o_part = static_cast<uint32_t *>(workspace);
  p.st_part = p.o_part + static_cast<size_t>(kMaxCtas) * p.G * D;
  p.out = reinterpret_cast<__nv_bfloat16 *>(out);
  p.err = err_word;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (D) {
    case 64: return launch_q8<64>(tmK, tmV, p, s);
    case 128: return launch_q8<128>(tmK, tmV, p, s);
    case 256: return launch_q8<256>(tmK, tmV, p, s);
    default: return launch_q8<512>(tmK, tmV, p, s);
  }
}

}  // extern "C"
