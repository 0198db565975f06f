// paged_tree_attn: attention of every row's tree of drafted tokens over the paged cache.
//
//   out[t][h] = sum_j softmax_j(scale q[t][h] . k_j) v_j
// over the keys j < ctx of the context and, among the row's own nodes (at cache positions ctx ..),
// those on t's path to its root, t included; with a window W only keys less than W positions
// behind t (a node's position is ctx + its depth).
//
// Bound by reading each key and value of a row's context once for all its nodes and the query
// heads of a kv head, until nodes x heads reach a few hundred. Those "columns" are the N of both
// products, at most 64 of them a unit of work, or 128 where the rows have more than 64 (and D <=
// 128), so that a small tree costs no more arithmetic than it has columns:
//   S^T = K q^T    M = 128 keys of a tile, N columns, both operands K-major,
//   O^T = V^T P^T  M = 128 columns of D, N columns, K = the tile's 128 keys, both MN-major: V as
//                  it lies in the cache, P as the threads write it, a key's columns in a row.
// An MMA with M = 128 takes 43 cycles for 32 columns, 51 for 64, 67 for 128, in either order of
// the operands: their way from shared memory at 128 bytes a cycle. With the queries as M, 32 rows
// would pay for 128.
// In S^T a thread owns a key. Its columns' maxima run across threads, so they are not taken tile
// by tile: a column keeps a reference, every thread checks that none of its scores passes it by
// more than 2^8, and only where one does (a unit's first tile, and few others) the maxima are
// reduced, the references moved and O scaled. The weights' sums are a third product, with ones in
// V's place: every lane of TMEM has them, and no thread keeps a sum for each column. Weights are
// rounded to bf16, V's type, for both operands of a product have one (an error of 0.0022 of the
// outputs' size, not the 0.0017 of rounding those alone), and summed as rounded; scores, references
// and O are fp32.
//
// Work: the units' tiles and one or two more places for each unit's start lie on one line, cut into
// equal shares for one persistent CTA an SM from the lengths, on the device. A unit that is cut
// leaves its parts (O, reference and sum, fp32) in the workspace, and whoever writes the last of
// them, or a second kernel, joins them in their order: results do not depend on timing and no CTA
// waits for another. (Shares that begin at a unit's edge where that is near, to cut fewer: 56 -> 71
// us for 64 nodes at D = 512, 39 -> 42 for the rollout batch.) The line is planned from row_start,
// ctx_lens and batch_idx before the prior kernel has ended, and the first tiles, which the table
// names, are then on their way to L2 (the rollout batch 37.3 -> 36.2 us, one row of 41 tokens 4.6
// -> 4.4).
//   warps 0-7 (softmax): D <= 128 with 64 columns, two units at a time, four warps each, so that
//     one unit's start and end overlap the other's tiles; else one unit, its columns in two
//     halves. Warp w has the keys of TMEM lanes 32 (w % 4) ..: masks, weights, references, a
//     unit's output or part;
//   warps 8, 9: K and V tiles by TMA, each into a ring of its own;
//   warp 10: a unit's queries by TMA, and which columns see a key: sets of 64 bits, from the
//     parents by pointer doubling;
//   warps 11, 12: the MMAs of S and of P V. With one warp for both, and one ring, each waited
//     while the other could have been issued; and an entry of 32 KB a barrier, not 16, halves the
//     waits (16 rows with trees of 64: one head of 512 55 -> 52 us).
// Rows of V that no node sees are cleared in shared memory (0 x NaN would reach every column);
// one that is not finite and seen by some nodes only is cleared too and those nodes' results
// are NaN: nothing of it reaches the others. So that this is between a tile's arrival and its
// product, the warp of P V says when a masked tile's V is there and waits until it is clean.
//
// What costs most next to memory is code: a first form with its loops unrolled had 120 KB, a third
// of its warps' time went into waiting for instructions, and the rollout batch took 70 us. Hence
// the loops kept as loops, the short waits, and one site of each product.
//
// Measured (6769 GB/s measured): 16 rows of 16k to 32k tokens, 8-node chains, 8 heads of 128,
// 241 us, 0.99 of reading them; 64 rows of 100 to 1024 tokens, trees of 8, 36 us, 0.64: its start
// (launch, plan, the rings' first fill) and its end (last tiles, join) are 6 us each; 64 rows of
// 256 to 2048 tokens in a window of 512, trees of 16, one head of 256, 26 us, 0.22, and 16 rows
// with trees of 64, one head of 512, 48 us, 0.16: they write and read as many bytes in parts as
// in keys, at D = 512 every 8 nodes read the keys again, and a tile's weights, P V and the next
// one's weights stand behind one another (at 512 there is no room for a second P); one row of 41
// tokens 4.4 us.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <mutex>

#include "pkv_internal.h"
#include "tcgen05.cuh"
#include "tree.cuh"

namespace {

constexpr int kTile = 128;               // keys of a tile
constexpr int kMaxCtas = 160;            // CTAs the workspace has room for
constexpr float kLazyLog2 = 8.f;
constexpr int kMostPlaces = 0x7fffffff;  // as many and more are reported, not computed
constexpr float kUnset = 1e30f;          // stands for -reference of a column without one
constexpr int kFan = 4;                  // parts that are joined at a time
constexpr int kLevels = 4;               // of joins: 4^4 parts
static_assert(kMaxCtas <= 256, "levels");
constexpr size_t kArrivedBytes = sizeof(int) * kLevels * 2 * kMaxCtas;   // their counters
constexpr int kJoinWarps = 8;            // of a joining CTA

template <int D, int MOST>
struct Cfg {
  static constexpr int COLS = MOST;                     // columns of a unit, at most
  // Units at work at a time, each with softmax warps, MMA warp, queries, P and TMEM of its own;
  // where there is room for one only, its softmax warps come in two groups of half the columns.
  static constexpr int UNITS = D <= 128 && COLS == 64 ? 2 : 1;
  static constexpr int GROUPS = 2 / UNITS;              // groups of four softmax warps a unit
  static constexpr int HALF = COLS / GROUPS;            // columns of a softmax warp, at most
  // Parts are joined by whoever is the last to write one; where units have two groups, by a second
  // kernel. By the last to write, a row of 41 tokens went from 8.4 to 4.8 us and the rollout batch
  // from 38.7 to 37.4; but the window of 512 at D = 256 from 30 to 38 and trees of 64 at D = 512
  // from 56 to 61, where one CTA's few warps read up to 128 KB a part.
  static constexpr bool JOINS = UNITS == 2;
  // Places on the line for a unit's start and end: where units go in twos one's overlap the other's
  // tiles (2 and 3: 40 and 42 us for the rollout batch, not 39, at the time), else they take as
  // long as two tiles (16 rows with trees of 64, one head of 512 51 -> 48 us; 64 rows of up to 1k
  // tokens with trees of 24, eight heads of 128 64 -> 56).
  static constexpr int START = UNITS == 2 ? 1 : 2;
  static constexpr int SOFT = 8;                        // softmax warps of all units
  static constexpr int PROD = SOFT, PREP = SOFT + 2, MMA = SOFT + 3;
  static constexpr int THREADS = (SOFT + 5) * 32;
  // A ring entry: 128 columns of D of a K tile in two atoms of 64, or of a V tile, in halves of 64
  // keys with two atoms each. (D = 64: an atom, all its keys.)
  static constexpr int ATOM = kTile * 128, ATOMS = D == 64 ? 1 : 2;   // bytes of 64 columns
  static constexpr int ENTRY = ATOMS * ATOM;
  static constexpr int E = D == 64 ? 1 : D / 128;       // entries of a K tile, and of a V tile
  static constexpr int KEYS = kTile / ATOMS;            // of a half of V, one after the other
  // as many as shared memory holds, in a ring for K and one for V
  static constexpr int NS = D == 64 ? (COLS == 128 ? 9 : 10) : 4;
  static constexpr int NK = NS / 2, NV = NS - NK;
  static constexpr int Q_ATOM = COLS * 128;
  static constexpr int Q_BYTES = D / 64 * Q_ATOM;
  static constexpr int P_ATOM = kTile * 128;            // 64 columns of every key
  static constexpr int P_BYTES = COLS / 64 * P_ATOM;
  static constexpr int OFF_Q = NS * ENTRY;              // [UNITS]
  static constexpr int OFF_P = OFF_Q + UNITS * Q_BYTES; // [UNITS]
  static constexpr int OFF_ONES = OFF_P + UNITS * P_BYTES;  // one swizzle atom of ones
  static constexpr int OFF_SMALL = OFF_ONES + 1024;
  // of a unit: S of two tiles, O^T's blocks, the sums of the weights (in every lane)
  static constexpr int SB = 2;
  static constexpr int S_COL = 0, O_COL = SB * COLS, L_COL = O_COL + E * COLS;
  static constexpr int UNIT_COLS = 512 / UNITS;
  static_assert(L_COL + COLS <= UNIT_COLS, "TMEM");
  static constexpr size_t RECORD = static_cast<size_t>(COLS) * (D + 2);   // floats of a part
};

// Which of a unit's columns see a key, a bit each, for each group of softmax warps its own.
template <int GROUPS>
struct Prep {
  uint64_t below[GROUPS][kTreeMax];    // those of the nodes that have node i on their path
  uint64_t shallow[GROUPS][kTreeMax];  // those of the nodes of depth <= i
  int depth[kTreeMax];
  unsigned poison[GROUPS][2];          // those that see some value that is not finite
};

// A unit cut into parts, for the joining kernel.
struct Cut {
  int token0, cols, head, parts;
};

struct Rows {
  int pre[kTreeRows + 1];           // first place of every row on the line
  int n0[kTreeRows], ctx[kTreeRows], slot[kTreeRows];
  uint8_t n[kTreeRows];             // (the top bit: padding, only zeros to write)
};

template <typename C>
struct Small {
  static constexpr int COLS = C::UNITS * C::COLS;
  Prep<C::GROUPS> prep[2];
  // of the columns, group g's from g * HALF on (the groups may be at different units)
  alignas(16) float mneg[COLS];     // a column's reference's negative, kUnset: none yet; -inf: an
                                    // unused column, of whatever scores: none is out of its reach
  float ref[COLS];                  // its reference, -inf: none yet
  float alpha[COLS];                // what a new one scales O and sums by; NaN: poisoned
  long long dst[COLS];              // its place in out, -1: none
  alignas(16) float red[kFan][COLS];   // maxima of the four warps of a group; parts' weights
  int last[2];                      // whether a unit's part was the last of some to arrive
  int scan[16];
  uint64_t bars[48];
  uint32_t tmem;
  Rows rows;
};

template <typename C>
constexpr size_t smem_bytes() {
  static_assert(1024 + C::OFF_SMALL + sizeof(Small<C>) <= 232448, "shared memory");
  return 1024 + C::OFF_SMALL + sizeof(Small<C>);
}

struct Args {
  const int32_t *table, *batch_idx, *ctx_lens, *row_start, *parents;
  const __nv_bfloat16 *k, *v;   // (what the maps name, for prefetches)
  __nv_bfloat16 *out;
  float *parts;
  int *arrived;   // [kLevels][2 kMaxCtas]
  Cut *cuts;      // [kMaxCtas]
  int32_t *err;
  int n_slots, max_pages, page_size, log_page, n_pages, window, B, N, Hq, Hkv, G;
  int unit_tokens, box_nodes;   // nodes of a unit at most, and of a box of queries
  float scale_log2;
};

// instruction descriptor, kind::f16: f32 accumulator, bf16 A and B, both K-major or both MN-major
__device__ __forceinline__ uint32_t idesc(int N, bool mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (mn ? (1u << 15) | (1u << 16) : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(kTcM >> 4) << 24);
}
// (d0, d1) = (a0, a1) * b + (c0, c1)
__device__ __forceinline__ void fma2(float &d0, float &d1, float a0, float a1, float b, float c0,
                                     float c1) {
  asm("{\n.reg .b64 ra, rb, rc, rd;\nmov.b64 ra, {%2, %3};\nmov.b64 rb, {%4, %4};\n"
      "mov.b64 rc, {%5, %6};\nfma.rn.f32x2 rd, ra, rb, rc;\nmov.b64 {%0, %1}, rd;\n}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}
// Waits for completion number k of a barrier's phases, a lane or a whole warp with one answer;
// false if it gave up, after about two seconds. (A loop of few instructions: the waits are many,
// and a kernel that does not fit the instruction caches waits for its code instead.)
__device__ __forceinline__ bool lane_wait(uint32_t bar, int k) {
  uint32_t done;
  asm volatile(
      "{\n.reg .pred p, q;\n.reg .u32 n;\nmov.u32 n, 0;\n"
      "WAIT:\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1024;\n"
      "@p bra DONE;\nadd.u32 n, n, 1;\nsetp.lt.u32 q, n, %3;\n@q bra WAIT;\n"
      "DONE:\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(bar), "r"(static_cast<uint32_t>(k) & 1u), "n"(1 << 21)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ bool wait_for(uint32_t bar, int k) {
  return __all_sync(0xffffffffu, lane_wait(bar, k));
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(r));
  return r != 0;
}
// reads of TMEM are a whole warp's, which may have come here by the ways of its lanes
__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t (&r)[16]) {
  __syncwarp();
  t_ld16(taddr, r);
}
// barrier of the 128 threads of a group, and whether any of them says yes
__device__ __forceinline__ bool group_any(int grp, bool mine) {
  uint32_t r;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.b32 q, %1, 0;\n"
      "barrier.cta.red.or.pred p, %2, 128, q;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(mine)), "r"(1 + grp)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int grp) {
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + grp) : "memory");
}
// the maximum over the 32 lanes (NaN only where all are); volatile, for it names all lanes and must
// not be moved under the branch of the one that uses it
__device__ __forceinline__ float lane_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// N of a unit's products: a multiple of 16 columns for each group of softmax warps
template <int GROUPS>
__device__ __forceinline__ int columns(int cols) {
  return (cols + 16 * GROUPS - 1) / (16 * GROUPS) * (16 * GROUPS);
}

// sums of places stop at kMostPlaces
__device__ __forceinline__ int add_places(int a, int b) {
  return static_cast<int>(min(static_cast<unsigned>(a) + static_cast<unsigned>(b),
                              static_cast<unsigned>(kMostPlaces)));
}

// A unit, or the part of it that this CTA has: tiles [t0, t1) of ntiles.
struct Part {
  int b, head, tok0, toks, n0, n, ctx, lo, tile0, ntiles, t0, t1;
  int start;   // the unit's first place on the line
  __device__ bool whole() const { return t0 == 0 && t1 == ntiles; }
};

// Goes through a CTA's share of the line, part by part.
template <int START>
struct Line {
  const Rows *sm;
  const Args *a;
  int pos, end, off;   // off: where in its unit pos is
  Part p;              // the unit at pos (all but t0 and t1)
  __device__ void row(int b) {
    p.b = b;
    p.n0 = sm->n0[b];
    p.n = sm->n[b] & 127;
    p.ctx = sm->ctx[b];
    p.lo = a->window > 0 ? max(0, p.ctx - a->window + 1) : 0;
    p.tile0 = p.lo / kTile;
    p.ntiles = sm->n[b] & 128 ? 0 : (p.ctx + p.n - 1) / kTile - p.tile0 + 1;
  }
  __device__ void begin(const Rows &s, const Args &args, int x0, int x1) {
    sm = &s;
    a = &args;
    pos = x0;
    end = x1;
    off = 0;
    if (x0 >= x1) return;
    int l = 0, r = args.B;   // the last row that starts at or before x0
#pragma unroll 1
    while (r - l > 1) {
      const int m = (l + r) / 2;
      if (s.pre[m] <= x0) l = m;
      else r = m;
    }
    row(l);
    const int cost = p.ntiles + START, units = (p.n + args.unit_tokens - 1) / args.unit_tokens;
    const int u = (x0 - s.pre[l]) / cost;
    off = x0 - s.pre[l] - u * cost;
    p.head = u / units;
    p.tok0 = (u - p.head * units) * args.unit_tokens;
  }
  // the next part, in p
  __device__ bool next() {
    if (pos >= end) return false;
    if (off == p.ntiles + START) {   // behind a unit: the next nodes, head or row with nodes
      off = 0;
      p.tok0 += a->unit_tokens;
      if (p.tok0 >= p.n) {
        p.tok0 = 0;
        if (++p.head == a->Hkv) {
          p.head = 0;
          int b = p.b + 1;
#pragma unroll 1
          while (sm->pre[b + 1] == pos) ++b;
          row(b);
        }
      }
    }
    p.toks = min(a->unit_tokens, p.n - p.tok0);
    const int to = min(p.ntiles + START, off + (end - pos));
    p.t0 = max(0, off - START);
    p.t1 = max(0, to - START);
    p.start = pos - off;
    pos += to - off;
    off = to;
    return true;
  }
};

// The line's W places in equal shares for n CTAs, the first ones one longer where need be: the
// first place of CTA c's, and the CTA that has a place.
__device__ __forceinline__ int share(int W, int c, int n) { return W / n * c + min(c, W % n); }
__device__ __forceinline__ int share_of(int W, int at, int n) {
  const int q = W / n, r = W % n, head = r * (q + 1);
  return at < head ? at / (q + 1) : r + (at - head) / q;
}

template <int D, int MOST>
__global__ void __launch_bounds__(Cfg<D, MOST>::THREADS, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Args a) {
  using C = Cfg<D, MOST>;
  extern __shared__ uint8_t raw[];
  uint8_t *sm = raw + ((1024u - (t_smem(raw) & 1023u)) & 1023u);
  Small<C> &s = *reinterpret_cast<Small<C> *>(sm + C::OFF_SMALL);
  Rows &rows = s.rows;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;
  const uint32_t sRing = t_smem(sm), sQ = t_smem(sm + C::OFF_Q), sP = t_smem(sm + C::OFF_P),
                 sOnes = t_smem(sm + C::OFF_ONES);
  const uint32_t bars = t_smem(s.bars);
  constexpr int U = C::UNITS;
  // the rings', then unit x's (S buffer b, preparation b)
  const uint32_t full = bars, empty = full + 8 * C::NS, drain = empty + 8 * C::NS,
                 prepfull = drain + 16, prepempty = prepfull + 16, unit0 = prepempty + 16;
  constexpr int UB = 9 + 2 * C::E;
  auto sfull = [&](int x, int b) { return unit0 + 8 * (UB * x + b); };
  auto sfree = [&](int x, int b) { return unit0 + 8 * (UB * x + 2 + b); };
  auto pfull = [&](int x) { return unit0 + 8 * (UB * x + 4); };
  auto pvdone = [&](int x) { return unit0 + 8 * (UB * x + 5); };
  auto ofree = [&](int x) { return unit0 + 8 * (UB * x + 6); };
  auto qfull = [&](int x) { return unit0 + 8 * (UB * x + 7); };
  auto qempty = [&](int x) { return unit0 + 8 * (UB * x + 8); };
  // of a masked tile, block by block of 128 columns of V: it is there, it is clean
  auto vthere = [&](int x, int blk) { return unit0 + 8 * (UB * x + 9 + blk); };
  auto vclean = [&](int x, int blk) { return unit0 + 8 * (UB * x + 9 + C::E + blk); };
  static_assert(2 * C::NS + 6 + U * UB <= 48, "barriers");

  if (tid == 32) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmQ)));
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmK)));
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmV)));
  }
  if (tid == 0) {
#pragma unroll 1
    for (int i = 0; i < C::NS; ++i) {
      t_bar_init(full + 8 * i, 1);
      t_bar_init(empty + 8 * i, 1);
    }
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      t_bar_init(drain + 8 * i, 1);
      t_bar_init(prepfull + 8 * i, 1);
      t_bar_init(prepempty + 8 * i, C::SOFT / U);
    }
#pragma unroll 1
    for (int x = 0; x < U; ++x) {
      for (int b = 0; b < 2; ++b) {
        t_bar_init(sfull(x, b), 1);
        t_bar_init(sfree(x, b), C::SOFT / U);
      }
      t_bar_init(pfull(x), C::SOFT / U);
      t_bar_init(pvdone(x), 1);
      t_bar_init(ofree(x), C::SOFT / U);
      t_bar_init(qfull(x), 1);
      t_bar_init(qempty(x), 1);
      for (int b = 0; b < C::E; ++b) {
        t_bar_init(vthere(x, b), 1);
        t_bar_init(vclean(x, b), C::SOFT / U);
      }
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
#pragma unroll 1
  for (int i = tid; i < 256; i += C::THREADS)
    reinterpret_cast<uint32_t *>(sm + C::OFF_ONES)[i] = 0x3f803f80u;
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  if (warp == 0) {
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     t_smem(&s.tmem)),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pkv_allow_next_grid();

  // the line: places of every row, summed up over the rows
  {
    constexpr int R = (kTreeRows + C::THREADS) / C::THREADS;   // rows of a thread, and the end
    int mine[R], sum = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int b = R * tid + i;
      mine[i] = 0;
      if (b < a.B) {
        const TreeRow r = tree_row(b, a.N, a.row_start, a.batch_idx, a.ctx_lens, a.n_slots,
                                   a.max_pages, a.page_size);
        if (r.bits && cta == 0) tree_report(a.err, r.bits);
        rows.n0[b] = r.n0;
        rows.ctx[b] = r.ctx;
        rows.slot[b] = r.slot;
        rows.n[b] = static_cast<uint8_t>(r.n | (r.slot == 0 ? 128 : 0));
        if (r.n > 0) {
          const int lo = a.window > 0 ? max(0, r.ctx - a.window + 1) : 0;
          const int tiles = r.slot == 0 ? 0 : (r.ctx + r.n - 1) / kTile - lo / kTile + 1;
          mine[i] = static_cast<int>(min(static_cast<long long>(kMostPlaces),
                                         static_cast<long long>(tiles + C::START) *
                                             (a.Hkv * ((r.n + a.unit_tokens - 1) /
                                                       a.unit_tokens))));
        }
      }
      sum = add_places(sum, mine[i]);
    }
    int upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto = add_places(upto, v);
    }
    if (lane == 31) s.scan[warp] = upto;
    t_fence_before();
    __syncthreads();
    t_fence_after();
#pragma unroll
    for (int w = 0; w < C::THREADS / 32 - 1; ++w)
      upto = w < warp ? add_places(upto, s.scan[w]) : upto;
    // (where the sum ran over, only its end counts)
    sum = upto - sum;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (R * tid + i <= a.B) rows.pre[R * tid + i] = sum;
      sum = add_places(sum, mine[i]);
    }
    __syncthreads();
  }
  const uint32_t tmem = s.tmem;
  const bool too_long = rows.pre[a.B] == kMostPlaces;
  const int W = too_long ? 0 : rows.pre[a.B];
  if (too_long && cta == 0 && tid == 0) tree_report(a.err, PKV_ERR_POS);
  const int ctas = min(static_cast<int>(gridDim.x), W);
  const int x0 = cta < ctas ? share(W, cta, ctas) : 0;
  const int x1 = cta < ctas ? share(W, cta + 1, ctas) : 0;
  Line<C::START> line;
  line.begin(rows, a, x0, x1);
  const Part &p = line.p;
  // (what the prior kernel may write or read - caches, queries, workspace, output - from here on;
  // the producers wait below)
  const bool producer = warp == C::PROD || warp == C::PROD + 1;
  if (!producer) pkv_wait_prior_grid();
  if (!C::JOINS && tid == 0) a.cuts[cta].cols = 0;

  // whether some columns do not see some keys of the unit's tile t
  auto is_masked = [&](int t) {
    const int j0 = (p.tile0 + t) * kTile;
    return j0 + kTile > p.ctx || (a.window > 0 && j0 <= p.ctx + p.n - 1 - a.window);
  };
  if (producer) {
    // ==================== producers, of K and of V ====================
    // (a warp goes through its boxes as one, and an elected lane issues them, as the MMAs)
    const bool is_v = warp != C::PROD;
    const int slots = is_v ? C::NV : C::NK, slot0 = is_v ? C::NK : 0;
    const int k_rows = min(a.page_size, kTile);             // tokens of a K box
    const int v_rows = min(a.page_size, C::KEYS);
    const int per_tile = kTile / k_rows;         // pages of a tile (1 where they are larger)
    const int split = is_v && per_tile == 1 ? C::ATOMS : 1;   // boxes of a page
    int at = 0, round = 0;                       // the next entry, how often the ring has been full
    int bits = 0;
    bool ok = true;
    // an entry of so many bytes; its number
    auto take = [&](int bytes) -> uint32_t {
      const uint32_t e = __shfl_sync(0xffffffffu, slot0 + at, 0);
      if (round > 0) ok = wait_for(empty + 8 * e, round - 1);
      if (ok && elect_one()) t_expect_tx(full + 8 * e, bytes);
      if (++at == slots) at = 0, ++round;
      return e;
    };
    // a K tile's boxes [first, last); lane i knows box i's row
    auto load_k = [&](int at_row, int head, int first, int last) {
#pragma unroll 1
      for (int c = 0; c < C::E; ++c) {
        const uint32_t e = take((last - first) * C::ATOMS * k_rows * 128);
        if (!ok) break;
#pragma unroll 1
        for (int i = first; i < last; ++i) {
          const int r = __shfl_sync(0xffffffffu, at_row, i);
          if (elect_one()) {
#pragma unroll
            for (int b = 0; b < C::ATOMS; ++b)
              t_tma_4d(sRing + e * C::ENTRY + b * C::ATOM + i * k_rows * 128, &tmK, 0, r, head,
                       C::ATOMS * c + b, full + 8 * e);
          }
          __syncwarp();
        }
      }
    };
    // a V tile's; a box has two atoms where its keys are a half's
    auto load_v = [&](int at_row, int head, int first, int last) {
      const int per = C::KEYS / v_rows;               // boxes (or pairs of them) of a half
      const int step = v_rows == C::KEYS ? C::ATOMS : 1;   // atoms of a box
#pragma unroll 1
      for (int c = 0; c < C::E; ++c) {
        const uint32_t e = take((last - first) * C::ATOMS * v_rows * 128);
        if (!ok) break;
#pragma unroll 1
        for (int i = first; i < last; ++i) {
          const int r = __shfl_sync(0xffffffffu, at_row, i);
          const int half = i >= per;
          const uint32_t to =
              sRing + e * C::ENTRY + half * C::ATOM + (i - half * per) * v_rows * 128;
          if (elect_one()) {
#pragma unroll 1
            for (int b = 0; b < C::ATOMS; b += step)
              t_tma_4d(to + b * C::KEYS * 128, &tmV, 0, r, head, C::ATOMS * c + b, full + 8 * e);
          }
          __syncwarp();
        }
      }
    };
    bool waited = false;
    while (ok && line.next()) {
      if (p.t0 == p.t1) continue;
      const int32_t *row = a.table + static_cast<long long>(rows.slot[p.b]) * a.max_pages;
      const int last_page = (p.ctx + p.n - 1) >> a.log_page;
      const int first_page = p.lo >> a.log_page;
      const int head = __shfl_sync(0xffffffffu, p.head, 0);
      // page numbers 32 at a time, the next ones on their way
      auto fetch = [&](int i) -> int {
        return i >= first_page && i <= last_page ? row[i] : 0;
      };
      int base = ((p.tile0 + p.t0) * kTile) >> a.log_page;
      int now = fetch(base + lane), then = fetch(base + 32 + lane);
      if (!waited) {
        // The first tiles' way to L2 begins before the prior kernel has ended: nothing is read
        // that it may still write.
        constexpr int kRows = D <= 128 ? 32768 / D : kTile;        // of 64 KB, or a tile
        const int from = ((p.tile0 + p.t0) * kTile) & (a.page_size - 1);   // (large pages)
        const int n = min(kRows, (p.t1 - p.t0) * kTile), size = min(a.page_size - from, n);
        if (lane * a.page_size < n && base + lane >= first_page && base + lane <= last_page &&
            now >= 0 && now < a.n_pages) {
          const long long at =
              static_cast<long long>(p.head) * a.n_pages * a.page_size +
              static_cast<long long>(now) * a.page_size + from;
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                           (is_v ? a.v : a.k) + at * D),
                       "r"(size * D * 2));
        }
        __syncwarp();
        pkv_wait_prior_grid();
        waited = true;
      }
#pragma unroll 1
      for (int t = p.t0; t < p.t1 && ok; ++t) {
        const int j0 = (p.tile0 + t) * kTile, page0 = j0 >> a.log_page;
        if (page0 >= base + 32) {
          base += 32;
          now = then;
          then = fetch(base + 32 + lane);
        }
        // boxes [first, last), and lane i knows box i's row
        const int first = __shfl_sync(0xffffffffu, max(0, first_page - page0) * split, 0);
        const int last =
            __shfl_sync(0xffffffffu, min(per_tile, last_page - page0 + 1) * split, 0);
        int page = __shfl_sync(0xffffffffu, now, (page0 - base + lane / split) & 31);
        if (lane >= first && lane < last && (page < 0 || page >= a.n_pages)) {
          bits |= page < 0 ? PKV_ERR_PAGE_NEG : PKV_ERR_PAGE_RANGE;
          page = 0;
        }
        const int at_row = page * a.page_size + (j0 & (a.page_size - 1)) +   // (large pages)
                           lane % split * C::KEYS;
        if (is_v) load_v(at_row, head, first, last);
        else load_k(at_row, head, first, last);
      }
    }
    tree_report(a.err, bits);
    if (!ok) {
      // what is on its way lands before the CTA leaves
#pragma unroll 1
      for (int i = 0; i < slots; ++i) {
        const int fills = round + (i < at ? 1 : 0);
#pragma unroll 1
        for (int k = 0; k < kSpin && fills && !t_test(full + 8 * (slot0 + i), fills - 1); ++k) {
        }
      }
    }
  } else if (warp >= C::MMA) {
    // ==================== MMA: a warp for S, one for P V ====================
    // A tile is one elected lane's, its waits too: a vote, an election and an address for each
    // entry took half as long as its products (1 to 2% of every call). Elected, not under a lane's
    // own branch: so the compiler knows that descriptors and addresses are the warp's; an MMA took
    // 90 to 150 cycles to issue otherwise. The warp meets between tiles.
    const bool is_pv = warp != C::MMA;
    static_assert(C::E == 1 || (C::E % C::NK == 0 && C::E % C::NV == 0), "slots of a tile");
    int at = 0, round = 0;                  // the next entry, how often the ring has been used up
    int segs = 0, done[2] = {0, 0}, masked[2] = {0, 0};   // tiles of each unit, masked ones
    bool ok = true;
    // (a tile's entries: the next one, or as many as the ring has, or a multiple)
    auto used = [&](int slots) {
      if (C::E > 1) round += C::E / slots;
      else if (++at == slots) at = 0, ++round;
    };
    const uint64_t dOne = t_desc(sOnes, 0, 0);
    while (ok && line.next()) {
      if (p.t0 == p.t1) continue;
      const int x = __shfl_sync(0xffffffffu, segs % U, 0), own = segs / U;
      ++segs;
      const int N = __shfl_sync(0xffffffffu, columns<C::GROUPS>(p.toks * a.G), 0);
      const uint32_t tx = __shfl_sync(0xffffffffu, tmem + x * C::UNIT_COLS, 0);
      int tiles = x ? done[1] : done[0];
      if (!is_pv) {
        const uint64_t dQ = t_desc(sQ + x * C::Q_BYTES, 16, 1024);
        const uint32_t id = idesc(N, false);
        ok = wait_for(qfull(x), own);
#pragma unroll 1
        for (int t = p.t0; t < p.t1 && ok; ++t, ++tiles) {
          const int buf = tiles % C::SB;
          const uint32_t to = __shfl_sync(0xffffffffu, tx + C::S_COL + buf * C::COLS, 0);
          const uint32_t slot = __shfl_sync(0xffffffffu, at, 0);
          if (elect_one()) {
            ok = tiles < C::SB || lane_wait(sfree(x, buf), tiles / C::SB - 1);
#pragma unroll
            for (int c = 0; c < C::E; ++c) {
              const uint32_t e = C::E > 1 ? c % C::NK : slot;
              ok = ok && lane_wait(full + 8 * e, round + (C::E > 1 ? c / C::NK : 0));
              t_fence_after();
              if (!ok) break;
#pragma unroll
              for (int b = 0; b < C::ATOMS; ++b) {
                const uint64_t ka = t_desc(sRing + e * C::ENTRY + b * C::ATOM, 16, 1024);
                const uint64_t qb = dQ + (C::ATOMS * c + b) * (C::Q_ATOM >> 4);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  t_mma(to, ka + k * 2, qb + k * 2, id, c > 0 || b > 0 || k > 0);
              }
              t_commit(empty + 8 * e);
            }
            if (ok) t_commit(sfull(x, buf));
            if (ok && t == p.t1 - 1) t_commit(qempty(x));
          }
          ok = __all_sync(0xffffffffu, ok);
          used(C::NK);
        }
      } else {
        const uint64_t dP = t_desc(sP + x * C::P_BYTES, C::P_ATOM, 1024);
        const uint32_t id = idesc(N, true);
        int masks = x ? masked[1] : masked[0];
#pragma unroll 1
        for (int t = p.t0; t < p.t1 && ok; ++t, ++tiles) {
          const bool mask = is_masked(t);
          const uint32_t slot = C::NK + __shfl_sync(0xffffffffu, at, 0);
          if (elect_one()) {
            // a masked tile's V is looked at block by block, as soon as it is there
            auto there = [&](int c) {
              const uint32_t e = C::E > 1 ? C::NK + c % C::NV : slot;
              ok = ok && lane_wait(full + 8 * e, round + (C::E > 1 ? c / C::NV : 0));
              if (ok && mask) t_arrive(vthere(x, c));
            };
            if (mask) there(0);
            ok = ok && lane_wait(pfull(x), tiles);
            if (t == p.t0 && own >= 1) ok = ok && lane_wait(ofree(x), own - 1);
            const uint32_t add = t > p.t0;
            t_fence_after();
            // the weights' sums: a row of ones, 128 times (they need no V, which may be on its way)
            if (ok) {
#pragma unroll
              for (int k = 0; k < kTile / 16; ++k)
                t_mma(tx + C::L_COL, dOne, dP + k * (2048 >> 4), id, k > 0 ? 1u : add);
            }
#pragma unroll
            for (int c = 0; c < C::E; ++c) {
              if (!mask) there(c);
              else if (c + 1 < C::E) there(c + 1);
              if (mask) ok = ok && lane_wait(vclean(x, c), masks);
              t_fence_after();
              if (!ok) break;
              const uint32_t e = C::E > 1 ? C::NK + c % C::NV : slot;
              const uint32_t to = tx + C::O_COL + c * C::COLS;
#pragma unroll
              for (int b = 0; b < C::ATOMS; ++b) {
                // (D = 64: rows 64 .. 127 of the product repeat rows 0 .. 63)
                const uint64_t va = t_desc(sRing + e * C::ENTRY + b * C::ATOM,
                                           D == 64 ? 0 : C::KEYS * 128, 1024);
                const uint64_t pb = dP + b * (C::KEYS * 128 >> 4);
#pragma unroll
                for (int k = 0; k < C::KEYS / 16; ++k)
                  t_mma(to, va + k * (2048 >> 4), pb + k * (2048 >> 4), id,
                        b > 0 || k > 0 ? 1u : add);
              }
              t_commit(empty + 8 * e);
            }
            if (ok) t_commit(pvdone(x));
          }
          ok = __all_sync(0xffffffffu, ok);
          used(C::NV);
          masks += mask;
        }
        if (x) masked[1] = masks;
        else masked[0] = masks;
      }
      if (x) done[1] = tiles;
      else done[0] = tiles;
    }
    if (elect_one()) {
      t_commit(drain + 8 * is_pv);
      t_wait_drain(drain + 8 * is_pv);
    }
    __syncwarp();
  } else if (warp == C::PREP) {
    // ====================== queries and who sees whom ======================
    int segs = 0, bits = 0;
    const int box = a.box_nodes * a.G * 128;      // bytes of a box: nodes x heads, one atom
    while (line.next()) {
      if (p.t0 == p.t1) continue;
      const int x = segs % U;
      if (segs >= U && !wait_for(qempty(x), segs / U - 1)) break;
      const int boxes = __shfl_sync(0xffffffffu, (p.toks + a.box_nodes - 1) / a.box_nodes, 0);
      const int head = __shfl_sync(0xffffffffu, p.head * a.G, 0);
      const int node = __shfl_sync(0xffffffffu, p.n0 + p.tok0, 0);
      if (elect_one()) {
        t_expect_tx(qfull(x), boxes * box * (D / 64));
#pragma unroll 1
        for (int i = 0; i < boxes; ++i)
#pragma unroll 1
          for (int at = 0; at < D / 64; ++at)
            t_tma_4d(sQ + x * C::Q_BYTES + at * C::Q_ATOM + i * box, &tmQ, 0, head,
                     node + a.box_nodes * i, at, qfull(x));
      }
      __syncwarp();
      Prep<C::GROUPS> &w = s.prep[segs & 1];
      if (segs >= 2 && !wait_for(prepempty + 8 * (segs & 1), (segs >> 1) - 1)) break;
      // paths: each node's set of ancestors and itself, twice as far every time
      uint64_t *path = w.below[0];
      int *jump = w.depth;
#pragma unroll
      for (int i = lane; i < kTreeMax; i += 32) {
        path[i] = 1ull << i;
        jump[i] = i < p.n ? tree_parent(a.parents, p.n0, i, bits) : -1;
      }
      __syncwarp();
#pragma unroll 1
      for (int r = 0; r < 6; ++r) {
        uint64_t v[2];
        int j[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int i = lane + 32 * q;
          v[q] = path[i];
          j[q] = jump[i];
          if (j[q] >= 0) {
            v[q] |= path[j[q]];
            j[q] = jump[j[q]];
          }
        }
        const bool more = __any_sync(0xffffffffu, j[0] >= 0 || j[1] >= 0);
        __syncwarp();   // all have read
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          path[lane + 32 * q] = v[q];
          jump[lane + 32 * q] = j[q];
        }
        __syncwarp();
        if (!more) break;
      }
      uint64_t below[2][2] = {{0, 0}, {0, 0}}, shallow[2][2] = {{0, 0}, {0, 0}};   // [group][node]
      int depth[2] = {0, 0};
      const int hn = columns<C::GROUPS>(p.toks * a.G) / C::GROUPS;
#pragma unroll 1
      for (int t = 0; t < p.n; ++t) {
        const uint64_t v = path[t];
        const int d = __popcll(v) - 1;
        const int first = (t - p.tok0) * a.G;          // the node's columns
        const bool here = t >= p.tok0 && t < p.tok0 + p.toks;
#pragma unroll
        for (int q = 0; q < 2; ++q)
          if (t == lane + 32 * q) depth[q] = d;
#pragma unroll
        for (int gr = 0; gr < C::GROUPS; ++gr) {
          // those of them that are the group's
          const int lo = max(0, first - gr * hn), hi = min(hn, first + a.G - gr * hn);
          const uint64_t mine = here && lo < hi ? ((1ull << (hi - lo)) - 1) << lo : 0;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int i = lane + 32 * q;
            below[gr][q] |= (v >> i) & 1 ? mine : 0;
            shallow[gr][q] |= d <= i ? mine : 0;
          }
        }
      }
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 2; ++q) {
#pragma unroll
        for (int gr = 0; gr < C::GROUPS; ++gr) {
          w.below[gr][lane + 32 * q] = below[gr][q];
          w.shallow[gr][lane + 32 * q] = shallow[gr][q];
        }
        w.depth[lane + 32 * q] = depth[q];
      }
      if (lane < 2 * C::GROUPS) w.poison[lane >> 1][lane & 1] = 0;
      __syncwarp();
      if (lane == 0) t_arrive(prepfull + 8 * (segs & 1));
      ++segs;
    }
    // (should the others have given up: what is on its way lands before the CTA leaves)
#pragma unroll 1
    for (int i = max(0, segs - U); i < segs; ++i) wait_for(qfull(i % U), i / U);
    tree_report(a.err, bits);
  } else {
    // ============================ softmax =============================
    const int quad = warp & 3, sub = warp >> 2;      // (sub: which four warps)
    const int x = U == 2 ? sub : 0, grp = U == 2 ? 0 : sub;   // unit, group of its columns
    const uint32_t sfull_x = sfull(x, 0), sfree_x = sfree(x, 0), pvdone_x = pvdone(x);
    const int row = 32 * quad + lane;           // the key of a tile, or the column of D
    const uint32_t trow = tmem + x * C::UNIT_COLS + (static_cast<uint32_t>(32 * quad) << 16);
    const int h0 = sub * C::HALF;               // where the warps' columns are in shared memory
    uint8_t *pbuf = sm + C::OFF_P + x * C::P_BYTES + row * 128;   // this key's row of P
    const int mine = 32 * quad + lane;          // the column that this thread looks after
    int tiles = 0, segs = 0, seg = 0, masks = 0, g = 0;   // g: where in V's ring
    bool ok = true, gone = false;
    // The parts of a unit are joined by fours: who is the last of four to write its own joins them
    // into the first's place, goes on with four such, and writes the output in the end. In the
    // parts' order whoever it is; nobody waits.
    auto join = [&](int cols) {
      const int first_cta = p.t0 == 0 ? cta : share_of(W, p.start + C::START, ctas);
      const int parts = share_of(W, p.start + C::START + p.ntiles - 1, ctas) - first_cta + 1;
      auto place = [&](int i) { return 2 * (first_cta + i) + (i == 0 ? 1 : 0); };
      int i = cta - first_cta;
#pragma unroll 1
      for (int span = 1, level = 0; span < parts; span *= kFan, ++level) {
        i -= i % (span * kFan);                       // the first of the four
        const int n = min(kFan, (parts - i + span - 1) / span);
        if (n == 1) continue;
        __threadfence();
        group_sync(sub);
        if (mine == 0) {
          int *count = a.arrived + level * 2 * kMaxCtas + place(i);
          const int last = atomicAdd(count, 1) == n - 1;
          if (last) *count = 0;                       // as it was
          s.last[sub] = last;
        }
        group_sync(sub);
        if (!s.last[sub]) return;
        __threadfence();
        const bool all = span * kFan >= parts;
        auto rec = [&](int k) { return a.parts + place(i + k * span) * C::RECORD; };
        float *to = rec(0);
        // a thread a column: the parts' weights
        float ref = -INFINITY, sum = 0.f;
        if (mine < cols) {
          float m[kFan];
#pragma unroll
          for (int k = 0; k < kFan; ++k) {
            m[k] = k < n ? __ldcg(rec(k) + C::COLS * D + mine) : -INFINITY;
            ref = fmaxf(ref, m[k]);
          }
#pragma unroll
          for (int k = 0; k < kFan; ++k) {
            const float w = m[k] == -INFINITY ? 0.f : exp2f(m[k] - ref);
            s.red[k][h0 + mine] = w;
            if (k < n) sum = fmaf(w, __ldcg(rec(k) + C::COLS * (D + 1) + mine), sum);
          }
          s.alpha[h0 + mine] = 1.f / sum;
        }
        group_sync(sub);
        constexpr int Q = D / 4, kAhead = 4;   // reads in flight
#pragma unroll 1
        for (int j0 = mine; j0 < cols * Q; j0 += kAhead * 128) {
          float4 y[kAhead];
#pragma unroll
          for (int h = 0; h < kAhead; ++h) y[h] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
          for (int k = 0; k < n; ++k) {
            const float *from = rec(k);
            float4 v[kAhead];
#pragma unroll
            for (int h = 0; h < kAhead; ++h)
              if (j0 + h * 128 < cols * Q)
                v[h] = __ldcg(reinterpret_cast<const float4 *>(from + (j0 + h * 128) * 4));
#pragma unroll
            for (int h = 0; h < kAhead; ++h) {
              if (j0 + h * 128 >= cols * Q) break;
              const float w = s.red[k][h0 + (j0 + h * 128) / Q];
              y[h].x = fmaf(w, v[h].x, y[h].x);
              y[h].y = fmaf(w, v[h].y, y[h].y);
              y[h].z = fmaf(w, v[h].z, y[h].z);
              y[h].w = fmaf(w, v[h].w, y[h].w);
            }
          }
#pragma unroll
          for (int h = 0; h < kAhead; ++h) {
            const int j = j0 + h * 128, c = j / Q;
            if (j >= cols * Q) break;
            if (all) {
              const float f = s.alpha[h0 + c];
              *reinterpret_cast<uint2 *>(a.out + s.dst[h0 + c] + j % Q * 4) =
                  make_uint2(t_pack(y[h].x * f, y[h].y * f), t_pack(y[h].z * f, y[h].w * f));
            } else {
              __stcg(reinterpret_cast<float4 *>(to + j * 4), y[h]);
            }
          }
        }
        if (!all && mine < cols) {
          __stcg(to + C::COLS * D + mine, ref);
          __stcg(to + C::COLS * (D + 1) + mine, sum);
        }
        if (all) return;
      }
    };
    // A unit, or the part of it that is this CTA's. Loops over chunks of 16 columns stay loops:
    // unrolled, the warps waited for instructions a third of the time.
    auto unit = [&]() {
      const int cols = p.toks * a.G;
      const int hn = columns<C::GROUPS>(cols) / C::GROUPS, c0 = grp * hn;   // this warp's columns
      Prep<C::GROUPS> &w = s.prep[seg & 1];
      // a group's columns in use
      auto used = [&](int gr) -> uint64_t {
        const int k = min(hn, cols - gr * hn);
        return k <= 0 ? 0 : ~0ull >> (64 - k);
      };
      bool any_masked = false;
#pragma unroll 1
      for (int t = p.t0; t < p.t1; ++t, ++tiles) {
        const int buf = tiles % C::SB;
        const int j0 = (p.tile0 + t) * kTile, j = j0 + row;
        const bool masked = is_masked(t);
        const bool first = t == p.t0;
        uint64_t sees = ~0ull;                  // the columns that see this thread's key
        bool none_sees = false, all_see = true;
        any_masked |= masked;
        // (S first: the unit's queries are there then, and the preparations before its own)
        ok = ok && wait_for(sfull_x + 8 * buf, tiles / C::SB);
        if (masked) {
          ok = ok && wait_for(prepfull + 8 * (seg & 1), seg >> 1);
          const int node = j - p.ctx;
          const int reach = node < 0 ? node + a.window - 1
                                     : min(static_cast<long long>(kTreeMax),
                                           static_cast<long long>(w.depth[min(node, p.n - 1)]) +
                                               a.window - 1);
          none_sees = true;
#pragma unroll
          for (int gr = 0; gr < C::GROUPS; ++gr) {
            uint64_t v = node >= p.n ? 0 : node >= 0 ? w.below[gr][node] : ~0ull;
            if (a.window > 0) v &= reach < 0 ? 0 : w.shallow[gr][min(reach, kTreeMax - 1)];
            if (gr == grp) sees = v;
            none_sees = none_sees && !(v & used(gr));
            all_see = all_see && !(~v & used(gr));
          }
        }
        t_fence_after();
        const uint32_t scol = trow + C::S_COL + buf * C::COLS + c0;
        // 16 scores of this thread's key, -inf where a node does not see it
        auto scores = [&](int c, float (&y)[16]) {
          uint32_t r[16];
          ld16(scol + c, r);
          t_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] = __uint_as_float(r[e]);
          if (masked) {
            const uint32_t bits = static_cast<uint32_t>(sees >> c);
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = bits & (1u << e) ? y[e] : -INFINITY;
          }
        };
        // P's place is free, and O is there, once the tile before has been multiplied. A unit that
        // is alone has its weights wait for it in registers, so that only their way to shared
        // memory is between two products (16 rows with trees of 64, eight heads of 128 77 -> 71
        // us; a row of 41 tokens by units in twos, though, 5.0 -> 5.3: more code).
        bool at_hand = tiles == 0;
        auto wait_pv = [&]() {
          if (!at_hand) {
            ok = ok && wait_for(pvdone_x, tiles - 1);
            t_fence_after();
          }
          at_hand = true;
        };
        uint32_t weights[C::HALF / 2];
        // of 16 columns, under the references at hand
        auto weigh = [&](int c, uint32_t *w, float &top) {
          float y[16];
          scores(c, y);
          const float4 *m4 = reinterpret_cast<const float4 *>(s.mneg + h0 + c);
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 m = m4[e / 4];
            fma2(y[e], y[e + 1], y[e], y[e + 1], a.scale_log2, m.x, m.y);
            fma2(y[e + 2], y[e + 3], y[e + 2], y[e + 3], a.scale_log2, m.z, m.w);
            top = t_max3(top, y[e], y[e + 1]);
            top = t_max3(top, y[e + 2], y[e + 3]);
            w[e / 2] = t_pack(t_ex2(y[e]), t_ex2(y[e + 1]));
            w[e / 2 + 1] = t_pack(t_ex2(y[e + 2]), t_ex2(y[e + 3]));
          }
        };
        // a key's columns in a row of 128 bytes as the swizzle has them
        auto put = [&](int c, const uint32_t *w) {
          const int at = ((c0 + c) & 63) >> 3;
          uint8_t *to = pbuf + (c0 + c) / 64 * C::P_ATOM;
          *reinterpret_cast<uint4 *>(to + ((at ^ (row & 7)) << 4)) =
              make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4 *>(to + (((at + 1) ^ (row & 7)) << 4)) =
              make_uint4(w[4], w[5], w[6], w[7]);
        };
        if (U == 2) wait_pv();
        // A first tile begins with the columns' maxima, others when a score is out of reach. (A
        // first guess without maxima, 2^4 above the first key's scores, gained nothing.)
        for (bool exact = first;;) {
          if (exact) {
            if (group_any(sub, !ok)) {
              gone = true;
              return;
            }
#pragma unroll 1
            for (int c = 0; c < hn; c += 16) {
              float y[16];
              scores(c, y);
#pragma unroll
              for (int e = 0; e < 16; ++e) y[e] = lane_max(y[e]);
              if (lane == 0) {
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                  *reinterpret_cast<float4 *>(&s.red[quad][h0 + c + e]) =
                      make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
              }
            }
            group_sync(sub);
            if (mine < hn) {
              const int c = h0 + mine;
              const float old = first ? -INFINITY : s.ref[c];
              const float top = fmaxf(fmaxf(s.red[0][c], s.red[1][c]),
                                      fmaxf(s.red[2][c], s.red[3][c])) * a.scale_log2;
              const float ref = fmaxf(old, top);
              s.ref[c] = ref;
              s.mneg[c] = c0 + mine >= cols ? -INFINITY : ref == -INFINITY ? kUnset : -ref;
              s.alpha[c] = old == ref ? 1.f : exp2f(old - ref);
            }
            group_sync(sub);
            if (!first) {
              wait_pv();
#pragma unroll 1
              for (int c = 0; c < hn; c += 16) {
#pragma unroll 1
                for (int blk = 0; blk <= C::E; ++blk) {   // (the last: the sums)
                  uint32_t r[16];
                  const uint32_t at = trow + C::O_COL + blk * C::COLS + c0 + c;
                  ld16(at, r);
                  t_wait_ld();
#pragma unroll
                  for (int e = 0; e < 16; ++e)
                    r[e] = __float_as_uint(__uint_as_float(r[e]) * s.alpha[h0 + c + e]);
                  t_st16(at, r);
                }
              }
              t_wait_st();
            }
          }
          float top = -INFINITY;
          if (ok) {
            if constexpr (U == 2) {
#pragma unroll 1
              for (int c = 0; c < hn; c += 16) {
                uint32_t w[8];
                weigh(c, w, top);
                put(c, w);
              }
            } else {
#pragma unroll
              for (int c = 0; c < C::HALF; c += 16)
                if (c < hn) weigh(c, weights + c / 2, top);
            }
          }
          if (exact || !group_any(sub, top > kLazyLog2 || !ok)) break;
          exact = true;
        }
        t_fence_before();
        __syncwarp();
        if (lane == 0) t_arrive(sfree_x + 8 * buf);
        wait_pv();
        if (U == 1 && ok) {
#pragma unroll
          for (int c = 0; c < C::HALF; c += 16)
            if (c < hn) put(c, weights + c / 2);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        t_fence_before();
        __syncwarp();
        if (lane == 0) t_arrive(pfull(x));
        if (masked) {
          // Rows of V seen by no column are cleared, and those seen by some only if they are not
          // finite, block by block between its being there and its product.
          const unsigned none = __ballot_sync(0xffffffffu, none_sees);
          const unsigned part = __ballot_sync(0xffffffffu, !none_sees && !all_see);
          // (a single atom is the first group's)
          const bool looks = (none | part) && (D > 64 || grp == 0);
          // this warp's share of a row of an entry: 8 lanes an atom, both atoms or its group's
          constexpr int AT = D == 64 || C::GROUPS == 2 ? 1 : 2;
          constexpr int STEP = 4 / AT;                 // rows at a time
          const int in = (lane & 7) * 16 +
                         (D == 64            ? 0
                          : C::GROUPS == 2 ? grp
                                           : (lane >> 3) & 1) * C::KEYS * 128;
          const int which = lane / (8 * AT);           // of the rows at a time
#pragma unroll 1
          for (int blk = 0; blk < C::E && ok; ++blk) {
            if (looks) ok = wait_for(vthere(x, blk), masks);
            if (looks && ok) {
              const int e = C::NK + (g + (t - p.t0) * C::E + blk) % C::NV;
              uint8_t *v = sm + e * C::ENTRY + 32 * quad / C::KEYS * C::ATOM + in +
                           (32 * quad % C::KEYS) * 128;
              unsigned clear = none;
              if (part) {
#pragma unroll 1
                for (int r0 = 0; r0 < 32; r0 += 4 * STEP) {
                  if (!(part >> r0 & ((1u << (4 * STEP - 1) << 1) - 1))) continue;
                  uint4 y[4];
#pragma unroll
                  for (int i = 0; i < 4; ++i)
                    y[i] = *reinterpret_cast<const uint4 *>(v + (r0 + i * STEP + which) * 128);
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    // 0 times what is finite stays 0
                    const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
                    __nv_bfloat162 z = zero;
                    z = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&y[i].x), zero, z);
                    z = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&y[i].y), zero, z);
                    z = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&y[i].z), zero, z);
                    z = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&y[i].w), zero, z);
                    const unsigned who = __ballot_sync(
                        0xffffffffu, (*reinterpret_cast<const uint32_t *>(&z) & 0x7fff7fffu) != 0);
#pragma unroll
                    for (int q = 0; q < STEP; ++q)
                      if (who >> (8 * AT * q) & ((1u << (8 * AT - 1) << 1) - 1))
                        clear |= part & (1u << (r0 + i * STEP + q));
                  }
                }
              }
              const unsigned poisoned = clear & part;
              if (poisoned >> lane & 1) {
                // (this row's node, for all groups: each has looked at columns of D of its own)
                const int node = j - p.ctx;
                const int reach =
                    node < 0 ? node + a.window - 1
                             : min(kTreeMax - 1, w.depth[node] + min(a.window, kTreeMax) - 1);
#pragma unroll
                for (int gr = 0; gr < C::GROUPS; ++gr) {
                  uint64_t u = node >= 0 ? w.below[gr][node] : ~0ull;
                  if (a.window > 0) u &= w.shallow[gr][min(reach, kTreeMax - 1)];
                  atomicOr(&w.poison[gr][0], static_cast<unsigned>(u));
                  atomicOr(&w.poison[gr][1], static_cast<unsigned>(u >> 32));
                }
              }
              if (clear) {
                const unsigned mine_of = clear >> which;
#pragma unroll
                for (int r = 0; r < 32; r += STEP)
                  if (mine_of >> r & 1)
                    *reinterpret_cast<uint4 *>(v + (r + which) * 128) = make_uint4(0, 0, 0, 0);
              }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) t_arrive(vclean(x, blk));
          }
          ++masks;
        }
      }
      ok = ok && wait_for(pvdone_x, tiles - 1);
      t_fence_after();
      const bool whole = p.whole();
      float *rec = a.parts + (2 * cta + (p.t0 == 0 ? 1 : 0)) * C::RECORD;
      if (mine < hn) {
        const int c = c0 + mine, k = h0 + mine, tok = p.tok0 + c / a.G;
        const bool bad = any_masked && (w.poison[grp][mine >> 5] >> (mine & 31) & 1);
        const long long q_row = static_cast<long long>(p.n0 + tok) * a.Hq + p.head * a.G + c % a.G;
        s.dst[k] = c < cols ? q_row * D : -1;
        s.alpha[k] = bad ? NAN : 1.f;
        if (!whole && c < cols) rec[C::COLS * D + c] = s.ref[k];
      }
      group_sync(sub);
      if (ok) {
#pragma unroll 1
        for (int c = 0; c < hn; c += 16) {
          float l[16];
          {
            uint32_t r[16];
            ld16(trow + C::L_COL + c0 + c, r);
            t_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) l[e] = __uint_as_float(r[e]) * s.alpha[h0 + c + e];
          }
          if (whole) {
#pragma unroll
            for (int e = 0; e < 16; ++e) l[e] = __fdividef(1.f, l[e]);
          } else if (row == 0) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (c0 + c + e < cols) rec[C::COLS * (D + 1) + c0 + c + e] = l[e];
          }
#pragma unroll 1
          for (int blk = 0; blk < C::E; ++blk) {
            const int d = blk * 128 + row;
            uint32_t r[16];
            ld16(trow + C::O_COL + blk * C::COLS + c0 + c, r);
            t_wait_ld();
            if (D == 64 && quad >= 2) continue;
            if (whole) {
              // two columns a step: even lanes store one, odd lanes the other, two places each
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                const float y0 = __uint_as_float(r[e]) * l[e];
                const float y1 = __uint_as_float(r[e + 1]) * l[e + 1];
                const float got = __shfl_xor_sync(0xffffffffu, lane & 1 ? y0 : y1, 1);
                const uint32_t v = lane & 1 ? t_pack(got, y1) : t_pack(y0, got);
                const long long dst = s.dst[h0 + c + e + (lane & 1)];
                if (dst >= 0) *reinterpret_cast<uint32_t *>(a.out + dst + (d & ~1)) = v;
              }
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int col = c0 + c + e;
                if (col < cols) rec[col * D + d] = __uint_as_float(r[e]);
              }
            }
          }
        }
      }
      if (!C::JOINS && tid == 0 && !whole && p.t0 == 0) {
        // the CTA of the unit's last tile
        const int c = share_of(W, p.start + C::START + p.ntiles - 1, ctas);
        const Cut cut = {p.n0 + p.tok0, cols, p.head, c - cta + 1};
        a.cuts[cta] = cut;
      }
      t_fence_before();
      __syncwarp();
      if (lane == 0) {
        t_arrive(ofree(x));
        t_arrive(prepempty + 8 * (seg & 1));
      }
      if constexpr (C::JOINS) {
        if (!whole && !group_any(sub, !ok)) join(cols);
      }
    };
    while (!gone && line.next()) {
      const int cols = p.toks * a.G;
      if (p.ntiles == 0) {                      // padding
#pragma unroll 1
        for (int i = warp; i < cols; i += C::SOFT) {   // all units' warps share them
          const long long o = (static_cast<long long>(p.n0 + p.tok0 + i / a.G) * a.Hq +
                               p.head * a.G + i % a.G) * D;
#pragma unroll 1
          for (int d = 2 * lane; d < D; d += 64)
            *reinterpret_cast<uint32_t *>(a.out + o + d) = 0;
        }
        continue;
      }
      if (p.t0 == p.t1) continue;
      seg = segs++;
      if (seg % U != x) {
        g = (g + (p.t1 - p.t0) * C::E) % C::NV;
        continue;
      }
      unit();
      g = (g + (p.t1 - p.t0) * C::E) % C::NV;
    }
    if ((gone || !ok) && lane == 0) tree_report(a.err, PKV_ERR_TIMEOUT);
  }
  t_fence_before();
  __syncthreads();
  t_fence_after();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(512));
}

// Joins the parts of the unit that CTA blockIdx.x began and others went on with: a warp a
// column, the reads of a few parts in flight with those of their weights.
template <int D, int MOST>
__global__ void __launch_bounds__(kJoinWarps * 32)
    tree_join_kernel(const float *parts, const Cut *cuts, __nv_bfloat16 *out, int Hq, int G) {
  using C = Cfg<D, MOST>;
  pkv_wait_prior_grid();
  pkv_allow_next_grid();
  const Cut cut = cuts[blockIdx.x];
  const int item = blockIdx.y * kJoinWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int col = item, d = 4 * lane;
  if (col >= cut.cols) return;
  auto rec = [&](int i) -> const float * {
    return parts + (2 * (blockIdx.x + i) + (i == 0 ? 1 : 0)) * C::RECORD;
  };
  constexpr int kAhead = C::E > 2 ? 2 : 4;
  float4 v[kAhead][C::E];
  auto read = [&](int i) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (i + j < cut.parts && d < D)
#pragma unroll
        for (int b = 0; b < C::E; ++b)
          v[j][b] = *reinterpret_cast<const float4 *>(rec(i + j) + col * D + 128 * b + d);
  };
  read(0);
  float top = -INFINITY, sum = 0.f, ref = -INFINITY, l = 0.f;
  for (int i = lane; i < cut.parts; i += 32) {
    ref = rec(i)[C::COLS * D + col];
    l = rec(i)[C::COLS * (D + 1) + col];
    top = fmaxf(top, ref);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (top == -INFINITY) top = 0.f;
  float4 x[C::E];
#pragma unroll
  for (int b = 0; b < C::E; ++b) x[b] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < cut.parts; i0 += 32) {
    if (cut.parts > 32 && i0 + lane < cut.parts) {   // (else they are at hand)
      ref = rec(i0 + lane)[C::COLS * D + col];
      l = rec(i0 + lane)[C::COLS * (D + 1) + col];
    }
    const float w = i0 + lane < cut.parts ? exp2f(ref - top) : 0.f;
    float s = i0 + lane < cut.parts ? w * l : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    sum += s;
    const int n = min(32, cut.parts - i0);
    for (int i = 0; i < n; i += kAhead) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const float wj = __shfl_sync(0xffffffffu, w, (i + j) & 31);
        if (i + j < n) {
#pragma unroll
          for (int b = 0; b < C::E; ++b) {
            x[b].x = fmaf(wj, v[j][b].x, x[b].x);
            x[b].y = fmaf(wj, v[j][b].y, x[b].y);
            x[b].z = fmaf(wj, v[j][b].z, x[b].z);
            x[b].w = fmaf(wj, v[j][b].w, x[b].w);
          }
        }
      }
      read(i0 + i + kAhead);
    }
  }
  if (d >= D) return;
  const float inv = 1.f / sum;
  const int tok = col / G;
  __nv_bfloat16 *o = out + (static_cast<long long>(cut.token0 + tok) * Hq + cut.head * G +
                            (col - tok * G)) * D;
#pragma unroll
  for (int b = 0; b < C::E; ++b)
    *reinterpret_cast<uint2 *>(o + 128 * b + d) =
        make_uint2(t_pack(x[b].x * inv, x[b].y * inv), t_pack(x[b].z * inv, x[b].w * inv));
}

template <int D, int MOST>
int launch(const pkv_bf16 *q, const pkv_bf16 *k, const pkv_bf16 *v, Args a, void *workspace,
           cudaStream_t s) {
  using C = Cfg<D, MOST>;
  static std::mutex mu;
  static bool done[64] = {false};
  int dev = 0;
  PKV_CUDA_CHECK(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return pkv::fail(PKV_E_CUDA, "device id out of range");
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      PKV_CUDA_CHECK(cudaFuncSetAttribute(tree_attn_kernel<D, MOST>,
                                          cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          static_cast<int>(smem_bytes<C>())));
      done[dev] = true;
    }
  }
  const int sms = pkv::sm_count();
  const int grid = sms < 1 ? 1 : sms < kMaxCtas ? sms : kMaxCtas;
  // A Q box is so many nodes that its rows fill whole swizzle atoms of 8, times what the rows have
  // on average: one box an atom mostly. (A box a node of 8 heads kept 16 rows with trees of 64 at
  // D = 512 waiting 4 us for each unit's queries: 57 us, now 54.)
  const int least = a.G % 8 == 0 ? 1 : a.G % 4 == 0 ? 2 : a.G % 2 == 0 ? 4 : 8;
  const int most = C::COLS / (least * a.G);
  a.unit_tokens = most * least;
  int times = 1;
  while (times < most && (most % times || 1LL * times * least * a.B < a.N)) ++times;
  const int box_nodes = times * least;
  a.box_nodes = box_nodes;
  a.k = reinterpret_cast<const __nv_bfloat16 *>(k);
  a.v = reinterpret_cast<const __nv_bfloat16 *>(v);
  a.arrived = static_cast<int *>(workspace);
  a.cuts = reinterpret_cast<Cut *>(static_cast<char *>(workspace) + kArrivedBytes);
  a.parts = reinterpret_cast<float *>(a.cuts + kMaxCtas);
  CUtensorMap tmQ, tmK, tmV;
  const int rows = a.n_pages * a.page_size;
  const int k_box = a.page_size < kTile ? a.page_size : kTile;
  const int v_box = a.page_size < C::KEYS ? a.page_size : C::KEYS;
  int st = pkv::prefill_atoms_map(&tmQ, q, a.N, a.Hq, D, a.G, box_nodes, 1);
  if (st == PKV_OK) st = pkv::prefill_atoms_map(&tmK, k, a.Hkv, rows, D, k_box, 1, 1);
  // (two atoms of V in a box where its keys are a half's)
  const int v_atoms = v_box == C::KEYS ? C::ATOMS : 1;
  if (st == PKV_OK) st = pkv::prefill_atoms_map(&tmV, v, a.Hkv, rows, D, v_box, 1, v_atoms);
  if (st != PKV_OK) return st;
  PKV_CUDA_CHECK(pkv::launch_pdl(tree_attn_kernel<D, MOST>, dim3(grid), dim3(C::THREADS),
                                 smem_bytes<C>(), s, tmQ, tmK, tmV, a));
  if constexpr (!C::JOINS)
    PKV_CUDA_CHECK(pkv::launch_pdl(tree_join_kernel<D, MOST>, dim3(grid, C::COLS / kJoinWarps),
                                   dim3(kJoinWarps * 32), 0, s, static_cast<const float *>(a.parts),
                                   static_cast<const Cut *>(a.cuts), a.out, a.Hq, a.G));
  return pkv::ok();
}

// Units of 128 columns where the rows have more than 64, by the packed nodes a row: the keys of
// a row are then read half as often (16 rows of 1k to 3k tokens, 8 heads of 128: trees of 64
// 90 -> 78 us, of 32 58 -> 52, since then 67 and 43). At D >= 256 units have 64: at 512 TMEM holds
// no more, at 256 it would hold one buffer of S and shared memory three entries (16 rows of up to
// 8k tokens with trees of 64 82 us, not 84, in a window of 512 trees of 16 31, not 28).
template <int D>
int launch_for(const pkv_bf16 *q, const pkv_bf16 *k, const pkv_bf16 *v, const Args &a,
               void *workspace, cudaStream_t s) {
  if (D <= 128 && static_cast<long long>(a.N) * a.G > 64LL * a.B)
    return launch<D, D <= 128 ? 128 : 64>(q, k, v, a, workspace, s);
  return launch<D, 64>(q, k, v, a, workspace, s);
}

size_t record_floats(int D) { return static_cast<size_t>(D <= 128 ? 128 : 64) * (D + 2); }

}  // namespace

extern "C" size_t paged_tree_attn_workspace(int Hq, int Hkv, int D) {
  if ((D != 64 && D != 128 && D != 256 && D != 512) || Hkv < 1 || Hq < Hkv || Hq % Hkv ||
      Hq / Hkv > 8 || Hq > 65535)
    return 0;
  return kArrivedBytes + kMaxCtas * sizeof(Cut) + 2 * kMaxCtas * record_floats(D) * sizeof(float);
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
  Args a = {};
  a.table = dev_table;
  a.batch_idx = batch_idx;
  a.ctx_lens = ctx_lens;
  a.row_start = row_start;
  a.parents = parents;
  a.out = reinterpret_cast<__nv_bfloat16 *>(out);
  a.err = err_word;
  a.n_slots = n_slots;
  a.max_pages = max_pages_per_seq;
  a.page_size = page_size;
  for (a.log_page = 0; (1 << a.log_page) < page_size;) ++a.log_page;
  a.n_pages = n_pages;
  a.window = window;
  a.B = B;
  a.N = N;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.scale_log2 = scale * 1.4426950408889634f;
  return D == 64    ? launch_for<64>(q, k_cache, v_cache, a, workspace, s)
         : D == 128 ? launch_for<128>(q, k_cache, v_cache, a, workspace, s)
         : D == 256 ? launch_for<256>(q, k_cache, v_cache, a, workspace, s)
                    : launch_for<512>(q, k_cache, v_cache, a, workspace, s);
}
