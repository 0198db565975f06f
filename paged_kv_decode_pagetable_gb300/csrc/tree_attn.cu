// paged_tree_attn: attention of every row's tree of drafted tokens over the paged cache.
//
//   out[t][h] = sum_j softmax_j(scale q[t][h] . k_j) v_j
// over the keys j < ctx of the context and, among the row's own nodes (at cache positions ctx ..),
// those on t's path to its root, t included; with a window W only keys less than W positions
// behind t (a node's position is ctx + its depth).
//
// Bound by reading each key and value of a row's context once for all its nodes and the query
// heads of a kv head, until nodes x heads reach a few hundred; those "columns" (at most 128 of
// them a unit, 64 where D > 128) are the N of both products, so that a small tree costs no
// more arithmetic than it has columns:
//   S^T = K q^T    M = 128 keys of a tile, N columns, both operands K-major,
//   O^T = V^T P^T  M = 128 columns of D, N columns, K = the tile's 128 keys, both MN-major: V as
//                  it lies in the cache, P as the threads write it, a key's columns in a row.
// In S^T a thread owns a key. Its columns' maxima run across threads, so they are not taken
// tile by tile: a column keeps a reference, every thread checks that none of its scores passes
// it by more than 2^8, and only where one does (a unit's first tile, and few others) the maxima
// are reduced, the references moved and O scaled. The sums of the weights stay per thread until
// a unit's end.
//
// Work: the units' tiles, one more place for each unit's start, lie on one line, cut into equal
// shares for one persistent CTA an SM from the lengths, on the device. A unit that is cut leaves
// its parts (O, reference and sum, fp32) in the workspace and a second small kernel joins them
// in order, so results do not depend on timing and no CTA waits for another.
//   warps 0-7 (softmax): warp w the keys of TMEM lanes 32 (w % 4) .. and half w / 4 of the
//     columns; masks, weights, references, a unit's output or part;
//   warp 8: K and V tiles by TMA, one box a page and 64 columns, into a ring of [128 keys][128
//     columns of D] in the order in which the MMAs use them up: K(0), K(1), V(0), K(2), V(1) ..;
//   warp 9: the MMAs, S one tile ahead of P V;
//   warp 10: a unit's queries by TMA, and which nodes see a key: sets of 64 bits, from the
//     parents by pointer doubling.
// Rows of V that no node sees are cleared in shared memory (0 x NaN would reach every column);
// one that is not finite and seen by some nodes only is cleared too and those nodes' results
// are NaN, as theirs are: nothing of it reaches the others.
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
constexpr int kSoftWarps = 8;
constexpr int kProdWarp = 8, kMmaWarp = 9, kPrepWarp = 10;
constexpr int kThreads = 11 * 32;
constexpr int kStart = 1;                // places on the line for a unit's start
constexpr int kMaxCtas = 160;            // CTAs the workspace has room for
constexpr float kLazyLog2 = 8.f;
constexpr float kUnset = 1e30f;          // stands for -reference of a column without one
constexpr int kJoinCols = 8;             // columns of a joining CTA

template <int D>
struct Cfg {
  static constexpr int COLS = D <= 128 ? 128 : 64;      // columns of a unit, at most
  static constexpr int HALF = COLS / 2;                 // of a softmax warp
  static constexpr int BLOCKS = D <= 128 ? 1 : D / 128; // ring entries of a K or V tile
  static constexpr int ATOMS = D == 64 ? 1 : 2;         // 64-column atoms of an entry
  static constexpr int ATOM = kTile * 128;              // bytes
  static constexpr int ENTRY = ATOMS * ATOM;
  static constexpr int NS = D == 64 ? 8 : D == 256 ? 5 : 4;
  static constexpr int Q_ATOM = COLS * 128;
  static constexpr int OFF_Q = NS * ENTRY;
  static constexpr int OFF_P = OFF_Q + (D / 64) * Q_ATOM;
  static constexpr int P_ATOM = kTile * 128;            // 64 columns of every key
  static constexpr int OFF_PREP = OFF_P + (COLS / 64) * P_ATOM;
  static constexpr int S_COL = 0, O_COL = 2 * COLS;
  static constexpr int TMEM_COLS = O_COL + BLOCKS * COLS <= 256 ? 256 : 512;
  static constexpr size_t RECORD = static_cast<size_t>(COLS) * (D + 2);   // floats of a part
};

// Which nodes see a key, of a unit's row.
struct Prep {
  uint64_t below[kTreeMax];    // nodes that have node i on their path
  uint64_t shallow[kTreeMax];  // nodes of depth <= i
  int depth[kTreeMax];
  unsigned poison[2];          // nodes that see a value that is not finite
};

// A unit cut into parts, for the joining kernel.
struct Cut {
  int token0, cols, head, parts;
};

struct Small {
  Prep prep[2];
  long long pre[kTreeRows + 1];     // first place of every row on the line
  int n0[kTreeRows], ctx[kTreeRows];
  uint8_t n[kTreeRows];
  float ref[128];                   // a column's reference, -inf: none yet
  alignas(16) float mneg[128];                  // its negative, kUnset: none yet
  float alpha[128];
  float red[4][128];                // of the four warps of a half: maxima, sums
  int pages[2][16];
  long long scan[kThreads / 32];
  uint64_t bars[48];
  uint32_t tmem;
  int abort;
};

template <int D>
constexpr size_t smem_bytes() {
  return 1024 + Cfg<D>::OFF_PREP + sizeof(Small);
}
static_assert(smem_bytes<64>() <= 232448 && smem_bytes<128>() <= 232448 &&
                  smem_bytes<256>() <= 232448 && smem_bytes<512>() <= 232448,
              "shared memory");

struct Args {
  const int32_t *table, *batch_idx, *ctx_lens, *row_start, *parents;
  __nv_bfloat16 *out;
  float *parts;
  Cut *cuts;
  int32_t *err;
  int n_slots, max_pages, page_size, log_page, n_pages, window, B, N, Hq, Hkv, G, unit_tokens;
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
// barrier of the 128 threads of a half, and whether any of them says yes
__device__ __forceinline__ bool half_any(int half, bool mine) {
  uint32_t r;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.b32 q, %1, 0;\n"
      "barrier.cta.red.or.pred p, %2, 128, q;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(mine)), "r"(1 + half)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void half_sync(int half) {
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + half) : "memory");
}

// A unit, or the part of it that this CTA has: tiles [t0, t1) of ntiles.
struct Part {
  int b, head, tok0, toks, n0, n, ctx, lo, tile0, ntiles, t0, t1;
  long long start;   // the unit's first place on the line
  __device__ bool whole() const { return t0 == 0 && t1 == ntiles; }
};

struct Line {
  const Small *sm;
  const Args *a;
  long long pos, end;
  int b;
  __device__ void begin(const Small &s, const Args &args, long long x0, long long x1) {
    sm = &s;
    a = &args;
    pos = x0;
    end = x1;
    int l = 0, r = args.B;   // the last row that starts at or before x0
    while (r - l > 1) {
      const int m = (l + r) / 2;
      if (s.pre[m] <= x0) l = m;
      else r = m;
    }
    b = l;
  }
  __device__ bool next(Part &p) {
    if (pos >= end) return false;
    while (pos >= sm->pre[b + 1]) ++b;
    p.b = b;
    p.n0 = sm->n0[b];
    p.n = sm->n[b] & 127;
    p.ctx = sm->ctx[b];
    p.lo = a->window > 0 ? max(0, p.ctx - a->window + 1) : 0;
    p.tile0 = p.lo / kTile;
    p.ntiles = sm->n[b] & 128 ? 0 : (p.ctx + p.n - 1) / kTile - p.tile0 + 1;
    const int cost = p.ntiles + kStart;
    const long long local = pos - sm->pre[b];
    const long long u = (local >> 31) ? local / cost
                                      : static_cast<uint32_t>(local) / static_cast<uint32_t>(cost);
    const int off = static_cast<int>(local - u * cost);
    const int units = (p.n + a->unit_tokens - 1) / a->unit_tokens;
    p.head = static_cast<int>(u) / units;
    p.tok0 = (static_cast<int>(u) - p.head * units) * a->unit_tokens;
    p.toks = min(a->unit_tokens, p.n - p.tok0);
    const int to = static_cast<int>(min(static_cast<long long>(cost), off + (end - pos)));
    p.t0 = max(0, off - kStart);
    p.t1 = max(0, to - kStart);
    p.start = pos - off;
    pos += to - off;
    return true;
  }
};

// first place of CTA c's share of W places among n CTAs
__device__ __forceinline__ long long share(long long W, int c, int n) { return W * c / n; }

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Args a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t raw[];
  uint8_t *sm = raw + ((1024u - (t_smem(raw) & 1023u)) & 1023u);
  Small &s = *reinterpret_cast<Small *>(sm + C::OFF_PREP);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;
  const uint32_t sRing = t_smem(sm), sQ = t_smem(sm + C::OFF_Q), sP = t_smem(sm + C::OFF_P);
  const uint32_t bars = t_smem(s.bars);
  const uint32_t full = bars, empty = full + 8 * C::NS, sfull = empty + 8 * C::NS,
                 sfree = sfull + 16, pfull = sfree + 16, pvdone = pfull + 8, ofree = pvdone + 8,
                 qfull = ofree + 8, qempty = qfull + 8, prepfull = qempty + 8,
                 prepempty = prepfull + 16, drain = prepempty + 16;
  volatile int *abort_flag = &s.abort;
  static_assert(2 * C::NS + 14 <= 48, "barriers");

  if (tid == 0) {
    for (int i = 0; i < C::NS; ++i) {
      t_bar_init(full + 8 * i, 1);
      t_bar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      t_bar_init(sfull + 8 * i, 1);
      t_bar_init(sfree + 8 * i, kSoftWarps);
      t_bar_init(prepfull + 8 * i, 1);
      t_bar_init(prepempty + 8 * i, kSoftWarps);
    }
    t_bar_init(pfull, kSoftWarps);
    t_bar_init(pvdone, 1);
    t_bar_init(ofree, kSoftWarps);
    t_bar_init(qfull, 1);
    t_bar_init(qempty, 1);
    t_bar_init(drain, 1);
    s.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     t_smem(&s.tmem)),
                 "r"(C::TMEM_COLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pkv_wait_prior_grid();
  pkv_allow_next_grid();

  // the line: places of every row, summed up over the rows
  {
    long long mine[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int b = 2 * tid + i;
      mine[i] = 0;
      if (b < a.B) {
        const TreeRow r = tree_row(b, a.N, a.row_start, a.batch_idx, a.ctx_lens, a.n_slots,
                                   a.max_pages, a.page_size);
        if (r.bits && cta == 0) tree_report(a.err, r.bits);
        s.n0[b] = r.n0;
        s.ctx[b] = r.ctx;
        // the top bit: padding, only zeros to write
        s.n[b] = static_cast<uint8_t>(r.n | (r.slot == 0 ? 128 : 0));
        if (r.n > 0) {
          const int lo = a.window > 0 ? max(0, r.ctx - a.window + 1) : 0;
          const int tiles = r.slot == 0 ? 0 : (r.ctx + r.n - 1) / kTile - lo / kTile + 1;
          mine[i] = static_cast<long long>(tiles + kStart) * a.Hkv *
                    ((r.n + a.unit_tokens - 1) / a.unit_tokens);
        }
      }
    }
    long long sum = mine[0] + mine[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) s.scan[warp] = sum;
    t_fence_before();
    __syncthreads();
    t_fence_after();
    for (int w = 0; w < warp; ++w) sum += s.scan[w];
    const int b = 2 * tid;
    if (b <= a.B) s.pre[b] = sum - mine[0] - mine[1];
    if (b + 1 <= a.B) s.pre[b + 1] = sum - mine[1];
    __syncthreads();
  }
  const uint32_t tmem = s.tmem;
  const long long W = s.pre[a.B];
  const int ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), W));
  const long long x0 = cta < ctas ? share(W, cta, ctas) : 0;
  const long long x1 = cta < ctas ? share(W, cta + 1, ctas) : 0;
  Line line;
  line.begin(s, a, x0, x1);
  Part p;
  if (tid == 0) a.cuts[cta].cols = 0;

  if (warp == kProdWarp) {
    // ============================ producer ============================
    const int box_rows = min(a.page_size, kTile);
    const int per_tile = kTile / box_rows;         // pages of a tile (1 where they are larger)
    int g = 0;                                     // ring entries so far
    int bits = 0;
    bool ok = true;
    // one K or V tile: its pages' boxes, BLOCKS entries
    auto load = [&](const CUtensorMap *tm, int which, int head, int j0, int first, int last) {
      const int row0 = j0 & (a.page_size - 1);     // (page_size > 128: place inside the page)
      for (int blk = 0; blk < C::BLOCKS && ok; ++blk, ++g) {
        const int e = g % C::NS;
        if (g >= C::NS && !t_wait_warp(empty + 8 * e, g / C::NS - 1, abort_flag)) {
          ok = false;
          break;
        }
        if (lane == 0)
          t_expect_tx(full + 8 * e, (last - first) * box_rows * 128 * C::ATOMS);
        __syncwarp();
        if (lane >= first && lane < last) {
          const int page = s.pages[which][lane];
          const int row = page * a.page_size + (per_tile == 1 ? row0 : 0);
#pragma unroll
          for (int at = 0; at < C::ATOMS; ++at)
            t_tma_4d(sRing + e * C::ENTRY + at * C::ATOM + lane * box_rows * 128, tm, 0, row, head,
                     blk * C::ATOMS + at, full + 8 * e);
        }
        __syncwarp();
      }
    };
    while (ok && line.next(p)) {
      if (p.t0 == p.t1) continue;
      const int slot = a.batch_idx ? a.batch_idx[p.b] : p.b;
      const int32_t *row = a.table + static_cast<long long>(slot) * a.max_pages;
      const int last_page = (p.ctx + p.n - 1) >> a.log_page;
      const int first_page = p.lo >> a.log_page;
      // page numbers 32 at a time, the next ones on their way
      const int base0 = ((p.tile0 + p.t0) * kTile) >> a.log_page;
      auto fetch = [&](int i) -> int {
        return i >= first_page && i <= last_page ? row[i] : 0;
      };
      int base = base0, now = fetch(base + lane), then = fetch(base + 32 + lane);
      int kf = 0, kl = 0;      // pages of the last K tile that are there
      for (int t = p.t0; t <= p.t1 && ok; ++t) {
        const int pf = kf, pl = kl;
        if (t < p.t1) {
          const int j0 = (p.tile0 + t) * kTile;
          const int page0 = j0 >> a.log_page;
          if (page0 >= base + 32) {
            base += 32;
            now = then;
            then = fetch(base + 32 + lane);
          }
          kf = max(0, first_page - page0);
          kl = min(per_tile, last_page - page0 + 1);
          int page = __shfl_sync(0xffffffffu, now, (page0 - base + lane) & 31);
          if (lane >= kf && lane < kl) {
            if (page < 0 || page >= a.n_pages) {
              bits |= page < 0 ? PKV_ERR_PAGE_NEG : PKV_ERR_PAGE_RANGE;
              page = 0;
            }
            s.pages[t & 1][lane] = page;
          }
          __syncwarp();
          load(&tmK, t & 1, p.head, j0, kf, kl);
        }
        if (t > p.t0 && ok)
          load(&tmV, (t - 1) & 1, p.head, (p.tile0 + t - 1) * kTile, pf, pl);
      }
    }
    tree_report(a.err, bits);
    if (!ok || *abort_flag) {
      // what is on its way lands before the CTA leaves
      for (int i = max(0, g - C::NS); i < g; ++i) {
        for (int k = 0; k < kSpin && !t_test(full + 8 * (i % C::NS), i / C::NS); ++k) {
        }
      }
    }
  } else if (warp == kMmaWarp) {
    // ============================== MMA ===============================
    if (lane == 0) {
      int g = 0, tiles = 0, segs = 0, pv = 0;
      bool ok = true;
      auto entry = [&]() -> int {   // the next ring entry, once it is there
        const int e = g % C::NS;
        if (!t_wait(full + 8 * e, g / C::NS, abort_flag)) ok = false;
        return e;
      };
      while (ok && line.next(p)) {
        if (p.t0 == p.t1) continue;
        const int N = (p.toks * a.G + 31) & ~31;
        const uint32_t idS = idesc(N, false), idO = idesc(N, true);
        if (!t_wait(qfull, segs, abort_flag)) break;
        auto do_pv = [&](bool first) {
          if (!t_wait(pfull, pv, abort_flag)) ok = false;
          if (ok && first && segs >= 1 && !t_wait(ofree, segs - 1, abort_flag)) ok = false;
          for (int blk = 0; blk < C::BLOCKS && ok; ++blk, ++g) {
            const int e = entry();
            if (!ok) break;
            t_fence_after();
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k) {
              // (D = 64: rows 64 .. 127 of the product repeat rows 0 .. 63)
              const uint64_t va = t_desc(sRing + e * C::ENTRY + k * 2048,
                                         C::ATOMS == 1 ? 0 : C::ATOM, 1024);
              const uint64_t pb = t_desc(sP + k * 2048, C::P_ATOM, 1024);
              t_mma(tmem + C::O_COL + blk * C::COLS, va, pb, idO, (k > 0 || !first) ? 1u : 0u);
            }
            t_commit(empty + 8 * e);
          }
          if (ok) t_commit(pvdone);
          ++pv;
        };
        for (int t = p.t0; t < p.t1 && ok; ++t, ++tiles) {
          const int buf = tiles & 1;
          if (tiles >= 2 && !t_wait(sfree + 8 * buf, (tiles >> 1) - 1, abort_flag)) {
            ok = false;
            break;
          }
          for (int blk = 0; blk < C::BLOCKS && ok; ++blk, ++g) {
            const int e = entry();
            if (!ok) break;
            t_fence_after();
#pragma unroll
            for (int k = 0; k < 4 * C::ATOMS; ++k) {
              const uint64_t ka =
                  t_desc(sRing + e * C::ENTRY + (k >> 2) * C::ATOM + (k & 3) * 32, 16, 1024);
              const uint64_t qb = t_desc(
                  sQ + (blk * C::ATOMS + (k >> 2)) * C::Q_ATOM + (k & 3) * 32, 16, 1024);
              t_mma(tmem + C::S_COL + buf * C::COLS, ka, qb, idS, (blk > 0 || k > 0) ? 1u : 0u);
            }
            t_commit(empty + 8 * e);
          }
          if (!ok) break;
          t_commit(sfull + 8 * buf);
          if (t == p.t1 - 1) t_commit(qempty);
          if (t > p.t0) do_pv(t == p.t0 + 1);
        }
        if (ok) do_pv(p.t1 - p.t0 == 1);
        ++segs;
      }
      t_commit(drain);
      t_wait_drain(drain);
    }
  } else if (warp == kPrepWarp) {
    // ====================== queries and who sees whom ======================
    int segs = 0, bits = 0;
    bool ok = true;
    const int box = 8 * a.G * 128;      // bytes of 8 nodes' heads, one atom
    while (ok && line.next(p)) {
      if (p.t0 == p.t1) continue;
      if (segs >= 1 && !t_wait_warp(qempty, segs - 1, abort_flag)) break;
      if (lane == 0) {
        const int boxes = (p.toks + 7) / 8;
        t_expect_tx(qfull, boxes * box * (D / 64));
        for (int i = 0; i < boxes; ++i)
          for (int at = 0; at < D / 64; ++at)
            t_tma_4d(sQ + at * C::Q_ATOM + i * box, &tmQ, 0, p.head * a.G, p.n0 + p.tok0 + 8 * i, at,
                     qfull);
      }
      Prep &w = s.prep[segs & 1];
      if (segs >= 2 && !t_wait_warp(prepempty + 8 * (segs & 1), (segs >> 1) - 1, abort_flag)) break;
      // paths: each node's set of ancestors and itself, twice as far every time
      uint64_t *path = w.below;
      int *jump = w.depth;
#pragma unroll
      for (int i = lane; i < kTreeMax; i += 32) {
        path[i] = 1ull << i;
        jump[i] = i < p.n ? tree_parent(a.parents, p.n0, i, bits) : -1;
      }
      __syncwarp();
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
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          path[lane + 32 * q] = v[q];
          jump[lane + 32 * q] = j[q];
        }
        __syncwarp();
        if (!more) break;
      }
      uint64_t below[2] = {0, 0}, shallow[2] = {0, 0};
      int depth[2];
      for (int t = 0; t < p.n; ++t) {
        const uint64_t v = path[t];
        const int d = __popcll(v) - 1;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int i = lane + 32 * q;
          below[q] |= ((v >> i) & 1) << t;
          shallow[q] |= static_cast<uint64_t>(d <= i) << t;
          if (t == i) depth[q] = d;
        }
      }
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        w.below[lane + 32 * q] = below[q];
        w.shallow[lane + 32 * q] = shallow[q];
        w.depth[lane + 32 * q] = lane + 32 * q < p.n ? depth[q] : 0;
      }
      if (lane < 2) w.poison[lane] = 0;
      __syncwarp();
      if (lane == 0) t_arrive(prepfull + 8 * (segs & 1));
      ++segs;
    }
    tree_report(a.err, bits);
  } else {
    // ============================ softmax =============================
    const int quad = warp & 3, half = warp >> 2;
    const int row = 32 * quad + lane;           // the key of a tile, or the column of D
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * quad) << 16);
    int tiles = 0, segs = 0, g = 0;             // g: ring entries of the units so far
    bool ok = true, gone = false;
    float l[C::HALF];
    while (!gone && line.next(p)) {
      const int cols = p.toks * a.G;
      if (p.ntiles == 0) {                      // padding
        for (int i = warp; i < cols; i += kSoftWarps) {
          const long long o = (static_cast<long long>(p.n0 + p.tok0 + i / a.G) * a.Hq +
                               p.head * a.G + i % a.G) * D;
          for (int d = 2 * lane; d < D; d += 64)
            *reinterpret_cast<uint32_t *>(a.out + o + d) = 0;
        }
        continue;
      }
      if (p.t0 == p.t1) continue;
      const int N = (cols + 31) & ~31;
      const int hn = N / 2, c0 = half * hn;     // this warp's columns c0 .. c0 + hn
      // (in shared memory from h0 on: the halves may be at different units)
      const int h0 = half * C::HALF;
      Prep &w = s.prep[segs & 1];
      const int nt = p.t1 - p.t0;
      bool any_masked = false;
#pragma unroll
      for (int c = 0; c < C::HALF; ++c) l[c] = 0.f;
      for (int t = p.t0; t < p.t1; ++t, ++tiles) {
        const int buf = tiles & 1, i = t - p.t0;
        const int j0 = (p.tile0 + t) * kTile, j = j0 + row;
        const bool masked = j0 + kTile > p.ctx ||
                            (a.window > 0 && j0 <= p.ctx + p.n - 1 - a.window);
        const bool first = i == 0;
        uint64_t sees = ~0ull;                  // nodes that see this thread's key
        any_masked |= masked;
        if (masked) {
          ok = ok && t_wait_warp(prepfull + 8 * (segs & 1), segs >> 1, abort_flag);
          const int node = j - p.ctx;
          if (node >= p.n) sees = 0;
          else if (node >= 0) {
            sees = w.below[node];
            if (a.window > 0)
              sees &= w.shallow[min(static_cast<long long>(kTreeMax - 1),
                                    static_cast<long long>(w.depth[node]) + a.window - 1)];
          } else if (a.window > 0) {
            const int d = node + a.window - 1;
            sees = d < 0 ? 0 : w.shallow[min(d, kTreeMax - 1)];
          }
          sees >>= p.tok0;
        }
        ok = ok && t_wait_warp(sfull + 8 * buf, tiles >> 1, abort_flag);
        t_fence_after();
        const uint32_t scol = trow + C::S_COL + buf * C::COLS + c0;
        // 16 scores of this thread's key, -inf where a node does not see it
        auto scores = [&](int c, float (&x)[16]) {
          uint32_t r[16];
          t_ld16(scol + c, r);
          t_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(r[e]);
          if (masked) {
            int tok = (c0 + c) / a.G, k = (c0 + c) - tok * a.G;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              if (!((sees >> (tok & 63)) & 1)) x[e] = -INFINITY;
              if (++k == a.G) {
                k = 0;
                ++tok;
              }
            }
          }
        };
        uint32_t pk[C::HALF / 2];
        // the weights under the references at hand; whether one is out of reach
        auto weights = [&]() -> bool {
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < C::HALF; c += 16) {
            if (c < hn) {
              float x[16];
              scores(c, x);
              const float4 *m4 = reinterpret_cast<const float4 *>(s.mneg + h0 + c);
#pragma unroll
              for (int e = 0; e < 16; e += 4) {
                const float4 m = m4[e / 4];
                fma2(x[e], x[e + 1], x[e], x[e + 1], a.scale_log2, m.x, m.y);
                fma2(x[e + 2], x[e + 3], x[e + 2], x[e + 3], a.scale_log2, m.z, m.w);
                top = t_max3(top, x[e], x[e + 1]);
                top = t_max3(top, x[e + 2], x[e + 3]);
              }
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                x[e] = t_ex2(x[e]);
                x[e + 1] = t_ex2(x[e + 1]);
                pk[(c + e) / 2] = t_pack(x[e], x[e + 1]);
              }
            }
          }
          return top > kLazyLog2;
        };
        bool slow = first;
        if (!first) slow = ok && weights();
        if (half_any(half, slow || !ok)) {
          if (half_any(half, !ok)) {
            gone = true;
            break;
          }
          // the columns' maxima over the tile
#pragma unroll
          for (int c = 0; c < C::HALF; c += 16) {
            if (c < hn) {
              float x[16];
              scores(c, x);
              // 16 columns over 32 lanes: halves change places until a lane pair has one
#pragma unroll
              for (int o = 16, n = 8; o >= 2; o >>= 1, n >>= 1) {
                const bool up = lane & o;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  if (e < n) {
                    const float give = up ? x[e] : x[e + n];
                    const float got = __shfl_xor_sync(0xffffffffu, give, o);
                    x[e] = fmaxf(up ? x[e + n] : x[e], got);
                  }
                }
              }
              const float v = fmaxf(x[0], __shfl_xor_sync(0xffffffffu, x[0], 1));
              const int col = (lane & 16 ? 8 : 0) + (lane & 8 ? 4 : 0) + (lane & 4 ? 2 : 0) +
                              (lane & 2 ? 1 : 0);
              if (!(lane & 1)) s.red[quad][h0 + c + col] = v;
            }
          }
          half_sync(half);
          if (32 * quad + lane < hn) {
            const int c = h0 + 32 * quad + lane;
            const float old = first ? -INFINITY : s.ref[c];
            const float top = fmaxf(fmaxf(s.red[0][c], s.red[1][c]),
                                    fmaxf(s.red[2][c], s.red[3][c])) * a.scale_log2;
            const float ref = fmaxf(old, top);
            s.ref[c] = ref;
            s.mneg[c] = ref == -INFINITY ? kUnset : -ref;
            s.alpha[c] = old == ref ? 1.f : exp2f(old - ref);
          }
          half_sync(half);
          if (!first) {
            ok = t_wait_warp(pvdone, tiles - 1, abort_flag);
            t_fence_after();
            if (ok) {
#pragma unroll
              for (int c = 0; c < C::HALF; c += 16) {
                if (c < hn) {
                  float al[16];
#pragma unroll
                  for (int e = 0; e < 16; ++e) al[e] = s.alpha[h0 + c + e];
#pragma unroll
                  for (int e = 0; e < 16; ++e) l[c + e] *= al[e];
                  for (int blk = 0; blk < C::BLOCKS; ++blk) {
                    uint32_t r[16];
                    const uint32_t at = trow + C::O_COL + blk * C::COLS + c0 + c;
                    t_ld16(at, r);
                    t_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                      r[e] = __float_as_uint(__uint_as_float(r[e]) * al[e]);
                    t_st16(at, r);
                  }
                }
              }
              t_wait_st();
            }
          }
          weights();
        }
        // the sums of the weights as they enter the product
#pragma unroll
        for (int c = 0; c < C::HALF; c += 2) {
          if (c < hn)
            t_add2(l[c], l[c + 1], __uint_as_float(pk[c / 2] << 16),
                   __uint_as_float(pk[c / 2] & 0xffff0000u));
        }
        t_fence_before();
        __syncwarp();
        if (lane == 0) t_arrive(sfree + 8 * buf);
        if (tiles >= 1) ok = ok && t_wait_warp(pvdone, tiles - 1, abort_flag);
        // this key's columns in a row of 128 bytes for each 64, as the swizzle has them
#pragma unroll
        for (int c = 0; c < C::HALF; c += 8) {
          if (c < hn) {
            const int col = c0 + c;
            uint8_t *to = sm + C::OFF_P + (col >> 6) * C::P_ATOM + row * 128 +
                          ((((col & 63) >> 3) ^ (row & 7)) << 4);
            *reinterpret_cast<uint4 *>(to) =
                make_uint4(pk[c / 2], pk[c / 2 + 1], pk[c / 2 + 2], pk[c / 2 + 3]);
          }
        }
        if (masked) {
          // the tile's V entries: V(i) stands behind K(i + 1) in the ring. Rows seen by no node
          // are cleared, and those seen by some only if they are not finite
          const int e0 = g + (2 * i + (i == nt - 1 ? 1 : 2)) * C::BLOCKS;
          const uint64_t unit = ~0ull >> (kTreeMax - p.toks);
          const bool some = (sees & unit) != 0, all = (sees & unit) == unit;
          // a phase is told from the one before only, so the entries' previous tiles have to be
          // there: they stand at or before K(i) or V(i - 1) in the ring, whose products are done,
          // but for rings no longer than a tile, where they are K(i + 1)
          static_assert(C::NS == C::BLOCKS || C::NS > 2 * C::BLOCKS, "previous tiles");
          if (C::NS == C::BLOCKS && i < nt - 1)
            ok = ok && t_wait_warp(sfull + 8 * (buf ^ 1), (tiles + 1) >> 1, abort_flag);
          bool bad = false;
          for (int blk = 0; blk < C::BLOCKS; ++blk) {
            const int n = e0 + blk, e = n % C::NS, k = n / C::NS;
            ok = ok && t_wait_warp(full + 8 * e, k, abort_flag);
            // each half one atom; D = 64 has one, shared by halves of its row
            constexpr int WORDS = C::ATOMS == 1 ? 4 : 8;
            uint8_t *v = sm + e * C::ENTRY + (C::ATOMS == 1 ? 0 : half * C::ATOM) + row * 128 +
                         (C::ATOMS == 1 ? half * 64 : 0);
            if (some && !all) {
#pragma unroll
              for (int x = 0; x < WORDS; ++x) {
                const uint4 y = *reinterpret_cast<const uint4 *>(v + 16 * x);
                const uint32_t u[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int z = 0; z < 4; ++z)
                  bad |= (u[z] & 0x7f80u) == 0x7f80u || (u[z] & 0x7f800000u) == 0x7f800000u;
              }
            }
          }
          if (bad) {
            const uint64_t who = (sees & unit) << p.tok0;
            atomicOr(&w.poison[0], static_cast<unsigned>(who));
            atomicOr(&w.poison[1], static_cast<unsigned>(who >> 32));
          }
          if ((bad || !some) && ok) {
            for (int blk = 0; blk < C::BLOCKS; ++blk) {
              const int e = (e0 + blk) % C::NS;
              constexpr int WORDS = C::ATOMS == 1 ? 4 : 8;
              uint8_t *v = sm + e * C::ENTRY + (C::ATOMS == 1 ? 0 : half * C::ATOM) + row * 128 +
                           (C::ATOMS == 1 ? half * 64 : 0);
              for (int x = 0; x < WORDS; ++x)
                *reinterpret_cast<uint4 *>(v + 16 * x) = make_uint4(0, 0, 0, 0);
            }
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        t_fence_before();
        __syncwarp();
        if (lane == 0) t_arrive(pfull);
      }
      if (gone) break;
      g += 2 * nt * C::BLOCKS;
      // the weights' sums of the columns, over the lanes and the half's warps
#pragma unroll
      for (int c = 0; c < C::HALF; c += 16) {
        if (c < hn) {
          float x[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = l[c + e];
#pragma unroll
          for (int o = 16, n = 8; o >= 2; o >>= 1, n >>= 1) {
            const bool up = lane & o;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if (e < n) {
                const float give = up ? x[e] : x[e + n];
                x[e] = (up ? x[e + n] : x[e]) + __shfl_xor_sync(0xffffffffu, give, o);
              }
            }
          }
          const float v = x[0] + __shfl_xor_sync(0xffffffffu, x[0], 1);
          const int col = (lane & 16 ? 8 : 0) + (lane & 8 ? 4 : 0) + (lane & 4 ? 2 : 0) +
                          (lane & 2 ? 1 : 0);
          if (!(lane & 1)) s.red[quad][h0 + c + col] = v;
        }
      }
      ok = ok && t_wait_warp(pvdone, tiles - 1, abort_flag);
      t_fence_after();
      half_sync(half);
      const bool whole = p.whole();
      const int place = 2 * cta + (p.t0 == 0 ? 1 : 0);
      float *rec = a.parts + place * C::RECORD;
      if (32 * quad + lane < hn) {
        const int c = c0 + 32 * quad + lane, k = h0 + 32 * quad + lane;
        float sum = (s.red[0][k] + s.red[1][k]) + (s.red[2][k] + s.red[3][k]);
        if (c < cols) {
          const int tok = p.tok0 + c / a.G;
          if (any_masked && (w.poison[tok >> 5] >> (tok & 31) & 1)) sum = NAN;
          if (!whole) {
            rec[C::COLS * D + c] = s.ref[k];
            rec[C::COLS * (D + 1) + c] = sum;
          }
        }
        s.alpha[k] = sum == 0.f ? 0.f : 1.f / sum;
      }
      half_sync(half);
      if (ok) {
#pragma unroll
        for (int blk = 0; blk < C::BLOCKS; ++blk) {
          const int d = blk * 128 + row;
#pragma unroll 1
          for (int c = 0; c < hn; c += 16) {
            uint32_t r[16];
            t_ld16(trow + C::O_COL + blk * C::COLS + c0 + c, r);
            t_wait_ld();
            if (D == 64 && quad >= 2) continue;
            if (whole) {
              // two columns a step: even lanes store one, odd lanes the other, two places each
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                const int col = c0 + c + e;
                const float y0 = __uint_as_float(r[e]) * s.alpha[h0 + c + e];
                const float y1 = __uint_as_float(r[e + 1]) * s.alpha[h0 + c + e + 1];
                const float got = __shfl_xor_sync(0xffffffffu, lane & 1 ? y0 : y1, 1);
                const int mine = col + (lane & 1);
                const uint32_t v = lane & 1 ? t_pack(got, y1) : t_pack(y0, got);
                if (mine < cols) {
                  const int tok = mine / a.G;
                  const long long o = static_cast<long long>(p.n0 + p.tok0 + tok) * a.Hq +
                                      p.head * a.G + (mine - tok * a.G);
                  *reinterpret_cast<uint32_t *>(a.out + o * D + (d & ~1)) = v;
                }
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
      if (tid == 0 && !whole && p.t0 == 0) {
        // the CTA of the unit's last tile
        const long long at = p.start + kStart + p.ntiles - 1;
        int c = static_cast<int>(at * ctas / W);
        while (c > 0 && share(W, c, ctas) > at) --c;
        while (share(W, c + 1, ctas) <= at) ++c;
        Cut cut = {p.n0 + p.tok0, cols, p.head, c - cta + 1};
        a.cuts[cta] = cut;
      }
      t_fence_before();
      __syncwarp();
      if (lane == 0) {
        t_arrive(ofree);
        t_arrive(prepempty + 8 * (segs & 1));
      }
      ++segs;
    }
    if ((gone || !ok) && lane == 0) tree_report(a.err, PKV_ERR_TIMEOUT);
  }
  t_fence_before();
  __syncthreads();
  t_fence_after();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(C::TMEM_COLS));
}

// Joins the parts of the unit that CTA blockIdx.x began and others went on with: a warp a column.
template <int D>
__global__ void __launch_bounds__(kJoinCols * 32)
    tree_join_kernel(const float *parts, const Cut *cuts, __nv_bfloat16 *out, int Hq, int G) {
  using C = Cfg<D>;
  pkv_wait_prior_grid();
  pkv_allow_next_grid();
  const Cut cut = cuts[blockIdx.x];
  const int col = blockIdx.y * kJoinCols + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (col >= cut.cols) return;
  auto rec = [&](int i) -> const float * {
    return parts + (2 * (blockIdx.x + i) + (i == 0 ? 1 : 0)) * C::RECORD;
  };
  float m = -INFINITY;
  for (int i = lane; i < cut.parts; i += 32) m = fmaxf(m, rec(i)[C::COLS * D + col]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (m == -INFINITY) m = 0.f;
  constexpr int E = D / 32;
  float x[E], l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = 0.f;
  for (int i = 0; i < cut.parts; ++i) {
    const float *r = rec(i);
    const float w = exp2f(r[C::COLS * D + col] - m);
    l = fmaf(w, r[C::COLS * (D + 1) + col], l);
    const float *y = r + col * D + (E == 2 ? 2 : 4) * lane;
#pragma unroll
    for (int e = 0; e < E; e += (E == 2 ? 2 : 4)) {
      if (E == 2) {
        const float2 v = *reinterpret_cast<const float2 *>(y);
        x[0] = fmaf(w, v.x, x[0]);
        x[1] = fmaf(w, v.y, x[1]);
      } else {
        const float4 v = *reinterpret_cast<const float4 *>(y + 32 * e);
        x[e] = fmaf(w, v.x, x[e]);
        x[e + 1] = fmaf(w, v.y, x[e + 1]);
        x[e + 2] = fmaf(w, v.z, x[e + 2]);
        x[e + 3] = fmaf(w, v.w, x[e + 3]);
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int tok = col / G;
  __nv_bfloat16 *o = out + (static_cast<long long>(cut.token0 + tok) * Hq + cut.head * G +
                            (col - tok * G)) * D;
  if (E == 2) {
    *reinterpret_cast<uint32_t *>(o + 2 * lane) = t_pack(x[0] * inv, x[1] * inv);
  } else {
#pragma unroll
    for (int e = 0; e < E; e += 4)
      *reinterpret_cast<uint2 *>(o + 32 * e + 4 * lane) =
          make_uint2(t_pack(x[e] * inv, x[e + 1] * inv), t_pack(x[e + 2] * inv, x[e + 3] * inv));
  }
}

template <int D>
int launch(const pkv_bf16 *q, const pkv_bf16 *k, const pkv_bf16 *v, Args a, void *workspace,
           cudaStream_t s) {
  using C = Cfg<D>;
  static std::mutex mu;
  static bool done[64] = {false};
  int dev = 0;
  PKV_CUDA_CHECK(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return pkv::fail(PKV_E_CUDA, "device id out of range");
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      PKV_CUDA_CHECK(cudaFuncSetAttribute(tree_attn_kernel<D>,
                                          cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          static_cast<int>(smem_bytes<D>())));
      done[dev] = true;
    }
  }
  const int sms = pkv::sm_count();
  const int grid = sms < 1 ? 1 : sms < kMaxCtas ? sms : kMaxCtas;
  a.unit_tokens = C::COLS / (8 * a.G) * 8;
  a.cuts = static_cast<Cut *>(workspace);
  a.parts = reinterpret_cast<float *>(static_cast<char *>(workspace) + kMaxCtas * sizeof(Cut));
  CUtensorMap tmQ, tmK, tmV;
  const int rows = a.n_pages * a.page_size, box = a.page_size < kTile ? a.page_size : kTile;
  int st = pkv::prefill_atoms_map(&tmQ, q, a.N, a.Hq, D, a.G, 8, 1);
  if (st == PKV_OK) st = pkv::prefill_atoms_map(&tmK, k, a.Hkv, rows, D, box, 1, 1);
  if (st == PKV_OK) st = pkv::prefill_atoms_map(&tmV, v, a.Hkv, rows, D, box, 1, 1);
  if (st != PKV_OK) return st;
  PKV_CUDA_CHECK(pkv::launch_pdl(tree_attn_kernel<D>, dim3(grid), dim3(kThreads), smem_bytes<D>(),
                                 s, tmQ, tmK, tmV, a));
  PKV_CUDA_CHECK(pkv::launch_pdl(tree_join_kernel<D>, dim3(grid, C::COLS / kJoinCols),
                                 dim3(kJoinCols * 32), 0, s, static_cast<const float *>(a.parts),
                                 static_cast<const Cut *>(a.cuts), a.out, a.Hq, a.G));
  return pkv::ok();
}

size_t record_floats(int D) {
  return D == 64    ? Cfg<64>::RECORD
         : D == 128 ? Cfg<128>::RECORD
         : D == 256 ? Cfg<256>::RECORD
                    : Cfg<512>::RECORD;
}

}  // namespace

extern "C" size_t paged_tree_attn_workspace(int Hq, int Hkv, int D) {
  if ((D != 64 && D != 128 && D != 256 && D != 512) || Hkv < 1 || Hq < Hkv || Hq % Hkv ||
      Hq / Hkv > 8 || Hq > 65535)
    return 0;
  return kMaxCtas * sizeof(Cut) + 2 * kMaxCtas * record_floats(D) * sizeof(float);
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
  return D == 64    ? launch<64>(q, k_cache, v_cache, a, workspace, s)
         : D == 128 ? launch<128>(q, k_cache, v_cache, a, workspace, s)
         : D == 256 ? launch<256>(q, k_cache, v_cache, a, workspace, s)
                    : launch<512>(q, k_cache, v_cache, a, workspace, s);
}
