// tree_verify: which drafted tokens stay, and the token behind them, from given random numbers.
//
// A row's walk starts at node 0. With p the target's probabilities after the current node, q the
// draft's, and its children in index order, after k refusals what the target has left is
//   w_k = max(p - a_k q, 0),  S_k = sum w_k,   a_0 = 0, S_0 = 1, a_{k+1} = a_k + S_k
// (subtracting q from the normalised w_k / S_k, max(w_k / S_k - q, 0) is w_{k+1} / S_k: the
// differences add up in the single number a). Child k with token x is accepted when
// u q(x) S_k < w_k(x), and the walk goes on from it; when no child is left, the next token is
// the least i with w(0) + .. + w(i) > u_pick S. Without q the drafts are certain ones (q is 1
// at x): w_k is p without the refused tokens, S_k = 1 - their sum.
// The scheme keeps the target's distribution if a node's children are independent samples of q
// (or, without q, any tokens that p does not depend on).
//
// Sums are kept in fixed point, in units of 2^-43: each probability is rounded to one once (fp32
// ones below 2^-20 lose up to 2^-44, far below what moves a threshold past a token), the sums
// are whole numbers. So they do not depend on how the vocabulary is divided, and the row's CTAs,
// which all do the same walk, cannot disagree on a decision.
//
// Bound by reading the last node's row of p (and of q where something was refused) once: a pass
// over a row is one of the target's V words. A cluster of up to 8 CTAs shares a row: each sums
// a contiguous part, the sums cross through distributed shared memory, and the warp whose part
// holds the threshold reads the group of words with it again for the token. Measured (floors at
// 6769 GB/s): 64 rows of 5 sampled drafts, 151936 words, 20.1 us (11.5), where a row's 4 CTAs meet
// after each pass; 16 trees of the likeliest tokens, 262144 words, 12.2 us (2.5): a chain of
// dependent steps down the path, each a few words, then one pass; one row of 3 drafts, 32000
// words, 6.5 us. With 64-bit conversions for the sums and a search through a warp's whole part the
// 64 rows took 44 us.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "pkv_internal.h"
#include "tree.cuh"

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kUnit = 128;      // words a warp reads at a time: four a lane
constexpr int kDeep = 4;        // such reads in flight
constexpr int kGroups = 32;     // sums that a warp keeps of its part
constexpr int kBits = 43;       // sums are in units of 2^-43
constexpr double kUnitSize = 1.0 / (1ull << kBits);
constexpr uint64_t kMaxA = uint64_t(127) << kBits;   // a stays below 2^7 (64 refusals of 1)

struct VerifyArgs {
  const float *p, *q;
  long long sp, sq;   // words from one row to the next
  const int32_t *tokens, *row_start, *parents;
  const float *u_accept, *u_pick;
  int32_t *accepted, *path, *next, *err;
  int N, V, path_cols;
};

// probabilities outside [0, 1] and NaN count as the nearest of the two ends (NaN as 0)
__device__ __forceinline__ float clean(float x) { return __saturatef(x); }

// x in [0, 1] in units of 2^-43, to the nearest, in two steps of fp32: added to 12, whose last
// place is 2^-20, x leaves its rounding to that in the sum's last bits; what remains, exact, is
// scaled and added to 1.5 * 2^23, whose last place is 1. hi and lo take the sums' bits, each
// kHi0 or kLo0 too large.
constexpr int kHi0 = 0x41400000, kLo0 = 0x4b400000;
__device__ __forceinline__ void fixed(float x, int &hi, int &lo) {
  const float y = __fadd_rn(x, 12.f);
  const float rest = __fsub_rn(x, __fsub_rn(y, 12.f));
  hi = __float_as_int(y);
  lo = __float_as_int(__fmaf_rn(rest, 0x1p43f, 0x1.8p23f));
}
__device__ __forceinline__ int64_t fixed(float x) {
  int hi, lo;
  fixed(x, hi, lo);
  return (static_cast<int64_t>(hi - kHi0) << 23) + (lo - kLo0);
}

// How a pass weighs a token: p itself, p - q (a = 1, the first refusal), or p - a q; none below 0.
enum { kPlain = 0, kFirst = 1, kLater = 2 };
template <int KIND>
__device__ __forceinline__ uint64_t weight(float p, float q, uint64_t a) {
  p = clean(p), q = clean(q);
  if (KIND == kPlain) return fixed(p);
  if (KIND == kFirst) return p > q ? fixed(p) - fixed(q) : 0;
  const uint64_t w = fixed(p), f = __umul64hi(static_cast<uint64_t>(fixed(q)) << 14, a << 7);
  return w > f ? w - f : 0;
}

// Adds the weights of N tokens to s.
template <int KIND, int N>
__device__ __forceinline__ void add_weights(const float (&p)[N], const float (&q)[N], uint64_t a,
                                            uint64_t &s) {
  if (KIND == kLater) {
#pragma unroll
    for (int i = 0; i < N; ++i) s += weight<KIND>(p[i], q[i], a);
    return;
  }
  int hi = 0, lo = 0;   // (terms up to 2^20 and 2^23)
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float x = clean(p[i]);
    int h, l;
    if (KIND == kFirst) {
      const float y = clean(q[i]);
      const bool more = x > y;
      int h2, l2;
      fixed(more ? x : 0.f, h, l);
      fixed(more ? y : 0.f, h2, l2);
      hi += h - h2;
      lo += l - l2;
    } else {
      fixed(x, h, l);
      hi += h - kHi0;
      lo += l - kLo0;
    }
  }
  s += (static_cast<int64_t>(hi) << 23) + lo;
}

struct Row {
  const float *p, *q;
  bool vec_p, vec_q;
};

// Four consecutive words of a row from index i on, 0 past V.
__device__ __forceinline__ float4 four(const float *row, bool vec, int i, int V) {
  if (vec && i + 3 < V) return __ldg(reinterpret_cast<const float4 *>(row + i));
  float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
  if (i < V) r.x = __ldg(row + i);
  if (i + 1 < V) r.y = __ldg(row + i + 1);
  if (i + 2 < V) r.z = __ldg(row + i + 2);
  if (i + 3 < V) r.w = __ldg(row + i + 3);
  return r;
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}
__device__ __forceinline__ uint64_t warp_before(uint64_t s, int lane) {   // exclusive scan
  uint64_t t = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t v = __shfl_up_sync(0xffffffffu, t, o);
    if (lane >= o) t += v;
  }
  return t - s;
}

struct Shared {
  int tok[kTreeMax], par[kTreeMax];
  float p[kTreeMax], q[kTreeMax], u[kTreeMax];
  int path[kTreeMax];
  int gone[kTreeMax];              // refused tokens of the current node (drafts without q)
  uint64_t group[kWarps][kGroups]; // sums of the groups of units of this CTA's warps
  uint64_t warp[kWarps];           // and of the warps
  uint64_t rank[2][kMaxCluster];   // sums of the row's CTAs, by turns
  uint64_t a;
  int node, n_gone, last, n_path;
};

// kDeep units from u on (below u1), all their reads in flight: what this lane has of them
template <int KIND>
__device__ __forceinline__ void read_units(const Row &r, int u, int u1, int V, int lane,
                                           float (&p)[4 * kDeep], float (&q)[4 * kDeep]) {
#pragma unroll
  for (int d = 0; d < kDeep; ++d) {
    const int i = u + d < u1 ? (u + d) * kUnit + 4 * lane : V;
    const float4 x = four(r.p, r.vec_p, i, V);
    p[4 * d] = x.x, p[4 * d + 1] = x.y, p[4 * d + 2] = x.z, p[4 * d + 3] = x.w;
    if (KIND != kPlain) {
      const float4 y = four(r.q, r.vec_q, i, V);
      q[4 * d] = y.x, q[4 * d + 1] = y.y, q[4 * d + 2] = y.z, q[4 * d + 3] = y.w;
    }
  }
}

// Sums of the groups of `size` units that units [u0, u1) make up; returns their sum.
template <int KIND>
__device__ __forceinline__ uint64_t sum_units(const Row &r, uint64_t a, Shared &sh, int size,
                                              int u0, int u1, int V, int warp, int lane) {
  uint64_t total = 0;
  int g = 0;
  for (int first = u0; first < u1; first += size, ++g) {
    const int end = min(u1, first + size);
    uint64_t s = 0;
    for (int u = first; u < end; u += kDeep) {
      float p[4 * kDeep], q[4 * kDeep];
      read_units<KIND>(r, u, end, V, lane, p, q);
      add_weights<KIND>(p, q, a, s);
    }
    // refused tokens among them
    for (int k = lane; k < sh.n_gone; k += 32) {
      const int unit = sh.gone[k] / kUnit;
      if (unit >= first && unit < end) s -= fixed(clean(r.p[sh.gone[k]]));
    }
    s = warp_sum(s);
    if (lane == 0) sh.group[warp][g] = s;
    total += s;
  }
  if (lane >= g) sh.group[warp][lane] = 0;
  return total;
}

// The token on which the threshold t falls, among the warp's units.
template <int KIND>
__device__ __forceinline__ int find(const Row &r, uint64_t a, const Shared &sh, uint64_t before,
                                    uint64_t t, int size, int u0, int u1, int V, int warp,
                                    int lane) {
  const uint64_t mine = sh.group[warp][lane];
  const uint64_t start = before + warp_before(mine, lane);
  const unsigned hit = __ballot_sync(0xffffffffu, t >= start && t < start + mine);
  if (!hit) return -1;
  const int g = __ffs(hit) - 1;
  before = __shfl_sync(0xffffffffu, start, g);
  const int first = u0 + g * size, end = min(u1, first + size);
  for (int u = first; u < end; u += kDeep) {
    float p[4 * kDeep], q[4 * kDeep];
    read_units<KIND>(r, u, end, V, lane, p, q);
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      const int i = (u + d) * kUnit + 4 * lane;
      uint64_t w[4], sum = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = weight<KIND>(p[4 * d + e], q[4 * d + e], a);
      for (int k = 0; k < sh.n_gone; ++k) {
        const int at = sh.gone[k] - i;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (at == e) w[e] = 0;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sum += w[e];
      uint64_t c = before + warp_before(sum, lane);
      int here = -1;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        c += w[e];
        if (here < 0 && c > t) here = i + e;
      }
      const unsigned who = __ballot_sync(0xffffffffu, here >= 0);
      if (who) return __shfl_sync(0xffffffffu, here, __ffs(who) - 1);
      before = __shfl_sync(0xffffffffu, c, 31);
    }
  }
  return -1;
}

__global__ void __launch_bounds__(kThreads, 2) tree_verify_kernel(const VerifyArgs a) {
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
  const int b = blockIdx.x / ranks;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pkv_wait_prior_grid();
  const int n0 = a.row_start[b], n1 = a.row_start[b + 1], n = n1 - n0;
  const bool bad = n0 < 0 || n1 < n0 || n1 > a.N || n > kTreeMax || n > a.path_cols;
  if (bad || n == 0) {   // the whole cluster leaves together
    if (rank == 0) {
      for (int t = tid; t < a.path_cols; t += kThreads)
        a.path[static_cast<long long>(b) * a.path_cols + t] = -1;
      if (tid == 0) {
        a.accepted[b] = 0;
        a.next[b] = -1;
        if (bad) tree_report(a.err, PKV_ERR_TREE);
      }
    }
    return;
  }
  // The row's CTAs write into one another's shared memory, which exists once they have started:
  // each tells the others here and hears of them before its first such write. (Relaxed: nothing
  // was written for them to see.)
  asm volatile("barrier.cluster.arrive.relaxed;");
  if (tid < n) {
    int bits = 0;
    const int t = a.tokens[n0 + tid];
    int up = tree_parent(a.parents, n0, tid, bits);
    if (tid == 0) up = -1;
    float p = 0.f, q = 1.f;
    if (up >= 0) {
      if (t < 0 || t >= a.V) {
        bits |= PKV_ERR_PROB;
        up = -1;   // never tried
      } else {
        p = clean(a.p[(n0 + up) * a.sp + t]);
        if (a.q) q = clean(a.q[(n0 + up) * a.sq + t]);
      }
    }
    sh.tok[tid] = t;
    sh.par[tid] = up;
    sh.p[tid] = p;
    sh.q[tid] = q;
    sh.u[tid] = a.u_accept[n0 + tid];
    if (bits && rank == 0) tree_report(a.err, bits);
  }
  __syncthreads();

  // the vocabulary's units, in equal contiguous parts for the row's warps
  const int units = (a.V + kUnit - 1) / kUnit;
  const int each = (units + ranks * kWarps - 1) / (ranks * kWarps);
  const int u0 = min(units, (rank * kWarps + warp) * each), u1 = min(units, u0 + each);
  const int size = (each + kGroups * kDeep - 1) / (kGroups * kDeep) * kDeep;   // of a group

  // state of the walk (warp 0's, the same in every CTA of the row)
  int cur = 0, i = 1, n_path = 1;
  double left = 1.0, s_k = 1.0;   // S_k without and with q
  uint64_t a_k = 0;
  int n_gone = 0;
  if (tid == 0) sh.path[0] = 0;
  bool retry = false;
  for (int turn = 0;; ++turn) {
    if (warp == 0) {
      bool pass = false;
      while (!pass && !retry) {
        // the next child of the current node
        const int c0 = lane, c1 = lane + 32;
        unsigned long long kids =
            __ballot_sync(0xffffffffu, c0 >= i && c0 < n && sh.par[c0] == cur) |
            static_cast<unsigned long long>(
                __ballot_sync(0xffffffffu, c1 >= i && c1 < n && sh.par[c1] == cur)) << 32;
        if (!kids) break;
        const int c = __ffsll(kids) - 1;
        i = c + 1;
        const double u = sh.u[c], p = sh.p[c], q = sh.q[c];
        bool good;
        if (a.q) {
          const double w = fmax(p - static_cast<double>(a_k) * kUnitSize * q, 0.0);
          good = u * q * s_k < w;
        } else {
          bool twice = false;
          for (int g = lane; g < n_gone; g += 32) twice |= sh.gone[g] == sh.tok[c];
          twice = __any_sync(0xffffffffu, twice);
          good = !twice && u * left < p;
          if (!good && !twice) {
            left -= p;
            if (lane == 0) sh.gone[n_gone] = sh.tok[c];
            ++n_gone;
            __syncwarp();
          }
        }
        if (good) {
          cur = c;
          if (lane == 0) sh.path[n_path] = c;
          ++n_path;
          left = 1.0;
          s_k = 1.0;
          a_k = 0;
          n_gone = 0;
        } else if (a.q) {
          // what is left after this refusal
          const uint64_t s = static_cast<uint64_t>(s_k * (1ull << kBits));
          a_k = a_k + s < kMaxA ? a_k + s : kMaxA;
          pass = true;
        }
      }
      // the pass is the walk's last unless a further child waits for its sum
      const int c0 = lane, c1 = lane + 32;
      const bool more = __any_sync(0xffffffffu, (c0 >= i && c0 < n && sh.par[c0] == cur) ||
                                                    (c1 >= i && c1 < n && sh.par[c1] == cur));
      if (lane == 0) {
        sh.node = cur;
        sh.a = a_k;
        sh.n_gone = n_gone;
        sh.last = !(pass && more);
        sh.n_path = n_path;
      }
    }
    __syncthreads();
    const uint64_t ak = sh.a;
    Row r;
    r.p = a.p + (n0 + sh.node) * a.sp;
    r.q = a.q ? a.q + (n0 + sh.node) * a.sq : nullptr;
    r.vec_p = (reinterpret_cast<uintptr_t>(r.p) & 15) == 0;
    r.vec_q = (reinterpret_cast<uintptr_t>(r.q) & 15) == 0;
    const bool last = sh.last;
    const int kind = ak == 0 ? kPlain : ak == 1ull << kBits ? kFirst : kLater;
    const uint64_t s =
        kind == kPlain   ? sum_units<kPlain>(r, ak, sh, size, u0, u1, a.V, warp, lane)
        : kind == kFirst ? sum_units<kFirst>(r, ak, sh, size, u0, u1, a.V, warp, lane)
                         : sum_units<kLater>(r, ak, sh, size, u0, u1, a.V, warp, lane);
    if (lane == 0) sh.warp[warp] = s;
    __syncthreads();
    if (turn == 0) asm volatile("barrier.cluster.wait;" ::: "memory");   // (all threads arrived)
    if (warp == 0) {
      const uint64_t mine = warp_sum(lane < kWarps ? sh.warp[lane] : 0);
      if (lane < ranks) *cluster.map_shared_rank(&sh.rank[turn & 1][rank], lane) = mine;
    }
    cluster.sync();
    uint64_t total = 0, before = 0;
    for (int k = 0; k < ranks; ++k) {
      if (k < rank) before += sh.rank[turn & 1][k];
      total += sh.rank[turn & 1][k];
    }
    if (!last) {
      s_k = static_cast<double>(total) * kUnitSize;
      continue;
    }
    if (total == 0 && (ak || sh.n_gone)) {   // nothing left but rounding: the target's own row
      a_k = 0;
      n_gone = 0;
      retry = true;
      __syncthreads();   // sh.n_gone has been read
      continue;
    }
    // the threshold: floor(u S), with u in units of 2^-64
    const float uf = a.u_pick[b];
    const float u = uf > 0.f ? fminf(uf, 0x1.fffffep-1f) : 0.f;
    const uint64_t u64 = static_cast<uint64_t>(u * 0x1p32f * 0x1p32f);
    const uint64_t t = __umul64hi(total, u64);
    if (rank == 0) {
      for (int k = tid; k < a.path_cols; k += kThreads)
        a.path[static_cast<long long>(b) * a.path_cols + k] = k < sh.n_path ? sh.path[k] : -1;
      if (tid == 0) a.accepted[b] = sh.n_path - 1;
      if (tid == 0 && total == 0) {
        a.next[b] = -1;
        tree_report(a.err, PKV_ERR_PROB);
      }
    }
    // this warp's part of the line
    for (int k = 0; k < warp; ++k) before += sh.warp[k];
    if (t >= before && t < before + sh.warp[warp]) {
      const int tok =
          kind == kPlain   ? find<kPlain>(r, ak, sh, before, t, size, u0, u1, a.V, warp, lane)
          : kind == kFirst ? find<kFirst>(r, ak, sh, before, t, size, u0, u1, a.V, warp, lane)
                           : find<kLater>(r, ak, sh, before, t, size, u0, u1, a.V, warp, lane);
      if (lane == 0) a.next[b] = tok;
    }
    return;   // every CTA's words were read before the last cluster barrier, or are its own
  }
}

}  // namespace

extern "C" int tree_verify(const float *target_probs, int64_t target_stride,
                           const float *draft_probs, int64_t draft_stride, const int32_t *tokens,
                           const int32_t *row_start, const int32_t *parents,
                           const float *u_accept, const float *u_pick, int B, int N, int V,
                           int path_cols, int32_t *accepted, int32_t *path, int32_t *next_token,
                           int32_t *err_word, void *stream) {
  static const char *fn = "tree_verify";
  if (B < 0 || B > 65535 || N < 0 || V < 1 || V > (1 << 22) || path_cols < 1)
    return pkv::fail(PKV_E_BAD_ARG, "%s: bad size argument (at most 65535 rows, 2^22 tokens)", fn);
  if (B == 0) return pkv::ok();
  if (!row_start || !u_pick || !accepted || !path || !next_token ||
      (N > 0 && (!target_probs || !tokens || !parents || !u_accept)))
    return pkv::fail(PKV_E_BAD_ARG, "%s: NULL tensor", fn);
  const int64_t most = int64_t(1) << 40;
  if (target_stride < V || target_stride > most ||
      (draft_probs && (draft_stride < V || draft_stride > most)))
    return pkv::fail(PKV_E_BAD_ARG, "%s: row strides must be at least V", fn);
  const int sms = pkv::sm_count();
  int ranks = kMaxCluster;
  while (ranks > 1 && (1LL * B * ranks > 2LL * sms || (ranks / 2) * kWarps * kUnit >= V))
    ranks /= 2;
  const VerifyArgs a = {target_probs, draft_probs, target_stride, draft_stride, tokens, row_start,
                        parents, u_accept, u_pick, accepted, path, next_token, err_word, N, V,
                        path_cols};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(B * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  PKV_CUDA_CHECK(cudaLaunchKernelEx(&cfg, tree_verify_kernel, a));
  return pkv::ok();
}
