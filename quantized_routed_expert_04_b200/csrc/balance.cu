// Balance loss of a batch's routing, its per-expert counts, and the loss's
// gradient in the logits.
//
// With p[t] = softmax(logits[t]) (or, with sigmoid routing, the scores divided
// by their sum), and for each sequence b of n_b counted tokens
//   counts[b][e] = number of (token, j) with idx[t][j] = e,
//   f_e = counts[b][e] E / (k n_b),   P_e = sum_t p[t][e] / n_b:
//   loss = coef / n_seq * sum_b sum_e f_e P_e.
// f is a constant of the gradient, so with u_b = dloss coef / (n_seq n_b):
//   softmax: dlogits[t][e] = u p_e (f_e - sum_j f_j p_j)
//   sigmoid: dlogits[t][e] = u s_e (1 - s_e) / S (f_e - sum_j f_j p_j).
//
// Both passes read each row of logits once and are bound by HBM (large
// batches) or by launch latency (small ones).  A row is held by kLanes lanes,
// 8 consecutive experts each, so a warp works on 32 / kLanes tokens at once
// and reduces over log2(kLanes) shuffles.  A block takes `chunk` consecutive
// tokens and walks the pieces of sequences among them; in the forward, each
// (block, sequence) piece has a slot of its own, block + sequence, for its
// partial sums, which the second kernel adds in block order: the result does
// not depend on timing.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "launch.h"

namespace strata {

namespace {

constexpr int kSumThreads = 1024;    // forward: one block per multiprocessor
constexpr int kGradThreads = 256;
constexpr int kFinishThreads = 1024;
constexpr int kFinishSeqs = 4;       // sequences of a cluster of the finishing kernel

__device__ __forceinline__ int clamp_int(int v, int lo, int hi) { return min(max(v, lo), hi); }

// Tokens [a, e) of sequence b, whatever the offsets hold.
struct Span {
  int a, e;
};
__device__ __forceinline__ Span seq_span(const BalanceParams &p, int b) {
  if (!p.seq_off) return {0, p.T};
  Span s;
  s.a = clamp_int(p.seq_off[b], 0, p.T);
  s.e = clamp_int(p.seq_off[b + 1], s.a, p.T);
  return s;
}

// First sequence that ends after token t (n_seq if none).
__device__ __forceinline__ int first_seq(const BalanceParams &p, int t) {
  if (!p.seq_off) return 0;
  int lo = 0, hi = p.n_seq;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (p.seq_off[mid + 1] > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// Expert i < 8 of lane j of a row: eight consecutive ones, or (rows that 16-byte
// loads cannot walk) every kLanes-th, so that neighbouring lanes load neighbours.
template <int kLanes, bool kVec>
__device__ __forceinline__ int expert_of(int j, int i) {
  return kVec ? 8 * j + i : j + kLanes * i;
}

// The lane's experts of a row (-inf past the last, or all of them if !use), in
// pairs: the arithmetic below runs two to an instruction.
template <int kLanes, bool kVec>
__device__ __forceinline__ void load_row8(const float *row, int j, int E, bool use, float2 v[4]) {
  const float none = __int_as_float(0xff800000);
  if (kVec) {
    float4 a = make_float4(none, none, none, none), b = a;
    if (use && 8 * j < E) a = __ldg(reinterpret_cast<const float4 *>(row + 8 * j));
    if (use && 8 * j + 4 < E) b = __ldg(reinterpret_cast<const float4 *>(row + 8 * j + 4));
    v[0] = make_float2(a.x, a.y);
    v[1] = make_float2(a.z, a.w);
    v[2] = make_float2(b.x, b.y);
    v[3] = make_float2(b.z, b.w);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e0 = expert_of<kLanes, kVec>(j, 2 * i), e1 = expert_of<kLanes, kVec>(j, 2 * i + 1);
      v[i].x = use && e0 < E ? __ldg(row + e0) : none;
      v[i].y = use && e1 < E ? __ldg(row + e1) : none;
    }
  }
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The double at v's place in the shared memory of block `rank` of the cluster.
__device__ __forceinline__ double cluster_read(const double *v, int rank) {
  uint32_t at;
  double d;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(v)), "r"(rank));
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(d) : "r"(at) : "memory");
  return d;
}

template <int kLanes>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int kLanes>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

__device__ __forceinline__ float2 pair(float v) { return make_float2(v, v); }
__device__ __forceinline__ float min_nan(float a, float b) {   // a NaN stays one
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
  return a;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
  return a;
}
__device__ __forceinline__ float exp2_approx(float v) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v));
  return e;
}
__device__ __forceinline__ float rcp_approx(float v) {   // within 1 unit; 0 from 2^126 on
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// e^-y for y in [-88, 110], as 2^(t - r): t = -y log2 e rounded, r what the
// rounding left out (the product's error by an FMA, plus y times the low part of
// log2 e), 2^-r = 1 - r ln 2.  The instruction's own error of 2^-22 is all that
// remains; below 2^-126 the result is 0.
__device__ __forceinline__ float2 exp_minus(float2 y) {
  constexpr double kLog2e = 1.4426950408889634074;
  constexpr float kHi = (float)kLog2e, kLo = (float)(kLog2e - (double)kHi);
  const float2 t = __fmul2_rn(y, pair(-kHi));
  float2 r = __ffma2_rn(y, pair(kHi), t);
  r = __ffma2_rn(y, pair(kLo), r);
  const float2 e = make_float2(exp2_approx(t.x), exp2_approx(t.y));
  return __ffma2_rn(e, __fmul2_rn(r, pair(-0.69314718f)), e);
}

// v: logits of the lane's experts -> terms proportional to p; returns the
// factor that makes them p (0 for a row without any probability: every logit
// -inf, or every sigmoid zero).  slope (if wanted): the same multiple of the
// factor of u (f_e - sum f p) in the gradient.
template <int kLanes, bool kSlope>
__device__ __forceinline__ float probabilities(float2 v[4], bool sigmoid, float2 slope[4]) {
  float2 z = make_float2(0.0f, 0.0f);
  if (!sigmoid) {
    float m = fmaxf(v[0].x, v[0].y);
#pragma unroll
    for (int i = 1; i < 4; ++i) m = fmaxf(m, fmaxf(v[i].x, v[i].y));
    m = lanes_max<kLanes>(m);
    if (m == __int_as_float(0xff800000)) m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = __ffma2_rn(v[i], pair(-1.0f), pair(m));   // >= 0
      v[i] = exp_minus(make_float2(min_nan(y.x, 110.0f), min_nan(y.y, 110.0f)));
      z = __fadd2_rn(z, v[i]);
      if (kSlope) slope[i] = v[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // ex = e^-l; s = 1 / (1 + ex) (0 from 2^126 on) and 1 - s = ex s
      const float2 ex = exp_minus(make_float2(max_nan(min_nan(v[i].x, 110.0f), -88.0f),
                                              max_nan(min_nan(v[i].y, 110.0f), -88.0f)));
      const float2 d = __fadd2_rn(ex, pair(1.0f));
      v[i] = make_float2(rcp_approx(d.x), rcp_approx(d.y));
      if (kSlope) slope[i] = __fmul2_rn(v[i], __fmul2_rn(ex, v[i]));
      z = __fadd2_rn(z, v[i]);
    }
  }
  const float total = lanes_sum<kLanes>(z.x + z.y);
  return total == 0.0f ? 0.0f : rcp_approx(total);
}

// The block's share of one sequence's tokens [a, e): sums of p per expert into
// s_p[0], counts into s_cnt, counted tokens into s_tok.
template <int kLanes, bool kVec>
__device__ __forceinline__ void sum_piece(const BalanceParams &p, int a, int e, float (*s_p)[kLanes * 8],
                                          int *s_cnt, int *s_tok) {
  constexpr int kTok = 32 / kLanes;   // tokens a warp works on at once
  constexpr int kWarps = kSumThreads / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int j = lane % kLanes, sub = lane / kLanes;
  const int E = p.E, k = p.k;
  for (int i = tid; i < E; i += kSumThreads) s_cnt[i] = 0;
  if (tid == 0) *s_tok = 0;
  __syncthreads();
  float2 acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = pair(0.0f);
  int n = 0;
  // Three tokens are in flight: this one's terms, the next one's row and first
  // id, and the mask of the one after (so that no load waits for another).
  constexpr int kStep = kWarps * kTok;
  auto mask_of = [&](int tok) { return tok < e && (!p.mask || p.mask[tok] != 0); };
  auto first_id = [&](int tok, bool use) {
    return use && j < k ? p.idx[(size_t)tok * k + j] : -1;
  };
  auto count = [&](int id) {   // integers: any order
    if (id < 0 || id >= E)
      set_status(p.status, STATUS_BAD_ROUTING);
    else
      atomicAdd(&s_cnt[id], 1);
  };
  float2 next[4];
  int tok = a + warp * kTok + sub;
  bool next_live = mask_of(tok), later = mask_of(tok + kStep);
  load_row8<kLanes, kVec>(p.logits + (size_t)tok * E, j, E, next_live, next);
  int next_id = first_id(tok, next_live);
  for (int t0 = a + warp * kTok; t0 < e; t0 += kStep, tok += kStep) {
    const bool live = next_live;
    const int id = next_id;
    float2 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = next[i];
    next_live = later;
    load_row8<kLanes, kVec>(p.logits + (size_t)(tok + kStep) * E, j, E, next_live, next);
    next_id = first_id(tok + kStep, next_live);
    later = mask_of(tok + 2 * kStep);
    if (live && j < k) {
      count(id);
      for (int i = j + kLanes; i < k; i += kLanes) count(p.idx[(size_t)tok * k + i]);
    }
    __syncwarp();
    // (a token that does not count was not loaded: its terms are finite)
    float r = probabilities<kLanes, false>(v, p.sigmoid, nullptr);
    r = live ? r : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = __ffma2_rn(v[i], pair(r), acc[i]);
    n += live && j == 0;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a1 = i % 2 ? acc[i / 2].y : acc[i / 2].x;
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1) a1 += __shfl_xor_sync(0xffffffffu, a1, o);
    if (sub == 0) s_p[warp][expert_of<kLanes, kVec>(j, i)] = a1;
  }
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0 && n) atomicAdd(s_tok, n);
  __syncthreads();
  for (int i = tid; i < E; i += kSumThreads) {
    float s = s_p[0][i];
#pragma unroll 8
    for (int w = 1; w < kWarps; ++w) s += s_p[w][i];
    s_p[0][i] = s;
  }
}

// kWhole: one block takes the whole batch, one sequence, and writes the
// results itself.
template <int kLanes, bool kVec, bool kWhole>
__global__ void __launch_bounds__(kSumThreads) balance_sum_kernel(const BalanceParams p) {
  __shared__ float s_p[kSumThreads / 32][kLanes * 8];
  __shared__ int s_cnt[kLanes * 8];
  __shared__ int s_tok;
  grid_dependency_wait();
  grid_dependency_launch();
  const int tid = threadIdx.x, E = p.E;
  if (kWhole) {
    const Span sp = seq_span(p, 0);
    if (p.seq_off && tid == 0 && (p.seq_off[0] != sp.a || p.seq_off[1] != sp.e))
      set_status(p.status, STATUS_BOUNDS);
    sum_piece<kLanes, kVec>(p, sp.a, sp.e, s_p, s_cnt, &s_tok);
    __syncthreads();
    if (tid < 32) {
      const int nb = s_tok;
      double all = 0.0;
      for (int i = tid; i < E; i += 32) {
        p.counts[i] = s_cnt[i];
        all += (double)s_cnt[i] * (double)s_p[0][i];
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
      if (tid == 0) {
        p.tokens[0] = nb;
        p.loss[0] = nb > 0 ? (float)((double)p.coef * all * E / ((double)p.k * nb * nb)) : 0.0f;
      }
    }
    return;
  }
  int t = blockIdx.x * p.chunk;
  const int t_end = min(p.T, t + p.chunk);
  for (int b = first_seq(p, t); b < p.n_seq && t < t_end; ++b) {
    const Span sp = seq_span(p, b);
    const int a = max(sp.a, t), e = min(sp.e, t_end);
    if (a >= e) continue;
    sum_piece<kLanes, kVec>(p, a, e, s_p, s_cnt, &s_tok);
    // (each thread wrote the s_p[0] that it reads here)
    const size_t slot = (size_t)blockIdx.x + b;
    for (int i = tid; i < E; i += kSumThreads) {
      p.part_p[slot * E + i] = s_p[0][i];
      p.part_cnt[slot * E + i] = s_cnt[i];
    }
    if (tid == 0) p.part_tok[slot] = s_tok;
    __syncthreads();
    t = e;
  }
  // Offsets that decrease have no such pieces, and the slots that the next kernel
  // would read were not all written: it is told to count nothing.  (By the last
  // block, whose chunk is the shortest.)
  if (p.seq_off && blockIdx.x == gridDim.x - 1) {
    int falls = 0;
#pragma unroll 4
    for (int b = tid; b < p.n_seq; b += kSumThreads) falls |= p.seq_off[b] > p.seq_off[b + 1];
    falls = __syncthreads_or(falls);
    if (tid == 0) *p.falls = falls;
  }
}

// Adds the slots of each sequence's pieces.  A cluster takes up to 4 sequences
// (kOne: the only one), each of its blocks 32 experts; of a block's 32 warps, as
// many as there are sequences for share one sequence's slots.  The kernel is
// nothing but latency (packed batch of 37 sequences, whole pass: 84.8 us with 4
// sequences a cluster, 85.5 with 16, 92.7 with 64, which saves the last launch
// but takes two turns).  Writes the counts, and
// adds sum over experts of counts x (sum of p), which is f P up to
// E / (k n^2), over the cluster: its first block writes the loss (one cluster)
// or each sequence's sum.
template <bool kOne>
__global__ void __launch_bounds__(kFinishThreads) balance_finish_kernel(const BalanceParams p) {
  constexpr int kWarps = kFinishThreads / 32;
  __shared__ double s_p[kWarps][32];
  __shared__ int s_c[kWarps][32], s_t[kWarps];
  __shared__ double s_term[kFinishSeqs];
  __shared__ int s_tok[kFinishSeqs];
  grid_dependency_wait();
  grid_dependency_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = p.E;
  const int b0 = kOne ? 0 : blockIdx.y * kFinishSeqs;
  const int nb = kOne ? 1 : min(kFinishSeqs, p.n_seq - b0);
  const int x = blockIdx.x * 32 + lane;              // the lane's expert
  // warp: share warp % shares of sequence q
  const int shares = kOne ? kWarps : kWarps / nb;
  const int q = kOne ? 0 : warp / shares, share = kOne ? warp : warp % shares;
  const bool mine = q < nb;
  double sum = 0.0;
  int cnt = 0, tok = 0;
  if (mine) {
    const int b = b0 + q;
    const Span sp = seq_span(p, b);
    if (p.seq_off && share == 0 && lane == 0 && (p.seq_off[b] != sp.a || p.seq_off[b + 1] != sp.e))
      set_status(p.status, STATUS_BOUNDS);
    const int c0 = sp.a / p.chunk;
    const bool none = sp.e <= sp.a || (p.seq_off && *p.falls != 0);
    const int n = none ? 0 : (sp.e - 1) / p.chunk - c0 + 1;
    // (at most 148 slots: five loads a lane; they are waited for at the end)
    int t[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      const int i = share + (lane + 32 * k) * shares;
      t[k] = i < n ? p.part_tok[c0 + i + b] : 0;
    }
    // several slots at a time, each load under its own condition (a loop's
    // remainder would take them one by one)
    constexpr int kAtOnce = kOne ? 5 : 8;
    for (int i0 = share; i0 < n; i0 += kAtOnce * shares) {
      float v[kAtOnce];
      int c[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int i = i0 + k * shares;
        const size_t at = ((size_t)c0 + i + b) * E + x;
        const bool in = i < n && x < E;
        v[k] = in ? p.part_p[at] : 0.0f;
        c[k] = in ? p.part_cnt[at] : 0;
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        sum += (double)v[k];
        cnt += c[k];
      }
    }
#pragma unroll
    for (int k = 0; k < 5; ++k) tok += t[k];
  }
  tok = __reduce_add_sync(0xffffffffu, tok);
  s_p[warp][lane] = sum;
  s_c[warp][lane] = cnt;
  if (lane == 0) s_t[warp] = tok;
  __syncthreads();
  if (mine && share == 0) {
#pragma unroll 8
    for (int w = 1; w < kWarps; ++w) {
      if (w >= shares) break;
      sum += s_p[warp + w][lane];
      cnt += s_c[warp + w][lane];
      tok += s_t[warp + w];
    }
    if (x < E) p.counts[(size_t)(b0 + q) * E + x] = cnt;
    double term = (double)cnt * sum;   // 0 for lanes without an expert
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(0xffffffffu, term, o);
    if (lane == 0) {
      s_term[q] = term;
      s_tok[q] = tok;
    }
  }
  __syncthreads();
  cluster_sync();
  if (blockIdx.x == 0) {
    for (int q = threadIdx.x; q < nb; q += kFinishThreads) {
      double all = 0.0;
      for (int r = 0; r < (int)gridDim.x; ++r) all += cluster_read(&s_term[q], r);
      const int n = s_tok[q];
      p.tokens[b0 + q] = n;
      all = n > 0 ? all * E / ((double)p.k * n * n) : 0.0;
      s_p[0][q] = all;
      if (gridDim.y > 1) p.seq_loss[b0 + q] = all;
    }
    __syncthreads();
    if (gridDim.y == 1 && warp == 0) {
      double all = lane < nb ? s_p[0][lane] : 0.0;
#pragma unroll
      for (int o = kFinishSeqs / 2; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
      if (lane == 0) p.loss[0] = (float)(all * (double)p.coef / p.n_seq);
    }
  }
  cluster_sync();   // no block leaves while its s_term may still be read
}

// The mean of the sequences' sums, in a fixed order.
__global__ void __launch_bounds__(256) balance_mean_kernel(const BalanceParams p) {
  __shared__ double s[8];
  grid_dependency_wait();
  grid_dependency_launch();
  double v = 0.0;
  for (int b = threadIdx.x; b < p.n_seq; b += 256) v += p.seq_loss[b];
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) v += s[w];
    p.loss[0] = (float)(v * (double)p.coef / p.n_seq);
  }
}

template <int kLanes, bool kVec>
__global__ void __launch_bounds__(kGradThreads) balance_grad_kernel(const BalanceGradParams g) {
  grid_dependency_wait();
  grid_dependency_launch();
  const BalanceParams &p = g.p;
  constexpr int kTok = 32 / kLanes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int j = lane % kLanes, sub = lane / kLanes;
  const int E = p.E;
  int t = blockIdx.x * p.chunk;
  const int t_end = min(p.T, t + p.chunk);
  const float dloss = g.dloss ? *g.dloss : 1.0f;
  // tokens [a, e) with the weights f and the factor u (zeros if !counted)
  auto piece = [&](int a, int e, bool counted, const float2 f[4], float u) {
    // last token first: the forward's last rows are still in L2, where the
    // batch as a whole does not fit.  The next row and the mask after it are
    // loaded ahead
    constexpr int kStep = kGradThreads / 32 * kTok;
    auto mask_of = [&](int tok) {
      return counted && tok >= a && (!p.mask || p.mask[tok] != 0);
    };
    int tok = e - 1 - warp * kTok - sub;
    float2 next[4];
    bool next_live = mask_of(tok), later = mask_of(tok - kStep);
    load_row8<kLanes, kVec>(p.logits + (long long)tok * E, j, E, next_live, next);
    for (int t1 = e - 1 - warp * kTok; t1 >= a; t1 -= kStep, tok -= kStep) {
      const bool in = tok >= a;
      const bool live = next_live;
      float2 v[4], slope[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = next[i];
      next_live = later;
      later = mask_of(tok - 2 * kStep);
      load_row8<kLanes, kVec>(p.logits + ((long long)tok - kStep) * E, j, E, next_live, next);
      const float r = probabilities<kLanes, true>(v, p.sigmoid, slope);
      float2 d2 = pair(0.0f);
#pragma unroll
      for (int i = 0; i < 4; ++i) d2 = __ffma2_rn(f[i], v[i], d2);
      const float dot = lanes_sum<kLanes>(d2.x + d2.y) * r;
      const float ur = live ? u * r : 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = __fmul2_rn(__fmul2_rn(slope[i], pair(ur)), __fadd2_rn(f[i], pair(-dot)));
      float *out = g.dlogits + (long long)tok * E;
      if (kVec) {
        float4 *o4 = reinterpret_cast<float4 *>(out + 8 * j);
        if (in && 8 * j < E) o4[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
        if (in && 8 * j + 4 < E) o4[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int x = expert_of<kLanes, kVec>(j, i);
          if (in && x < E) out[x] = i % 2 ? v[i / 2].y : v[i / 2].x;
        }
      }
    }
  };
  float2 f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = pair(0.0f);
  for (int b = first_seq(p, t); b < p.n_seq && t < t_end; ++b) {
    const Span sp = seq_span(p, b);
    const int a = max(sp.a, t), e = min(sp.e, t_end);
    if (a >= e) continue;
    piece(t, a, false, f, 0.0f);   // tokens in front of the sequence
    const int nb = p.tokens[b];
    const float inv = nb > 0 ? __fdiv_rn(1.0f, (float)nb) : 0.0f;
    const float per = (float)E / (float)p.k * inv;
    float2 fb[4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int x = expert_of<kLanes, kVec>(j, i);
      const float one = x < E ? (float)p.counts[(size_t)b * E + x] * per : 0.0f;
      if (i % 2) fb[i / 2].y = one;
      else fb[i / 2].x = one;
    }
    piece(a, e, true, fb, dloss * (p.coef / (float)p.n_seq) * inv);
    t = e;
  }
  piece(t, t_end, false, f, 0.0f);   // tokens behind the last sequence
}

// Forward: tokens per block, a multiple of 32, that give each of the 148
// multiprocessors one block of 32 warps.
int sum_chunk(int T) { return std::max(32, ((T + 147) / 148 + 31) & ~31); }
int sum_blocks(int T) { return (T + sum_chunk(T) - 1) / sum_chunk(T); }   // <= 148
// Backward: up to four blocks of 8 warps each, at least two rows a warp.
int grad_chunk(int T) {
  const int per = (T + 591) / 592;
  return ((per < 16 ? 16 : per) + 7) & ~7;
}
// Batches that one block passes over in at most four steps take one launch
// (forward and backward together, one block against the others: 256 experts 9.3
// against 9.9 us with 128 tokens, 12.7 against 10.1 with 256; 64 experts 8.0
// against 9.0 with 512, 11.1 against 9.3 with 1024; 8 experts 8.3 against 9.5
// with 2048, 11.8 against 10.0 with 4096).
bool whole_batch(const BalanceParams &p) {
  int lanes = 1;
  while (8 * lanes < p.E) lanes *= 2;
  return p.n_seq == 1 && p.T <= std::min(2048, 4 * (kSumThreads / lanes));
}

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// kLanes: the power of two of lanes that holds E experts, 8 a lane.
template <template <int, bool> class Launch, typename... A>
cudaError_t by_shape(int E, bool vec, A... a) {
#define STRATA_CASE(n) \
  if (E <= 8 * n) return vec ? Launch<n, true>::run(a...) : Launch<n, false>::run(a...);
  STRATA_CASE(1)
  STRATA_CASE(2)
  STRATA_CASE(4)
  STRATA_CASE(8)
  STRATA_CASE(16)
  STRATA_CASE(32)
#undef STRATA_CASE
  return cudaErrorInvalidValue;
}

template <int kLanes, bool kVec>
struct LaunchSum {
  static cudaError_t run(const BalanceParams *p, bool whole, cudaStream_t stream) {
    if (whole)
      return launch_pdl(balance_sum_kernel<kLanes, kVec, true>, dim3(1), dim3(kSumThreads), 0, stream, *p);
    return launch_pdl(balance_sum_kernel<kLanes, kVec, false>, dim3(sum_blocks(p->T)),
                      dim3(kSumThreads), 0, stream, *p);
  }
};
template <int kLanes, bool kVec>
struct LaunchGrad {
  static cudaError_t run(const BalanceGradParams *g, cudaStream_t stream) {
    const int chunk = g->p.chunk;
    return launch_pdl(balance_grad_kernel<kLanes, kVec>, dim3((g->p.T + chunk - 1) / chunk),
                      dim3(kGradThreads), 0, stream, *g);
  }
};

inline bool vec_rows(const void *p, int E) {
  return E % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

}  // namespace

size_t balance_workspace(int T, int E, int n_seq) {
  const size_t slots = (size_t)sum_blocks(T) + n_seq;
  return 2 * up256(slots * E * 4) + up256(slots * 4) + up256((size_t)n_seq * 8) + up256(4);
}

cudaError_t run_balance(BalanceParams p, void *workspace, cudaStream_t stream) {
  const size_t slots = (size_t)sum_blocks(p.T) + p.n_seq;
  char *w = static_cast<char *>(workspace);
  p.part_p = reinterpret_cast<float *>(w);
  p.part_cnt = reinterpret_cast<int *>(w += up256(slots * p.E * 4));
  p.part_tok = reinterpret_cast<int *>(w += up256(slots * p.E * 4));
  p.seq_loss = reinterpret_cast<double *>(w += up256(slots * 4));
  p.falls = reinterpret_cast<int *>(w += up256((size_t)p.n_seq * 8));
  p.chunk = sum_chunk(p.T);
  const bool whole = whole_batch(p);
  cudaError_t e =
      by_shape<LaunchSum>(p.E, vec_rows(p.logits, p.E), (const BalanceParams *)&p, whole, stream);
  if (whole || e != cudaSuccess) return e;
  const int groups = (p.E + 31) / 32, clusters = (p.n_seq + kFinishSeqs - 1) / kFinishSeqs;
  e = launch_pdl_cluster(p.n_seq == 1 ? balance_finish_kernel<true> : balance_finish_kernel<false>,
                         dim3(groups, clusters), groups, dim3(kFinishThreads), 0, stream, p);
  if (e == cudaSuccess && clusters > 1)
    e = launch_pdl(balance_mean_kernel, dim3(1), dim3(256), 0, stream, p);
  return e;
}

cudaError_t run_balance_grad(BalanceGradParams g, cudaStream_t stream) {
  g.p.chunk = grad_chunk(g.p.T);
  const bool vec = vec_rows(g.p.logits, g.p.E) && vec_rows(g.dlogits, g.p.E);
  return by_shape<LaunchGrad>(g.p.E, vec, (const BalanceGradParams *)&g, stream);
}

}  // namespace strata
