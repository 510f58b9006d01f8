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
// tokens and walks the pieces of sequences among them; each (block, sequence)
// piece has a slot of its own, block + sequence, for its partial sums, which
// the second kernel adds in block order: the result does not depend on timing.
#include "common.cuh"
#include "kernels.h"
#include "launch.h"

namespace strata {

namespace {

constexpr int kBalThreads = 256;
constexpr int kBalWarps = kBalThreads / 32;
constexpr int kFinishThreads = 1024;

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

// Experts 8 j .. 8 j + 7 of a row (-inf past the last).
template <bool kVec>
__device__ __forceinline__ void load_row8(const float *row, int j, int E, bool use, float v[8]) {
  const float none = __int_as_float(0xff800000);
  if (kVec) {
    float4 a = make_float4(none, none, none, none), b = a;
    if (use && 8 * j < E) {
      a = __ldg(reinterpret_cast<const float4 *>(row + 8 * j));
      b = __ldg(reinterpret_cast<const float4 *>(row + 8 * j + 4));
    }
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = use && 8 * j + i < E ? __ldg(row + 8 * j + i) : none;
  }
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

// v: logits of the lane's experts -> p.  slope (if wanted): the factor of
// u (f_e - sum f p) in the gradient.  A row without any probability (every
// logit -inf, or every sigmoid zero) gives zeros.
template <int kLanes, bool kSlope>
__device__ __forceinline__ void probabilities(float v[8], bool sigmoid, float slope[8]) {
  if (!sigmoid) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) m = fmaxf(m, v[i]);
    m = lanes_max<kLanes>(m);
    const bool none = m == __int_as_float(0xff800000);
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = none && v[i] == m ? 0.0f : expf(v[i] - m);
      z += v[i];
    }
    z = lanes_sum<kLanes>(z);
    const float r = z == 0.0f ? 0.0f : __fdiv_rn(1.0f, z);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] *= r;
      if (kSlope) slope[i] = v[i];
    }
  } else {
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float ex = expf(-v[i]);
      const float s = __fdiv_rn(1.0f, 1.0f + ex);
      // s (1 - s) with 1 - s = ex s, or 1 where ex is beyond fp32 (s = 0)
      if (kSlope) slope[i] = s == 0.0f ? 0.0f : s * (ex * s);
      v[i] = s;
      z += s;
    }
    z = lanes_sum<kLanes>(z);
    const float r = z == 0.0f ? 0.0f : __fdiv_rn(1.0f, z);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] *= r;
      if (kSlope) slope[i] *= r;
    }
  }
}

template <int kLanes, bool kVec>
__global__ void __launch_bounds__(kBalThreads) balance_partial_kernel(const BalanceParams p) {
  __shared__ float s_p[kBalWarps][kLanes * 8];
  __shared__ int s_cnt[kLanes * 8];
  __shared__ int s_tok;
  grid_dependency_wait();
  grid_dependency_launch();
  constexpr int kTok = 32 / kLanes;   // tokens a warp works on at once
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int j = lane % kLanes, sub = lane / kLanes;
  const int E = p.E, k = p.k;
  int t = blockIdx.x * p.chunk;
  const int t_end = min(p.T, t + p.chunk);
  for (int b = first_seq(p, t); b < p.n_seq && t < t_end; ++b) {
    const Span sp = seq_span(p, b);
    const int a = max(sp.a, t), e = min(sp.e, t_end);
    if (a >= e) continue;
    for (int i = tid; i < E; i += kBalThreads) s_cnt[i] = 0;
    if (tid == 0) s_tok = 0;
    __syncthreads();
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
    int n = 0;
    for (int t0 = a + warp * kTok; t0 < e; t0 += kBalWarps * kTok) {
      const int tok = t0 + sub;
      const bool live = tok < e && (!p.mask || p.mask[tok] != 0);
      float v[8];
      load_row8<kVec>(p.logits + (size_t)tok * E, j, E, live, v);
      probabilities<kLanes, false>(v, p.sigmoid, nullptr);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += live ? v[i] : 0.0f;
      n += live && j == 0;
    }
    // counts: one pair a thread, added up in shared memory (integers: any order)
    const long long q1 = (long long)e * k;
    for (long long q = (long long)a * k + tid; q < q1; q += kBalThreads) {
      if (p.mask && !p.mask[q / k]) continue;
      const int id = p.idx[q];
      if (id < 0 || id >= E)
        set_status(p.status, STATUS_BAD_ROUTING);
      else
        atomicAdd(&s_cnt[id], 1);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int o = kLanes; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
      if (sub == 0) s_p[warp][8 * j + i] = acc[i];
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0 && n) atomicAdd(&s_tok, n);
    __syncthreads();
    const size_t slot = (size_t)blockIdx.x + b;
    for (int i = tid; i < E; i += kBalThreads) {
      float s = s_p[0][i];
#pragma unroll
      for (int w = 1; w < kBalWarps; ++w) s += s_p[w][i];
      p.part_p[slot * E + i] = s;
      p.part_cnt[slot * E + i] = s_cnt[i];
    }
    if (tid == 0) p.part_tok[slot] = s_tok;
    __syncthreads();
    t = e;
  }
}

// One block per sequence: adds its pieces' slots, writes its counts and its
// sum of f P.
__global__ void __launch_bounds__(kFinishThreads) balance_finish_kernel(const BalanceParams p) {
  __shared__ double s_p[kFinishThreads];
  __shared__ int s_c[kFinishThreads];
  __shared__ int s_tok;
  grid_dependency_wait();
  grid_dependency_launch();
  const int b = blockIdx.x, tid = threadIdx.x, E = p.E;
  const Span sp = seq_span(p, b);
  if (p.seq_off && tid == 0 && (p.seq_off[b] != sp.a || p.seq_off[b + 1] != sp.e))
    set_status(p.status, STATUS_BOUNDS);
  const int c0 = sp.a / p.chunk;
  const int n = sp.e > sp.a ? (sp.e - 1) / p.chunk - c0 + 1 : 0;
  if (tid == 0) s_tok = 0;
  __syncthreads();
  const int x = tid % kMaxExperts, y = tid / kMaxExperts;   // expert, share of the slots
  constexpr int kShares = kFinishThreads / kMaxExperts;
  double sum = 0.0;
  int cnt = 0, tok = 0;
  for (int i = tid; i < n; i += kFinishThreads) tok += p.part_tok[c0 + i + b];
  if (x < E)
    for (int i = y; i < n; i += kShares) {
      const size_t slot = (size_t)c0 + i + b;
      sum += (double)p.part_p[slot * E + x];
      cnt += p.part_cnt[slot * E + x];
    }
  tok = __reduce_add_sync(0xffffffffu, tok);
  if ((tid & 31) == 0 && tok) atomicAdd(&s_tok, tok);
  s_p[tid] = sum;
  s_c[tid] = cnt;
  __syncthreads();
  const int nb = s_tok;
  double term = 0.0;
  if (y == 0 && x < E) {
    for (int i = 1; i < kShares; ++i) {
      sum += s_p[i * kMaxExperts + x];
      cnt += s_c[i * kMaxExperts + x];
    }
    p.counts[(size_t)b * E + x] = cnt;
    if (nb > 0) term = (double)cnt * E / ((double)p.k * nb) * (sum / nb);
  }
  __syncthreads();
  for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(0xffffffffu, term, o);
  if ((tid & 31) == 0) s_p[tid >> 5] = term;
  __syncthreads();
  if (tid == 0) {
    double all = 0.0;
    for (int w = 0; w < kMaxExperts / 32; ++w) all += s_p[w];
    p.tokens[b] = nb;
    if (p.n_seq == 1)
      p.loss[0] = (float)((double)p.coef * all);
    else
      p.seq_loss[b] = all;
  }
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
__global__ void __launch_bounds__(kBalThreads) balance_grad_kernel(const BalanceGradParams g) {
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
  auto piece = [&](int a, int e, bool counted, const float f[8], float u) {
    for (int t0 = a + warp * kTok; t0 < e; t0 += kBalWarps * kTok) {
      const int tok = t0 + sub;
      const bool in = tok < e;
      const bool live = counted && in && (!p.mask || p.mask[tok] != 0);
      float v[8], slope[8];
      load_row8<kVec>(p.logits + (size_t)tok * E, j, E, live, v);
      probabilities<kLanes, true>(v, p.sigmoid, slope);
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) dot = fmaf(f[i], v[i], dot);
      dot = lanes_sum<kLanes>(dot);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = live ? u * slope[i] * (f[i] - dot) : 0.0f;
      float *out = g.dlogits + (size_t)tok * E + 8 * j;
      if (kVec) {
        if (in && 8 * j < E) {
          reinterpret_cast<float4 *>(out)[0] = make_float4(v[0], v[1], v[2], v[3]);
          reinterpret_cast<float4 *>(out)[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (in && 8 * j + i < E) out[i] = v[i];
      }
    }
  };
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = 0.0f;
  for (int b = first_seq(p, t); b < p.n_seq && t < t_end; ++b) {
    const Span sp = seq_span(p, b);
    const int a = max(sp.a, t), e = min(sp.e, t_end);
    if (a >= e) continue;
    piece(t, a, false, f, 0.0f);   // tokens in front of the sequence
    const int nb = p.tokens[b];
    const float inv = nb > 0 ? __fdiv_rn(1.0f, (float)nb) : 0.0f;
    const float per = (float)E / (float)p.k * inv;
    float fb[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      fb[i] = 8 * j + i < E ? (float)p.counts[(size_t)b * E + 8 * j + i] * per : 0.0f;
    piece(a, e, true, fb, dloss * (p.coef / (float)p.n_seq) * inv);
    t = e;
  }
  piece(t, t_end, false, f, 0.0f);   // tokens behind the last sequence
}

// Tokens per block: a multiple of 8 that gives the 148 multiprocessors up to
// four blocks each.
int balance_chunk(int T) {
  const int per = (T + 591) / 592;
  return ((per < 16 ? 16 : per) + 7) & ~7;
}
int balance_blocks(int T) { return (int)(((long long)T + balance_chunk(T) - 1) / balance_chunk(T)); }

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
struct LaunchPartial {
  static cudaError_t run(const BalanceParams *p, cudaStream_t stream) {
    return launch_pdl(balance_partial_kernel<kLanes, kVec>, dim3(balance_blocks(p->T)),
                      dim3(kBalThreads), 0, stream, *p);
  }
};
template <int kLanes, bool kVec>
struct LaunchGrad {
  static cudaError_t run(const BalanceGradParams *g, cudaStream_t stream) {
    return launch_pdl(balance_grad_kernel<kLanes, kVec>, dim3(balance_blocks(g->p.T)),
                      dim3(kBalThreads), 0, stream, *g);
  }
};

inline bool vec_rows(const void *p, int E) {
  return E % 8 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

}  // namespace

size_t balance_workspace(int T, int E, int n_seq) {
  const size_t slots = (size_t)balance_blocks(T) + n_seq;
  return 2 * up256(slots * E * 4) + up256(slots * 4) + up256((size_t)n_seq * 8);
}

cudaError_t run_balance(BalanceParams p, void *workspace, cudaStream_t stream) {
  const size_t slots = (size_t)balance_blocks(p.T) + p.n_seq;
  char *w = static_cast<char *>(workspace);
  p.part_p = reinterpret_cast<float *>(w);
  p.part_cnt = reinterpret_cast<int *>(w += up256(slots * p.E * 4));
  p.part_tok = reinterpret_cast<int *>(w += up256(slots * p.E * 4));
  p.seq_loss = reinterpret_cast<double *>(w += up256(slots * 4));
  p.chunk = balance_chunk(p.T);
  cudaError_t e = by_shape<LaunchPartial>(p.E, vec_rows(p.logits, p.E), (const BalanceParams *)&p, stream);
  if (e == cudaSuccess)
    e = launch_pdl(balance_finish_kernel, dim3(p.n_seq), dim3(kFinishThreads), 0, stream, p);
  if (e == cudaSuccess && p.n_seq > 1)
    e = launch_pdl(balance_mean_kernel, dim3(1), dim3(256), 0, stream, p);
  return e;
}

cudaError_t run_balance_grad(BalanceGradParams g, cudaStream_t stream) {
  g.p.chunk = balance_chunk(g.p.T);
  const bool vec = vec_rows(g.p.logits, g.p.E) && vec_rows(g.dlogits, g.p.E);
  return by_shape<LaunchGrad>(g.p.E, vec, (const BalanceGradParams *)&g, stream);
}

}  // namespace strata
