// Gradient of the router: from the gradients of the routing weights and of
// the logits to the router's weights, its bias and the activations.
//
//   dl = dlogits + (dw through the routing weights)
//        softmax: w_j = softmax over the selected logits:
//                 dl[idx_j] += w_j (dw_j - sum_i w_i dw_i)
//        sigmoid: w_j = scale s_j / S, S the sum of the selected scores:
//                 dl[idx_j] += scale s_j (1 - s_j) / S (dw_j - sum_i s_i / S dw_i)
//   dW = dl^T x,   db = sum_t dl,   dx = dl W.
#include "common.cuh"
#include "kernels.h"
#include "launch.h"

namespace strata {

namespace {

// One warp per token: the token's row of dl.
__global__ void __launch_bounds__(256) route_grad_logits_kernel(const RouteGradParams p) {
  grid_dependency_wait();
  grid_dependency_launch();
  const int lane = threadIdx.x & 31, E = p.E, k = p.k;
  const long long t = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= p.T) return;
  // lane j < k: selection j
  int id = -1;
  float g = 0.0f;
  if (p.dw) {
    const bool sel = lane < k;
    id = sel ? p.idx[t * k + lane] : -1;
    const bool bad = sel && (id < 0 || id >= E);
    if (__any_sync(0xffffffffu, bad)) {
      // the forward writes a zero row for such a token: dw has no meaning
      if (bad) set_status(p.status, STATUS_BAD_ROUTING);
      id = -1;
    } else {
      const float l = sel ? p.logits[t * E + id] : 0.0f;
      const float dw = sel ? p.dw[t * k + lane] : 0.0f;
      float w, slope;   // w_j / scale, and its factor in the gradient
      if (p.mode.sigmoid) {
        const float ex = expf(-l);
        const float s = sel ? __fdiv_rn(1.0f, 1.0f + ex) : 0.0f;
        float z = s;
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        // (a true division: one selected expert has w = 1 and no gradient)
        w = z == 0.0f ? 0.0f : __fdiv_rn(s, z);
        slope = s == 0.0f ? 0.0f : p.mode.scale * w * (ex * s);
      } else {
        float m = sel ? l : __int_as_float(0xff800000);
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const bool none = m == __int_as_float(0xff800000);
        const float ex = !sel || (none && l == m) ? 0.0f : expf(l - m);
        float z = ex;
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        w = z == 0.0f ? 0.0f : __fdiv_rn(ex, z);
        slope = w;
      }
      float dot = sel ? w * dw : 0.0f;
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      g = sel ? slope * (dw - dot) : 0.0f;
    }
  }
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    float v = p.dlogits && e < E ? p.dlogits[t * E + e] : 0.0f;
    for (int j = 0; j < k; ++j) {
      const int ij = __shfl_sync(0xffffffffu, id, j);
      const float gj = __shfl_sync(0xffffffffu, g, j);
      if (ij == e) v += gj;
    }
    if (e < E) p.dl[t * E + e] = v;
  }
}

// C[m][n] = sum_k A(k, m) B[k][n] in fp32, 64 x 64 a block.  A(k, m) is
// A[k * lda + m] or, transposed, A[m * lda + k].
template <bool kTransA, typename TB, typename TC>
__global__ void __launch_bounds__(256) route_grad_gemm_kernel(const float *A, int lda, const TB *B,
                                                              int M, int N, int K, TC *C) {
  grid_dependency_wait();
  grid_dependency_launch();
  __shared__ float as[16][65], bs[16][65];
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64, tid = threadIdx.x;
  const int tm = (tid / 16) * 4, tn = (tid % 16) * 4;
  float c[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += 16) {
    for (int i = tid; i < 16 * 64; i += 256) {
      const int kk = kTransA ? i % 16 : i / 64, mm = kTransA ? i / 16 : i % 64;
      const bool in = k0 + kk < K && m0 + mm < M;
      as[kk][mm] = !in ? 0.0f
                       : kTransA ? A[(size_t)(m0 + mm) * lda + k0 + kk]
                                 : A[(size_t)(k0 + kk) * lda + m0 + mm];
      const int kb = i / 64, nb = i % 64;
      bs[kb][nb] = k0 + kb < K && n0 + nb < N ? (float)B[(size_t)(k0 + kb) * N + n0 + nb] : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 16; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) c[i][j] = fmaf(as[kk][tm + i], bs[kk][tn + j], c[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j)
      if (m0 + tm + i < M && n0 + tn + j < N)
        C[(size_t)(m0 + tm + i) * N + n0 + tn + j] = (TC)c[i][j];
}

__global__ void __launch_bounds__(256) route_grad_bias_kernel(const float *dl, int T, int E,
                                                              float *db) {
  grid_dependency_wait();
  grid_dependency_launch();
  __shared__ double s[8];
  double v = 0.0;
  for (int t = threadIdx.x; t < T; t += 256) v += dl[(size_t)t * E + blockIdx.x];
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) v += s[w];
    db[blockIdx.x] = (float)v;
  }
}

}  // namespace

size_t route_grad_workspace(int T, int E, int H) { return sizeof(float) * (size_t)T * E; }

cudaError_t run_route_grad(RouteGradParams p, void *workspace, cudaStream_t stream) {
  p.dl = static_cast<float *>(workspace);
  const float *dl = p.dl;
  cudaError_t e = launch_pdl(route_grad_logits_kernel, dim3((p.T + 7) / 8), dim3(256), 0, stream, p);
  if (e == cudaSuccess && p.dW)
    e = launch_pdl(route_grad_gemm_kernel<false, __nv_bfloat16, float>,
                   dim3((p.H + 63) / 64, (p.E + 63) / 64), dim3(256), 0, stream, dl, p.E, p.x, p.E,
                   p.H, p.T, p.dW);
  if (e == cudaSuccess && p.dx)
    e = launch_pdl(route_grad_gemm_kernel<true, float, __nv_bfloat16>,
                   dim3((p.H + 63) / 64, (p.T + 63) / 64), dim3(256), 0, stream, dl, p.E, p.W, p.T,
                   p.H, p.E, p.dx);
  if (e == cudaSuccess && p.db)
    e = launch_pdl(route_grad_bias_kernel, dim3(p.E), dim3(256), 0, stream, dl, p.T, p.E, p.db);
  return e;
}

}  // namespace strata
