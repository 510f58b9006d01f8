// RMS norm with the residual's addition, its output in 16 or 32 bits and/or
// in e4m3 with scales, and its gradient.
//
// Forward, per row: s = x + r, y = s * rsqrt(mean(s^2) + eps) * g.  Gradient,
// with i = rsqrt(mean(h^2) + eps) of the saved sum h and gy = dy * g:
//   dx = i gy - h i^3 mean(gy h) + ds,   dg = sum over rows of dy h i.
// Everything between the loads and the stores is fp32: s (not its rounding)
// is what is squared and normalised, and each output is rounded once.
//
// Both are bound by HBM: a row is read once, kept in registers through its
// reduction, and written once.  Element mapping: with 16-byte aligned rows
// (kVec) a thread holds groups of 8 consecutive elements, one 16-byte access
// each (two for fp32); otherwise the block's threads take consecutive
// elements one by one, which keeps every access of a warp contiguous.
#include <cuda_fp8.h>

#include <algorithm>
#include <cstdlib>

#include "common.cuh"
#include "kernels.h"
#include "launch.h"

namespace strata {

namespace {

constexpr int kNormMaxH = 16384;
constexpr int kMaxStages = 8;

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32(float v) { return v; }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_f32(float v) { return v; }

// Eight elements as they are stored.
template <typename T>
struct Vec8 {
  uint4 q[sizeof(T) / 2];
};

// Plain loads and stores (never the read-only path: an output may be the same
// buffer as an input).
template <typename T>
__device__ __forceinline__ Vec8<T> load8(const T *p) {
  Vec8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.q[i] = reinterpret_cast<const uint4 *>(p)[i];
  return r;
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const Vec8<T> &r) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4 *>(p)[i] = r.q[i];
}

__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __half) { return __half22float2(bits_h2(w)); }
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  return h2_bits(__floats2half2_rn(a, b));
}
template <typename T>
__device__ __forceinline__ void unpack8(const Vec8<T> &r, float v[8]) {
  const uint32_t w[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2(w[i], T());
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
template <>
__device__ __forceinline__ void unpack8(const Vec8<float> &r, float v[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[4 * i] = __uint_as_float(r.q[i].x);
    v[4 * i + 1] = __uint_as_float(r.q[i].y);
    v[4 * i + 2] = __uint_as_float(r.q[i].z);
    v[4 * i + 3] = __uint_as_float(r.q[i].w);
  }
}
template <typename T>
__device__ __forceinline__ Vec8<T> pack8(const float v[8]) {
  Vec8<T> r;
  r.q[0] = make_uint4(pack2(v[0], v[1], T()), pack2(v[2], v[3], T()), pack2(v[4], v[5], T()),
                      pack2(v[6], v[7], T()));
  return r;
}
template <>
__device__ __forceinline__ Vec8<float> pack8<float>(const float v[8]) {
  Vec8<float> r;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    r.q[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                        __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
  return r;
}

// max that keeps a NaN (a group with a NaN gets a NaN scale, so that it reads
// back as NaN)
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Four floats -> four e4m3 bytes (nearest even, saturating at 448, NaN kept).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Step of a group whose largest magnitude is amax: amax / 448, but never
// below the smallest normal fp32 (an all-zero group divides by it safely).
__device__ __forceinline__ float e4m3_step(float amax) {
  return max_nan(__fdiv_rn(amax, 448.0f), 1.17549435e-38f);
}

struct SumOp {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct MaxOp {
  __device__ __forceinline__ float operator()(float a, float b) const { return max_nan(a, b); }
};

// Reduction over the kTpr threads of a row, the result in every one of them.
// slots: kTpr / 32 floats of shared memory that no other reduction in flight
// uses.
template <int kTpr, typename Op>
__device__ __forceinline__ float row_reduce(float v, Op op, float *slots, int tid) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (kTpr > 32) {
    constexpr int kWarps = kTpr / 32;
    if ((tid & 31) == 0) slots[tid >> 5] = v;
    __syncthreads();
    v = slots[tid & (kWarps - 1)];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  }
  return v;
}

struct NormParams {
  const void *x, *residual;
  const float *weight;
  void *residual_out, *out;
  uint8_t *q8;
  float *scales;
  long long ldx, ldr, ldro, ldo;   // row strides in elements
  int T, H, group, n_groups;       // group: columns per scale, >= H for one scale a row
  float eps, inv_h;
};

// kTpr threads per row, kRows rows per block, kNe elements per thread.
template <typename T, int kTpr, int kRows, int kNe, bool kVec>
__global__ void __launch_bounds__(kTpr *kRows) norm_kernel(const NormParams p) {
  __shared__ float s_red[2][kTpr > 32 ? kTpr / 32 : 1];
  __shared__ float s_amax[kVec ? 1 : kRows * kNe * (kTpr / 32)];
  grid_dependency_wait();
  grid_dependency_launch();
  const int tid = threadIdx.x % kTpr;
  const long long row = (long long)blockIdx.x * kRows + threadIdx.x / kTpr;
  if (kRows > 1 && row >= p.T) return;   // whole warps (kTpr = 32)
  const int H = p.H;
  const T *x = static_cast<const T *>(p.x) + row * p.ldx;
  const T *r = p.residual ? static_cast<const T *>(p.residual) + row * p.ldr : nullptr;
  T *ro = p.residual_out ? static_cast<T *>(p.residual_out) + row * p.ldro : nullptr;
  T *out = p.out ? static_cast<T *>(p.out) + row * p.ldo : nullptr;
  uint8_t *q8 = p.q8 ? p.q8 + row * H : nullptr;
  float *scales = p.q8 ? p.scales + row * p.n_groups : nullptr;

  float v[kNe];
  float sq = 0.0f;
  if (kVec) {
    constexpr int kNv = kNe / 8;
    Vec8<T> a[kNv], b[kNv];
#pragma unroll
    for (int i = 0; i < kNv; ++i) {
      const int c = (tid + i * kTpr) * 8;
      if (c < H) {
        a[i] = load8(x + c);
        if (r) b[i] = load8(r + c);
      }
    }
#pragma unroll
    for (int i = 0; i < kNv; ++i) {
      float s[8], t[8];
      unpack8(a[i], s);
      if (r) {
        unpack8(b[i], t);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] += t[j];
      }
      const bool in = (tid + i * kTpr) * 8 < H;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[8 * i + j] = in ? s[j] : 0.0f;
        sq = fmaf(v[8 * i + j], v[8 * i + j], sq);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kNe; ++i) {
      const int c = tid + i * kTpr;
      v[i] = c < H ? to_f32(x[c]) : 0.0f;
    }
    if (r) {
#pragma unroll
      for (int i = 0; i < kNe; ++i) {
        const int c = tid + i * kTpr;
        if (c < H) v[i] += to_f32(r[c]);
      }
    }
#pragma unroll
    for (int i = 0; i < kNe; ++i) sq = fmaf(v[i], v[i], sq);
  }
  if (ro) {
    if (kVec) {
#pragma unroll
      for (int i = 0; i < kNe / 8; ++i) {
        const int c = (tid + i * kTpr) * 8;
        if (c < H) store8(ro + c, pack8<T>(v + 8 * i));
      }
    } else {
#pragma unroll
      for (int i = 0; i < kNe; ++i) {
        const int c = tid + i * kTpr;
        if (c < H) ro[c] = from_f32<T>(v[i]);
      }
    }
  }
  sq = row_reduce<kTpr>(sq, SumOp(), s_red[0], tid);
  const float inv = rsqrtf(fmaf(sq, p.inv_h, p.eps));

  // y, and the 16- or 32-bit output
  if (kVec) {
#pragma unroll
    for (int i = 0; i < kNe / 8; ++i) {
      const int c = (tid + i * kTpr) * 8;
      if (c < H) {
        const float4 w0 = __ldg(reinterpret_cast<const float4 *>(p.weight + c));
        const float4 w1 = __ldg(reinterpret_cast<const float4 *>(p.weight + c + 4));
        const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) v[8 * i + j] = v[8 * i + j] * inv * w[j];
        if (out) store8(out + c, pack8<T>(v + 8 * i));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[8 * i + j] = 0.0f;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kNe; ++i) {
      const int c = tid + i * kTpr;
      v[i] = c < H ? v[i] * inv * __ldg(p.weight + c) : 0.0f;
      if (out && c < H) out[c] = from_f32<T>(v[i]);
    }
  }
  if (!q8) return;

  // e4m3: per group of columns, the largest magnitude, the step and the bytes
  float row_amax = 0.0f;
  const bool per_row = p.group >= H;
  if (per_row) {
#pragma unroll
    for (int i = 0; i < kNe; ++i) row_amax = max_nan(row_amax, fabsf(v[i]));
    row_amax = row_reduce<kTpr>(row_amax, MaxOp(), s_red[1], tid);
    if (tid == 0) scales[0] = e4m3_step(row_amax);
  }
  if (kVec) {
    const int lanes = p.group / 8;   // lanes per group: 4, 8 or 16
#pragma unroll
    for (int i = 0; i < kNe / 8; ++i) {
      const int c = (tid + i * kTpr) * 8;
      float amax = row_amax;
      if (!per_row) {
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = max_nan(amax, fabsf(v[8 * i + j]));
        for (int o = 1; o < lanes; o <<= 1)
          amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      }
      const float step = e4m3_step(amax), mul = __fdiv_rn(1.0f, step);
      if (c < H) {
        uint2 q;
        q.x = e4m3x4(v[8 * i] * mul, v[8 * i + 1] * mul, v[8 * i + 2] * mul, v[8 * i + 3] * mul);
        q.y = e4m3x4(v[8 * i + 4] * mul, v[8 * i + 5] * mul, v[8 * i + 6] * mul,
                     v[8 * i + 7] * mul);
        *reinterpret_cast<uint2 *>(q8 + c) = q;
        if (!per_row && c % p.group == 0) scales[c / p.group] = step;
      }
    }
  } else {
    // a warp's 32 lanes hold columns 32 m .. 32 m + 31 of m = i * kTpr / 32 +
    // warp: the largest magnitude of each such run, then a step per group
    float *run = s_amax + (threadIdx.x / kTpr) * kNe * (kTpr / 32);
    auto meet = [] {
      if (kTpr > 32)
        __syncthreads();
      else
        __syncwarp();
    };
    const float row_mul = per_row ? __fdiv_rn(1.0f, e4m3_step(row_amax)) : 0.0f;
    if (!per_row) {
#pragma unroll
      for (int i = 0; i < kNe; ++i) {
        float a = fabsf(v[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
        if ((tid & 31) == 0) run[i * (kTpr / 32) + (tid >> 5)] = a;
      }
      meet();
      // group g: its runs' largest, its step, and 1 / step back to the runs
      const int per = p.group / 32, runs = (H + 31) / 32;
      for (int g = tid; g < p.n_groups; g += kTpr) {
        float amax = 0.0f;
        for (int m = g * per; m < min(g * per + per, runs); ++m) amax = max_nan(amax, run[m]);
        const float step = e4m3_step(amax), mul = __fdiv_rn(1.0f, step);
        scales[g] = step;
        for (int m = g * per; m < min(g * per + per, runs); ++m) run[m] = mul;
      }
      meet();
    }
#pragma unroll
    for (int i = 0; i < kNe; ++i) {
      const int c = tid + i * kTpr;
      const float mul = per_row ? row_mul : run[i * (kTpr / 32) + (tid >> 5)];
      if (c < H) q8[c] = __nv_cvt_float_to_fp8(v[i] * mul, __NV_SATFINITE, __NV_E4M3);
    }
  }
}

// Threads per row: 16 elements each at the widths where a row has the threads to
// itself (8192 x 4096 bf16 with residual and 8-bit output: 49.5 us with 256
// threads, 50.3 with 128 of 32 elements, 51.8 with 512 of 8), fewer on short
// rows, where a warp has one.  Rows that 16-byte accesses cannot walk go element by
// element: 8192 x 4095 91 us; 2048 x 16383 123 us, 67 with 16384.
template <typename T, bool kVec>
cudaError_t launch_norm(const NormParams &p, cudaStream_t stream) {
  const int H = p.H, T_ = p.T;
  auto rows = [&](int per) { return dim3(((long long)T_ + per - 1) / per); };
  if (H <= 256) return launch_pdl(norm_kernel<T, 32, 4, 8, kVec>, rows(4), dim3(128), 0, stream, p);
  if (H <= 512) return launch_pdl(norm_kernel<T, 32, 4, 16, kVec>, rows(4), dim3(128), 0, stream, p);
  if (H <= 1024) return launch_pdl(norm_kernel<T, 128, 1, 8, kVec>, rows(1), dim3(128), 0, stream, p);
  if (H <= 2048) return launch_pdl(norm_kernel<T, 256, 1, 8, kVec>, rows(1), dim3(256), 0, stream, p);
  if (H <= 4096) return launch_pdl(norm_kernel<T, 256, 1, 16, kVec>, rows(1), dim3(256), 0, stream, p);
  if (H <= 8192) return launch_pdl(norm_kernel<T, 512, 1, 16, kVec>, rows(1), dim3(512), 0, stream, p);
  return launch_pdl(norm_kernel<T, 1024, 1, 16, kVec>, rows(1), dim3(1024), 0, stream, p);
}

// ---------------------------------------------------------------- gradient
struct NormGradParams {
  const void *h, *dout, *dsum;
  const float *weight;
  void *dx;
  float *partial;                // [gridDim.x][H] sums over each block's rows, or null
  long long ldh, lddo, ldds, lddx;
  int T, H;
  float eps, inv_h;
  int stages;                    // rows in flight per block
};

// kRows groups of kTpr threads, each with rows of its own: group g of block b
// walks rows b kRows + g, + gridDim.x kRows, ...; a thread keeps its columns'
// weights (kKeepW) and weight-gradient sums in registers over all of them.
// With kVec the rows come through a ring of shared-memory stages per group,
// filled by bulk copies, so that several rows of all three inputs are in flight
// while one is reduced: on 8192 rows of 4096 bf16 with a direct gradient, plain
// loads with one row ahead in registers took 98 us (waiting for loads; and 88
// through the ring with elements converted one by one), now 44 us.  The barrier
// of the row's reduction also frees its stage: every thread has its elements in
// registers by then.  A copy that does not arrive within the limit of its wait
// ends the copies, after those in flight have had as long again each to land; its
// row and all the thread's rows behind it become NaN, and with them the weight's
// gradient.  Without kVec (rows that 16-byte copies cannot walk) the
// next row's elements are loaded into registers ahead, 2 or 4 bytes an access: 8192
// rows of 4095 bf16 78 us, 50 with 4096; and above 8192 columns a thread's 64
// registers do not hold both rows (556 to 668 bytes a thread are spilled: 2048 rows
// of 16383 bf16 220 us, 75 with 16384).
template <typename T, int kTpr, int kRows, int kNe, bool kVec, int kMinBlocks>
__global__ void __launch_bounds__(kTpr *kRows, kMinBlocks) norm_grad_kernel(const NormGradParams p) {
  constexpr int kWarps = kTpr / 32;
  // 1024 threads have 64 registers each: they keep only the sums in them and read
  // the row from its stage twice; !kVec's next row takes the weights' registers
  constexpr bool kHold = !kVec || kTpr < 1024;
  constexpr bool kKeepW = kVec && kHold;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float2 s_red[kRows][2][kWarps];
  __shared__ uint64_t s_full[kRows][kMaxStages];
  const int tid = threadIdx.x % kTpr, group = threadIdx.x / kTpr, H = p.H;
  uint64_t *full = s_full[group];
  const uint32_t row_bytes = (uint32_t)H * sizeof(T);
  const bool direct = p.dsum != nullptr;
  if (kVec) {
    if (tid == 0) {
      for (int s = 0; s < p.stages; ++s) mbar_init(&full[s], 1);
      fence_mbar_init();
    }
    __syncthreads();
  }
  grid_dependency_wait();
  grid_dependency_launch();
  // all threads of a row
  auto meet = [&] {
    if (kWarps == 1)
      __syncwarp();
    else if (kRows == 1)
      __syncthreads();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(kTpr) : "memory");
  };
  const long long row0 = (long long)blockIdx.x * kRows + group, step = (long long)gridDim.x * kRows;
  const uint32_t stage_bytes = row_bytes * (direct ? 3 : 2);
  uint8_t *ring = smem + (size_t)group * p.stages * stage_bytes;
  auto fetch = [&](long long row, int st) {
    if (row >= p.T) return;
    uint8_t *dst = ring + st * stage_bytes;
    mbar_arrive_expect_tx(&full[st], stage_bytes);
    bulk_g2s(dst, static_cast<const T *>(p.h) + row * p.ldh, row_bytes, &full[st]);
    bulk_g2s(dst + row_bytes, static_cast<const T *>(p.dout) + row * p.lddo, row_bytes, &full[st]);
    if (direct)
      bulk_g2s(dst + 2 * row_bytes, static_cast<const T *>(p.dsum) + row * p.ldds, row_bytes, &full[st]);
  };
  if (kVec && tid == 0)
    for (int s = 0; s < p.stages; ++s) fetch(row0 + s * step, s);
  auto col = [&](int i) { return kVec ? (tid + (i / 8) * kTpr) * 8 + i % 8 : tid + i * kTpr; };
  constexpr int kAhead = kVec ? 1 : kNe;
  T ha[kAhead], da[kAhead];   // !kVec: the next row
  auto load_row = [&](long long row) {
    if (kVec || row >= p.T) return;
    const T *h = static_cast<const T *>(p.h) + row * p.ldh;
    const T *dy = static_cast<const T *>(p.dout) + row * p.lddo;
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (col(i) < H) {
        ha[i] = h[col(i)];
        da[i] = dy[col(i)];
      }
  };
  load_row(row0);
  float dg[kNe], w[kKeepW ? kNe : 1];
#pragma unroll
  for (int i = 0; i < kNe; ++i) {
    dg[i] = 0.0f;
    if (kKeepW) w[i] = col(i) < H ? __ldg(p.weight + col(i)) : 0.0f;
  }
  auto weight = [&](int i) {
    return kKeepW ? w[kKeepW ? i : 0] : col(i) < H ? __ldg(p.weight + col(i)) : 0.0f;
  };
  auto weight8 = [&](int i, float w8[8]) {   // of columns col(i) ..
    if (kKeepW || !kVec) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w8[j] = weight(i + j);
    } else if (col(i) < H) {
      const float4 x = __ldg(reinterpret_cast<const float4 *>(p.weight + col(i)));
      const float4 y = __ldg(reinterpret_cast<const float4 *>(p.weight + col(i) + 4));
      w8[0] = x.x; w8[1] = x.y; w8[2] = x.z; w8[3] = x.w;
      w8[4] = y.x; w8[5] = y.y; w8[6] = y.z; w8[7] = y.w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w8[j] = 0.0f;
    }
  };
  int flip = 0, st = 0;
  uint32_t phase = 0;
  bool lost = false;   // (every thread takes every step all the same: no barrier is missed)
  for (long long row = row0; row < p.T; row += step, flip ^= 1) {
    float a[kHold ? kNe : 8], d[kHold ? kNe : 8];
    Vec8<T> sc[kVec && kHold ? kNe / 8 : 1];
    T sn[kAhead];
    float sq = 0.0f, dot = 0.0f;
    const T *sh = reinterpret_cast<const T *>(ring + st * stage_bytes);
    auto unpack_at = [&](int i, float *a8, float *d8) {
      if (col(i) < H) {
        unpack8(load8(sh + col(i)), a8);
        unpack8(load8(sh + H + col(i)), d8);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) a8[j] = d8[j] = 0.0f;
      }
    };
    if (kVec) {
      if (!lost && !mbar_wait(&full[st], phase, nullptr)) {
        lost = true;
        // (the ring's memory is used again below, and the block's after its end)
        if (tid == 0)
          for (int k = 0; k < p.stages && row + k * step < p.T; ++k) {
            const int s = st + k < p.stages ? st + k : st + k - p.stages;
            (void)mbar_wait(&full[s], s >= st ? phase : phase ^ 1u, nullptr);
          }
      }
#pragma unroll
      for (int i = 0; i < kNe; i += 8) {
        unpack_at(i, a + (kHold ? i : 0), d + (kHold ? i : 0));
        if (kHold) {
          if (direct && col(i) < H) sc[i / 8] = load8(sh + 2 * H + col(i));
        } else {
          float w8[8];
          weight8(i, w8);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            sq = fmaf(a[j], a[j], sq);
            dot = fmaf(d[j] * w8[j], a[j], dot);
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        a[kVec ? 0 : i] = col(i) < H ? to_f32(ha[i]) : 0.0f;
        d[kVec ? 0 : i] = col(i) < H ? to_f32(da[i]) : 0.0f;
      }
      if (direct) {
        const T *ds = static_cast<const T *>(p.dsum) + row * p.ldds;
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (col(i) < H) sn[i] = ds[col(i)];
      }
      load_row(row + step);
    }
    if (kHold) {
#pragma unroll
      for (int i = 0; i < (kHold ? kNe : 0); ++i) {
        sq = fmaf(a[i], a[i], sq);
        dot = fmaf(d[i] * weight(i), a[i], dot);
      }
    }
    if (kVec && lost) sq = __int_as_float(0x7fffffff);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sq += __shfl_xor_sync(0xffffffffu, sq, o);
      dot += __shfl_xor_sync(0xffffffffu, dot, o);
    }
    // (two slots in turn: a warp is at most one row ahead of the others)
    if (kWarps > 1 && (tid & 31) == 0) s_red[group][flip][tid >> 5] = make_float2(sq, dot);
    if (kWarps > 1 || kVec) meet();
    auto next_stage = [&] {
      if (tid == 0 && !lost) fetch(row + p.stages * step, st);
      if (++st == p.stages) {
        st = 0;
        phase ^= 1u;
      }
    };
    if (kVec && kHold) next_stage();
    if (kWarps > 1) {
      const float2 v = s_red[group][flip][tid & (kWarps - 1)];
      sq = v.x;
      dot = v.y;
#pragma unroll
      for (int o = kWarps / 2; o > 0; o >>= 1) {
        sq += __shfl_xor_sync(0xffffffffu, sq, o);
        dot += __shfl_xor_sync(0xffffffffu, dot, o);
      }
    }
    const float inv = rsqrtf(fmaf(sq, p.inv_h, p.eps));
    const float back = dot * p.inv_h * inv * inv;   // i^2 mean(gy h)
    T *dx = static_cast<T *>(p.dx) + row * p.lddx;
#pragma unroll
    for (int i = 0; i < kNe; i += 8) {
      float o[8], s[8], w8[8];
      if (!kHold) unpack_at(i, a, d);
      weight8(i, w8);
      if (kVec && direct && col(i) < H) unpack8(kHold ? sc[kHold ? i / 8 : 0] : load8(sh + 2 * H + col(i)), s);
#pragma unroll
      for (int j = i; j < i + 8; ++j) {
        const float aj = a[kHold ? j : j - i], dj = d[kHold ? j : j - i];
        dg[j] = fmaf(dj, aj * inv, dg[j]);
        o[j - i] = inv * (dj * w8[j - i] - aj * back);
        if (kVec) {
          if (direct) o[j - i] += s[j - i];
        } else if (col(j) < H) {
          dx[col(j)] = from_f32<T>(direct ? o[j - i] + to_f32(sn[kVec ? 0 : j]) : o[j - i]);
        }
      }
      if (kVec && col(i) < H) store8(dx + col(i), pack8<T>(o));
    }
    if (kVec && !kHold) {
      meet();
      next_stage();
    }
  }
  if (!p.partial) return;
  float *out = p.partial + (long long)blockIdx.x * H;
  // this thread's columns (as 16-byte stores: one row of 4096 6.2 -> 4.2 us, 1200
  // rows 13.9 -> 9.6)
  auto put = [&](float *to) {
    if (kVec) {
#pragma unroll
      for (int i = 0; i < kNe; i += 4)
        if (col(i) < H)
          *reinterpret_cast<float4 *>(to + col(i)) = make_float4(dg[i], dg[i + 1], dg[i + 2], dg[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < kNe; ++i)
        if (col(i) < H) to[col(i)] = dg[i];
    }
  };
  if (kRows == 1) {
    put(out);
    return;
  }
  // the groups' sums, in order, through shared memory (every stage has been read)
  float *rows = reinterpret_cast<float *>(smem);
  __syncthreads();
  put(rows + group * H);
  __syncthreads();
  for (int c = threadIdx.x; c < H; c += kTpr * kRows) {
    float v = rows[c];
#pragma unroll
    for (int g = 1; g < kRows; ++g) v += rows[g * H + c];
    out[c] = v;
  }
}

// Sum of n <= 296 rows of partial sums, in a fixed order: 32 columns a block,
// 32 rows at a time.
__global__ void __launch_bounds__(1024) norm_grad_sum_kernel(const float *partial, int n, int H,
                                                             float *out) {
  __shared__ float s[32][33];
  grid_dependency_wait();
  grid_dependency_launch();
  const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  // all of the thread's (at most 10) loads at once, each under its own condition
  float t[10];
#pragma unroll
  for (int k = 0; k < 10; ++k) {
    const int r = y + 32 * k;
    t[k] = r < n && c < H ? partial[(long long)r * H + c] : 0.0f;
  }
  float v = t[0];
#pragma unroll
  for (int k = 1; k < 10; ++k) v += t[k];
  s[y][lane] = v;
  __syncthreads();
  v = s[lane][y];   // row share lane of column y
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int cy = blockIdx.x * 32 + y;
  if (lane == 0 && cy < H) out[cy] = v;
}

// Rows that a block takes at once: 256 threads have a row of at most 4096
// elements, smaller ones share the block.
inline int grad_rows(int H) { return H <= 512 ? 8 : H <= 1024 ? 4 : H <= 2048 ? 2 : 1; }
// Blocks of the gradient kernel: two for each of the 148 multiprocessors, half
// as many where that leaves a group of threads fewer than four rows (each
// block's partial sums are as long as a row and are read again).
inline int grad_blocks(int T, int H) {
  const long long need = ((long long)T + grad_rows(H) - 1) / grad_rows(H);
  return need >= 1184 ? 296 : need < 148 ? (int)need : 148;
}

template <typename T, int kTpr, int kRows, int kNe, bool kVec, int kMinBlocks>
cudaError_t launch_norm_grad_as(NormGradParams p, cudaStream_t stream) {
  auto kern = norm_grad_kernel<T, kTpr, kRows, kNe, kVec, kMinBlocks>;
  int smem = kRows > 1 ? kRows * p.H * (int)sizeof(float) : 0;   // the groups' sums
  p.stages = 0;
  if (kVec) {
    // two blocks share a multiprocessor's 227 KB, or one takes it (a row of
    // 16384 fp32 elements and its two gradients are 192 KB).  The limit belongs to
    // the kernel, not to the launch: every call sets the same one, so that calls of
    // several threads do not lower it under one another.
    constexpr int kLimit = (kMinBlocks > 1 ? 110 : 220) * 1024;
    constexpr int kMostH = kTpr * kNe;
    static_assert(kRows * kMostH * 3 * (int)sizeof(T) <= kLimit, "one stage of the widest rows fits");
    const int stage = p.H * (int)sizeof(T) * (p.dsum ? 3 : 2);
    p.stages = std::min(kMaxStages, kLimit / (kRows * stage));
    smem = std::max(smem, kRows * p.stages * stage);
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kLimit);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, dim3(grad_blocks(p.T, p.H)), dim3(kTpr * kRows), smem, stream, p);
}

template <typename T, bool kVec>
cudaError_t launch_norm_grad(const NormGradParams &p, cudaStream_t stream) {
  if (p.H <= 256) return launch_norm_grad_as<T, 32, 8, 8, kVec, 2>(p, stream);
  if (p.H <= 512) return launch_norm_grad_as<T, 32, 8, 16, kVec, 2>(p, stream);
  if (p.H <= 1024) return launch_norm_grad_as<T, 64, 4, 16, kVec, 2>(p, stream);
  if (p.H <= 2048) return launch_norm_grad_as<T, 128, 2, 16, kVec, 2>(p, stream);
  if (p.H <= 4096) return launch_norm_grad_as<T, 256, 1, 16, kVec, 2>(p, stream);
  if (p.H <= 8192) return launch_norm_grad_as<T, 512, 1, 16, kVec, 1>(p, stream);
  return launch_norm_grad_as<T, 1024, 1, 16, kVec, 1>(p, stream);
}

// ---------------------------------------------------------------- unpack
// e4m3 rows and their scales -> bf16 activations (the reader of norm_kernel's
// 8-bit output): 16 elements a thread, always inside one group of scales
// (groups are multiples of 32; H is a multiple of 128).  The product of the
// exact e4m3 value and the scale is rounded once to bf16.
__global__ void __launch_bounds__(256) unpack_q8_kernel(const uint8_t *q8, const float *scales,
                                                        int group, int n_groups, int H,
                                                        long long n16, __nv_bfloat16 *x) {
  grid_dependency_wait();
  grid_dependency_launch();
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n16) return;
  const int per_row = H / 16;
  const long long t = i / per_row;
  const int c = (int)(i - t * per_row) * 16;
  const float s = scales[t * n_groups + c / group];
  const uint4 raw = reinterpret_cast<const uint4 *>(q8)[i];
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t o[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((uint16_t)(w[k / 2] >> (16 * (k & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
    o[k] = *reinterpret_cast<const uint32_t *>(&b);
  }
  uint4 *dst = reinterpret_cast<uint4 *>(x) + 2 * i;
  dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
  dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

int dtype_bytes(int dtype) {
  switch (dtype) {
    case STRATA_DTYPE_BF16: case STRATA_DTYPE_F16: return 2;
    case STRATA_DTYPE_F32: return 4;
  }
  return 0;
}

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// A row operand: present, aligned to its elements, rows that do not overlap.
bool rows_ok(const void *p, long long ld, int T, int H, int bytes) {
  return p && aligned(p, bytes) && (T <= 1 || ld >= H);
}
// Two row operands, one of them written, share elements other than by being in the
// same place (where each row is read before it is written): a block would write
// what another has yet to read.
bool rows_clash(const void *a, long long lda, const void *b, long long ldb, int T, int H, int bytes) {
  if (!a || !b) return false;
  if (T <= 1) lda = ldb = H;
  if (a == b && lda == ldb) return false;
  const long long d = (long long)(reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a));
  const long long row = (long long)H * bytes, sa = lda * bytes, sb = ldb * bytes;
  if (d >= (T - 1) * sa + row || -d >= (T - 1) * sb + row) return false;   // one ends before the other begins
  // row i of a begins i sa behind a's start and meets row j of b if |d + j sb - i sa|
  // is less than a row: with one stride that goes by i - j alone
  const int rows = sa == sb ? 1 : T;
  for (int i = 0; i < rows; ++i) {
    const long long at = i * sa - d;   // from b's start
    long long j = at >= 0 ? at / sb : -((-at + sb - 1) / sb);   // the row of b at or before it
    for (int k = 0; k < 2; ++k, ++j)
      if (llabs(at - j * sb) < row && (sa == sb ? llabs(j) < T : j >= 0 && j < T)) return true;
  }
  return false;
}
// ... that 16-byte accesses can walk.
bool rows_vec(const void *p, long long ld, int bytes) {
  return !p || (aligned(p, 16) && ld * bytes % 16 == 0);
}

}  // namespace

cudaError_t run_unpack_q8(const uint8_t *q8, const float *scales, int group, int T, int H,
                          __nv_bfloat16 *x, cudaStream_t stream) {
  const long long n16 = (long long)T * H / 16;
  const int g = group < H ? group : H;
  return launch_pdl(unpack_q8_kernel, dim3((unsigned)((n16 + 255) / 256)), dim3(256), 0, stream, q8,
                    scales, g, (H + g - 1) / g, H, n16, x);
}

}  // namespace strata

using namespace strata;

extern "C" {

strata_status strata_rmsnorm(int dtype, const void *x, long long x_stride, const void *residual,
                             long long residual_stride, const float *weight, float eps,
                             int n_tokens, int hidden, void *residual_out,
                             long long residual_out_stride, void *out, long long out_stride,
                             void *out_q8, float *scales, int group, strata_stream_t stream) {
  const int b = dtype_bytes(dtype);
  if (!b || n_tokens < 0 || hidden < 1 || !(eps >= 0.0f) || !(eps <= 3.0e38f))
    return STRATA_ERR_INVALID_ARG;
  if (hidden > kNormMaxH) return STRATA_ERR_UNSUPPORTED;
  if (residual_out && residual_out == out) return STRATA_ERR_INVALID_ARG;
  if (n_tokens == 1) x_stride = residual_stride = residual_out_stride = out_stride = hidden;
  if (out_q8 ? !scales || (group != 32 && group != 64 && group != 128 && group < hidden)
             : scales != nullptr)
    return STRATA_ERR_INVALID_ARG;
  if (n_tokens == 0) return STRATA_OK;
  if (!rows_ok(x, x_stride, n_tokens, hidden, b) || !weight || !aligned(weight, 4) ||
      !aligned(scales, 4) || (!out && !out_q8))
    return STRATA_ERR_INVALID_ARG;
  if ((residual && !rows_ok(residual, residual_stride, n_tokens, hidden, b)) ||
      (residual_out && !rows_ok(residual_out, residual_out_stride, n_tokens, hidden, b)) ||
      (out && !rows_ok(out, out_stride, n_tokens, hidden, b)))
    return STRATA_ERR_INVALID_ARG;
  auto clash = [&](const void *u, long long ldu, const void *v, long long ldv) {
    return rows_clash(u, ldu, v, ldv, n_tokens, hidden, b);
  };
  if (clash(residual_out, residual_out_stride, x, x_stride) ||
      clash(residual_out, residual_out_stride, residual, residual_stride) ||
      clash(residual_out, residual_out_stride, out, out_stride) || clash(out, out_stride, x, x_stride) ||
      clash(out, out_stride, residual, residual_stride))
    return STRATA_ERR_INVALID_ARG;
  NormParams p;
  p.x = x;
  p.residual = residual;
  p.weight = weight;
  p.residual_out = residual_out;
  p.out = out;
  p.q8 = static_cast<uint8_t *>(out_q8);
  p.scales = scales;
  p.ldx = x_stride;
  p.ldr = residual_stride;
  p.ldro = residual_out_stride;
  p.ldo = out_stride;
  p.T = n_tokens;
  p.H = hidden;
  p.group = out_q8 ? group : hidden;
  p.n_groups = (hidden + p.group - 1) / p.group;
  p.eps = eps;
  p.inv_h = (float)(1.0 / hidden);
  const bool vec = hidden % 8 == 0 && rows_vec(x, x_stride, b) &&
                   rows_vec(residual, residual_stride, b) &&
                   rows_vec(residual_out, residual_out_stride, b) && rows_vec(out, out_stride, b) &&
                   aligned(weight, 16) && aligned(out_q8, 8);
  cudaError_t e;
  switch (dtype) {
    case STRATA_DTYPE_BF16:
      e = vec ? launch_norm<__nv_bfloat16, true>(p, stream) : launch_norm<__nv_bfloat16, false>(p, stream);
      break;
    case STRATA_DTYPE_F16:
      e = vec ? launch_norm<__half, true>(p, stream) : launch_norm<__half, false>(p, stream);
      break;
    default:
      e = vec ? launch_norm<float, true>(p, stream) : launch_norm<float, false>(p, stream);
  }
  return status_of(e);
}

size_t strata_rmsnorm_backward_workspace(int n_tokens, int hidden) {
  if (n_tokens < 0 || hidden < 1 || hidden > kNormMaxH) return 0;
  const size_t blocks = grad_blocks(n_tokens > 0 ? n_tokens : 1, hidden);
  return blocks * hidden * sizeof(float);
}

strata_status strata_rmsnorm_backward(int dtype, const void *h, long long h_stride,
                                      const float *weight, float eps, const void *dout,
                                      long long dout_stride, const void *dsum,
                                      long long dsum_stride, int n_tokens, int hidden, void *dx,
                                      long long dx_stride, float *dweight, void *workspace,
                                      size_t workspace_bytes, strata_stream_t stream) {
  const int b = dtype_bytes(dtype);
  if (!b || n_tokens < 0 || hidden < 1 || !(eps >= 0.0f) || !(eps <= 3.0e38f))
    return STRATA_ERR_INVALID_ARG;
  if (hidden > kNormMaxH) return STRATA_ERR_UNSUPPORTED;
  if (!aligned(dweight, 4)) return STRATA_ERR_INVALID_ARG;
  if (n_tokens == 1) h_stride = dout_stride = dsum_stride = dx_stride = hidden;
  if (n_tokens == 0)
    return dweight ? status_of(cudaMemsetAsync(dweight, 0, sizeof(float) * hidden, stream)) : STRATA_OK;
  if (!rows_ok(h, h_stride, n_tokens, hidden, b) || !weight || !aligned(weight, 4) ||
      !rows_ok(dout, dout_stride, n_tokens, hidden, b) ||
      (dsum && !rows_ok(dsum, dsum_stride, n_tokens, hidden, b)) ||
      !rows_ok(dx, dx_stride, n_tokens, hidden, b))
    return STRATA_ERR_INVALID_ARG;
  if (rows_clash(dx, dx_stride, h, h_stride, n_tokens, hidden, b) ||
      rows_clash(dx, dx_stride, dout, dout_stride, n_tokens, hidden, b) ||
      rows_clash(dx, dx_stride, dsum, dsum_stride, n_tokens, hidden, b))
    return STRATA_ERR_INVALID_ARG;
  if (dweight && (!workspace || !aligned(workspace, 16) ||
                  workspace_bytes < strata_rmsnorm_backward_workspace(n_tokens, hidden)))
    return STRATA_ERR_INVALID_ARG;
  NormGradParams p;
  p.h = h;
  p.dout = dout;
  p.dsum = dsum;
  p.weight = weight;
  p.dx = dx;
  p.partial = dweight ? static_cast<float *>(workspace) : nullptr;
  p.ldh = h_stride;
  p.lddo = dout_stride;
  p.ldds = dsum_stride;
  p.lddx = dx_stride;
  p.T = n_tokens;
  p.H = hidden;
  p.eps = eps;
  p.inv_h = (float)(1.0 / hidden);
  const bool vec = hidden % 8 == 0 && rows_vec(h, h_stride, b) && rows_vec(dout, dout_stride, b) &&
                   rows_vec(dsum, dsum_stride, b) && rows_vec(dx, dx_stride, b) && aligned(weight, 16);
  cudaError_t e;
  switch (dtype) {
    case STRATA_DTYPE_BF16:
      e = vec ? launch_norm_grad<__nv_bfloat16, true>(p, stream)
              : launch_norm_grad<__nv_bfloat16, false>(p, stream);
      break;
    case STRATA_DTYPE_F16:
      e = vec ? launch_norm_grad<__half, true>(p, stream)
              : launch_norm_grad<__half, false>(p, stream);
      break;
    default:
      e = vec ? launch_norm_grad<float, true>(p, stream) : launch_norm_grad<float, false>(p, stream);
  }
  if (e == cudaSuccess && dweight)
    e = launch_pdl(norm_grad_sum_kernel, dim3((hidden + 31) / 32), dim3(1024), 0, stream,
                   (const float *)p.partial, grad_blocks(n_tokens, hidden), hidden, dweight);
  return status_of(e);
}

}  // extern "C"
