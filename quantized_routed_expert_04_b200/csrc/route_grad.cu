// Gradient of the router: from the gradients of the routing weights and of
// the logits to the router's weights, its bias and the activations.
//
//   dl = dlogits + (dw through the routing weights)
//        softmax: w_j = softmax over the selected logits:
//                 dl[idx_j] += w_j (dw_j - sum_i w_i dw_i)
//        sigmoid: w_j = scale s_j / S, S the sum of the selected scores:
//                 dl[idx_j] += scale s_j (1 - s_j) / S (dw_j - sum_i s_i / S dw_i)
//   dW = dl^T x,   db = sum_t dl,   dx = dl W.
//
// Four launches: the rows of dl (and W) as bf16 pieces; dW and dx on the
// tensor cores (tcgen05, accumulators in tensor memory); the sums of dW's and
// db's parts.
//
// fp32 operands on bf16 tensor cores: a number is the sum of its bf16
// rounding, the bf16 rounding of what is left, and so on; each piece keeps 8
// more bits.  dW needs fp32 accuracy: x is bf16 already, dl takes three pieces
// (24 bits), three exact products per element, added in fp32.  dx is rounded to
// bf16 at the end: dl and W take two pieces each, and hi hi + hi lo + lo hi
// leaves out 2^-18 of a product.
#include <cuda.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "launch.h"

namespace strata {

namespace {

constexpr int kPrepWarps = 8;

__device__ __forceinline__ uint32_t bf162_bits(__nv_bfloat162 v) {
  return *reinterpret_cast<uint32_t *>(&v);
}

// Eight floats -> their bf16 roundings (returned), v becomes what is left.
__device__ __forceinline__ uint4 take_bf16(float v[8]) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    const float2 f = __bfloat1622float2(b);
    v[2 * i] -= f.x;
    v[2 * i + 1] -= f.y;
    o[i] = bf162_bits(b);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Blocks 0 .. tok_blocks - 1: rows of dl, one warp per token at a time, each
// lane 8 consecutive experts, as three bf16 pieces, and the block's share of
// db.  The blocks behind them: W as two bf16 pieces.
__global__ void __launch_bounds__(32 * kPrepWarps) route_grad_prep_kernel(const RouteGradParams p) {
  __shared__ float s_db[kPrepWarps][kMaxExperts];
  grid_dependency_wait();
  grid_dependency_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = p.E, k = p.k;
  if ((int)blockIdx.x >= p.tok_blocks) {
    const size_t n8 = (size_t)E * p.H / 8;
    const size_t step = (size_t)(gridDim.x - p.tok_blocks) * blockDim.x;
    for (size_t i = (size_t)(blockIdx.x - p.tok_blocks) * blockDim.x + threadIdx.x; i < n8; i += step) {
      const float4 a = reinterpret_cast<const float4 *>(p.W)[2 * i];
      const float4 b = reinterpret_cast<const float4 *>(p.W)[2 * i + 1];
      float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      reinterpret_cast<uint4 *>(p.Wp)[i] = take_bf16(v);
      reinterpret_cast<uint4 *>(p.Wp)[n8 + i] = take_bf16(v);
    }
    return;
  }
  float db[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) db[i] = 0.0f;
  for (int t = blockIdx.x * kPrepWarps + warp; t < p.T; t += p.tok_blocks * kPrepWarps) {
    // lane j < k: selection j
    int id = -1;
    float g = 0.0f;
    if (p.dw) {
      const bool sel = lane < k;
      id = sel ? p.idx[(size_t)t * k + lane] : -1;
      const bool bad = sel && (id < 0 || id >= E);
      if (__any_sync(0xffffffffu, bad)) {
        // the forward writes a zero row for such a token: dw has no meaning
        if (bad) set_status(p.status, STATUS_BAD_ROUTING);
        id = -1;
      } else {
        const float l = sel ? p.logits[(size_t)t * E + id] : 0.0f;
        const float dw = sel ? p.dw[(size_t)t * k + lane] : 0.0f;
        float w, slope;   // w_j / scale, and its factor in the gradient
        if (p.mode.sigmoid) {
          const float ex = expf(-l);
          const float s = sel ? __fdiv_rn(1.0f, 1.0f + ex) : 0.0f;
          float z = s;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
          // (a true division: one selected expert has w = 1 and no gradient)
          w = z == 0.0f ? 0.0f : __fdiv_rn(s, z);
          slope = s == 0.0f ? 0.0f : p.mode.scale * w * (ex * s);
        } else {
          float m = sel ? l : __int_as_float(0xff800000);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          const bool none = m == __int_as_float(0xff800000);
          const float ex = !sel || (none && l == m) ? 0.0f : expf(l - m);
          float z = ex;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
          w = z == 0.0f ? 0.0f : __fdiv_rn(ex, z);
          slope = w;
        }
        float dot = sel ? w * dw : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        g = sel ? slope * (dw - dot) : 0.0f;
      }
    }
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = 8 * lane + i;
      v[i] = p.dlogits && e < E ? p.dlogits[(size_t)t * E + e] : 0.0f;
    }
    if (p.dw) {
      for (int j = 0; j < k; ++j) {
        const int at = __shfl_sync(0xffffffffu, id, j) - 8 * lane;
        const float gj = __shfl_sync(0xffffffffu, g, j);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += at == i ? gj : 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) db[i] += v[i];
    if (p.dlp && 8 * lane < E) {
      const size_t row = (size_t)p.T * p.Epad / 8;
      uint4 *out = reinterpret_cast<uint4 *>(p.dlp) + (size_t)t * (p.Epad / 8) + lane;
      out[0] = take_bf16(v);
      out[row] = take_bf16(v);
      out[2 * row] = take_bf16(v);
    }
  }
  if (p.db_part) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s_db[warp][8 * lane + i] = db[i];
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
      float s = s_db[0][e];
#pragma unroll
      for (int w = 1; w < kPrepWarps; ++w) s += s_db[w][e];
      p.db_part[(size_t)blockIdx.x * E + e] = s;
    }
  }
}

// ---------------------------------------------------------------- tensor cores
// Both GEMMs read at least one operand along its rows, the K index running
// down them ("MN-major"): a box of 64 elements x R rows lands as R rows of 128
// bytes, 128-byte swizzled in groups of 8 rows.  The descriptor's leading
// offset is the distance between such boxes (64 elements further along M or
// N), its stride offset that between groups of 8 rows (8 further along K).
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t smem_addr, uint32_t box_bytes) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr >> 4) & 0x3FFF);
  d |= (uint64_t)(box_bytes >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// bf16 A and B, f32 accumulator; a_mn, b_mn: the operand is MN-major.
__device__ __forceinline__ uint32_t umma_idesc_bf16(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void tma_load_3d(void *dst, const void *tmap, int c0, int c1, int c2,
                                            uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

struct Ring {
  uint32_t st = 0, ph = 0;
  __device__ __forceinline__ void next(uint32_t stages) {
    if (++st == stages) {
      st = 0;
      ph ^= 1u;
    }
  }
};

constexpr int kMaxStages = 6;
constexpr int kSmemLimit = 232448;
constexpr uint32_t kTmem = 512;

// dW[e][h] = sum_t dl[t][e] x[t][h]: M = 128 rows of h (two accumulators: 256
// h a block), N = the experts, K = tokens.  All experts sit in one tile, so x
// is read from memory once; the tokens are split over blocks until the
// multiprocessors are full.  Stages of 32 tokens: x as 4 boxes, each piece of
// dl as experts / 64 boxes.
constexpr int kDwTok = 32;
constexpr int kDwBox = kDwTok * 128;
constexpr int kDwH = 256;
constexpr int kDwThreads = 192;   // producer, MMA, 4 epilogue warps

struct DwParams {
  int T, H, E, splits, stages;
  float *out;         // [splits][E][H]
  int *status;
};

__global__ void __launch_bounds__(kDwThreads, 1)
    route_grad_dw_kernel(const DwParams p, const __grid_constant__ CUtensorMap map_x,
                         const __grid_constant__ CUtensorMap map_dl) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full;
  __shared__ uint32_t s_tmem;
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&acc_full, 1);
    fence_mbar_init();
    prefetch_tmap(&map_x);
    prefetch_tmap(&map_dl);
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  grid_dependency_wait();
  grid_dependency_launch();

  const int h0 = blockIdx.x * kDwH, split = blockIdx.y;
  const int n_acc = p.H - h0 >= kDwH ? 2 : 1;
  const int nb = (p.E + 63) / 64;                     // boxes of 64 experts
  const int n_kb = (p.T + kDwTok - 1) / kDwTok;
  const int kb0 = (int)((long long)split * n_kb / p.splits);
  const int kb1 = (int)((long long)(split + 1) * n_kb / p.splits);
  const int stage_bytes = (kDwH / 64 + 3 * nb) * kDwBox;
  if (warp == 0) {
    if (lane == 0) {
      Ring r;
      int issued = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&empty[r.st], r.ph ^ 1u, p.status)) { ok = false; break; }
        uint8_t *a = smem + r.st * stage_bytes, *b = a + kDwH / 64 * kDwBox;
        mbar_arrive_expect_tx(&full[r.st], (uint32_t)((2 * n_acc + 3 * nb) * kDwBox));
        for (int i = 0; i < 2 * n_acc; ++i)
          tma_load_2d(a + i * kDwBox, &map_x, h0 + 64 * i, kb * kDwTok, &full[r.st]);
        for (int c = 0; c < 3; ++c)
          for (int i = 0; i < nb; ++i)
            tma_load_3d(b + (c * nb + i) * kDwBox, &map_dl, 64 * i, kb * kDwTok, c, &full[r.st]);
        ++issued;
        r.next(p.stages);
      }
      if (!ok)   // let issued copies land before the block exits
        for (int m = issued > p.stages ? issued - p.stages : 0; m < issued; ++m)
          (void)mbar_wait(&full[m % p.stages], (m / p.stages) & 1u, p.status);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      Ring r;
      const uint32_t idesc = umma_idesc_bf16(128, 64 * nb, true, true);
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&full[r.st], r.ph, p.status)) { ok = false; break; }
        tc_fence_after();
        const uint32_t a = smem_u32(smem + r.st * stage_bytes), b = a + kDwH / 64 * kDwBox;
#pragma unroll
        for (int ks = 0; ks < kDwTok / 16; ++ks)
          for (int c = 0; c < 3; ++c) {
            const uint64_t bd = umma_desc_mn_sw128(b + c * nb * kDwBox + ks * 2048, kDwBox);
            for (int m = 0; m < n_acc; ++m)
              umma_f16(tmem + m * 256, umma_desc_mn_sw128(a + m * 2 * kDwBox + ks * 2048, kDwBox), bd,
                       idesc, kb > kb0 || ks > 0 || c > 0 ? 1u : 0u);
          }
        umma_commit(&empty[r.st]);
        r.next(p.stages);
      }
      if (ok) umma_commit(&acc_full);
    }
  } else {
    // lane: one h of its quarter; column: one expert -> 128 consecutive bytes
    const int qd = warp & 3;
    const int okw = lane == 0 ? (mbar_wait(&acc_full, 0u, p.status) ? 1 : 0) : 0;
    if (__shfl_sync(0xffffffffu, okw, 0)) {
      tc_fence_after();
      for (int m = 0; m < n_acc; ++m) {
        float *out = p.out + (size_t)split * p.E * p.H + h0 + 128 * m + 32 * qd + lane;
        for (int c0 = 0; c0 < p.E; c0 += 32) {
          float v[32];
          tmem_ld_32x32b_x32(tmem + ((uint32_t)(32 * qd) << 16) + m * 256 + c0, v);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c0 + i < p.E) out[(size_t)(c0 + i) * p.H] = v[i];
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmem);
  }
}

// dx[t][h] = sum_e dl[t][e] W[e][h]: M = 128 rows of h, N = 256 tokens, K = the
// experts.  The block's W (both pieces, every expert) stays in shared memory
// while blocks of 256 tokens of dl stream past it in stages of 64 experts of
// one piece.  Work items (h tile, token tile), h-major, in one contiguous run
// per block: W is loaded again only where a run crosses into the next h tile.
constexpr int kDxTok = 256, kDxH = 128;
constexpr int kDxStage = kDxTok * 128;
constexpr int kDxWBox = 64 * 128;
constexpr int kDxEpiWarps = 8;
constexpr int kDxThreads = 32 * (2 + kDxEpiWarps);

struct DxParams {
  int T, H, E, stages;
  __nv_bfloat16 *out;   // [T][H]
  int *status;
};

__global__ void __launch_bounds__(kDxThreads, 1)
    route_grad_dx_kernel(const DxParams p, const __grid_constant__ CUtensorMap map_dl,
                         const __grid_constant__ CUtensorMap map_w) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], w_full, w_empty;
  __shared__ uint32_t s_tmem;
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], kDxEpiWarps);
    }
    mbar_init(&w_full, 1);
    mbar_init(&w_empty, 1);
    fence_mbar_init();
    prefetch_tmap(&map_dl);
    prefetch_tmap(&map_w);
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  grid_dependency_wait();
  grid_dependency_launch();

  const int n_kb = (p.E + 63) / 64;
  const int t_tiles = (p.T + kDxTok - 1) / kDxTok;
  const long long items = (long long)t_tiles * (p.H / kDxH);
  const long long i0 = items * blockIdx.x / gridDim.x, i1 = items * (blockIdx.x + 1) / gridDim.x;
  uint8_t *w_smem = smem;                              // [piece][k block][h half]
  uint8_t *ring = smem + 2 * n_kb * 2 * kDxWBox;
  if (warp == 0) {
    if (lane == 0) {
      Ring r;
      long long issued = 0;
      int cur = -1, w_uses = 0;
      bool ok = true;
      for (long long i = i0; i < i1 && ok; ++i) {
        const int h = (int)(i / t_tiles), t = (int)(i - (long long)h * t_tiles);
        if (h != cur) {
          if (cur >= 0 && !mbar_wait(&w_empty, (w_uses - 1) & 1u, p.status)) { ok = false; break; }
          cur = h;
          ++w_uses;
          mbar_arrive_expect_tx(&w_full, (uint32_t)(2 * n_kb * 2 * kDxWBox));
          for (int c = 0; c < 2; ++c)
            for (int kb = 0; kb < n_kb; ++kb)
              for (int m = 0; m < 2; ++m)
                tma_load_3d(w_smem + ((c * n_kb + kb) * 2 + m) * kDxWBox, &map_w, h * kDxH + 64 * m,
                            64 * kb, c, &w_full);
        }
        for (int q = 0; q < 2 * n_kb; ++q) {
          if (!mbar_wait(&empty[r.st], r.ph ^ 1u, p.status)) { ok = false; break; }
          mbar_arrive_expect_tx(&full[r.st], kDxStage);
          tma_load_3d(ring + r.st * kDxStage, &map_dl, 64 * (q >> 1), t * kDxTok, q & 1, &full[r.st]);
          ++issued;
          r.next(p.stages);
        }
      }
      if (!ok) {
        for (long long m = issued > p.stages ? issued - p.stages : 0; m < issued; ++m)
          (void)mbar_wait(&full[m % p.stages], (uint32_t)(m / p.stages) & 1u, p.status);
        if (w_uses) (void)mbar_wait(&w_full, (w_uses - 1) & 1u, p.status);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      Ring r;
      const uint32_t idesc = umma_idesc_bf16(kDxH, kDxTok, true, false);
      const uint32_t w0 = smem_u32(w_smem), b0 = smem_u32(ring);
      int cur = -1, w_uses = 0, n = 0;
      bool ok = true;
      for (long long i = i0; i < i1 && ok; ++i, ++n) {
        const int h = (int)(i / t_tiles);
        if (h != cur) {
          cur = h;
          if (!mbar_wait(&w_full, w_uses & 1u, p.status)) { ok = false; break; }
          ++w_uses;
        }
        const int buf = n & 1;
        if (!mbar_wait(&acc_empty[buf], ((n >> 1) & 1u) ^ 1u, p.status)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d = tmem + buf * 256;
        for (int kb = 0; kb < n_kb && ok; ++kb) {
          const int steps = min(4, (p.E - 64 * kb + 15) / 16);
          for (int c = 0; c < 2; ++c) {   // dl's piece: with both pieces of W, then with the first
            if (!mbar_wait(&full[r.st], r.ph, p.status)) { ok = false; break; }
            tc_fence_after();
            const uint64_t bd = umma_desc_sw128(b0 + r.st * kDxStage);
            for (int wc = 0; wc < 2 - c; ++wc) {
              const uint64_t ad = umma_desc_mn_sw128(w0 + (wc * n_kb + kb) * 2 * kDxWBox, kDxWBox);
              for (int ks = 0; ks < steps; ++ks)
                umma_f16(d, ad + ks * (2048 >> 4), bd + ks * (32 >> 4), idesc,
                         kb > 0 || c > 0 || wc > 0 || ks > 0 ? 1u : 0u);
            }
            umma_commit(&empty[r.st]);
            r.next(p.stages);
          }
        }
        if (!ok) break;
        umma_commit(&acc_full[buf]);
        if (i + 1 < i1 && (int)((i + 1) / t_tiles) != cur) umma_commit(&w_empty);
      }
    }
  } else {
    // lane: one h; column: one token.  Two steps of pairwise exchange give each
    // lane 4 consecutive h of one token of every four: 8-byte stores, 64
    // consecutive bytes a token.
    const int qd = warp & 3, half = (warp - 2) >> 2;
    int n = 0;
    for (long long i = i0; i < i1; ++i, ++n) {
      const int h = (int)(i / t_tiles), t0 = (int)(i - (long long)h * t_tiles) * kDxTok;
      const int buf = n & 1;
      const int okw = lane == 0 ? (mbar_wait(&acc_full[buf], (n >> 1) & 1u, p.status) ? 1 : 0) : 0;
      if (!__shfl_sync(0xffffffffu, okw, 0)) break;
      tc_fence_after();
      __nv_bfloat16 *out = p.out + (size_t)h * kDxH + 32 * qd + (lane & ~3);
      for (int c0 = 32 * half; c0 < kDxTok; c0 += 64) {
        float v[32];
        tmem_ld_32x32b_x32(tmem + ((uint32_t)(32 * qd) << 16) + buf * 256 + c0, v);
#pragma unroll
        for (int q = 0; q < 32; q += 4) {
          // lanes 4 l + s, columns q + s: transpose 4 x 4
          const bool odd = lane & 1, high = lane & 2;
          const float a = __shfl_xor_sync(0xffffffffu, odd ? v[q] : v[q + 1], 1);
          const float b = __shfl_xor_sync(0xffffffffu, odd ? v[q + 2] : v[q + 3], 1);
          // column q (even lanes) or q + 1 (odd): this pair of h; the same for q + 2, q + 3
          const __nv_bfloat162 lo = odd ? __floats2bfloat162_rn(a, v[q + 1]) : __floats2bfloat162_rn(v[q], a);
          const __nv_bfloat162 hi = odd ? __floats2bfloat162_rn(b, v[q + 3]) : __floats2bfloat162_rn(v[q + 2], b);
          const uint32_t keep = high ? bf162_bits(hi) : bf162_bits(lo);
          const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? bf162_bits(lo) : bf162_bits(hi), 2);
          const int t = t0 + c0 + q + (lane & 3);
          if (t < p.T)
            *reinterpret_cast<uint2 *>(out + (size_t)t * p.H) =
                high ? make_uint2(got, keep) : make_uint2(keep, got);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[buf]);
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmem);
  }
}

// dW = sum of its splits, db = sum of the prep blocks' parts, in order.
__global__ void __launch_bounds__(256) route_grad_sum_kernel(const RouteGradParams p, int splits,
                                                             int dw_blocks) {
  grid_dependency_wait();
  grid_dependency_launch();
  if ((int)blockIdx.x < dw_blocks) {
    const size_t n4 = (size_t)p.E * p.H / 4;
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n4) return;
    const float4 *part = reinterpret_cast<const float4 *>(p.dW_part) + i;
    float4 s = part[0];
    for (int k = 1; k < splits; ++k) {
      const float4 v = part[k * n4];
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    reinterpret_cast<float4 *>(p.dW)[i] = s;
    return;
  }
  // db: one warp per expert
  const int e = (blockIdx.x - dw_blocks) * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (e >= p.E) return;
  double s = 0.0;
  for (int b = lane; b < p.tok_blocks; b += 32) s += p.db_part[(size_t)b * p.E + e];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) p.db[e] = (float)s;
}

// ---------------------------------------------------------------- host
constexpr int kSms = 148;

int prep_blocks(int T) {
  const int n = (T + kPrepWarps - 1) / kPrepWarps;
  return n < 2 * kSms ? n : 2 * kSms;
}
int dw_tiles(int H) { return (H + kDwH - 1) / kDwH; }
// Shares of the tokens: as many as fill the multiprocessors, each of at least
// one stage.
int dw_splits(int T, int H) {
  const int n_kb = (T + kDwTok - 1) / kDwTok;
  int s = kSms / dw_tiles(H);
  if (s < 1) s = 1;
  return s < n_kb ? s : n_kb;
}

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct Layout {
  size_t dlp, wp, db, dw, total;
};
Layout layout(int T, int E, int H) {
  const int Epad = (E + 7) / 8 * 8;
  Layout L;
  size_t off = 0;
  L.dlp = off;
  off += up256((size_t)3 * T * Epad * 2);
  L.wp = off;
  off += up256((size_t)2 * E * H * 2);
  L.db = off;
  off += up256((size_t)prep_blocks(T) * E * 4);
  L.dw = off;
  const int splits = dw_splits(T, H);
  off += splits > 1 ? up256((size_t)splits * E * H * 4) : 0;
  L.total = off;
  return L;
}

// bf16 [planes][rows][cols], row stride ld elements, as boxes of 64 x box_rows
// (one plane), 128-byte swizzle; elements outside read as zero.
bool encode_planes(CUtensorMap *m, const void *base, int cols, int rows, int ld, int planes,
                   int box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)planes};
  cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)ld * 2 * rows};
  cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, planes > 1 ? 3 : 2, const_cast<void *>(base), dims,
             strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t route_grad_workspace(int T, int E, int H) { return layout(T > 0 ? T : 1, E, H).total; }

cudaError_t run_route_grad(RouteGradParams p, void *workspace, cudaStream_t stream) {
  const Layout L = layout(p.T, p.E, p.H);
  char *w = static_cast<char *>(workspace);
  p.Epad = (p.E + 7) / 8 * 8;
  p.tok_blocks = prep_blocks(p.T);
  p.dlp = p.dW || p.dx ? reinterpret_cast<__nv_bfloat16 *>(w + L.dlp) : nullptr;
  p.Wp = reinterpret_cast<__nv_bfloat16 *>(w + L.wp);
  p.db_part = p.db ? reinterpret_cast<float *>(w + L.db) : nullptr;
  const int splits = dw_splits(p.T, p.H);
  p.dW_part = splits > 1 ? reinterpret_cast<float *>(w + L.dw) : p.dW;
  const size_t n8 = (size_t)p.E * p.H / 8;
  const int w_blocks = p.dx ? (int)std::min<size_t>((n8 + 255) / 256, 4 * kSms) : 0;
  cudaError_t e = launch_pdl(route_grad_prep_kernel, dim3(p.tok_blocks + w_blocks),
                             dim3(32 * kPrepWarps), 0, stream, p);
  const int nb = (p.E + 63) / 64;
  if (e == cudaSuccess && p.dW) {
    CUtensorMap mx, md;
    if (!encode_planes(&mx, p.x, p.H, p.T, p.H, 1, kDwTok) ||
        !encode_planes(&md, p.dlp, p.E, p.T, p.Epad, 3, kDwTok))
      return cudaErrorInvalidValue;
    const int stage = (kDwH / 64 + 3 * nb) * kDwBox;
    DwParams d{p.T, p.H, p.E, splits, std::min(kMaxStages, (kSmemLimit - 2048) / stage), p.dW_part,
               p.status};
    const int smem = d.stages * stage + 1024;
    e = cudaFuncSetAttribute(route_grad_dw_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
      e = launch_pdl(route_grad_dw_kernel, dim3(dw_tiles(p.H), splits), dim3(kDwThreads), smem, stream,
                     d, mx, md);
  }
  if (e == cudaSuccess && p.dx) {
    CUtensorMap md, mw;
    if (!encode_planes(&md, p.dlp, p.E, p.T, p.Epad, 3, kDxTok) ||
        !encode_planes(&mw, p.Wp, p.H, p.E, p.H, 2, 64))
      return cudaErrorInvalidValue;
    const int wb = 2 * nb * 2 * kDxWBox;
    DxParams d{p.T, p.H, p.E, std::min(kMaxStages, (kSmemLimit - 2048 - wb) / kDxStage), p.dx, p.status};
    const int smem = wb + d.stages * kDxStage + 1024;
    const long long items = (long long)((p.T + kDxTok - 1) / kDxTok) * (p.H / kDxH);
    e = cudaFuncSetAttribute(route_grad_dx_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
      e = launch_pdl(route_grad_dx_kernel, dim3((unsigned)std::min<long long>(items, kSms)),
                     dim3(kDxThreads), smem, stream, d, md, mw);
  }
  const int dw_blocks = p.dW && splits > 1 ? (int)(((size_t)p.E * p.H / 4 + 255) / 256) : 0;
  const int db_blocks = p.db ? (p.E + 7) / 8 : 0;
  if (e == cudaSuccess && dw_blocks + db_blocks > 0)
    e = launch_pdl(route_grad_sum_kernel, dim3(dw_blocks + db_blocks), dim3(256), 0, stream, p, splits,
                   dw_blocks);
  return e;
}

}  // namespace strata
