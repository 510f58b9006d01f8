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
// Three launches: the operands in 16 bits; dW on the tensor cores (tcgen05,
// accumulators in tensor memory); dx on the tensor cores, whose spare warps, and
// after dx the others, add up the parts of dW and db.  A few tokens take one launch
// on the fp32 units instead (few_tokens below).
//
// 8192 tokens x 256 experts x 4096: 89 us replayed, 106 with fresh inputs (alone
// and with caches flushed the preparation takes 13, dW 45, dx 44).  Both products
// are bound by the tensor cores: 51.5 GFLOP each for three pieces, dW's on 64 of
// the 74 pairs of blocks.  2048 x 32 x 4096: 20.6 us replayed, the latency of three
// launches over 35 MB.
//
// fp32 operands on 16-bit tensor cores.  dW needs fp32 accuracy: x is bf16
// already, and dl is taken as the sum of three bf16 numbers (its rounding, the
// rounding of what is left, and again: 24 bits): three exact products per
// element, added in fp32.  dx is rounded to bf16 at the end, but rows of dl that
// come from a softmax sum to zero, so that whatever the rows of W have in common
// cancels in dl W, and what a rounding of the operands loses of it does not: with
// one f16 number (11 bits) for each, a common part of 16 times the rows' spread
// made dx three times less exact than its last rounding, one of 64 eleven times.
// So dl and W are two f16 numbers each (22 bits), three products per element (the
// two small parts' left out): 18 us more than with one of 8192 tokens x 256 experts
// x 4096, 0.6 to 1 with 32 experts.  Each row of dl and each 32 columns of W is first
// multiplied by the power of two that puts its largest magnitude in [2^14, 2^15),
// the top of f16's range: whatever the sizes of the weights, what is lost below
// f16's normal range is 2^-39 of the largest.

#include <cuda.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "launch.h"

namespace strata {

namespace {

constexpr int kPrepWarps = 16;

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

// Over groups of `lanes` (a power of two) lanes.
__device__ __forceinline__ float group_sum(float v, int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < lanes) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float group_max(float v, int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < lanes) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// A token's inputs, over the lanes of its group: lane j < k its selection j, lane j
// the gradients of logits 8 j ..
struct TokenIn {
  int id;
  float dw, l;
  float dl[8];
};
// Everything but the selected logit (whose place the id gives).
__device__ __forceinline__ void load_token(const RouteGradParams &p, long long t, int j, bool vec,
                                           TokenIn &in) {
  in.id = -1;
  in.dw = in.l = 0.0f;
  if (p.dw && t < p.T && j < p.k) {
    in.id = p.idx[t * p.k + j];
    in.dw = p.dw[t * p.k + j];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) in.dl[i] = 0.0f;
  if (!p.dlogits || t >= p.T) return;
  const float *row = p.dlogits + t * p.E + 8 * j;
  if (vec) {
    if (8 * j < p.E) {
      const float4 a = reinterpret_cast<const float4 *>(row)[0];
      const float4 b = reinterpret_cast<const float4 *>(row)[1];
      in.dl[0] = a.x; in.dl[1] = a.y; in.dl[2] = a.z; in.dl[3] = a.w;
      in.dl[4] = b.x; in.dl[5] = b.y; in.dl[6] = b.z; in.dl[7] = b.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (8 * j + i < p.E) in.dl[i] = row[i];
  }
}
// The selected logits; a token with an id out of range (the forward writes it a
// zero row, so dw has no meaning) loses its selections.  group: its lanes.
__device__ __forceinline__ void load_selected(const RouteGradParams &p, long long t, int j, unsigned group,
                                              TokenIn &in) {
  if (!p.dw) return;
  const bool sel = t < p.T && j < p.k;
  const bool bad = sel && (in.id < 0 || in.id >= p.E);
  const unsigned any_bad = __ballot_sync(0xffffffffu, bad) & group;
  if (bad) set_status(p.status, STATUS_BAD_ROUTING);
  if (any_bad) in.id = -1;
  if (sel && in.id >= 0) in.l = p.logits[t * p.E + in.id];
}

// Lane j of a token's group of lanes: the gradient of selection j's logit
// through the routing weights, from the logit l and dw (id < 0: no selection).
__device__ __forceinline__ float weight_grad(const RouteMode &mode, int id, float l, float dw, int lanes) {
  const bool use = id >= 0;
  float w, slope;   // w_j / scale, and its factor in the gradient
  if (mode.sigmoid) {
    const float ex = expf(-l);
    const float s = use ? __fdiv_rn(1.0f, 1.0f + ex) : 0.0f;
    const float z = group_sum(s, lanes);
    // (a true division: one selected expert has w = 1 and no gradient)
    w = z == 0.0f ? 0.0f : __fdiv_rn(s, z);
    slope = s == 0.0f ? 0.0f : mode.scale * w * (ex * s);
  } else {
    const float m = group_max(use ? l : __int_as_float(0xff800000), lanes);
    const bool none = m == __int_as_float(0xff800000);
    const float ex = !use || (none && l == m) ? 0.0f : expf(l - m);
    const float z = group_sum(ex, lanes);
    w = z == 0.0f ? 0.0f : __fdiv_rn(ex, z);
    slope = w;
  }
  const float dot = group_sum(use ? w * dw : 0.0f, lanes);
  return use ? slope * (dw - dot) : 0.0f;
}

// Two floats -> their f16 roundings and those of what is left.
__device__ __forceinline__ void split_f16(float a, float b, uint32_t &hi, uint32_t &lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  hi = h2_bits(h);
  lo = h2_bits(__floats2half2_rn(a - f.x, b - f.y));
}
// What takes a largest magnitude m to [2^14, 2^15), and back (m below 2^-112: as
// far as a power of two goes, 2^126).
struct F16Scale {
  float mul, back;
};
__device__ __forceinline__ F16Scale f16_scale(float m) {
  const int ex = min(max((int)(__float_as_uint(m) >> 23) - 127, -112), 127);
  return {__uint_as_float((uint32_t)(127 + 14 - ex) << 23), __uint_as_float((uint32_t)(127 - 14 + ex) << 23)};
}
constexpr int kWCols = 32;             // columns of W that share a scale
// Router weights from here on are reported (STATUS_RANGE) where dx is wanted.
constexpr float kWLimit = kF16Overflow / 256.0f;

// Blocks 0 .. tok_blocks - 1: rows of dl, a group of kG lanes per token, each lane
// 8 consecutive experts, as three bf16 pieces and as two of scaled f16, and the
// block's share of db.  The blocks behind them: 32 columns of W likewise, all experts
// in registers between the search for the largest and the rounding.  (kG holds the
// experts and the selections; a warp per token whatever their number made the whole
// call over 8192 tokens x 32 experts x 4096 take 44.1 us, 42.2 with 8 lanes each, both
// with dx in one product.  Two blocks a multiprocessor: with 72 registers a thread
// and one, 8192 tokens x 256 experts took 4 us more.)
template <int kG>
__global__ void __launch_bounds__(32 * kPrepWarps, 2) route_grad_prep_kernel(const RouteGradParams p) {
  constexpr int kTok = 32 / kG;   // tokens a warp works on at once
  // a row per group: the scattered selections, at the end the sums for db
  __shared__ __align__(16) float s_row[kPrepWarps * kTok][8 * kG];
  for (int i = threadIdx.x; i < kPrepWarps * kMaxExperts; i += blockDim.x) (&s_row[0][0])[i] = 0.0f;
  __syncthreads();
  grid_dependency_wait();
  grid_dependency_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = p.E;
  if ((int)blockIdx.x >= p.tok_blocks) {
    constexpr int kRows = 32 * kPrepWarps / (kWCols / 4);   // experts at once
    constexpr int kTurns = kMaxExperts / kRows;
    const int tile = (int)blockIdx.x - p.tok_blocks, e0 = threadIdx.x / (kWCols / 4);
    const size_t at = (size_t)e0 * p.H + kWCols * tile + 4 * (threadIdx.x % (kWCols / 4));
    float4 v[kTurns];
#pragma unroll
    for (int k = 0; k < kTurns; ++k)
      v[k] = e0 + k * kRows < E ? *reinterpret_cast<const float4 *>(p.W + at + (size_t)k * kRows * p.H)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < kTurns; ++k)
      m = fmaxf(m, fmaxf(fmaxf(fabsf(v[k].x), fabsf(v[k].y)), fmaxf(fabsf(v[k].z), fabsf(v[k].w))));
    const bool over = m >= kWLimit;
    m = group_max(m, 32);
    float *most = &s_row[0][0];
    if (lane == 0) most[warp] = m;
    __syncthreads();
    const F16Scale scale = f16_scale(group_max(most[lane % kPrepWarps], kPrepWarps));
#pragma unroll
    for (int k = 0; k < kTurns; ++k)
      if (e0 + k * kRows < E) {
        uint2 hi, lo;
        split_f16(v[k].x * scale.mul, v[k].y * scale.mul, hi.x, lo.x);
        split_f16(v[k].z * scale.mul, v[k].w * scale.mul, hi.y, lo.y);
        __half *out = p.W16 + at + (size_t)k * kRows * p.H;
        *reinterpret_cast<uint2 *>(out) = hi;
        *reinterpret_cast<uint2 *>(out + (size_t)E * p.H) = lo;
      }
    if (threadIdx.x == 0) p.w_scale[tile] = scale.back;
    if (over) set_status(p.status, STATUS_RANGE);
    return;
  }
  const int j = lane % kG, base = lane - j;   // the group's lanes: base ..
  const unsigned group = (kG == 32 ? 0xffffffffu : (1u << (kG & 31)) - 1u) << base;
  float *row = s_row[warp * kTok + lane / kG];
  const bool vec = E % 8 == 0 && (reinterpret_cast<uintptr_t>(p.dlogits) & 15) == 0;
  float db[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) db[i] = 0.0f;
  auto finish = [&](long long t, TokenIn &in) {   // (all lanes of the warp, past the last token too)
    float (&v)[8] = in.dl;
    if (p.dw) {
      // scattered through a row of shared memory that is zero in between; of
      // lanes with the same expert the first adds up all, in lane order
      float g = weight_grad(p.mode, in.id, in.l, in.dw, kG);
      const unsigned same = __match_any_sync(0xffffffffu, in.id) & group;
      const bool first = (same & ((1u << lane) - 1u)) == 0u && in.id >= 0;
      if (__any_sync(0xffffffffu, in.id >= 0 && (same & (same - 1u)) != 0u)) {
        float sum = 0.0f;
        for (int q = 0; q < p.k; ++q) {
          const float gq = __shfl_sync(0xffffffffu, g, base + q);
          if ((same >> (base + q)) & 1u) sum += gq;
        }
        g = sum;
      }
      if (first) row[in.id] = g;
      __syncwarp();
      const float4 a = reinterpret_cast<const float4 *>(row)[2 * j];
      const float4 b = reinterpret_cast<const float4 *>(row)[2 * j + 1];
      v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
      v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
      __syncwarp();
      if (first) row[in.id] = 0.0f;
      __syncwarp();   // before another lane writes there: the next token's, or db's sums
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) db[i] += v[i];
    const size_t at = (size_t)t * (p.Epad / 8) + j;
    const bool out_here = t < p.T && 8 * j < E;
    if (p.dl16) {
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
      m = group_max(m, kG);
      const F16Scale scale = f16_scale(m);
      if (out_here) {
        uint4 hi, lo;
        split_f16(v[0] * scale.mul, v[1] * scale.mul, hi.x, lo.x);
        split_f16(v[2] * scale.mul, v[3] * scale.mul, hi.y, lo.y);
        split_f16(v[4] * scale.mul, v[5] * scale.mul, hi.z, lo.z);
        split_f16(v[6] * scale.mul, v[7] * scale.mul, hi.w, lo.w);
        uint4 *out = reinterpret_cast<uint4 *>(p.dl16) + at;
        out[0] = hi;
        out[(size_t)p.T * p.Epad / 8] = lo;
      }
      if (t < p.T && j == 0) p.t_scale[t] = scale.back;
    }
    if (p.dlp && out_here) {
      const size_t plane = (size_t)p.T * p.Epad / 8;
      uint4 *out = reinterpret_cast<uint4 *>(p.dlp) + at;
      out[0] = take_bf16(v);
      out[plane] = take_bf16(v);
      out[2 * plane] = take_bf16(v);
    }
  };
  // two tokens a turn: their loads are in flight together
  const long long step = (long long)p.tok_blocks * kPrepWarps * kTok;
  for (long long t0 = ((long long)blockIdx.x * kPrepWarps + warp) * kTok; t0 < p.T; t0 += 2 * step) {
    const long long t = t0 + lane / kG;
    TokenIn a, b;
    load_token(p, t, j, vec, a);
    load_token(p, t + step, j, vec, b);
    load_selected(p, t, j, group, a);
    load_selected(p, t + step, j, group, b);
    finish(t, a);
    if (t0 + step < p.T) finish(t + step, b);
  }
  if (p.db_part) {
#pragma unroll
    for (int i = 0; i < 8; ++i) row[8 * j + i] = db[i];
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
      float s = s_row[0][e];
#pragma unroll
      for (int w = 1; w < kPrepWarps * kTok; ++w) s += s_row[w][e];
      p.db_part[(size_t)blockIdx.x * E + e] = s;
    }
  }
}

// ---------------------------------------------------------------- tensor cores
// Both products run on pairs of blocks (clusters of two, tcgen05 cta_group::2):
// one MMA covers M = 256 rows of h, 128 in each block's tensor memory, and up
// to N = 256 columns, whose operand each block loads half of.  So the streamed
// operand crosses from L2 half as often as with one block per tile, which is
// what bounded that form.  Every block loads its own share into its own shared
// memory and counts the bytes on the first block's barrier; the first block's
// MMA thread issues for both, and its commits arrive at both.
//
// Both read at least one operand along its rows, the K index running down them
// ("MN-major"): a box of 64 elements x R rows lands as R rows of 128 bytes,
// 128-byte swizzled in groups of 8 rows.  The descriptor's leading offset is
// the distance between such boxes (64 elements further along M or N), its
// stride offset that between groups of 8 rows (8 further along K).
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t smem_addr, uint32_t box_bytes) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr >> 4) & 0x3FFF);
  d |= (uint64_t)(box_bytes >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// f32 accumulator, A and B both bf16 or both f16; a_mn, b_mn: the operand is
// MN-major.
__device__ __forceinline__ uint32_t umma_idesc_16(bool bf16, int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// The MMA warp runs its loop as a whole and one elected lane (always the same)
// issues: control flow and descriptors stay uniform, so that they live in
// uniform registers as the instruction wants them.  With a loop under
// `lane == 0` issuing took longer than the 128 cycles that the MMA itself takes
// (dx: 162-190 cycles each).
__device__ __forceinline__ void umma2_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on the barrier at this place in both blocks once all earlier MMAs of
// the elected lane have completed.
__device__ __forceinline__ void umma2_commit(uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive(uint32_t bar_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_addr) : "memory");
}
// Loads into this block's shared memory, counted on a barrier of either block
// of the pair (a shared::cluster address); issued, like the MMAs, by one lane of
// a warp that runs as a whole.
__device__ __forceinline__ void tma2_load_2d(void *dst, const void *tmap, int c0, int c1, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(smem_u32(dst)),
      "l"(tmap), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma2_load_3d(void *dst, const void *tmap, int c0, int c1, int c2,
                                             uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(smem_u32(dst)),
      "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// 16 columns of this warp's 32 tensor-memory lanes (one lane a thread).
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, float v[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// A tile of this block's shared memory -> global memory; rows and columns
// outside the tensor are left out.
__device__ __forceinline__ void tma_store_2d(const void *tmap, const void *src, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n\t"
      "cp.async.bulk.commit_group;" ::"l"(tmap),
      "r"(c0), "r"(c1), "r"(smem_u32(src))
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

constexpr int kMaxStages = 8;
constexpr int kSmemLimit = 232448;
constexpr uint32_t kTmem = 512;       // two accumulators of 256 columns
constexpr int kTileH = 256;           // rows of h per pair of blocks
constexpr int kEpiWarps = 8;
constexpr int kTcThreads = 32 * (2 + kEpiWarps);   // producer, MMA, epilogue

// Barriers of a block (those that count arrivals of both blocks live in the
// first one) and the pair's tensor memory.
struct PairShared {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], w_full[4], w_empty;
  uint32_t tmem;
};

__device__ __forceinline__ void pair_begin(PairShared &s, int stages, int epi_warps, int warp) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.acc_full[i], 1);
      mbar_init(&s.acc_empty[i], 2 * epi_warps);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&s.w_full[i], 1);
    mbar_init(&s.w_empty, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s.tmem)),
                 "r"(kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both blocks' barriers are set up before either signals
  tc_fence_after();
}
__device__ __forceinline__ void pair_end(PairShared &s, int warp) {
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // neither block leaves while the other may still reach it
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(s.tmem), "r"(kTmem)
                 : "memory");
  }
}
// Every lane tests the barrier and the warp votes; only if the phase is not
// complete yet does one lane wait, within its limit, and tell the others.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, int lane, int *status) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const int ok = lane == 0 ? (mbar_wait(bar, parity, status) ? 1 : 0) : 0;
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// dW[e][h] = sum_t dl[t][e] x[t][h]: M = 256 rows of h, N = the experts (all of
// them, so x is read from memory once), K = tokens in stages of 32 or 64.  The
// stages of all h tiles in one row are cut into equal runs, one per pair of
// blocks; a run's part of a tile goes to slot run + tile of the workspace (or
// straight to dW if it is the whole tile), and the last kernel adds the slots in
// order.
//
// The tensor core cuts its running sum at every MMA (2^-23 relative, always
// towards zero): over one chain of 910 tokens, 168 MMAs, dW came out 2.7e-6 too
// small.  So a chain is 48 MMAs long; the epilogue warps add the
// chains in fp32 registers, rounding to nearest, while the other accumulator
// takes the next chain.
//
// An MMA costs about 115 cycles at N = 128 and 128 at N = 256, so the pieces of
// dl share MMAs where the experts leave room (the pair's first block loads the
// first half of the columns, the second the rest):
//   form 0, up to 64 experts:   one MMA: hi 64 | mid 64 | lo 64 | (not used)
//   form 1, up to 128 experts:  two: hi 128 | mid 128, then lo 128 on top of hi
//   form 2, up to 256 experts:  three: hi, mid, lo, 256 columns each
// and the epilogue adds the columns of an expert.  Whole calls over 4096 h, in
// form 2 and in their own: 32 experts x 2048 tokens 26.5 and 19.9 us, 128 experts
// 29.0 and 23.2, 64 experts x 8192 tokens 59.4 and 43.2 (with dx in one product).
//
// A stage is 32 tokens in form 2 (7 stages of 32 KB) and 64 in the others, whose
// MMAs take less time than issuing the copies of so small boxes: a pair with a
// tile to itself (4096 h) takes 0.19 us per 32 tokens with 32 experts, 0.31 in
// stages of 32; with 128 experts 0.29 and 0.32, with 256 0.505 (3 stages of 64)
// and 0.50.
__host__ __device__ constexpr int dw_tok(int E) { return E <= 128 ? 64 : 32; }
template <int kForm>
struct DwForm {
  static constexpr int kTok = dw_tok(64 << kForm);           // tokens per stage
  static constexpr int kBox = kTok * 128;                    // bytes of 64 columns
  static constexpr int kCols = 32 << kForm;                  // experts per epilogue warp
  static constexpr int kSums = 3 - kForm;                    // column groups to add per expert
  static constexpr int kBoxes = kForm == 0 ? 2 : 3 * kForm;  // of dl, per block and stage
  static constexpr int kChain = (kForm == 0 ? 768 : kForm == 1 ? 384 : 256) / kTok;   // stages: 48 MMAs on hi
};

struct DwParams {
  int T, H, E, pairs, stages;
  float *out;          // dW
  float *part;         // [pairs + tiles - 1][E][256]
  int *status;
};
__host__ __device__ inline long long run_begin(long long units, int pairs, int i) {
  return units * i / pairs;
}

template <int kForm>
__global__ void __launch_bounds__(kTcThreads, 1)
    route_grad_dw_kernel(const DwParams p, const __grid_constant__ CUtensorMap map_x,
                         const __grid_constant__ CUtensorMap map_dl) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ PairShared s;
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    prefetch_tmap(&map_x);
    prefetch_tmap(&map_dl);
  }
  pair_begin(s, p.stages, kEpiWarps, warp);
  const uint32_t tmem = s.tmem, rank = cluster_rank();
  grid_dependency_wait();
  grid_dependency_launch();

  using F = DwForm<kForm>;
  constexpr int kTok = F::kTok, kBox = F::kBox;
  constexpr int kStage = (2 + F::kBoxes) * kBox;   // per block
  const int n_kb = (p.T + kTok - 1) / kTok;
  const int tiles = (p.H + kTileH - 1) / kTileH;
  const int pair = blockIdx.x >> 1;
  const long long units = (long long)tiles * n_kb;
  const long long u0 = run_begin(units, p.pairs, pair), u1 = run_begin(units, p.pairs, pair + 1);
  if (warp == 0) {
    Ring r;
    const int n = (int)(u1 - u0);
    int tile = (int)(u0 / n_kb), kb = (int)(u0 - (long long)tile * n_kb), issued = 0;
    const uint32_t bar0 = cluster_addr(&s.full[0], 0);
    bool ok = true;
    for (; issued < n; ++issued) {
      if (!warp_wait(&s.empty[r.st], r.ph ^ 1u, lane, p.status)) { ok = false; break; }
      const int t = kb * kTok, h = tile * kTileH + 128 * (int)rank;
      uint8_t *a = smem + r.st * kStage, *b = a + 2 * kBox;
      const uint32_t bar = bar0 + 8 * r.st;
      if (rank == 0 && lane == 0)
        mbar_arrive_expect_tx(&s.full[r.st], 2 * kStage - (kForm == 0 ? kBox : 0));
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 2; ++i) tma2_load_2d(a + i * kBox, &map_x, h + 64 * i, t, bar);
      const int rk = (int)rank;
      auto piece = [&](int box, int c, int e) { tma2_load_3d(b + box * kBox, &map_dl, e, t, c, bar); };
      if (kForm == 0) {
        piece(0, 2 * rk, 0);
        if (rk == 0) piece(1, 1, 0);
      } else if (kForm == 1) {
        piece(0, rk, 0);
        piece(1, rk, 64);
        piece(2, 2, 64 * rk);
      } else {
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          piece(2 * c, c, 128 * rk);
          piece(2 * c + 1, c, 128 * rk + 64);
        }
      }
      if (++kb == n_kb) {
        kb = 0;
        ++tile;
      }
      r.next(p.stages);
    }
    if (!ok && rank == 0 && lane == 0)   // let issued copies land
      for (int m = issued > p.stages ? issued - p.stages : 0; m < issued; ++m)
        (void)mbar_wait(&s.full[m % p.stages], (uint32_t)(m / p.stages) & 1u, p.status);
  } else if (warp == 1) {
    if (rank == 0) {
      Ring r;
      const uint32_t idesc = umma_idesc_16(true, 256, 256, true, true);
      const uint32_t idesc_lo = umma_idesc_16(true, 256, 128, true, true);   // form 1
      int n = 0;   // chains
      bool ok = true;
      for (long long u = u0; u < u1 && ok; ++n) {
        const int tile = (int)(u / n_kb);
        const long long end = min(min(u1, (long long)(tile + 1) * n_kb), u + F::kChain);
        const int buf = n & 1;
        if (!warp_wait(&s.acc_empty[buf], ((n >> 1) & 1u) ^ 1u, lane, p.status)) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * 256;
        uint32_t more = 0u;
        for (; u < end; ++u) {
          if (!warp_wait(&s.full[r.st], r.ph, lane, p.status)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a = smem_u32(smem + r.st * kStage);
          const uint64_t ad = umma_desc_mn_sw128(a, kBox);
          const uint64_t bd = umma_desc_mn_sw128(a + 2 * kBox, kBox);
#pragma unroll
          for (int ks = 0; ks < kTok / 16; ++ks) {
            const uint64_t ak = ad + ks * (2048 >> 4), bk = bd + ks * (2048 >> 4);
            umma2_f16(d, ak, bk, idesc, ks > 0 ? 1u : more);
            if (kForm == 1) umma2_f16(d, ak, bk + (2 * kBox >> 4), idesc_lo, 1u);
            if (kForm == 2) {
              umma2_f16(d, ak, bk + (2 * kBox >> 4), idesc, 1u);
              umma2_f16(d, ak, bk + (4 * kBox >> 4), idesc, 1u);
            }
          }
          more = 1u;
          umma2_commit(&s.empty[r.st]);
          r.next(p.stages);
        }
        if (ok) umma2_commit(&s.acc_full[buf]);
      }
    }
  } else {
    // lane: one h; column: one expert.  Each warp holds a quarter of the lanes
    // and half of the experts.
    constexpr int kCols = F::kCols;
    const int qd = warp & 3, half = (warp - 2) >> 2;
    const int hh = 128 * (int)rank + 32 * qd + lane;
    const uint32_t empty_bar[2] = {cluster_addr(&s.acc_empty[0], 0), cluster_addr(&s.acc_empty[1], 0)};
    int n = 0;
    bool ok = true;
    for (long long u = u0; u < u1 && ok;) {
      const int tile = (int)(u / n_kb);
      const long long tile0 = (long long)tile * n_kb, end = min(u1, tile0 + n_kb);
      const bool whole = u == tile0 && end == tile0 + n_kb;
      float acc[kCols];
#pragma unroll
      for (int i = 0; i < kCols; ++i) acc[i] = 0.0f;
      for (; u < end; u += F::kChain, ++n) {
        const int buf = n & 1;
        if (!warp_wait(&s.acc_full[buf], (n >> 1) & 1u, lane, p.status)) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int g = 0; g < F::kSums; ++g)   // (the small pieces' columns last)
#pragma unroll
          for (int c = 0; c < kCols; c += 16) {
            float v[16];
            tmem_ld_32x32b_x16(tmem + ((uint32_t)(32 * qd) << 16) + buf * 256 + 2 * kCols * g +
                                   half * kCols + c, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[c + i] += v[i];
          }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) cluster_arrive(empty_bar[buf]);
      }
      u = end;
      const int h = tile * kTileH + hh;
      if (!ok || h >= p.H) continue;
      float *out = whole ? p.out + h : p.part + ((size_t)(pair + tile) * p.E) * kTileH + hh;
      const size_t ld = whole ? p.H : kTileH;
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        if (half * kCols + i < p.E) out[(size_t)(half * kCols + i) * ld] = acc[i];
    }
  }
  pair_end(s, warp);
}

// ---- the last sums: dW from the runs' parts, db from the prep blocks' parts
struct SumParams {
  RouteGradParams g;
  int pairs;          // runs of the dW kernel
  int dw_rows;        // rows of 256 h to add up: tiles * E, or 0
};

// One warp: expert e's 256 h of one tile, 8 a lane.
__device__ __forceinline__ void sum_dw(const SumParams &q, int tile, int e, int lane) {
  const RouteGradParams &p = q.g;
  const int tiles = (p.H + kTileH - 1) / kTileH, n_kb = (p.T + dw_tok(p.E) - 1) / dw_tok(p.E);
  // the runs that hold units of this tile (run r starts at unit units r / pairs)
  const long long units = (long long)tiles * n_kb, first = (long long)tile * n_kb;
  const int r0 = (int)(((first + 1) * q.pairs - 1) / units);
  const int r1 = (int)(((first + n_kb) * q.pairs - 1) / units);
  if (r0 == r1) return;   // one run had the whole tile and wrote it
  const float4 *part =
      reinterpret_cast<const float4 *>(p.dW_part + ((size_t)(r0 + tile) * p.E + e) * kTileH) + lane;
  const size_t step = (size_t)p.E * kTileH / 4;
  float4 s[2] = {};
  for (int r = r0; r <= r1; r += 4) {
    float4 v[4][2];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        v[k][c] = r + k <= r1 ? __ldcg(part + k * step + 32 * c) : make_float4(0.f, 0.f, 0.f, 0.f);
    part += 4 * step;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        s[c].x += v[k][c].x;
        s[c].y += v[k][c].y;
        s[c].z += v[k][c].z;
        s[c].w += v[k][c].w;
      }
  }
  float4 *out = reinterpret_cast<float4 *>(p.dW + (size_t)e * p.H + tile * kTileH) + lane;
#pragma unroll
  for (int c = 0; c < 2; ++c)
    if (tile * kTileH + 128 * c < p.H) out[32 * c] = s[c];
}
// One warp: expert e.
__device__ __forceinline__ void sum_db(const RouteGradParams &p, int e, int lane) {
  double s = 0.0;
  float v[10];   // at most 296 blocks
#pragma unroll
  for (int k = 0; k < 10; ++k) {
    const int b = lane + 32 * k;
    v[k] = b < p.tok_blocks ? __ldcg(p.db_part + (size_t)b * p.E + e) : 0.0f;
  }
#pragma unroll
  for (int k = 0; k < 10; ++k) s += (double)v[k];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) p.db[e] = (float)s;
}
// Rows of all this: db's experts, then dW's rows of 256 h.
__host__ __device__ inline int sum_rows(const SumParams &q) { return (q.g.db ? q.g.E : 0) + q.dw_rows; }
// Rows [begin, end), by warp `warp` of `warps`.
__device__ __forceinline__ void sum_parts(const SumParams &q, int begin, int end, int warp, int warps, int lane) {
  const int n_db = q.g.db ? q.g.E : 0;
  for (int r = begin + warp; r < end; r += warps) {
    if (r < n_db) {
      sum_db(q.g, r, lane);
    } else {
      const int i = r - n_db, tile = i / q.g.E;
      sum_dw(q, tile, i - tile * q.g.E, lane);
    }
  }
}
// ... in a launch of its own, where dx is not wanted.
__global__ void __launch_bounds__(256) route_grad_sum_kernel(const SumParams q) {
  grid_dependency_wait();
  grid_dependency_launch();
  sum_parts(q, 0, sum_rows(q), blockIdx.x * 8 + (threadIdx.x >> 5), gridDim.x * 8, threadIdx.x & 31);
}

// dx[t][h] = sum_e dl[t][e] W[e][h]: M = 256 tokens, N = 256 rows of h, K = the
// experts, in f16: dl's large part by both parts of W, its small part by W's
// large one.  W's share of the tile (every expert, both parts) stays in shared
// memory while tokens stream past it in stages of 64 experts of one part.  Work
// items (h tile, token tile), h-major, in one contiguous run per pair: W is loaded
// again only where a run crosses into the next h tile.  With 256 experts an item
// is 48 MMAs (6144 cycles), below 64 hardly any: there writing dx is what counts.
// Each lane scales its token's row, writes bf16 to a swizzled tile of its warp, and
// a bulk store takes the 64 h out; above 192 experts, where W leaves no room for
// four stages of tokens beside such tiles, 32 h at a time.  (Stores straight from
// registers, 32 bytes each: 8192 tokens x 32 experts x 4096 50.0 us, 44.1 this way;
// with 256 experts the same.)  Every index is kept by adding: with a 64-bit
// division for each item in every warp an item began 700 cycles later.
constexpr int kDxTok = 256;
constexpr int kDxStage = kDxTok / 2 * 128;   // per block
constexpr int kDxWBox = 64 * 128;
constexpr int kDxOut = 32 * 64;              // 32 tokens x 32 h of bf16: half of a tile
constexpr int kDxEpiWarps = 16;
constexpr int kSumWarps = 4;
constexpr int kDxThreads = 32 * (2 + kDxEpiWarps + kSumWarps);

struct DxParams {
  int T, H, E, stages;
  int out_halves;         // of a tile, per epilogue warp: 1 or 2
  int t_tiles;            // of 256 tokens
  int per, extra;         // items of a pair; that many pairs take one more
  int after_dw;           // the kernel before this one on the stream is dW's
  int spare_rows;         // rows of the sums that the spare warps take
  const float *t_scale;   // [T]
  const float *w_scale;   // [H / 32]
  int *status;
};

__global__ void __launch_bounds__(kDxThreads, 1)
    route_grad_dx_kernel(const DxParams p, const SumParams q, const __grid_constant__ CUtensorMap map_dl,
                         const __grid_constant__ CUtensorMap map_w,
                         const __grid_constant__ CUtensorMap map_dx) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ PairShared s;
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    prefetch_tmap(&map_dl);
    prefetch_tmap(&map_w);
    prefetch_tmap(&map_dx);
  }
  pair_begin(s, p.stages, kDxEpiWarps, warp);
  const uint32_t tmem = s.tmem, rank = cluster_rank();
  // dx needs what the preparation wrote, and the dW kernel lets this grid start
  // only once all its blocks have waited for the preparation, whose writes are then
  // in L2: only the warps that add up dW's parts wait for the dW kernel itself, so
  // that dx runs beside it wherever multiprocessors are free (128 tokens x 64
  // experts x 2048: 10.5 us, 13.4 with every warp waiting; both with dx in one
  // product).  The programming model promises those writes only to a thread that
  // waits itself; here they are read by bulk tensor loads and __ldcg, which go to
  // L2, never through an L1 that could hold older lines.  What this needs: every
  // block of dW waits before it lets this grid start, the warps above read nothing
  // that dW's kernel writes, and dx shares no memory with x (the host refuses it).
  if (!p.after_dw || warp >= 2 + kDxEpiWarps) {
    grid_dependency_wait();
    grid_dependency_launch();
  }

  const int n_kb = (p.E + 63) / 64;
  const int pair = blockIdx.x >> 1, items = p.per + (pair < p.extra);
  const int first = pair * p.per + min(pair, p.extra);
  int h = first / p.t_tiles, t = first - h * p.t_tiles;   // the item's tiles of h and of tokens
  auto next_item = [&] {
    if (++t == p.t_tiles) {
      t = 0;
      ++h;
    }
  };
  uint8_t *w_smem = smem;                              // [part][k block][half of the block's 128 h]
  const int w_part = n_kb * 2 * kDxWBox;
  uint8_t *ring = smem + 2 * w_part;
  uint8_t *out_smem = ring + p.stages * kDxStage;      // [epilogue warp]
  if (warp == 0) {
    Ring r;
    int issued = 0, cur = -1, w_uses = 0;
    const uint32_t bar0 = cluster_addr(&s.full[0], 0), w_bar0 = cluster_addr(&s.w_full[0], 0);
    bool ok = true;
    for (int n = 0; n < items && ok; ++n, next_item()) {
      const bool fresh = h != cur;
      if (fresh) {
        if (cur >= 0 && !warp_wait(&s.w_empty, (w_uses - 1) & 1u, lane, p.status)) { ok = false; break; }
        cur = h;
        ++w_uses;
      }
      for (int kb = 0; kb < n_kb; ++kb) {
        if (fresh) {
          if (rank == 0 && lane == 0) mbar_arrive_expect_tx(&s.w_full[kb], 8 * kDxWBox);
          __syncwarp();
#pragma unroll
          for (int m = 0; m < 4; ++m)
            tma2_load_3d(w_smem + (m / 2) * w_part + (kb * 2 + m % 2) * kDxWBox, &map_w,
                         h * kTileH + 128 * (int)rank + 64 * (m % 2), 64 * kb, m / 2, w_bar0 + 8 * kb);
        }
        for (int part = 0; part < 2; ++part) {
          if (ok && !warp_wait(&s.empty[r.st], r.ph ^ 1u, lane, p.status)) ok = false;
          if (!ok) break;   // (every copy of W that a barrier expects is still issued)
          if (rank == 0 && lane == 0) mbar_arrive_expect_tx(&s.full[r.st], 2 * kDxStage);
          __syncwarp();
          tma2_load_3d(ring + r.st * kDxStage, &map_dl, 64 * kb, t * kDxTok + kDxTok / 2 * (int)rank, part,
                       bar0 + 8 * r.st);
          ++issued;
          r.next(p.stages);
        }
      }
    }
    if (!ok && rank == 0 && lane == 0) {   // let issued copies land
      for (int m = issued > p.stages ? issued - p.stages : 0; m < issued; ++m)
        (void)mbar_wait(&s.full[m % p.stages], (uint32_t)(m / p.stages) & 1u, p.status);
      for (int kb = 0; w_uses && kb < n_kb; ++kb) (void)mbar_wait(&s.w_full[kb], (w_uses - 1) & 1u, p.status);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      Ring r;
      const uint32_t idesc = umma_idesc_16(false, kDxTok, kTileH, false, true);
      const uint64_t bd0 = umma_desc_mn_sw128(smem_u32(w_smem), kDxWBox);
      const uint64_t ad0 = umma_desc_sw128(smem_u32(ring));
      int cur = -1, w_uses = 0;
      bool ok = true;
      for (int n = 0; n < items && ok; ++n, next_item()) {
        const bool fresh = h != cur;
        if (fresh) {
          cur = h;
          ++w_uses;
        }
        const int buf = n & 1;
        if (!warp_wait(&s.acc_empty[buf], ((n >> 1) & 1u) ^ 1u, lane, p.status)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d = tmem + buf * 256;
        for (int kb = 0; kb < n_kb; ++kb) {
          if (fresh && !warp_wait(&s.w_full[kb], (w_uses - 1) & 1u, lane, p.status)) { ok = false; break; }
          const int steps = min(4, (p.E - 64 * kb + 15) / 16);
          const uint64_t bd = bd0 + (uint64_t)(kb * (2 * kDxWBox >> 4)), bd_lo = bd + (uint64_t)(w_part >> 4);
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            if (!warp_wait(&s.full[r.st], r.ph, lane, p.status)) { ok = false; break; }
            tc_fence_after();
            const uint64_t ad = ad0 + (uint64_t)(r.st * (kDxStage >> 4));
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              if (ks < steps) {
                umma2_f16(d, ad + ks * (32 >> 4), bd + ks * (2048 >> 4), idesc, part || kb > 0 || ks > 0 ? 1u : 0u);
                if (part == 0) umma2_f16(d, ad + ks * (32 >> 4), bd_lo + ks * (2048 >> 4), idesc, 1u);
              }
            umma2_commit(&s.empty[r.st]);
            r.next(p.stages);
          }
          if (!ok) break;
        }
        if (!ok) break;
        umma2_commit(&s.acc_full[buf]);
        if (n + 1 < items && t + 1 == p.t_tiles) umma2_commit(&s.w_empty);
      }
    }
  } else if (warp < 2 + kDxEpiWarps) {
    // lane: one token; column: one h.  Each warp: a quarter of the block's 128
    // tokens and 64 of the columns.
    const int qd = warp & 3, col = 64 * ((warp - 2) >> 2);
    const uint32_t empty_bar[2] = {cluster_addr(&s.acc_empty[0], 0), cluster_addr(&s.acc_empty[1], 0)};
    uint8_t *tile = out_smem + (warp - 2) * p.out_halves * kDxOut;
    const bool half = p.out_halves == 1;
    for (int n = 0; n < items; ++n, next_item()) {
      const int tok0 = t * kDxTok + kDxTok / 2 * (int)rank + 32 * qd;
      const float scale = tok0 + lane < p.T ? __ldcg(p.t_scale + tok0 + lane) : 0.0f;
      // of the warp's two 32 columns (H is a multiple of 128)
      const int h0 = h * kTileH + col;
      const float2 w_scale =
          h0 < p.H ? __ldcg(reinterpret_cast<const float2 *>(p.w_scale + h0 / kWCols)) : make_float2(0.f, 0.f);
      const int buf = n & 1;
      if (!warp_wait(&s.acc_full[buf], (n >> 1) & 1u, lane, p.status)) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float v[32];
        tmem_ld_32x32b_x32(tmem + ((uint32_t)(32 * qd) << 16) + buf * 256 + col + 32 * c, v);
        const float ws = c == 0 ? w_scale.x : w_scale.y;
        if (c == 1) {   // the accumulator is in registers
          tc_fence_before();
          __syncwarp();
          if (lane == 0) cluster_arrive(empty_bar[buf]);
        }
        if (c == 0 || half) {   // the tile's last store has read it
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            // (one after the other: the product of the two may leave fp32's range)
            o[j] = bf162_bits(__floats2bfloat162_rn(v[8 * k + 2 * j] * scale * ws,
                                                    v[8 * k + 2 * j + 1] * scale * ws));
          const int at = half ? lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)
                              : lane * 128 + (((4 * c + k) ^ (lane & 7)) << 4);
          *reinterpret_cast<uint4 *>(tile + at) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        if (c == 1 || half) {
          fence_async_smem();
          __syncwarp();
          if (lane == 0 && h0 < p.H && tok0 < p.T) tma_store_2d(&map_dx, tile, half ? h0 + 32 * c : h0, tok0);
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
    if (p.spare_rows < sum_rows(q)) {
      grid_dependency_wait();
      sum_parts(q, p.spare_rows, sum_rows(q), blockIdx.x * kDxEpiWarps + warp - 2, gridDim.x * kDxEpiWarps, lane);
    }
  } else {
    sum_parts(q, 0, p.spare_rows, blockIdx.x * kSumWarps + warp - 2 - kDxEpiWarps, gridDim.x * kSumWarps, lane);
  }
  pair_end(s, warp);
}

// ---------------------------------------------------------------- few tokens
// The whole of it in one launch on the fp32 units: a block per 16 or 32 h
// computes dl (every block the same) into shared memory and takes its columns of
// dW and dx.  The three launches of the other form take 9 to 15 us however small
// the batch is; this one takes 5 us with one token.
constexpr int kSmallThreads = 1024;

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(void *dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Threads that share a tile of dW (four experts x one h; n tiles).
__host__ __device__ inline int small_parts(int n) {
  int parts = 1;
  while (parts < 16 && 2 * parts * n <= kSmallThreads) parts *= 2;
  return parts;
}
// Shared memory: dl [T][Ep] and W [Ep][hs] in fp32, x [T][hs] in bf16, the parts
// of dW; Ep: the experts rounded up to four.
struct SmallSmem {
  size_t red, total;
};
// h a block: 16, or 32 where that would be more blocks than multiprocessors.
inline int small_hs(int H) { return H / 16 > 148 ? 32 : 16; }
SmallSmem small_smem(int T, int E, int H) {
  const int hs = small_hs(H);
  const size_t Ep = (E + 3) / 4 * 4;
  const int n = (int)Ep / 4 * hs, parts = small_parts(n);
  const size_t red = 4 * (T * Ep + Ep * hs) + (size_t)2 * T * hs;
  return {red, red + (parts > 1 ? (size_t)n * parts * 16 : 0)};
}

template <int kSmallH>
__global__ void __launch_bounds__(kSmallThreads) route_grad_small_kernel(const RouteGradParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  grid_dependency_wait();
  grid_dependency_launch();
  const int T = p.T, E = p.E, k = p.k, H = p.H, Ep = (E + 3) & ~3;
  float *dl = reinterpret_cast<float *>(smem_raw);
  float *ws = dl + (size_t)T * Ep;
  __nv_bfloat16 *xs = reinterpret_cast<__nv_bfloat16 *>(ws + Ep * kSmallH);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h0 = blockIdx.x * kSmallH;
  // everything that is read as it is, in flight at once
  if (p.dlogits && Ep == E && (reinterpret_cast<uintptr_t>(p.dlogits) & 15) == 0) {
    for (int i = tid; i < T * E / 4; i += kSmallThreads) cp_async16(dl + 4 * i, p.dlogits + 4 * i);
  } else {
    for (int t = warp; t < T; t += kSmallThreads / 32)
      for (int e = lane; e < Ep; e += 32) {
        if (p.dlogits && e < E)
          cp_async4(dl + t * Ep + e, p.dlogits + (size_t)t * E + e);
        else
          dl[t * Ep + e] = 0.0f;
      }
  }
  if (p.dW)
    for (int i = tid; i < T * (kSmallH / 8); i += kSmallThreads)
      cp_async16(xs + 8 * i, p.x + (size_t)(i / (kSmallH / 8)) * H + h0 + 8 * (i % (kSmallH / 8)));
  if (p.dx)
    for (int i = tid; i < Ep * (kSmallH / 4); i += kSmallThreads) {
      const int e = i / (kSmallH / 4);
      if (e < E)
        cp_async16(ws + 4 * i, p.W + (size_t)e * H + h0 + 4 * (i % (kSmallH / 4)));
      else
        *reinterpret_cast<float4 *>(ws + 4 * i) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  // meanwhile the gradient through the routing weights: a group of lanes (the
  // power of two that holds k) per token
  int lanes = 1;
  while (lanes < k) lanes *= 2;
  const int at_once = kSmallThreads / lanes;
  bool met = false;
  auto meet = [&] {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    met = true;
  };
  if (p.dw) {
    const int j = lane & (lanes - 1);
    const unsigned group = (lanes == 32 ? 0xffffffffu : (1u << lanes) - 1u) << (lane - j);
    for (int t0 = 0; t0 < T; t0 += at_once) {
      const int t = t0 + tid / lanes;
      const bool sel = t < T && j < k;
      int id = sel ? p.idx[(size_t)t * k + j] : -1;
      const float dw = sel ? p.dw[(size_t)t * k + j] : 0.0f;
      const bool bad = sel && (id < 0 || id >= E);
      if (bad) set_status(p.status, STATUS_BAD_ROUTING);
      if (__ballot_sync(0xffffffffu, bad) & group) id = -1;   // (as the other form)
      const float l = id >= 0 ? p.logits[(size_t)t * E + id] : 0.0f;
      const float g = weight_grad(p.mode, id, l, dw, lanes);
      // of lanes of the token with the same expert the first adds up all
      float sum = 0.0f;
      bool first = id >= 0;
      for (int q = 0; q < k; ++q) {
        const int from = lane - j + q;
        const int other = __shfl_sync(0xffffffffu, id, from);
        const float og = __shfl_sync(0xffffffffu, g, from);
        if (other == id) {
          sum += og;
          first = first && q >= j;
        }
      }
      if (!met) meet();
      if (first) dl[t * Ep + id] += sum;
    }
  }
  if (!met) meet();
  __syncthreads();
  if (p.dx) {   // (the limit of the other form: what is refused does not go by the batch)
    bool over = false;
    for (int i = tid; i < E * kSmallH; i += kSmallThreads) over |= fabsf(ws[i]) >= kWLimit;
    if (over) set_status(p.status, STATUS_RANGE);
  }
  // dW: four experts of one h a thread; where that leaves threads over, the
  // tokens are split between up to 16 of them, whose sums meet below
  const int n = Ep / 4 * kSmallH, parts = small_parts(n);
  float4 *red = reinterpret_cast<float4 *>(smem_raw + p.small_red);   // [parts][n]
  auto put = [&](int tile, const float4 &a) {
    const int h = tile % kSmallH, e = tile / kSmallH * 4;
    float *out = p.dW + (size_t)e * H + h0 + h;
    out[0] = a.x;
    if (e + 1 < E) out[H] = a.y;
    if (e + 2 < E) out[2 * (size_t)H] = a.z;
    if (e + 3 < E) out[3 * (size_t)H] = a.w;
  };
  if (p.dW) {
    for (int q = tid; q < n * parts; q += kSmallThreads) {
      const int part = q / n, tile = q - part * n;
      const int h = tile % kSmallH, e = tile / kSmallH * 4;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int t = part; t < T; t += parts) {
        const float4 d = *reinterpret_cast<const float4 *>(dl + t * Ep + e);
        const float x = __bfloat162float(xs[t * kSmallH + h]);
        a.x = fmaf(d.x, x, a.x);
        a.y = fmaf(d.y, x, a.y);
        a.z = fmaf(d.z, x, a.z);
        a.w = fmaf(d.w, x, a.w);
      }
      if (parts == 1)
        put(tile, a);
      else
        red[q] = a;
    }
  }
  // dx: two h of a token a thread (the threads in reverse, so that those without
  // a part of dW go first)
  if (p.dx) {
    for (int q = kSmallThreads - 1 - tid; q < T * (kSmallH / 2); q += kSmallThreads) {
      const int h = q % (kSmallH / 2) * 2, t = q / (kSmallH / 2);
      float a0 = 0.0f, a1 = 0.0f;
#pragma unroll 2
      for (int e = 0; e < Ep; e += 4) {
        const float4 d = *reinterpret_cast<const float4 *>(dl + t * Ep + e);
        const float dv[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 w = *reinterpret_cast<const float2 *>(ws + (e + i) * kSmallH + h);
          a0 = fmaf(dv[i], w.x, a0);
          a1 = fmaf(dv[i], w.y, a1);
        }
      }
      *reinterpret_cast<__nv_bfloat162 *>(p.dx + (size_t)t * H + h0 + h) = __floats2bfloat162_rn(a0, a1);
    }
  }
  if (p.dW && parts > 1) {
    __syncthreads();
    for (int tile = tid; tile < n; tile += kSmallThreads) {
      float4 a = red[tile];
      for (int part = 1; part < parts; ++part) {
        const float4 v = red[part * n + tile];
        a.x += v.x;
        a.y += v.y;
        a.z += v.z;
        a.w += v.w;
      }
      put(tile, a);
    }
  }
  // db: a warp per expert, the experts spread over the blocks
  if (p.db)
    for (int e = blockIdx.x + gridDim.x * warp; e < E; e += gridDim.x * (kSmallThreads / 32)) {
      float v = 0.0f;
      for (int t = lane; t < T; t += 32) v += dl[t * Ep + e];
      v = group_sum(v, 32);
      if (lane == 0) p.db[e] = v;
    }
}

// ---------------------------------------------------------------- host
constexpr int kPairs = 74;   // 148 multiprocessors
// Limits of dynamic shared memory, the same in every call whatever it needs: they
// belong to the kernel, and calls of several threads must not lower them under one
// another.
constexpr int kTcSmem = kSmemLimit - 1024;
constexpr int kSmallSmem = 116 * 1024;
static_assert(4 * kPairs <= 320, "sum_db reads up to 320 blocks' parts");

// Lanes of the preparation per token: the power of two that holds the experts, 8 a
// lane, and the selections.
int prep_lanes(int E, int k) {
  int g = 8;
  while (8 * g < E || g < k) g *= 2;
  return g;
}
// (the selections of 32 lanes at the most: what the workspace's size goes by)
int prep_blocks(int T, int lanes) {
  const int per = kPrepWarps * 32 / lanes, n = (T + per - 1) / per;
  return n < 4 * kPairs ? n : 4 * kPairs;
}
int h_tiles(int H) { return (H + kTileH - 1) / kTileH; }
// Pairs of blocks for dW.  Each tile of h takes the same number m of runs (so
// that no run has parts of two tiles), or the stages of all tiles are cut into 74
// runs wherever that falls.  More runs are shorter, but every part of a tile is
// written and read again, only then can dW be added up, and pairs that dW leaves
// free have dx to do.  The costs below, in us, follow measurements of whole calls
// at 256 to 7168 h, 32 to 256 experts, 64 to 8192 tokens.  E.g. 4096 h x 256
// experts: 256 tokens 17.7 us with m = 1, 27.0 with 4, 27.9 with 74 runs; 1024
// tokens 35.6, 29.6 (29.2 with 3, which is taken) and 30.8; 8192 tokens 163, 87.6
// and 85.8.  1024 h x 32 experts: 1024 tokens 11.6 with m = 8, 13.4 with 18; 8192
// tokens 21.4 and 20.0.  7168 h x 256 experts: 8192 tokens 141 with m = 2, 137
// with 74 runs.
int dw_pairs(int T, int E, int H) {
  const int tiles = h_tiles(H);
  const long long n_kb = (T + dw_tok(E) - 1) / dw_tok(E);
  const double share = E / 256.0;
  const double tile = T / 32.0 * (0.15 + 0.35 * share);   // one pair alone
  const double part = 0.03 + 0.10 * share;
  const double cut = 1.9;                                  // any parts at all
  const long long most = std::min<long long>(kPairs, tiles * n_kb);
  // (a run with parts of two tiles writes twice: 4 us with 256 experts)
  int best = (int)most;
  double cost = tile * tiles / most + (tiles % most == 0 ? 0.0 : cut + part * (most + tiles) + 0.5 + 4.0 * share);
  for (long long m = 1; m * tiles <= most; ++m) {
    const double c = tile / m + (m > 1 ? cut + part * m * tiles : 0.0);
    if (c < cost) {
      cost = c;
      best = (int)(m * tiles);
    }
  }
  return best;
}

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct Layout {
  size_t dlp, dl16, t_scale, w16, w_scale, db, dw, total;
};
Layout layout(int T, int E, int H) {
  const int Epad = (E + 7) / 8 * 8;
  Layout L;
  size_t off = 0;
  L.dlp = off;
  off += up256((size_t)3 * T * Epad * 2);
  L.dl16 = off;
  off += up256((size_t)2 * T * Epad * 2);
  L.t_scale = off;
  off += up256((size_t)T * 4);
  L.w16 = off;
  off += up256((size_t)2 * E * H * 2);
  L.w_scale = off;
  off += up256((size_t)H / kWCols * 4);
  L.db = off;
  off += up256((size_t)prep_blocks(T, 32) * E * 4);
  L.dw = off;
  off += up256((size_t)(dw_pairs(T, E, H) + h_tiles(H)) * E * kTileH * 4);
  L.total = off;
  return L;
}

// 16-bit elements [planes][rows][cols], row stride ld elements, as boxes of
// box_cols (64 or 32) x box_rows (one plane), swizzled over their 128 or 64 bytes;
// elements outside read as zero.
bool encode_planes(CUtensorMap *m, CUtensorMapDataType type, const void *base, int cols, int rows, int ld, int planes,
                   int box_cols, int box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)planes};
  cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)ld * 2 * rows};
  cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, type, planes > 1 ? 3 : 2, const_cast<void *>(base), dims,
             strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t route_grad_workspace(int T, int E, int H) { return layout(T > 0 ? T : 1, E, H).total; }

// One launch on the fp32 units while it is the shorter of the two, by times, in
// us, that follow measurements of both forms from 8 to 256 experts and 256 to
// 16384 h: a block's products, its rows of dl, and as many rounds of blocks as
// there are; the other form's launches, and its preparation of more experts.  E.g.
// 2048 h: 8 experts 9.5 against 10.8 us with 320 tokens, 14.2 against 11.8 with
// 640; 64 experts 8.5 against 11.0 with 80, 13.3 against 11.3 with 160; 128
// experts 10.1 against 11.8 with 60, 18.5 against 12.4 with 140; 7168 h x 64
// experts 8.8 against 10.1 with 10, 12.9 against 10.7 with 40.  In between it is up
// to 1.5 us off (2048 h x 64 experts x 110 tokens: 9.8 against 11.3, taken).  (At
// most 78 KB of shared memory.)
bool few_tokens(int T, int E, int H) {
  const int hs = small_hs(H);
  const double rounds = std::max(1.0, H / hs / 148.0);
  const double products = (double)T * ((E + 3) / 4 * 4) * hs / 1024;
  return rounds * (4.6 + 0.042 * products + 0.0105 * T) < 10.1 + 0.027 * std::max(0, E - 64) + 0.0018 * T;
}

cudaError_t run_route_grad(RouteGradParams p, void *workspace, cudaStream_t stream) {
  if (few_tokens(p.T, p.E, p.H)) {
    const SmallSmem layout = small_smem(p.T, p.E, p.H);
    const int smem = (int)layout.total, hs = small_hs(p.H);
    p.small_red = (int)layout.red;
    auto kern = hs == 16 ? route_grad_small_kernel<16> : route_grad_small_kernel<32>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmallSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(p.H / hs), dim3(kSmallThreads), smem, stream, p);
  }
  const Layout L = layout(p.T, p.E, p.H);
  char *w = static_cast<char *>(workspace);
  p.Epad = (p.E + 7) / 8 * 8;
  const int lanes = prep_lanes(p.E, p.k);
  p.tok_blocks = prep_blocks(p.T, lanes);
  p.dlp = p.dW ? reinterpret_cast<__nv_bfloat16 *>(w + L.dlp) : nullptr;
  p.dl16 = p.dx ? reinterpret_cast<__half *>(w + L.dl16) : nullptr;
  p.t_scale = reinterpret_cast<float *>(w + L.t_scale);
  p.W16 = reinterpret_cast<__half *>(w + L.w16);
  p.w_scale = reinterpret_cast<float *>(w + L.w_scale);
  p.db_part = p.db ? reinterpret_cast<float *>(w + L.db) : nullptr;
  p.dW_part = reinterpret_cast<float *>(w + L.dw);
  const int w_blocks = p.dx ? p.H / kWCols : 0;
  cudaError_t e = launch_pdl(lanes == 8    ? route_grad_prep_kernel<8>
                             : lanes == 16 ? route_grad_prep_kernel<16>
                                           : route_grad_prep_kernel<32>,
                             dim3(p.tok_blocks + w_blocks), dim3(32 * kPrepWarps), 0, stream, p);
  const auto kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kF16 = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const int pairs = dw_pairs(p.T, p.E, p.H), tiles = h_tiles(p.H);
  if (e == cudaSuccess && p.dW) {
    CUtensorMap mx, md;
    const int form = p.E <= 64 ? 0 : p.E <= 128 ? 1 : 2, tok = dw_tok(p.E);
    if (!encode_planes(&mx, kBf16, p.x, p.H, p.T, p.H, 1, 64, tok) ||
        !encode_planes(&md, kBf16, p.dlp, p.E, p.T, p.Epad, 3, 64, tok))
      return cudaErrorInvalidValue;
    const int stage = (2 + (form == 0 ? DwForm<0>::kBoxes : form == 1 ? DwForm<1>::kBoxes
                                                                      : DwForm<2>::kBoxes)) * tok * 128;
    DwParams d{p.T, p.H, p.E, pairs, std::min(kMaxStages, (kSmemLimit - 2048) / stage), p.dW, p.dW_part,
               p.status};
    const int smem = d.stages * stage + 1024;
    auto kern = form == 0   ? route_grad_dw_kernel<0>
                : form == 1 ? route_grad_dw_kernel<1>
                            : route_grad_dw_kernel<2>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmem);
    if (e == cudaSuccess)
      e = launch_pdl_cluster(kern, dim3(2 * pairs), 2, dim3(kTcThreads), smem, stream, d, mx, md);
  }
  const SumParams q{p, pairs, p.dW && tiles % pairs != 0 ? tiles * p.E : 0};
  if (e == cudaSuccess && p.dx) {
    const int halves = p.E > 192 ? 1 : 2;
    CUtensorMap md, mw, mo;
    if (!encode_planes(&md, kF16, p.dl16, p.E, p.T, p.Epad, 2, 64, kDxTok / 2) ||
        !encode_planes(&mw, kF16, p.W16, p.H, p.E, p.H, 2, 64, 64) ||
        !encode_planes(&mo, kBf16, p.dx, p.H, p.T, p.H, 1, halves == 1 ? 32 : 64, 32))
      return cudaErrorInvalidValue;
    const int fixed = (p.E + 63) / 64 * 4 * kDxWBox + kDxEpiWarps * halves * kDxOut;
    const int t_tiles = (p.T + kDxTok - 1) / kDxTok, items = t_tiles * tiles;
    DxParams d{p.T, p.H, p.E, std::min(kMaxStages, (kSmemLimit - 2048 - fixed) / kDxStage), halves, t_tiles,
               0, 0, p.dW ? 1 : 0, 0, p.t_scale, p.w_scale, p.status};
    const int smem = fixed + d.stages * kDxStage + 1024;
    // (pairs without an item of dx help with the sums, a row of 256 or an expert
    // per warp; not many more than dW leaves room for, since those start late: 1024
    // tokens x 256 h x 256 experts 18.5 us with 64 pairs, 18.2 with 37)
    const int sums = sum_rows(q);
    const int help = std::min((sums + 2 * kSumWarps - 1) / (2 * kSumWarps), std::max(kPairs - pairs, kPairs / 2));
    const int grid = std::min(std::max(items, help), kPairs);
    d.per = items / grid;
    d.extra = items % grid;
    // a row takes a spare warp about 1.2 us and an item of dx its pair 2.3 to 3.6: what the
    // spare warps would not have done by the end of dx, the epilogue's do then (2048
    // tokens x 1024 h x 256 experts: 21.3 us, 24.7 with the spare warps alone)
    d.spare_rows = (int)std::min<long long>(sums, 2LL * grid * kSumWarps * (1 + 2 * (items / grid)));
    e = cudaFuncSetAttribute(route_grad_dx_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmem);
    if (e == cudaSuccess)
      e = launch_pdl_cluster(route_grad_dx_kernel, dim3(2 * grid), 2, dim3(kDxThreads), smem, stream, d, q, md, mw, mo);
  } else if (e == cudaSuccess && sum_rows(q)) {
    const int blocks = (sum_rows(q) + 7) / 8;
    e = launch_pdl(route_grad_sum_kernel, dim3(blocks), dim3(256), 0, stream, q);
  }
  return e;
}

}  // namespace strata
