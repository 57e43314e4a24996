// Kernels 11 and 12: the adapters of short requests (up to kLoraShortRows rows: a decoding token, the one
// conditioning row of the adaptive normalisation).
//
// Mathematics.  out[m] = y[m] + sum_j w_j B_j (A_j x[m]); the plan has gathered rows with the same
// adapters, up to 16, into groups, so that a group's A and B are read once.  With so few rows the
// weights are the traffic: r (K + N) bf16 values per adapter against K + 2 N per row.
//
// Kernel 11 forms u = w A x of a group, 16 ranks per CTA: mma.sync m16n8k16 with the 16 adapter
// rows as M and the group's rows as N.  The k index of a fragment may be permuted as long as both
// operands agree, so a lane takes 8 neighbouring k of its row with one 16-byte load (two MMAs)
// and no shared memory is needed.  The warps share K; their sums are added in warp order.  A long
// K with few groups is also split over CTAs (ks): each writes its part, and kernel 12 adds the parts
// in order.  Kernel 12 forms B u the same way, 16 output columns per warp and step as M; u (32
// bits) enters as a high and a low bf16 part, which keeps it to 2^-16 relative.
#pragma once

#include "lora_plan.h"
#include "ptx.cuh"

namespace svdq {
namespace k11 {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int G = kLoraGroupRows;

struct Params {
  const __nv_bfloat16 *X, *A, *B, *Yin;
  __nv_bfloat16* Y;
  long long ldx, ldyin, ldy;
  const int32_t* groups;                   // the plan's group records
  float* part;                             // [groups][ks][16 rows][slots rank]
  int N, K, rank, slots, ks;
  int ngroups;                             // groups with adapters; groups after them are copied
  int early;                               // kernel 12: kernel 11 comes before it
};

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8), bf16: lane (g = lane / 4, t = lane % 4) holds rows g and
// g + 8 of A, column g of B, and columns 2 t, 2 t + 1 of D's rows g and g + 8.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The bits of u's bf16 rounding, and what is left of u (nothing where that is infinite, so that an
// overflow stays an infinity).
__device__ __forceinline__ uint16_t split_hi_lo(float u, float& lo) {
  const __nv_bfloat16 h = __float2bfloat16_rn(u);
  const float hf = __bfloat162float(h);
  lo = isinf(hf) ? 0.f : u - hf;
  return __bfloat16_as_ushort(h);
}

__global__ void __launch_bounds__(kThreads)
lora_short_down_kernel(const Params p) {
  __shared__ float red[kWarps][16][G + 1];
  grid_dependency_wait();                          // X may come from the previous kernel
  grid_launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int32_t* rec = p.groups + static_cast<size_t>(blockIdx.x) * lora_group_words(p.slots);
  const int nrows = rec[0];
  const int slot = blockIdx.y * 16 / p.rank, r0 = blockIdx.y * 16 % p.rank;
  const int id = rec[4 + slot];
  float d[2][4] = {};
  if (id >= 0) {
    const __nv_bfloat16* a_lo = p.A + (static_cast<size_t>(id) * p.rank + r0 + g) * p.K + 8 * t;
    const __nv_bfloat16* a_hi = a_lo + static_cast<size_t>(8) * p.K;
    const __nv_bfloat16* x_lo = g < nrows ? p.X + rec[12 + g] * p.ldx + 8 * t : nullptr;
    const __nv_bfloat16* x_hi = g + 8 < nrows ? p.X + rec[12 + g + 8] * p.ldx + 8 * t : nullptr;
    const int steps = p.K / 32;
    const int end = static_cast<int>(static_cast<long long>(steps) * (blockIdx.z + 1) / p.ks);
#pragma unroll 4
    for (int s = static_cast<int>(static_cast<long long>(steps) * blockIdx.z / p.ks) + warp; s < end; s += kWarps) {
      const uint4 z = make_uint4(0u, 0u, 0u, 0u);
      const uint4 al = __ldg(reinterpret_cast<const uint4*>(a_lo + 32 * s));
      const uint4 ah = __ldg(reinterpret_cast<const uint4*>(a_hi + 32 * s));
      const uint4 xl = x_lo ? __ldg(reinterpret_cast<const uint4*>(x_lo + 32 * s)) : z;
      mma16816(d[0], al.x, ah.x, al.y, ah.y, xl.x, xl.y);
      mma16816(d[0], al.z, ah.z, al.w, ah.w, xl.z, xl.w);
      if (nrows > 8) {
        const uint4 xh = x_hi ? __ldg(reinterpret_cast<const uint4*>(x_hi + 32 * s)) : z;
        mma16816(d[1], al.x, ah.x, al.y, ah.y, xh.x, xh.y);
        mma16816(d[1], al.z, ah.z, al.w, ah.w, xh.z, xh.w);
      }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    red[warp][g][8 * h + 2 * t] = d[h][0];
    red[warp][g][8 * h + 2 * t + 1] = d[h][1];
    red[warp][g + 8][8 * h + 2 * t] = d[h][2];
    red[warp][g + 8][8 * h + 2 * t + 1] = d[h][3];
  }
  __syncthreads();
  const int r = threadIdx.x % 16, i = threadIdx.x / 16;    // rank of the block, row of the group
  if (i < nrows) {
    float u = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) u += red[w][r][i];
    const float wt = __int_as_float(rec[12 + G + i * p.slots + slot]);
    const int jr = p.slots * p.rank;
    p.part[((static_cast<size_t>(blockIdx.x) * p.ks + blockIdx.z) * G + i) * jr + blockIdx.y * 16 + r] =
        id >= 0 ? u * wt : 0.f;
  }
}

constexpr int kUStride = kLoraMaxRank + 8;         // bf16 per row of u in shared memory

// kWide: 32 ranks per step, a lane's share of a row of B one 16-byte load (rank % 32 == 0); else 16 and an
// 8-byte load.  kSteps = slots rank / (32 or 16).  A warp's next 16 columns of B and y are in flight while it
// works on the present ones, and the first are requested before the grid's dependency: kernel 11 lets this
// grid start after its own dependency wait, so B, y and the plan are complete by then.
template <bool kWide, int kSteps>
__global__ void __launch_bounds__(kThreads)
lora_short_up_kernel(const Params p) {
  constexpr int kSpan = kWide ? 32 : 16;           // ranks per step
  constexpr int kWords = kWide ? 4 : 2;            // 32-bit words of a row of B per lane and step
  __shared__ __align__(16) uint16_t uh[G * kUStride], ul[G * kUStride];
  __shared__ __align__(16) float ds[kWarps][G][20];
  __shared__ int32_t head[4 + 8 + G];              // the record's rows, ids and row indexes
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int32_t* rec = p.groups + static_cast<size_t>(blockIdx.x) * lora_group_words(p.slots);
  if (!p.early) grid_dependency_wait();
  if (threadIdx.x < 4 + 8 + G) head[threadIdx.x] = __ldcg(rec + threadIdx.x);
  __syncthreads();
  const int nrows = head[0];
  const int jr = p.slots * p.rank;
  const int step_n = gridDim.y * kWarps * 16;
  const int yi = lane / 2, yc = 8 * (lane % 2);    // this lane's row of the group and columns of y
  const long long yrow = yi < nrows ? head[12 + yi] : 0;

  const bool copied = static_cast<int>(blockIdx.x) >= p.ngroups;   // rows that no adapter touches
  const uint32_t* brow[kSteps];                    // this lane's words of row g of each step's block of B
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int id = copied ? -1 : head[4 + s * kSpan / p.rank];
    brow[s] = id < 0 ? nullptr
                     : reinterpret_cast<const uint32_t*>(p.B + (static_cast<size_t>(id) * p.N + g) * p.rank +
                                                         s * kSpan % p.rank + kSpan / 4 * t);
  }
  uint32_t bl[kSteps][kWords], bh[kSteps][kWords]; // rows n0 + g and n0 + g + 8
  uint4 y = make_uint4(0u, 0u, 0u, 0u);
  auto fetch = [&](int n0) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (!brow[s]) {
#pragma unroll
        for (int w = 0; w < kWords; ++w) bl[s][w] = bh[s][w] = 0u;
        continue;
      }
      const uint32_t* lo = brow[s] + static_cast<size_t>(n0) * p.rank / 2;
      const uint32_t* hi = lo + 4 * p.rank;
      if constexpr (kWide) {
        const uint4 a = __ldcg(reinterpret_cast<const uint4*>(lo)), b = __ldcg(reinterpret_cast<const uint4*>(hi));
        bl[s][0] = a.x; bl[s][1] = a.y; bl[s][2] = a.z; bl[s][3] = a.w;
        bh[s][0] = b.x; bh[s][1] = b.y; bh[s][2] = b.z; bh[s][3] = b.w;
      } else {
        const uint2 a = __ldcg(reinterpret_cast<const uint2*>(lo)), b = __ldcg(reinterpret_cast<const uint2*>(hi));
        bl[s][0] = a.x; bl[s][1] = a.y;
        bh[s][0] = b.x; bh[s][1] = b.y;
      }
    }
    if (yi < nrows) y = __ldcg(reinterpret_cast<const uint4*>(p.Yin + yrow * p.ldyin + n0 + yc));
  };
  int n0 = (blockIdx.y * kWarps + warp) * 16;
  if (n0 < p.N) fetch(n0);
  if (p.early) grid_dependency_wait();             // the parts of u
  grid_launch_dependents();
  if (copied) {
    for (; n0 < p.N; n0 += step_n) {
      if (yi < nrows) *reinterpret_cast<uint4*>(p.Y + yrow * p.ldy + n0 + yc) = y;
      if (n0 + step_n < p.N) fetch(n0 + step_n);
    }
    return;
  }
  for (int i = threadIdx.x; i < G * jr; i += kThreads) {
    const int row = i / jr, c = i % jr;
    float u = 0.f;
    if (row < nrows) {
      const float* src = p.part + (static_cast<size_t>(blockIdx.x) * p.ks * G + row) * jr + c;
      for (int z = 0; z < p.ks; ++z) u += __ldcg(src + static_cast<size_t>(z) * G * jr);
    }
    float lo;
    uh[row * kUStride + c] = split_hi_lo(u, lo);
    ul[row * kUStride + c] = __bfloat16_as_ushort(__float2bfloat16_rn(lo));
  }
  __syncthreads();
  const int nt = nrows > 8 ? 2 : 1;
  for (; n0 < p.N; n0 += step_n) {
    float d[2][4] = {};
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int c = s * kSpan + kSpan / 4 * t;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h >= nt) continue;
#pragma unroll
        for (int w = 0; w < kWords; w += 2) {
          const uint2 vh = *reinterpret_cast<const uint2*>(uh + (8 * h + g) * kUStride + c + 2 * w);
          const uint2 vl = *reinterpret_cast<const uint2*>(ul + (8 * h + g) * kUStride + c + 2 * w);
          mma16816(d[h], bl[s][w], bh[s][w], bl[s][w + 1], bh[s][w + 1], vh.x, vh.y);
          mma16816(d[h], bl[s][w], bh[s][w], bl[s][w + 1], bh[s][w + 1], vl.x, vl.y);
        }
      }
    }
    const uint4 yv = y;
    if (n0 + step_n < p.N) fetch(n0 + step_n);
    // through shared memory: a lane adds 8 columns of one row
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      ds[warp][8 * h + 2 * t][g] = d[h][0];
      ds[warp][8 * h + 2 * t + 1][g] = d[h][1];
      ds[warp][8 * h + 2 * t][g + 8] = d[h][2];
      ds[warp][8 * h + 2 * t + 1][g + 8] = d[h][3];
    }
    __syncwarp();
    if (yi < nrows) {
      const float* v = &ds[warp][yi][yc];
      const float4 v0 = *reinterpret_cast<const float4*>(v), v1 = *reinterpret_cast<const float4*>(v + 4);
      uint4 o;
      o.x = pack_bf16x2(bf16lo_to_f32(yv.x) + v0.x, bf16hi_to_f32(yv.x) + v0.y);
      o.y = pack_bf16x2(bf16lo_to_f32(yv.y) + v0.z, bf16hi_to_f32(yv.y) + v0.w);
      o.z = pack_bf16x2(bf16lo_to_f32(yv.z) + v1.x, bf16hi_to_f32(yv.z) + v1.y);
      o.w = pack_bf16x2(bf16lo_to_f32(yv.w) + v1.z, bf16hi_to_f32(yv.w) + v1.w);
      *reinterpret_cast<uint4*>(p.Y + yrow * p.ldy + n0 + yc) = o;
    }
    __syncwarp();
  }
}

}  // namespace k11
}  // namespace svdq
