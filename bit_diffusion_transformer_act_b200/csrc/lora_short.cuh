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
// in order.  Kernel 12 forms B u the same way, with the group's rows as M; u (32 bits) enters as a high and a low
// bf16 part, which keeps it to 2^-16 relative.
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
  int depth;                               // kernel 12: pieces on their way per warp
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
    // Ordinary loads: X, or an adapter, may have been written while this grid was already resident, which the
    // read-only path (ld.global.nc, __ldg) does not allow.
    const int steps = p.K / 32;
    const int end = static_cast<int>(static_cast<long long>(steps) * (blockIdx.z + 1) / p.ks);
#pragma unroll 4
    for (int s = static_cast<int>(static_cast<long long>(steps) * blockIdx.z / p.ks) + warp; s < end; s += kWarps) {
      const uint4 z = make_uint4(0u, 0u, 0u, 0u);
      const uint4 al = *reinterpret_cast<const uint4*>(a_lo + 32 * s);
      const uint4 ah = *reinterpret_cast<const uint4*>(a_hi + 32 * s);
      const uint4 xl = x_lo ? *reinterpret_cast<const uint4*>(x_lo + 32 * s) : z;
      mma16816(d[0], al.x, ah.x, al.y, ah.y, xl.x, xl.y);
      mma16816(d[0], al.z, ah.z, al.w, ah.w, xl.z, xl.w);
      if (nrows > 8) {
        const uint4 xh = x_hi ? *reinterpret_cast<const uint4*>(x_hi + 32 * s) : z;
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
constexpr int kUpWarps = 4;
constexpr int kUpThreads = kUpWarps * 32;
constexpr int kUpCols = 32;                        // output columns per piece (a warp's step)
__host__ __device__ constexpr int up_piece_bytes(int jr) { return kUpCols * jr * 2; }   // of B
constexpr int kUpRingBytes = 45 * 1024;            // per CTA: four per SM (three where two stages need more)
constexpr int kUpMaxDepth = 8;

// kWide: 32 ranks per step, a lane's share of a row of B 16 bytes (rank % 32 == 0); else 16 ranks and 8 bytes.
// kSteps = slots rank / (32 or 16).  The group's rows are the MMAs' M here, and their operand, u's hi and lo
// fragments, stays in registers for all of a group's columns.  Four MMAs of 8 columns make a piece; column c of the
// j-th is the piece's column 8 (c / 2) + 2 j + c % 2, so that a lane's eight sums are neighbours in a row and
// y is read and written 16 bytes at a time without an exchange.  (With B's rows as M and the tile turned through
// shared memory a piece of 16 columns took 300 instructions.)
// A piece's rows of B lie together in memory: one bulk copy per slot brings them into the warp's ring.  A stage
// belongs to one warp, which refills it when it has read it.  The first ring's worth is requested before the grid's
// dependency: kernel 11 lets this grid start after its own dependency wait, so B, y and the plan are
// complete by then.
template <bool kWide, int kSteps>
__global__ void __launch_bounds__(kUpThreads, kSteps * (kWide ? 32 : 16) <= 64 ? 4 : 3)
lora_short_up_kernel(const Params p) {
  constexpr int kSpan = kWide ? 32 : 16;           // ranks per step
  constexpr int kWords = kWide ? 4 : 2;            // 32-bit words of a row of B per lane and step
  constexpr int kStage = up_piece_bytes(kSpan * kSteps);
  extern __shared__ __align__(128) uint8_t ring[];   // [warps][depth][slots][32 rows of B]
  __shared__ __align__(16) uint16_t uh[G * kUStride], ul[G * kUStride];
  __shared__ int32_t head[4 + 8 + G];              // the record's rows, ids and row indexes
  __shared__ __align__(8) uint64_t bars[kUpWarps][kUpMaxDepth];
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kUpWarps * kUpMaxDepth; ++i) mbar_init(smem_addr(&bars[0][0] + i), 1);
    abort_word = 0;
    fence_mbar_init();
  }
  if (!p.early) grid_dependency_wait();
  // This CTA's run of strips (kUpWarps pieces) of one group.
  const int group = blockIdx.x;
  const int strips = (p.N / kUpCols + kUpWarps - 1) / kUpWarps;
  const int item = static_cast<int>(static_cast<long long>(strips) * blockIdx.y / gridDim.y);
  const int end = static_cast<int>(static_cast<long long>(strips) * (blockIdx.y + 1) / gridDim.y);
  const int n_end = min(p.N, end * kUpWarps * kUpCols);
  const int32_t* rec = p.groups + static_cast<size_t>(group) * lora_group_words(p.slots);
  if (threadIdx.x < 4 + 8 + G) head[threadIdx.x] = __ldcg(rec + threadIdx.x);
  __syncthreads();
  const int nrows = head[0];
  const int jr = p.slots * p.rank;
  constexpr int step_n = kUpWarps * kUpCols;
  const bool on0 = g < nrows, on1 = g + 8 < nrows;   // this lane's rows of the group, and their columns 8 t .. + 7
  const long long row0 = on0 ? head[12 + g] : 0, row1 = on1 ? head[12 + g + 8] : 0;
  const bool copied = group >= p.ngroups;        // rows that no adapter touches
  uint8_t* mine = ring + warp * p.depth * kStage;
  int has = 0;                                   // slots with an adapter
  for (int j = 0; j < p.slots; ++j) has += !copied && head[4 + j] >= 0;
  auto request = [&](int n0, int st) {           // lane 0 of the warp
    if (n0 >= n_end || lane != 0 || has == 0) return;
    const uint32_t bar = smem_addr(&bars[warp][st]);
    mbar_arrive_expect_tx(bar, has * kUpCols * p.rank * 2);
    for (int j = 0; j < p.slots; ++j) {
      const int id = head[4 + j];
      if (id >= 0)
        bulk_load(smem_addr(mine + st * kStage + j * kUpCols * p.rank * 2),
                  p.B + (static_cast<size_t>(id) * p.N + n0) * p.rank, kUpCols * p.rank * 2, bar);
    }
  };
  auto fetch_y = [&](int n0, uint4 (&y)[2]) {
    if (n0 < n_end && on0) y[0] = __ldcg(reinterpret_cast<const uint4*>(p.Yin + row0 * p.ldyin + n0 + 8 * t));
    if (n0 < n_end && on1) y[1] = __ldcg(reinterpret_cast<const uint4*>(p.Yin + row1 * p.ldyin + n0 + 8 * t));
  };
  int n0 = (item * kUpWarps + warp) * kUpCols;
  for (int i = 0; i < p.depth; ++i) request(n0 + i * step_n, i);
  uint4 y[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  fetch_y(n0, y);
  if (p.early) grid_dependency_wait();           // the parts of u
  for (int i = threadIdx.x; !copied && i < G * jr / 4; i += kUpThreads) {
    const int row = 4 * i / jr, c = 4 * i % jr;
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < nrows) {
      const float* src = p.part + (static_cast<size_t>(group) * p.ks * G + row) * jr + c;
      for (int z = 0; z < p.ks; ++z) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(src + static_cast<size_t>(z) * G * jr));
        u.x += v.x;
        u.y += v.y;
        u.z += v.z;
        u.w += v.w;
      }
    }
    float l[4];
    const uint32_t h0 = split_hi_lo(u.x, l[0]), h1 = split_hi_lo(u.y, l[1]), h2 = split_hi_lo(u.z, l[2]),
                   h3 = split_hi_lo(u.w, l[3]);
    *reinterpret_cast<uint2*>(uh + row * kUStride + c) = make_uint2(h0 | (h1 << 16), h2 | (h3 << 16));
    *reinterpret_cast<uint2*>(ul + row * kUStride + c) = make_uint2(pack_bf16x2(l[0], l[1]), pack_bf16x2(l[2], l[3]));
  }
  __syncthreads();
  uint32_t fh[kSteps][2][kWords], fl[kSteps][2][kWords];   // u of rows g and g + 8
  uint32_t off[kSteps];                          // this lane's ranks of each step, at MMA column g, in a stage
  bool use[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int slot = s * kSpan / p.rank;
    use[s] = !copied && head[4 + slot] >= 0;
    off[s] = ((slot * kUpCols + 8 * (g / 2) + g % 2) * p.rank + s * kSpan % p.rank + kSpan / 4 * t) * 2;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int w = 0; w < kWords; w += 2) {
        const int at = (8 * r + g) * kUStride + s * kSpan + kSpan / 4 * t + 2 * w;
        const uint2 a = *reinterpret_cast<const uint2*>(uh + at), b = *reinterpret_cast<const uint2*>(ul + at);
        fh[s][r][w] = a.x;
        fh[s][r][w + 1] = a.y;
        fl[s][r][w] = b.x;
        fl[s][r][w + 1] = b.y;
      }
  }
  int stage = 0;                                 // the next to read, and the phase of its barrier
  uint32_t phase = 0;
  for (; n0 < n_end; n0 += step_n) {
    uint4 yn[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    fetch_y(n0 + step_n, yn);                    // the next piece's
    float d[4][4] = {};
    if (has > 0) {
      if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(smem_addr(&bars[warp][stage]), phase, abort_flag, 93))) break;
      const uint8_t* from = mine + stage * kStage;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        if (!use[s]) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t b[kWords];
          const uint8_t* at = from + off[s] + 4 * j * p.rank;   // two rows further per MMA
          if constexpr (kWide) {
            const uint4 v = *reinterpret_cast<const uint4*>(at);
            b[0] = v.x; b[1] = v.y; b[2] = v.z; b[3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(at);
            b[0] = v.x; b[1] = v.y;
          }
#pragma unroll
          for (int w = 0; w < kWords; w += 2) {
            mma16816(d[j], fh[s][0][w], fh[s][1][w], fh[s][0][w + 1], fh[s][1][w + 1], b[w], b[w + 1]);
            mma16816(d[j], fl[s][0][w], fl[s][1][w], fl[s][0][w + 1], fl[s][1][w + 1], b[w], b[w + 1]);
          }
        }
      }
      __syncwarp();                              // the stage has been read
      request(n0 + p.depth * step_n, stage);
      stage = stage + 1 == p.depth ? 0 : stage + 1;
      if (stage == 0) phase ^= 1u;
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (!(r ? on1 : on0)) continue;
      if (!copied) {                             // (copied rows keep their bits)
        uint32_t* w = reinterpret_cast<uint32_t*>(&y[r]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = pack_bf16x2(bf16lo_to_f32(w[j]) + d[j][2 * r], bf16hi_to_f32(w[j]) + d[j][2 * r + 1]);
      }
      *reinterpret_cast<uint4*>(p.Y + (r ? row1 : row0) * p.ldy + n0 + 8 * t) = y[r];
    }
    y[0] = yn[0];
    y[1] = yn[1];
  }
  grid_launch_dependents();
  __syncthreads();
  if (*abort_flag) {                               // let the copies already issued finish
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 2000000ull) { }
  }
}

}  // namespace k11
}  // namespace svdq
