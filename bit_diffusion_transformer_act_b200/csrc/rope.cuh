// Kernels 9 and 10: rotary positions with several axes -- applied to the normalised q and k of a
// projection (kernel 9), and as the cos / sin tables that the fused QKV projection reads
// (kernel 10).
//
// Mathematics.  A head's rotary pairs are dealt to the axes in order (axis a has d_a / 2 pairs);
// pair i of axis a turns by position[m, a] * theta_a^(-2 i / d_a).  Only the angle's fraction of a
// turn counts, so the host passes each pair's frequency in turns, f = theta_a^(-2 i / d_a) / (2 pi), and the
// kernels round the fraction to units of 2^-32 turns:
//   - integer positions: f as a 64-bit fixed-point fraction; position * f modulo one turn is the product modulo
//     2^64, of which the upper half is kept, rounded (f's own end is off by less than 2^-64 per unit of position);
//   - float positions: position * f in 64-bit floating point, less the nearest integer.
// So the angle is off by half a unit, 2 pi 2^-33 = 7.3e-10 radians (twice that at integer positions near 2^31),
// whatever its size: of a small angle that is more than 2^-24 of itself, of the rotated values it is far below
// their last bit.  (A product in 32 bits would be off by position * 2^-24 radians: 0.004 at position 65536.)  The
// fraction's upper two bits, rounded, are the quarter; the rest is an angle within pi / 4, as a float within
// 3 * 2^-24 of itself, whose sine and cosine are the Taylor polynomials of degree 9 and 8: their remainders are at
// most x^11 / 11! < 2^-29 and x^10 / 10! < 2^-25 there.  Sine and cosine come out within 4.5 * 2^-24 of themselves,
// beside the angle's 7.3e-10.  28 instructions per pair, where the 64-bit reduction and the library's sine and
// cosine of any argument took about 100.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ptx.cuh"

namespace svdq {
namespace k9 {

constexpr int kMaxAxes = 8;
constexpr int kMaxPairs = 128;             // head_dim <= 256
constexpr int kWarps = 8;                  // that rotate
constexpr int kThreads = (kWarps + 1) * 32;   // and one that loads
constexpr int kBlocksPerSm = 2;
constexpr int kMaxStages = 32;
constexpr int kRingBytes = 100 * 1024;     // two blocks per SM
constexpr int kUnitBytes = 6400;           // at most, where heads can be shared out
static_assert(2 * kWarps * kUnitBytes <= kRingBytes, "two stages per warp");
constexpr int kAfterBytes = 2 * kMaxStages * 8 + 16 + 2 * 2 * kMaxPairs * 2;   // barriers, flag, norm weights
constexpr int kTableThreads = 256;

struct Freqs {
  uint64_t f[kMaxPairs];                   // turns per unit of position, in pair order: for integer positions the
                                           // fraction in units of 2^-64, for float ones the bits of a double
  uint8_t axis[kMaxPairs];
};

struct View {                              // element (m, h, d) at ptr[m * row + h * head + d]
  __nv_bfloat16* ptr;
  long long row, head;
};

struct Params {
  View q, k, oq, ok;
  const __nv_bfloat16 *wq, *wk;            // [D] or null (no normalisation)
  const void* pos;                         // [P, axes] int32, or float32
  int axes, M, q_heads, k_heads;
  uint32_t P;
  int D, rot;                              // head width, rotated columns
  int q_groups, groups;                    // what a warp holds at once: groups of q's heads, of q's and k's
  int chunk;                               // groups per unit of work
  uint32_t units;                          // of a token
  int stage_log, stage_bytes;              // 1 << stage_log stages, a multiple of kWarps
  float eps;
};

template <bool kFloat>
using Position = std::conditional_t<kFloat, double, int>;

// The angle of one position and frequency, in 2^-32 turns.
__device__ __forceinline__ uint32_t turn_fraction(double pos, uint64_t f) {
  const double t = pos * __longlong_as_double(static_cast<long long>(f));
  // adding 1.5 * 2^20 to the fraction leaves it in units of 2^-32 in the low half of the result
  return static_cast<uint32_t>(__double2loint(t - rint(t) + 1572864.0));
}
__device__ __forceinline__ uint32_t turn_fraction(int pos, uint64_t f) {
  const uint32_t p = static_cast<uint32_t>(pos), hi = static_cast<uint32_t>(f >> 32), lo = static_cast<uint32_t>(f);
  // upper half of pos * f modulo 2^64, rounded (pos < 0: its unsigned value less 2^32, whose product with f's
  // low half comes back off the upper half)
  const uint64_t low = static_cast<uint64_t>(p) * lo + 0x80000000u;
  return p * hi + static_cast<uint32_t>(low >> 32) - (pos < 0 ? lo : 0u);
}

// Sine and cosine of `frac` * 2^-32 turns; NaN where `bad` is (else it is 0).
__device__ __forceinline__ void sincos_turns(uint32_t frac, float bad, float& s, float& c) {
  const uint32_t q = (frac + 0x20000000u) >> 30;   // nearest quarter turn
  const float x = fmaf(static_cast<float>(static_cast<int>(frac - (q << 30))), 1.46291807926715968e-9f, bad);   // 2 pi 2^-32
  const float z = x * x;
  const float sp = fmaf(fmaf(fmaf(fmaf(1.f / 362880.f, z, -1.f / 5040.f), z, 1.f / 120.f), z, -1.f / 6.f) * z, x, x);
  const float cp = fmaf(fmaf(fmaf(fmaf(1.f / 40320.f, z, -1.f / 720.f), z, 1.f / 24.f), z, -0.5f), z, 1.f);
  const float a = q & 1u ? cp : sp, b = q & 1u ? sp : cp;
  s = __uint_as_float(__float_as_uint(a) ^ ((q & 2u) << 30));
  c = __uint_as_float(__float_as_uint(b) ^ (((q + 1u) & 2u) << 30));
}

// A position; a float one that is not finite has no angle: `bad` is NaN for it, else 0.  (An ordinary load: the
// previous kernel may have written the positions while this grid was already resident, which the read-only path,
// ld.global.nc, does not allow.)
template <bool kFloat>
__device__ __forceinline__ Position<kFloat> position(const void* pos, long long i, float& bad) {
  if constexpr (kFloat) {
    const float x = static_cast<const float*>(pos)[i];
    bad = x * 0.f;
    return static_cast<double>(x);
  } else {
    bad = 0.f;
    return static_cast<const int*>(pos)[i];
  }
}

template <int V>
__device__ __forceinline__ void load_v(const __nv_bfloat16* p, uint32_t (&r)[V / 2]) {
  if constexpr (V == 8) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r[0] = v.x; r[1] = v.y;
  }
}
template <int V>
__device__ __forceinline__ void store_v(__nv_bfloat16* p, const uint32_t (&r)[V / 2]) {
  if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = make_uint4(r[0], r[1], r[2], r[3]);
  else *reinterpret_cast<uint2*>(p) = make_uint2(r[0], r[1]);
}

// A unit of work is a token's heads of q and of k, or a run of them.  One warp of a block requests units ahead
// into a ring of stages (bulk copies: one where the heads are contiguous, else one per head); the others take
// units in turn, read a stage and write the result straight to its place.
// Within a unit, V pairs are held by one lane as two runs of V elements; LPR lanes (a power of two, at least
// D / 2V) hold a head's row, and a warp 32 / LPR heads at a time.  A lane's place in the row does not change, so
// the token's sines and cosines are formed once for the unit's heads -- each lane forms its share of the pairs
// it needs, the lanes with the same place the rest -- and the norm weights are folded into them: with
// u = x / rms, pair (x0, x1) becomes (u0 w0 c - u1 w1 s, u0 w0 s + u1 w1 c), four factors per pair and one
// scale per head.
//
// Bound by memory (q and k read and written once: 4 bytes a value) if the instructions are few and enough
// bytes are on their way.  9216 tokens of 40 heads of 128 (floor 29 us): 61 us with the sines formed by every
// lane, the weights unpacked per head and scalar arithmetic (2940 warp instructions per token); 43 us without
// that, the next heads of a warp prefetched into registers (16 KB per SM on their way); 37 us as it is (the
// copies alone, without the arithmetic, 35.5).
template <int V, int LPR, bool kHalf, bool kFloat>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
qk_norm_rope_kernel(const __grid_constant__ Params p, const __grid_constant__ Freqs fr) {
  extern __shared__ __align__(128) uint8_t ring[];
  constexpr int HPW = 32 / LPR;
  constexpr int kShare = HPW >= V ? 1 : V / HPW;   // pairs of its place whose angle a lane forms
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int stages = 1 << p.stage_log;
  uint8_t* after = ring + stages * p.stage_bytes;
  const uint32_t bars = smem_addr(after);
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kMaxStages + s); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(after + 2 * kMaxStages * 8);
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) { mbar_init(full(s), 1); mbar_init(empty(s), 1); }
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  grid_dependency_wait();                          // q and k come from the previous kernel
  grid_launch_dependents();
  // This block's units are blockIdx.x, blockIdx.x + gridDim.x, ...: at any time the grid works on one region.
  const uint32_t total = static_cast<uint32_t>(p.M) * p.units;   // below 2^31
  const int count = static_cast<int>((total - blockIdx.x + gridDim.x - 1) / gridDim.x);
  const uint32_t w0 = blockIdx.x, step = gridDim.x;

  // Unit w: its token, and which heads of q and of k.  A token's units differ in length; turning their order with
  // the token deals the long ones out to all warps.
  struct Unit {
    uint32_t m;
    int q0, nq, k0, nk;                            // first head and heads
  };
  auto unit_of = [&](uint32_t w) {
    Unit t;
    t.m = w;
    int g0 = 0;
    if (p.units > 1) {
      t.m = w / p.units;
      g0 = static_cast<int>((w - t.m * p.units + t.m) % p.units) * p.chunk;
    }
    const int g1 = min(g0 + p.chunk, p.groups);
    t.q0 = g0 * HPW;
    t.nq = max(0, min(min(g1, p.q_groups) * HPW, p.q_heads) - t.q0);
    t.k0 = max(g0 - p.q_groups, 0) * HPW;
    t.nk = max(0, min((g1 - p.q_groups) * HPW, p.k_heads) - t.k0);
    return t;
  };

  if (warp == kWarps) {
    // ---------------------------------------------------------------- loads
    // Lane s refills stage s: the first requests go out together, and no stage waits for another.
    uint64_t seen = 0;                             // when the polls for a free stage last began
    int n = lane < stages ? lane : count;
    uint32_t phase = 1;
    for (uint32_t i = 1; __any_sync(0xFFFFFFFFu, n < count); ++i) {
      const bool go = n < count && mbar_test_wait(empty(lane), phase);
      if (go) {
        const Unit t = unit_of(w0 + n * step);
        const uint32_t bar = full(lane);
        mbar_arrive_expect_tx(bar, (t.nq + t.nk) * p.D * 2);
        auto load = [&](const View& v, int h0, int heads, uint32_t dst) {
          const __nv_bfloat16* src = v.ptr + t.m * v.row + h0 * v.head;
          if (heads > 0 && v.head == p.D) {
            bulk_load(dst, src, heads * p.D * 2, bar);
          } else {
            for (int h = 0; h < heads; ++h) bulk_load(dst + h * p.D * 2, src + h * v.head, p.D * 2, bar);
          }
        };
        const uint32_t dst = smem_addr(ring + lane * p.stage_bytes);
        load(p.q, t.q0, t.nq, dst);
        load(p.k, t.k0, t.nk, dst + t.nq * p.D * 2);
        n += stages;
        phase ^= 1u;
      }
      if (__any_sync(0xFFFFFFFFu, go)) {
        i = 0;
        continue;
      }
      __nanosleep(32);                             // the polls would take issue slots from the other warps
      if ((i & 63u) == 0) {
        const uint64_t now = global_timer_ns();
        if (i == 64) seen = now;
        const bool late = now - seen > kWaitLimitNs;
        if (__any_sync(0xFFFFFFFFu, late || *abort_flag)) {
          if (lane == 0 && late) atomicOr(&g_device_status, 1u | (91u << 8));
          *abort_flag = 1;
          break;
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- rotation
    const int u = lane % LPR, sub = lane / LPR;
    const bool active = u * 2 * V < p.D;           // lanes past the row's end hold nothing
    // The lane's runs, so that neighbouring lanes' runs are neighbours: the same V pairs' first and second
    // elements (halves), or V / 2 pairs of either half of the row.  Places past the rotated columns are only
    // normalised; interleaved, that may hold for the second run alone.
    const bool turned0 = kHalf ? u * 2 * V < p.rot : V * u < p.rot;
    const bool turned1 = kHalf ? turned0 : p.D / 2 + V * u < p.rot;
    const int e0 = kHalf && !turned0 ? 2 * V * u : V * u;
    const int run = !kHalf ? p.D / 2 : turned0 ? p.rot / 2 : V;   // from the first run to the second
    uint64_t f[kShare];
    int ax[kShare];
#pragma unroll
    for (int k = 0; k < kShare; ++k) {
      const int j = sub * kShare + k;              // (lanes with sub >= V have nothing to form)
      const bool first = kHalf || j < V / 2;
      const bool on = active && j < V && (first ? turned0 : turned1);
      const int i = kHalf ? V * u + j : (first ? V * u : p.D / 2 + V * u - V) / 2 + j;
      f[k] = on ? fr.f[i] : 0u;
      ax[k] = on ? fr.axis[i] : 0;
    }
    const float inv_d = 1.0f / static_cast<float>(p.D);
    __nv_bfloat16* weights = reinterpret_cast<__nv_bfloat16*>(after + 2 * kMaxStages * 8 + 16);   // of q, of k
    for (int i = threadIdx.x; i < 2 * p.D; i += kWarps * 32) {
      const __nv_bfloat16* w = i < p.D ? p.wq : p.wk;
      weights[i] = w ? w[i < p.D ? i : i - p.D] : __float2bfloat16_rn(1.f);
    }
    Position<kFloat> pos[kShare];
    float bad[kShare];
    auto fetch_position = [&](uint32_t w) {
      uint32_t m = p.units > 1 ? w / p.units : w;
      if (m >= p.P) m %= p.P;
#pragma unroll
      for (int j = 0; j < kShare; ++j)
        pos[j] = position<kFloat>(p.pos, static_cast<long long>(m) * p.axes + ax[j], bad[j]);
    };
    // The warps take units in turn.  The number of stages is a multiple of the warps', so a stage always belongs to
    // the same warp, which cannot wait for a stage's next phase before its present one is over.
    if (warp < count) fetch_position(w0 + warp * step);
    asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");   // the weights; these warps only
    for (int n = warp; n < count; n += kWarps) {
      const int s = n & (stages - 1);
      const Unit t = unit_of(w0 + n * step);
      float cs[kShare], sn[kShare];
#pragma unroll
      for (int j = 0; j < kShare; ++j) {
        sincos_turns(turn_fraction(pos[j], f[j]), bad[j], sn[j], cs[j]);
      }
      if (n + kWarps < count) fetch_position(w0 + (n + kWarps) * step);   // the next unit's, while this one is worked on
      if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(full(s), (n >> p.stage_log) & 1u, abort_flag, 92))) break;

      // Heads h0 .. h0 + heads - 1 of q or of k, at `at` in the stage.  Written twice into the code, so that
      // strides and pointers stay operands from the parameters instead of selected values.
      auto rotate = [&](const uint8_t* at, const View& vo, int h0, int heads, bool normed, const __nv_bfloat16* w) {
        uint32_t n0[V / 2], n1[V / 2];             // norm weights of this lane's runs
#pragma unroll
        for (int i = 0; i < V / 2; ++i) n0[i] = n1[i] = 0u;
        if (active) {
          load_v<V>(w + e0, n0);
          load_v<V>(w + e0 + run, n1);
        }
        // the factors of pairs 2 i and 2 i + 1 side by side: y0 = x0 f00 + x1 f01, y1 = x0 f10 + x1 f11
        uint64_t f00[V / 2], f01[V / 2], f10[V / 2], f11[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          float g[4][2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int j = 2 * i + k;
            const float c = __shfl_sync(0xFFFFFFFFu, cs[j % kShare], u + LPR * (j / kShare));
            const float s = __shfl_sync(0xFFFFFFFFu, sn[j % kShare], u + LPR * (j / kShare));
            // weights of the pair's two elements: of the two runs (halves), or neighbours
            const uint32_t a = kHalf ? n0[i] : (j < V / 2 ? n0[j % (V / 2)] : n1[j % (V / 2)]);
            const uint32_t b = kHalf ? n1[i] : a;
            const float wa = kHalf && k ? bf16hi_to_f32(a) : bf16lo_to_f32(a);
            const float wb = kHalf && !k ? bf16lo_to_f32(b) : bf16hi_to_f32(b);
            const bool turned = i < V / 4 ? turned0 : turned1;
            g[0][k] = turned ? wa * c : wa;
            g[1][k] = -wb * s;
            g[2][k] = wa * s;
            g[3][k] = turned ? wb * c : wb;
          }
          f00[i] = f32x2_pack(g[0][0], g[0][1]);
          f01[i] = f32x2_pack(g[1][0], g[1][1]);
          f10[i] = f32x2_pack(g[2][0], g[2][1]);
          f11[i] = f32x2_pack(g[3][0], g[3][1]);
        }
        const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(at) + sub * p.D + e0;
        __nv_bfloat16* dst = vo.ptr + t.m * vo.row + (h0 + sub) * vo.head + e0;
        const long long dst_step = HPW * vo.head;
        int left = active ? heads - sub : 0;       // > 0: this lane holds a head
        // Places past the rotated columns add no cross terms: an infinity must not reach its neighbour.
#pragma unroll 1
        for (int h = 0; h < heads; h += HPW) {
          uint32_t r0[V / 2], r1[V / 2];
#pragma unroll
          for (int j = 0; j < V / 2; ++j) r0[j] = r1[j] = 0u;
          if (left > 0) {
            load_v<V>(src, r0);
            load_v<V>(src + run, r1);
          }
          src += HPW * p.D;
          uint64_t x0[V / 2], x1[V / 2];           // first and second elements of pairs 2 i, 2 i + 1
#pragma unroll
          for (int i = 0; i < V / 2; ++i) {
            const uint32_t a = kHalf ? r0[i] : (i < V / 4 ? r0[(2 * i) % (V / 2)] : r1[(2 * i) % (V / 2)]);
            const uint32_t b = kHalf ? r1[i] : (i < V / 4 ? r0[(2 * i + 1) % (V / 2)] : r1[(2 * i + 1) % (V / 2)]);
            // halves: a, b hold (x0 of both pairs), (x1 of both pairs); interleaved: pair 2 i, pair 2 i + 1
            x0[i] = kHalf ? f32x2_pack(bf16lo_to_f32(a), bf16hi_to_f32(a)) : f32x2_pack(bf16lo_to_f32(a), bf16lo_to_f32(b));
            x1[i] = kHalf ? f32x2_pack(bf16lo_to_f32(b), bf16hi_to_f32(b)) : f32x2_pack(bf16hi_to_f32(a), bf16hi_to_f32(b));
          }
          float scale = 1.f;
          if (normed) {
            uint64_t q0 = f32x2_mul(x0[0], x0[0]), q1 = f32x2_mul(x1[0], x1[0]);
#pragma unroll
            for (int i = 1; i < V / 2; ++i) {
              q0 = f32x2_fma(x0[i], x0[i], q0);
              q1 = f32x2_fma(x1[i], x1[i], q1);
            }
            float sa, sb, sc, sd;
            f32x2_unpack(q0, sa, sb);
            f32x2_unpack(q1, sc, sd);
            float ss = (sa + sb) + (sc + sd);      // 0 for lanes past the row's end, which hold zeros
#pragma unroll
            for (int o = LPR / 2; o > 0; o /= 2) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
            scale = rsqrtf(fmaf(ss, inv_d, p.eps));
          }
          const uint64_t scale2 = f32x2_pack(scale, scale);
          uint32_t o0[V / 2], o1[V / 2];
#pragma unroll
          for (int i = 0; i < V / 2; ++i) {
            uint64_t y0 = f32x2_mul(x0[i], f00[i]), y1 = f32x2_mul(x1[i], f11[i]);
            if (i < V / 4 ? turned0 : turned1) {
              y0 = f32x2_fma(x1[i], f01[i], y0);
              y1 = f32x2_fma(x0[i], f10[i], y1);
            }
            y0 = f32x2_mul(y0, scale2);
            y1 = f32x2_mul(y1, scale2);
            float a0, a1, b0, b1;                  // y0 and y1 of pair 2 i, of pair 2 i + 1
            f32x2_unpack(y0, a0, b0);
            f32x2_unpack(y1, a1, b1);
            const uint32_t first = kHalf ? pack_bf16x2(a0, b0) : pack_bf16x2(a0, a1);
            const uint32_t second = kHalf ? pack_bf16x2(a1, b1) : pack_bf16x2(b0, b1);
            if (kHalf) {
              o0[i] = first;
              o1[i] = second;
            } else if (i < V / 4) {
              o0[(2 * i) % (V / 2)] = first;
              o0[(2 * i + 1) % (V / 2)] = second;
            } else {
              o1[(2 * i) % (V / 2)] = first;
              o1[(2 * i + 1) % (V / 2)] = second;
            }
          }
          if (left > 0) {
            store_v<V>(dst, o0);
            store_v<V>(dst + run, o1);
          }
          left -= HPW;
          dst += dst_step;
        }
      };
      const uint8_t* stage = ring + s * p.stage_bytes;
      if (t.nq > 0) rotate(stage, p.oq, t.q0, t.nq, p.wq != nullptr, weights);
      if (t.nk > 0) rotate(stage + t.nq * p.D * 2, p.ok, t.k0, t.nk, p.wk != nullptr, weights + p.D);
      __syncwarp();
      if (lane == 0) mbar_arrive_relaxed(empty(s));   // every value read is in registers; stores are not waited for
    }
  }
  __syncthreads();
  if (*abort_flag) {                               // a wait ran out: let the copies already issued finish
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 2000000ull) { }
  }
}

// Kernel 10: a thread owns kTokens positions (columns of the tables, kTableThreads apart) and walks over a share of
// the pairs; 32 neighbouring threads write one 128-byte line of each table.  Tokens m, m + P, m + 2P, ... have the
// same position and get the same values.  Bound by its stores, 8 bytes per (token, pair), if the instructions are
// few and its blocks fit at once.  131075 tokens, 64 pairs, float positions (floor 10.6 us): 27 us with a 64-bit
// reduction and the library's sine and cosine, 18.9 us with fixed-point turns and one token per thread (20 of 55
// instructions were the loop's), 15.2 us with four.  Float positions take 40 registers, so six blocks fit on an SM
// where the host asks for eight: the 1032 blocks of this case are a wave of 888 and a rest.
constexpr int kTokens = 4;
struct TableParams {
  const void* pos;
  int axes, P, M, pairs, rot_pairs;
  int per;                                 // pairs per grid row
  float *cos, *sin;                        // [pairs, M]
};

template <bool kFloat>
__global__ void __launch_bounds__(kTableThreads)
rope_tables_kernel(const __grid_constant__ TableParams p, const __grid_constant__ Freqs fr) {
  grid_dependency_wait();
  grid_launch_dependents();
  const long long m0 = static_cast<long long>(blockIdx.x) * (kTableThreads * kTokens) + threadIdx.x;
  const int i0 = blockIdx.y * p.per, i1 = min(i0 + p.per, p.pairs);
  float* cos = p.cos + static_cast<long long>(i0) * p.M + m0;
  float* sin = p.sin + static_cast<long long>(i0) * p.M + m0;
  Position<kFloat> x[kTokens];
  float bad[kTokens];
  bool on[kTokens];
#pragma unroll
  for (int t = 0; t < kTokens; ++t) {
    on[t] = m0 + t * kTableThreads < p.P;
    x[t] = 0;
    bad[t] = 0.f;
  }
  const int more = p.M / p.P - 1;                  // further tokens with the same position
  auto walk = [&](auto whole) {                    // whole: every token of the block, no further ones
    auto put = [&](int t, float s, float c) {
      if (!decltype(whole)::value && !on[t]) return;
      cos[t * kTableThreads] = c;
      sin[t * kTableThreads] = s;
      if (!decltype(whole)::value)
        for (int r = 1; r <= more; ++r) {
          cos[t * kTableThreads + static_cast<long long>(r) * p.P] = c;
          sin[t * kTableThreads + static_cast<long long>(r) * p.P] = s;
        }
    };
    int i = i0;
    while (i < min(i1, p.rot_pairs)) {             // axis by axis
      const int a = fr.axis[i];
#pragma unroll
      for (int t = 0; t < kTokens; ++t)
        if (on[t]) x[t] = position<kFloat>(p.pos, (m0 + t * kTableThreads) * p.axes + a, bad[t]);
      do {
        const uint64_t f = fr.f[i];
#pragma unroll
        for (int t = 0; t < kTokens; ++t) {
          float s, c;
          sincos_turns(turn_fraction(x[t], f), bad[t], s, c);
          put(t, s, c);
        }
        cos += p.M;
        sin += p.M;
        ++i;
      } while (i < min(i1, p.rot_pairs) && fr.axis[i] == a);
    }
    for (; i < i1; ++i, cos += p.M, sin += p.M) {  // pairs past the rotated columns stay as they are
#pragma unroll
      for (int t = 0; t < kTokens; ++t) put(t, 0.f, 1.f);
    }
  };
  if (more == 0 && (static_cast<long long>(blockIdx.x) + 1) * (kTableThreads * kTokens) <= p.P)
    walk(std::true_type{});
  else
    walk(std::false_type{});
}

}  // namespace k9
}  // namespace svdq
