// Kernels 9 and 10: rotary positions with several axes -- applied to the normalised q and k of a
// projection (kernel 9), and as the cos / sin tables that the fused QKV projection reads
// (kernel 10).
//
// Mathematics.  A head's rotary pairs are dealt to the axes in order (axis a has d_a / 2 pairs);
// pair i of axis a turns by position[m, a] * theta_a^(-2 i / d_a).  Only the angle's fraction of a
// turn counts, so the host passes each pair's frequency in turns, f = theta_a^(-2 i / d_a) / (2 pi), and the
// kernels form the fraction in units of 2^-32 turns:
//   - integer positions: f as a 64-bit fixed-point fraction; position * f modulo one turn is the
//     product modulo 2^64, of which the upper half is kept -- exact but for f's own rounding (2^-64);
//   - float positions: position * f in 64-bit floating point, less the nearest integer.
// (A product in 32 bits would be off by position * 2^-24 radians: 0.004 at position 65536.)  The fraction's
// upper two bits, rounded, are the quarter; the rest is an angle within pi / 4, exact to 2^-24 of itself
// as a float, whose sine and cosine are the Taylor polynomials of degree 9 and 8: their remainders are at
// most x^11 / 11! < 2^-29 and x^10 / 10! < 2^-25 there.  Thus 28 instructions per pair, where the 64-bit
// reduction and the library's sine and cosine of any argument took about 100.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ptx.cuh"

namespace svdq {
namespace k9 {

constexpr int kMaxAxes = 8;
constexpr int kMaxPairs = 128;             // head_dim <= 256
constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 3;

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
  int axes, P, M, q_heads, k_heads;
  int D, rot;                              // head width, rotated columns
  int parts;                               // warps that share a token's heads
  float eps;
};

// The angle of one position and frequency, in 2^-32 turns.
template <bool kFloat>
__device__ __forceinline__ uint32_t turn_fraction(uint32_t pos_bits, uint64_t f) {
  if constexpr (kFloat) {
    const double t = static_cast<double>(__uint_as_float(pos_bits)) * __longlong_as_double(static_cast<long long>(f));
    // adding 1.5 * 2^20 to the fraction leaves it in units of 2^-32 in the low half of the result
    return static_cast<uint32_t>(__double2loint(t - rint(t) + 1572864.0));
  } else {
    const int p = static_cast<int>(pos_bits);
    const uint32_t hi = static_cast<uint32_t>(f >> 32), lo = static_cast<uint32_t>(f);
    // upper half of p * f modulo 2^64 (p < 0: its unsigned value less 2^32, whose product with f's low
    // half comes back off the upper half)
    return static_cast<uint32_t>(p) * hi + __umulhi(static_cast<uint32_t>(p), lo) - (p < 0 ? lo : 0u);
  }
}

// Sine and cosine of `frac` * 2^-32 turns.
__device__ __forceinline__ void sincos_turns(uint32_t frac, float& s, float& c) {
  const uint32_t q = (frac + 0x20000000u) >> 30;   // nearest quarter turn
  const float x = static_cast<float>(static_cast<int>(frac - (q << 30))) * 1.46291807926715968e-9f;   // 2 pi 2^-32
  const float z = x * x;
  const float sp = fmaf(fmaf(fmaf(fmaf(1.f / 362880.f, z, -1.f / 5040.f), z, 1.f / 120.f), z, -1.f / 6.f) * z, x, x);
  const float cp = fmaf(fmaf(fmaf(fmaf(1.f / 40320.f, z, -1.f / 720.f), z, 1.f / 24.f), z, -0.5f), z, 1.f);
  const float a = q & 1u ? cp : sp, b = q & 1u ? sp : cp;
  s = __uint_as_float(__float_as_uint(a) ^ ((q & 2u) << 30));
  c = __uint_as_float(__float_as_uint(b) ^ (((q + 1u) & 2u) << 30));
}

// The position's bits; a float position that is not finite has no angle: `bad` is NaN for it, else 0.
template <bool kFloat>
__device__ __forceinline__ uint32_t position(const void* pos, long long i, float& bad) {
  const uint32_t bits = __ldg(static_cast<const uint32_t*>(pos) + i);
  bad = kFloat ? __uint_as_float(bits) * 0.f : 0.f;
  return bits;
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

// A unit is V pairs, held by one lane as two runs of V elements; LPR lanes (a power of two, at least D / 2V)
// hold a head's row, and a warp 32 / LPR heads of one token at a time.  A lane's unit does not change, so the
// token's sines and cosines are formed once for all its heads -- each lane forms its share of the pairs of
// its unit, the lanes that hold the unit for other heads the rest -- and the norm weights are folded into
// them: with u = x / rms, pair (x0, x1) becomes (u0 w0 c - u1 w1 s, u0 w0 s + u1 w1 c), four factors per pair
// and one scale per head.
//
// Bound by memory (q and k read and written once: 4 bytes a value) if the instructions are few: with the
// sines formed by every lane, the weights unpacked per head and scalar arithmetic the kernel issued
// 2940 warp instructions per token of 40 heads and took 61 us at 9216 tokens (floor 29 us).
template <int V, int LPR, bool kHalf, bool kFloat>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
qk_norm_rope_kernel(const __grid_constant__ Params p, const __grid_constant__ Freqs fr) {
  constexpr int HPW = 32 / LPR;
  constexpr int kShare = HPW >= V ? 1 : V / HPW;   // pairs of its unit whose angle a lane forms
  const int lane = threadIdx.x % 32;
  const int u = lane % LPR, sub = lane / LPR;
  const bool active = u * 2 * V < p.D;             // lanes past the row's end hold nothing
  const bool turned = u * 2 * V < p.rot;           // units past the rotated columns are only normalised
  const int e0 = turned && kHalf ? V * u : 2 * V * u;
  const int run = turned && kHalf ? p.rot / 2 : V;  // from the unit's first run to its second
  uint64_t f[kShare];
  int ax[kShare];
#pragma unroll
  for (int j = 0; j < kShare; ++j) {
    const int i = V * u + sub * kShare + j;        // (lanes with sub >= V have nothing to form)
    f[j] = turned && sub * kShare < V ? fr.f[i] : 0u;
    ax[j] = turned && sub * kShare < V ? fr.axis[i] : 0;
  }
  grid_dependency_wait();                          // q and k come from the previous kernel
  grid_launch_dependents();
  const int warps = gridDim.x * (kThreads / 32);
  const int wid = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  const int part = wid % p.parts;
  const float inv_d = 1.0f / static_cast<float>(p.D);
  const int step = p.parts * HPW;
  const long long m_step = warps / p.parts;
  for (long long m = wid / p.parts; m < p.M; m += m_step) {
    float cs[kShare], sn[kShare];
    const long long at = static_cast<long long>(static_cast<int>(m) % p.P) * p.axes;
#pragma unroll
    for (int j = 0; j < kShare; ++j) {
      float bad;
      const uint32_t x = position<kFloat>(p.pos, at + ax[j], bad);
      sincos_turns(turn_fraction<kFloat>(x, f[j]), sn[j], cs[j]);
      if (kFloat) {
        sn[j] += bad;
        cs[j] += bad;
      }
    }
    // This lane's heads of q or of k: written twice into the code, so that the strides and pointers stay
    // operands from the parameters instead of selected values.
    auto rotate = [&](const View& vi, const View& vo, const __nv_bfloat16* w, int heads) {
      const int h0 = part * HPW;
      if (h0 >= heads) return;
      const __nv_bfloat16* src = vi.ptr + m * vi.row + (h0 + sub) * vi.head + e0;
      __nv_bfloat16* dst = vo.ptr + m * vo.row + (h0 + sub) * vo.head + e0;
      const long long src_step = step * vi.head, dst_step = step * vo.head;
      int left = active ? heads - h0 - sub : 0;    // > 0: this lane holds a head
      uint32_t r0[V / 2], r1[V / 2];
#pragma unroll
      for (int j = 0; j < V / 2; ++j) r0[j] = r1[j] = 0u;
      if (left > 0) {
        load_v<V>(src, r0);
        load_v<V>(src + run, r1);
      }
      // the factors of pairs 2 i and 2 i + 1 side by side: y0 = x0 f00 + x1 f01, y1 = x0 f10 + x1 f11
      uint64_t f00[V / 2], f01[V / 2], f10[V / 2], f11[V / 2];
      {
        uint32_t w0[V / 2], w1[V / 2];
#pragma unroll
        for (int j = 0; j < V / 2; ++j) w0[j] = w1[j] = 0x3F803F80u;
        if (w && active) {
          load_v<V>(w + e0, w0);
          load_v<V>(w + e0 + run, w1);
        }
        float g[4][V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float c = __shfl_sync(0xFFFFFFFFu, cs[j % kShare], u + LPR * (j / kShare));
          const float s = __shfl_sync(0xFFFFFFFFu, sn[j % kShare], u + LPR * (j / kShare));
          // weights of the pair's two elements: of the two runs (halves), or neighbours
          const uint32_t a = kHalf ? w0[j / 2] : (j < V / 2 ? w0[j % (V / 2)] : w1[j % (V / 2)]);
          const uint32_t b = kHalf ? w1[j / 2] : a;
          const float wa = kHalf && j % 2 ? bf16hi_to_f32(a) : bf16lo_to_f32(a);
          const float wb = kHalf && j % 2 == 0 ? bf16lo_to_f32(b) : bf16hi_to_f32(b);
          g[0][j] = turned ? wa * c : wa;
          g[1][j] = -wb * s;
          g[2][j] = wa * s;
          g[3][j] = turned ? wb * c : wb;
        }
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          f00[i] = f32x2_pack(g[0][2 * i], g[0][2 * i + 1]);
          f01[i] = f32x2_pack(g[1][2 * i], g[1][2 * i + 1]);
          f10[i] = f32x2_pack(g[2][2 * i], g[2][2 * i + 1]);
          f11[i] = f32x2_pack(g[3][2 * i], g[3][2 * i + 1]);
        }
      }
      // Units past the rotated columns add no cross terms: an infinity must not reach its neighbour.
#pragma unroll 1
      for (int n = heads - h0; n > 0; n -= step) {
        uint64_t x0[V / 2], x1[V / 2];             // first and second elements of pairs 2 i, 2 i + 1
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          const uint32_t a = kHalf ? r0[i] : (i < V / 4 ? r0[(2 * i) % (V / 2)] : r1[(2 * i) % (V / 2)]);
          const uint32_t b = kHalf ? r1[i] : (i < V / 4 ? r0[(2 * i + 1) % (V / 2)] : r1[(2 * i + 1) % (V / 2)]);
          // halves: a, b hold (x0 of both pairs), (x1 of both pairs); interleaved: pair 2 i, pair 2 i + 1
          x0[i] = kHalf ? f32x2_pack(bf16lo_to_f32(a), bf16hi_to_f32(a)) : f32x2_pack(bf16lo_to_f32(a), bf16lo_to_f32(b));
          x1[i] = kHalf ? f32x2_pack(bf16lo_to_f32(b), bf16hi_to_f32(b)) : f32x2_pack(bf16hi_to_f32(a), bf16hi_to_f32(b));
        }
        const bool store = left > 0;
        left -= step;
        src += src_step;
        if (left > 0) {                            // the next heads, while these are worked on
          load_v<V>(src, r0);
          load_v<V>(src + run, r1);
        }
        float scale = 1.f;
        if (w) {
          uint64_t q0 = f32x2_mul(x0[0], x0[0]), q1 = f32x2_mul(x1[0], x1[0]);
#pragma unroll
          for (int i = 1; i < V / 2; ++i) {
            q0 = f32x2_fma(x0[i], x0[i], q0);
            q1 = f32x2_fma(x1[i], x1[i], q1);
          }
          float sa, sb, sc, sd;
          f32x2_unpack(q0, sa, sb);
          f32x2_unpack(q1, sc, sd);
          float ss = (sa + sb) + (sc + sd);
          if (LPR > 1 && !store) ss = 0.f;         // lanes past the row's end
#pragma unroll
          for (int o = LPR / 2; o > 0; o /= 2) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
          scale = rsqrtf(fmaf(ss, inv_d, p.eps));
        }
        const uint64_t scale2 = f32x2_pack(scale, scale);
        uint32_t o0[V / 2], o1[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          uint64_t y0 = f32x2_mul(x0[i], f00[i]), y1 = f32x2_mul(x1[i], f11[i]);
          if (turned) {
            y0 = f32x2_fma(x1[i], f01[i], y0);
            y1 = f32x2_fma(x0[i], f10[i], y1);
          }
          y0 = f32x2_mul(y0, scale2);
          y1 = f32x2_mul(y1, scale2);
          float a0, a1, b0, b1;                    // y0 and y1 of pair 2 i, of pair 2 i + 1
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
        if (store) {
          store_v<V>(dst, o0);
          store_v<V>(dst + run, o1);
        }
        dst += dst_step;
      }
    };
    rotate(p.q, p.oq, p.wq, p.q_heads);
    rotate(p.k, p.ok, p.wk, p.k_heads);
  }
}

// Kernel 10: a thread owns one position (a column of the tables) and walks over a share of the
// pairs; 32 neighbouring threads write one 128-byte line of each table.  Tokens m, m + P,
// m + 2P, ... have the same position and get the same values.
struct TableParams {
  const void* pos;
  int axes, P, M, pairs, rot_pairs;
  int per;                                 // pairs per grid row
  float *cos, *sin;                        // [pairs, M]
};

template <bool kFloat>
__global__ void __launch_bounds__(kThreads)
rope_tables_kernel(const __grid_constant__ TableParams p, const __grid_constant__ Freqs fr) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int m0 = blockIdx.x * kThreads + threadIdx.x;
  if (m0 >= p.P) return;
  const int i0 = blockIdx.y * p.per, i1 = min(i0 + p.per, p.pairs);
  float* cos = p.cos + static_cast<long long>(i0) * p.M + m0;
  float* sin = p.sin + static_cast<long long>(i0) * p.M + m0;
  int i = i0;
  while (i < min(i1, p.rot_pairs)) {               // axis by axis
    const int a = fr.axis[i];
    float bad;
    const uint32_t x = position<kFloat>(p.pos, static_cast<long long>(m0) * p.axes + a, bad);
    int end = i + 1;
    while (end < min(i1, p.rot_pairs) && fr.axis[end] == a) ++end;
#pragma unroll 4
    for (; i < end; ++i) {
      float s, c;
      sincos_turns(turn_fraction<kFloat>(x, fr.f[i]), s, c);
      if (kFloat) {
        s += bad;
        c += bad;
      }
      cos[0] = c;
      sin[0] = s;
      for (long long m = p.P; m < p.M - m0; m += p.P) {
        cos[m] = c;
        sin[m] = s;
      }
      cos += p.M;
      sin += p.M;
    }
  }
  for (; i < i1; ++i, cos += p.M, sin += p.M)      // pairs past the rotated columns stay as they are
    for (long long m = 0; m < p.M - m0; m += p.P) {
      cos[m] = 1.f;
      sin[m] = 0.f;
    }
}

}  // namespace k9
}  // namespace svdq
