// Kernels 9 and 10: rotary positions with several axes -- applied to the normalised q and k of a
// projection (kernel 9), and as the cos / sin tables that the fused QKV projection reads
// (kernel 10).
//
// Mathematics.  A head's rotary pairs are dealt to the axes in order (axis a has d_a / 2 pairs);
// pair i of axis a turns by position[m, a] * theta_a^(-2 i / d_a).  The host passes each pair's
// frequency in turns, f = theta_a^(-2 i / d_a) / (2 pi), in 64 bits; the kernel forms
// t = position * f in 64 bits, subtracts the nearest integer, and takes the sine and cosine of
// 2 pi (t - rint t) in 32 bits.  A product in 32 bits would be off by position * 2^-24 radians
// (0.004 at position 65536); here the angle is within 2^-52 |t| turns before its one rounding
// to 32 bits.
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

struct Freqs {
  double f[kMaxPairs];                     // turns per unit of position, in pair order
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
  int pos_float;
  int axes, P, M, q_heads, heads;          // heads: of q and k together
  int D, rot;                              // head width, rotated columns
  int parts;                               // warps that share a token's heads
  float eps;
};

__device__ __forceinline__ double position(const void* pos, int is_float, long long i) {
  return is_float ? static_cast<double>(__ldg(static_cast<const float*>(pos) + i))
                  : static_cast<double>(__ldg(static_cast<const int*>(pos) + i));
}

// Sine and cosine of `turns` turns.
__device__ __forceinline__ void sincos_turns(double turns, float& s, float& c) {
  sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &s, &c);
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

// A unit is V pairs, held by one lane as two runs of V elements; LPR lanes (a power of two, at
// least D / 2V) hold a head's row, and a warp 32 / LPR heads of one token at a time.  A lane's
// unit does not change, so its sines and cosines are formed once per token and used for all of
// the token's heads.
template <int V, int LPR, bool kHalf>
__global__ void __launch_bounds__(kThreads)
qk_norm_rope_kernel(const __grid_constant__ Params p, const __grid_constant__ Freqs fr) {
  constexpr int HPW = 32 / LPR;
  const int lane = threadIdx.x % 32;
  const int u = lane % LPR, sub = lane / LPR;
  const bool active = u * 2 * V < p.D;             // lanes past the row's end hold nothing
  const bool turned = u * 2 * V < p.rot;           // units past the rotated columns are only normalised
  const int e0 = turned && kHalf ? V * u : 2 * V * u;
  const int e1 = turned && kHalf ? p.rot / 2 + V * u : 2 * V * u + V;
  double f[V];
  int ax[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    f[j] = turned ? fr.f[V * u + j] : 0.0;
    ax[j] = turned ? fr.axis[V * u + j] : 0;
  }
  grid_dependency_wait();                          // q and k come from the previous kernel
  grid_launch_dependents();
  uint32_t w0[2][V / 2], w1[2][V / 2];             // norm weights of q and k
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const __nv_bfloat16* w = t ? p.wk : p.wq;
#pragma unroll
    for (int j = 0; j < V / 2; ++j) w0[t][j] = w1[t][j] = 0u;
    if (w && active) {
      load_v<V>(w + e0, w0[t]);
      load_v<V>(w + e1, w1[t]);
    }
  }
  const int warps = gridDim.x * (kThreads / 32);
  const int wid = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  const int part = wid % p.parts;
  const float inv_d = 1.0f / static_cast<float>(p.D);
  for (long long m = wid / p.parts; m < p.M; m += warps / p.parts) {
    float c[V], s[V];
    if (turned) {
      const long long at = static_cast<long long>(static_cast<int>(m) % p.P) * p.axes;
#pragma unroll
      for (int j = 0; j < V; ++j) sincos_turns(position(p.pos, p.pos_float, at + ax[j]) * f[j], s[j], c[j]);
    }
    for (int h0 = part * HPW; h0 < p.heads; h0 += p.parts * HPW) {
      const int h = h0 + sub;
      const bool on = active && h < p.heads;
      const bool is_k = h >= p.q_heads;
      const View& vi = is_k ? p.k : p.q;
      const View& vo = is_k ? p.ok : p.oq;
      const int hh = is_k ? h - p.q_heads : h;
      uint32_t r0[V / 2], r1[V / 2];
#pragma unroll
      for (int j = 0; j < V / 2; ++j) r0[j] = r1[j] = 0u;
      if (on) {
        const __nv_bfloat16* src = vi.ptr + m * vi.row + hh * vi.head;
        load_v<V>(src + e0, r0);
        load_v<V>(src + e1, r1);
      }
      float x0[V], x1[V];                          // the unit's two runs
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        x0[2 * j] = bf16lo_to_f32(r0[j]);
        x0[2 * j + 1] = bf16hi_to_f32(r0[j]);
        x1[2 * j] = bf16lo_to_f32(r1[j]);
        x1[2 * j + 1] = bf16hi_to_f32(r1[j]);
      }
      float ss = 0.f;                              // no branch here: lanes of q and of k may share a warp
#pragma unroll
      for (int j = 0; j < V; ++j) ss = fmaf(x0[j], x0[j], fmaf(x1[j], x1[j], ss));
#pragma unroll
      for (int o = LPR / 2; o > 0; o /= 2) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
      if (is_k ? p.wk != nullptr : p.wq != nullptr) {
        const float rstd = rsqrtf(fmaf(ss, inv_d, p.eps));
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          const uint32_t a = is_k ? w0[1][j] : w0[0][j], b = is_k ? w1[1][j] : w1[0][j];
          x0[2 * j] *= rstd * bf16lo_to_f32(a);
          x0[2 * j + 1] *= rstd * bf16hi_to_f32(a);
          x1[2 * j] *= rstd * bf16lo_to_f32(b);
          x1[2 * j + 1] *= rstd * bf16hi_to_f32(b);
        }
      }
      if (turned) {
        // pair j: halves (x0[j], x1[j]); interleaved (x[2j], x[2j + 1]) of the 2V contiguous elements
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float& a = kHalf ? x0[j] : (j < V / 2 ? x0[2 * j] : x1[2 * j - V]);
          float& b = kHalf ? x1[j] : (j < V / 2 ? x0[2 * j + 1] : x1[2 * j + 1 - V]);
          const float y0 = a * c[j] - b * s[j];
          const float y1 = a * s[j] + b * c[j];
          a = y0;
          b = y1;
        }
      }
      if (on) {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          r0[j] = pack_bf16x2(x0[2 * j], x0[2 * j + 1]);
          r1[j] = pack_bf16x2(x1[2 * j], x1[2 * j + 1]);
        }
        __nv_bfloat16* dst = vo.ptr + m * vo.row + hh * vo.head;
        store_v<V>(dst + e0, r0);
        store_v<V>(dst + e1, r1);
      }
    }
  }
}

// Kernel 10: a thread owns one position (a column of the tables) and walks over a share of the
// pairs; 32 neighbouring threads write one 128-byte line of each table.  Tokens m, m + P,
// m + 2P, ... have the same position and get the same values.
struct TableParams {
  const void* pos;
  int pos_float;
  int axes, P, M, pairs, rot_pairs;
  int per;                                 // pairs per grid row
  float *cos, *sin;                        // [pairs, M]
};

__global__ void __launch_bounds__(kThreads)
rope_tables_kernel(const __grid_constant__ TableParams p, const __grid_constant__ Freqs fr) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int m0 = blockIdx.x * kThreads + threadIdx.x;
  if (m0 >= p.P) return;
  const int i0 = blockIdx.y * p.per, i1 = min(i0 + p.per, p.pairs);
  int last = -1;
  double x = 0.0;
  for (int i = i0; i < i1; ++i) {
    float s = 0.f, c = 1.f;                        // pairs past the rotated columns stay as they are
    if (i < p.rot_pairs) {
      const int a = fr.axis[i];
      if (a != last) {
        x = position(p.pos, p.pos_float, static_cast<long long>(m0) * p.axes + a);
        last = a;
      }
      sincos_turns(x * fr.f[i], s, c);
    }
    for (long long m = m0; m < p.M; m += p.P) {
      p.cos[static_cast<long long>(i) * p.M + m] = c;
      p.sin[static_cast<long long>(i) * p.M + m] = s;
    }
  }
}

}  // namespace k9
}  // namespace svdq
