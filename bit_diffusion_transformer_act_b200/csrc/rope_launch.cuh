// Host side of the rotary calls: frequencies, checks, launches of kernels 9 and 10.  Part of libsvdq.cu, whose
// helpers it uses, and those of lora_launch.cuh.
#pragma once

#include <string.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>

#include "lora_launch.cuh"
#include "rope.cuh"

extern "C" {

// The pairs' frequencies in turns per unit of position, as the kernels read them (see Freqs).  Along an axis they
// are a geometric sequence, formed in extended precision (128 products of 2^-64 each).  They follow from the
// axes alone, and a model has one set: the last one of the thread is kept with what it was formed from
// (forming it costs as much as a launch).
struct RopeFreqs {
  int axes = 0, is_float = 0, rot = 0;
  int32_t dims[svdq::k9::kMaxAxes];
  double theta[svdq::k9::kMaxAxes];
  svdq::k9::Freqs fr;
};
static const RopeFreqs& rope_freqs(int axes, const int32_t* dims, const double* theta, bool is_float) {
  static thread_local RopeFreqs r;
  if (r.axes == axes && r.is_float == is_float && memcmp(r.dims, dims, axes * sizeof(int32_t)) == 0 &&
      memcmp(r.theta, theta, axes * sizeof(double)) == 0)
    return r;
  r.axes = axes;
  r.is_float = is_float;
  memcpy(r.dims, dims, axes * sizeof(int32_t));
  memcpy(r.theta, theta, axes * sizeof(double));
  int at = 0;
  for (int a = 0; a < axes; ++a) {
    const long double ratio = std::pow(static_cast<long double>(theta[a]), -2.0L / dims[a]);
    long double f = 0.159154943091895335768883763372514362L;   // 1 / (2 pi)
    for (int i = 0; i < dims[a] / 2; ++i, ++at) {
      if (is_float) {
        const double d = static_cast<double>(f);
        memcpy(&r.fr.f[at], &d, sizeof(d));
      } else {
        r.fr.f[at] = static_cast<uint64_t>(std::ldexp(f - std::floor(f), 64));   // whole turns do not count
      }
      r.fr.axis[at] = static_cast<uint8_t>(a);
      f *= ratio;
    }
  }
  r.rot = 2 * at;
  for (; at < svdq::k9::kMaxPairs; ++at) {
    r.fr.f[at] = 0;
    r.fr.axis[at] = 0;
  }
  return r;
}

// Checks of the arguments that both rotary calls share.
static int rope_check(const void* positions, int P, int axes, const int32_t* dims, const double* theta, int M,
                      int head_dim) {
  if (M < 0 || head_dim <= 0 || axes <= 0 || !dims || !theta) return SVDQ_ERR_INVALID_ARG;
  if (axes > svdq::k9::kMaxAxes || head_dim > 2 * svdq::k9::kMaxPairs) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  int64_t rot = 0;
  for (int a = 0; a < axes; ++a) {
    if (dims[a] <= 0 || !(theta[a] > 0.0) || !std::isfinite(theta[a])) return SVDQ_ERR_INVALID_ARG;
    if (dims[a] % 2 != 0) return SVDQ_ERR_UNSUPPORTED_SHAPE;
    rot += dims[a];
  }
  if (rot % 8 != 0 || rot > head_dim) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (M == 0) return SVDQ_OK;
  if (P <= 0 || M % P != 0) return SVDQ_ERR_INVALID_ARG;
  if (!positions || (reinterpret_cast<uintptr_t>(positions) & 3u)) return SVDQ_ERR_INVALID_ARG;
  return SVDQ_OK;
}

// A [M, heads, D] view with strides, made canonical where an extent is 1 (its stride then says nothing).
struct HeadsView {
  const void* ptr;
  int64_t row, head;
  int heads;
};
static HeadsView heads_view(const void* ptr, int64_t row, int64_t head, int heads, int M, int D) {
  if (heads <= 1) head = D;
  if (M <= 1) row = std::max<int64_t>(D, head * std::max(1, heads - 1) + D);
  return {ptr, row, head, heads};
}
static bool heads_ok(const HeadsView& v) {
  return v.ptr && aligned16(v.ptr) && v.row >= 0 && v.head >= 0 && v.row % 8 == 0 && v.head % 8 == 0;
}
// No two elements of the view are the same word.
static bool heads_distinct(const HeadsView& v, int M, int D) {
  const bool by_token = v.head >= D && v.row >= (v.heads - 1) * v.head + D;
  const bool by_head = v.row >= D && v.head >= (M - 1) * v.row + D;
  return by_token || by_head || (v.heads == 1 && v.row >= D);
}
static bool heads_overlap(const HeadsView& a, const HeadsView& b, int M, int D) {
  // token-major views are matrices of rows
  const int64_t wa = (a.heads - 1) * a.head + D, wb = (b.heads - 1) * b.head + D;
  if (!rows_overlap(a.ptr, a.row, wa, b.ptr, b.row, wb, M)) return false;
  // Rows that interlace (q and k of one head side by side) are told apart where the strides are the same:
  // heads m, h of a and m', h' of b meet where b's start is row (m - m') + head (h - h') from a's to within D.
  const int64_t head = a.heads > 1 ? a.head : b.head, row = a.row;
  if ((M > 1 && (row != b.row || row <= 0)) || (b.heads > 1 && b.head != head)) return true;   // others by their range
  const int64_t delta = (reinterpret_cast<intptr_t>(b.ptr) - reinterpret_cast<intptr_t>(a.ptr)) / 2;
  for (int64_t dh = 1 - b.heads; dh < a.heads; ++dh) {
    const int64_t left = delta - head * dh;
    const int64_t below = M > 1 ? left / row - (left % row < 0) : 0;   // floor
    for (int64_t dm = below; dm <= below + 1; ++dm)
      if (dm > -M && dm < M && std::abs(left - row * dm) < D) return true;
  }
  return false;
}

int svdq_qk_norm_rope(const void* Q, int64_t q_row_stride, int64_t q_head_stride, int q_heads, const void* K,
                      int64_t k_row_stride, int64_t k_head_stride, int k_heads, int M, int head_dim,
                      const void* norm_wq, const void* norm_wk, float eps, const void* positions, int positions_float,
                      int P, int axes, const int32_t* axis_dims, const double* axis_theta, int pairing, void* out_q,
                      int64_t oq_row_stride, int64_t oq_head_stride, void* out_k, int64_t ok_row_stride,
                      int64_t ok_head_stride, void* stream) {
  if (q_heads < 0 || k_heads < 0 || q_heads > (1 << 16) || k_heads > (1 << 16) || (pairing != 0 && pairing != 1))
    return SVDQ_ERR_INVALID_ARG;
  if ((norm_wq || norm_wk) && (!(eps >= 0.f) || !std::isfinite(eps))) return SVDQ_ERR_INVALID_ARG;
  if (int st = rope_check(positions, P, axes, axis_dims, axis_theta, M, head_dim)) return st;
  const int D = head_dim;
  if (D % 8 != 0) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (M == 0 || q_heads + k_heads == 0) return SVDQ_OK;
  if ((norm_wq && !aligned16(norm_wq)) || (norm_wk && !aligned16(norm_wk))) return SVDQ_ERR_INVALID_ARG;
  const HeadsView q = heads_view(Q, q_row_stride, q_head_stride, q_heads, M, D);
  const HeadsView k = heads_view(K, k_row_stride, k_head_stride, k_heads, M, D);
  const HeadsView oq = heads_view(out_q, oq_row_stride, oq_head_stride, q_heads, M, D);
  const HeadsView ok = heads_view(out_k, ok_row_stride, ok_head_stride, k_heads, M, D);
  auto same = [](const HeadsView& a, const HeadsView& b) { return a.ptr == b.ptr && a.row == b.row && a.head == b.head; };
  if (q_heads > 0 && (!heads_ok(q) || !heads_ok(oq) || !heads_distinct(oq, M, D) ||
                      (!same(q, oq) && heads_overlap(q, oq, M, D))))
    return SVDQ_ERR_INVALID_ARG;
  if (k_heads > 0 && (!heads_ok(k) || !heads_ok(ok) || !heads_distinct(ok, M, D) ||
                      (!same(k, ok) && heads_overlap(k, ok, M, D))))
    return SVDQ_ERR_INVALID_ARG;
  if (q_heads > 0 && k_heads > 0 &&
      (heads_overlap(oq, ok, M, D) || heads_overlap(oq, k, M, D) || heads_overlap(ok, q, M, D)))
    return SVDQ_ERR_INVALID_ARG;
  int dev;
  if (int st = current_device_ok(&dev)) return st;

  namespace k9 = svdq::k9;
  const RopeFreqs& rf = rope_freqs(axes, axis_dims, axis_theta, positions_float != 0);
  const k9::Freqs& fr = rf.fr;
  k9::Params p;
  p.rot = rf.rot;
  auto view = [](const HeadsView& v) {
    return k9::View{static_cast<__nv_bfloat16*>(const_cast<void*>(v.ptr)), v.row, v.head};
  };
  p.q = view(q);
  p.k = view(k);
  p.oq = view(oq);
  p.ok = view(ok);
  p.wq = static_cast<const __nv_bfloat16*>(norm_wq);
  p.wk = static_cast<const __nv_bfloat16*>(norm_wk);
  p.pos = positions;
  p.axes = axes;
  p.P = P;
  p.M = M;
  p.q_heads = q_heads;
  p.k_heads = k_heads;
  p.D = D;
  p.eps = eps;
  // 8 pairs per lane where runs of 8 fit the head and the rotated columns, else 4
  const int V = D % 16 == 0 && p.rot % 16 == 0 ? 8 : 4;
  int lpr = 1;
  while (lpr * 2 * V < D) lpr *= 2;
  // Groups of heads (what a warp holds at once) per unit: all of a token's, fewer where a unit would exceed
  // kUnitBytes (so that every warp has two stages), and fewer while there are less than two units for every warp
  // of the device.
  const int hpw = 32 / lpr;
  p.q_groups = (q_heads + hpw - 1) / hpw;
  p.groups = p.q_groups + (k_heads + hpw - 1) / hpw;
  const int group_bytes = hpw * D * 2;               // at most 1 KB
  const int64_t warps = static_cast<int64_t>(k9::kBlocksPerSm) * sm_count(dev) * k9::kWarps;
  const int64_t least = std::max<int64_t>((p.groups + k9::kUnitBytes / group_bytes - 1) / (k9::kUnitBytes / group_bytes),
                                          std::min<int64_t>(p.groups, 2 * warps / M));
  p.chunk = static_cast<int>((p.groups + least - 1) / std::max<int64_t>(1, least));
  p.units = static_cast<uint32_t>((p.groups + p.chunk - 1) / p.chunk);
  if (static_cast<int64_t>(M) * p.units > INT32_MAX) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  p.stage_bytes = (p.chunk * group_bytes + 127) / 128 * 128;
  p.stage_log = 4;
  static_assert(2 * k9::kWarps == 1 << 4, "the least stage_log");
  while ((2 << p.stage_log) <= k9::kMaxStages && (2 << p.stage_log) * p.stage_bytes <= k9::kRingBytes) ++p.stage_log;
  const int smem = (p.stage_bytes << p.stage_log) + k9::kAfterBytes;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(static_cast<int64_t>(M) * p.units, static_cast<int64_t>(k9::kBlocksPerSm) * sm_count(dev))));
  const int kind = (pairing ? 2 : 0) + (positions_float ? 1 : 0);
#define SVDQ_ROPE_LAUNCH(V_, L_, H_, F_)                                                               \
  (set_smem_once<k9::qk_norm_rope_kernel<V_, L_, H_, F_>>(k9::kRingBytes + k9::kAfterBytes, dev) &&         \
           launch_pdl(k9::qk_norm_rope_kernel<V_, L_, H_, F_>, grid, k9::kThreads, smem, stream, p, fr) \
       ? launch_status()                                                                                  \
       : SVDQ_ERR_CUDA)
#define SVDQ_ROPE_CASE(V_, L_)                                                                            \
  if (V == V_ && lpr == L_)                                                                               \
    return kind == 0   ? SVDQ_ROPE_LAUNCH(V_, L_, false, false)                                           \
           : kind == 1 ? SVDQ_ROPE_LAUNCH(V_, L_, false, true)                                            \
           : kind == 2 ? SVDQ_ROPE_LAUNCH(V_, L_, true, false)                                            \
                       : SVDQ_ROPE_LAUNCH(V_, L_, true, true)
  SVDQ_ROPE_CASE(8, 1);
  SVDQ_ROPE_CASE(8, 2);
  SVDQ_ROPE_CASE(8, 4);
  SVDQ_ROPE_CASE(8, 8);
  SVDQ_ROPE_CASE(8, 16);
  SVDQ_ROPE_CASE(4, 1);
  SVDQ_ROPE_CASE(4, 2);
  SVDQ_ROPE_CASE(4, 4);
  SVDQ_ROPE_CASE(4, 8);
  SVDQ_ROPE_CASE(4, 16);
  SVDQ_ROPE_CASE(4, 32);
#undef SVDQ_ROPE_CASE
#undef SVDQ_ROPE_LAUNCH
  return SVDQ_ERR_UNSUPPORTED_SHAPE;
}

int svdq_rope_axes_tables(const void* positions, int positions_float, int P, int axes, const int32_t* axis_dims,
                          const double* axis_theta, int M, int head_dim, void* rope_cos, void* rope_sin,
                          void* stream) {
  if (int st = rope_check(positions, P, axes, axis_dims, axis_theta, M, head_dim)) return st;
  if (head_dim % 2 != 0) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (M == 0) return SVDQ_OK;
  if (!rope_cos || !rope_sin || !aligned16(rope_cos) || !aligned16(rope_sin)) return SVDQ_ERR_INVALID_ARG;
  int dev;
  if (int st = current_device_ok(&dev)) return st;
  namespace k9 = svdq::k9;
  const RopeFreqs& rf = rope_freqs(axes, axis_dims, axis_theta, positions_float != 0);
  const k9::Freqs& fr = rf.fr;
  k9::TableParams p;
  p.pos = positions;
  p.axes = axes;
  p.P = P;
  p.M = M;
  p.pairs = head_dim / 2;
  p.rot_pairs = rf.rot / 2;
  p.cos = static_cast<float*>(rope_cos);
  p.sin = static_cast<float*>(rope_sin);
  const int bx = (P - 1) / (k9::kTableThreads * k9::kTokens) + 1;
  // pairs per thread: the fewest that keep the grid within eight blocks per SM (integer positions; with float ones
  // six fit)
  const int by = std::max(1, std::min(p.pairs, 8 * sm_count(dev) / bx));
  p.per = (p.pairs + by - 1) / by;
  if (!launch_pdl(positions_float ? k9::rope_tables_kernel<true> : k9::rope_tables_kernel<false>, dim3(bx, (p.pairs + p.per - 1) / p.per), k9::kTableThreads, 0, stream, p, fr))
    return SVDQ_ERR_CUDA;
  return launch_status();
}

}  // extern "C"
