// Host side of the adapters' call: checks, workspace, launches of kernels 11 to 14.  Part of libsvdq.cu, whose
// helpers (device checks, tensor maps, shared-memory limits) it uses.
#pragma once

#include <algorithm>

#include "lora_plan.h"
#include "lora_short.cuh"
#include "lora_tile.cuh"

namespace {

// Two row-strided bf16 matrices (elements (m, c) at ptr[m * ld + c], c < width): whether they may share an
// element.  Windows of one matrix (equal row strides) are told apart by their columns.
bool rows_overlap(const void* a, int64_t lda, int64_t wa, const void* b, int64_t ldb, int64_t wb, int64_t rows) {
  const intptr_t pa = reinterpret_cast<intptr_t>(a) / 2, pb = reinterpret_cast<intptr_t>(b) / 2;
  if (pa + (rows - 1) * lda + wa <= pb || pb + (rows - 1) * ldb + wb <= pa) return false;
  if (lda != ldb || wa > lda || wb > lda) return true;
  const int64_t d = ((pb - pa) % lda + lda) % lda;        // b's first column in a's rows
  return !(d >= wa && d + wb <= lda);
}

// Launches `kernel` with programmatic dependent launch.
template <class... KArgs, class... Args>
bool launch_pdl(void (*kernel)(KArgs...), dim3 grid, int threads, int smem, void* stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;   // see grid_dependency_wait
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
    (void)cudaGetLastError();
    return false;
  }
  return true;
}

}  // namespace

extern "C" {

// CTAs over which a group's K is split in kernel 11: as many as keep the grid within about four CTAs
// per SM, each with at least 16 steps of 32 K (two per warp).
static int lora_short_splits(int groups, int K, int jr, int dev) {
  const int64_t ctas = static_cast<int64_t>(groups) * (jr / 16);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({4 * sm_count(dev) / ctas, K / 512, 16})));
}

static bool lora_plan_ok(const svdq_lora_plan* p) {
  return p && p->M >= 0 && p->requests >= 0 && p->slots >= 1 && p->slots <= svdq::kLoraMaxSlots && p->adapters >= 0 &&
         p->tiles >= 0 && p->copy_tiles >= 0 && p->groups >= 0 && p->copy_groups >= 0 &&
         p->bytes == static_cast<int64_t>(4 * svdq::lora_layout(p->slots, static_cast<size_t>(p->tiles) + p->copy_tiles,
                                                                static_cast<size_t>(p->groups) + p->copy_groups).words);
}

// Slices of K in kernel 13: as many as keep the grid within one CTA per SM (its ring then takes all of the
// shared memory), at least one, at most the 64-column chunks of K and four (kernel 14 reads every part).
// 4608 x 2560 -> 7680, 64 ranks, both kernels: 45.6, 39.3, 38.2, 38.8, 42.4, 44.2 us with 1, 2, 3, 4, 6, 8
// slices; 9001 x 10240 -> 2560, 128 ranks: 92, 69, 82, 77 us with 1, 2, 3, 4 (two is one CTA per SM).
static int lora_tile_splits(int tiles, int K, int dev) {
  return std::max(1, std::min({sm_count(dev) / std::max(1, tiles), K / 64, 4}));
}

// The workspace: kernel 13's parts, then kernel 11's.
struct LoraWorkspace {
  size_t part, total;
};
static LoraWorkspace lora_workspace(const svdq_lora_plan* p, int K, int jr, int dev) {
  LoraWorkspace w;
  w.part = static_cast<size_t>(p->tiles) * lora_tile_splits(p->tiles, K, dev) * svdq::kLoraTileRows * jr * sizeof(float);
  w.total = w.part;
  if (p->groups > 0)
    w.total += static_cast<size_t>(p->groups) * lora_short_splits(p->groups, K, jr, dev) * svdq::kLoraGroupRows * jr *
               sizeof(float);
  w.total = std::max<size_t>(w.total, 16);
  return w;
}

size_t svdq_lora_workspace_bytes(const svdq_lora_plan* plan, int K, int rank) {
  if (!lora_plan_ok(plan) || K <= 0 || K % 64 != 0 || rank <= 0 || rank % 16 != 0 ||
      plan->slots * static_cast<int64_t>(rank) > svdq::kLoraMaxRank)
    return 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    (void)cudaGetLastError();
    return 0;
  }
  return lora_workspace(plan, K, plan->slots * rank, dev).total;
}

// One call's arguments, checked.
struct LoraCall {
  const void *X, *Yin, *A, *B;
  void *Y, *ws, *stream;
  int64_t ldx, ldyin, ldy;
  const svdq_lora_plan* plan;
  const int32_t *tiles, *groups;                    // the plan's sections on the device
  int M, N, K, rank, jr, dev;
};

// Kernels 13 and 14: the tiles of long requests, and (copy) of the rows to copy.
static int lora_tiles_launch(const LoraCall& c, bool copy) {
  namespace k13 = svdq::k13;
  namespace k14 = svdq::k14;
  const int tiles = c.plan->tiles, all = tiles + (copy ? c.plan->copy_tiles : 0);
  const int jr = c.jr;
  const int sms = sm_count(c.dev);
  const auto bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (tiles > 0) {
    k13::Params p;
    p.tiles = c.tiles;
    p.parts = static_cast<float*>(c.ws);
    p.K = c.K;
    p.rank = c.rank;
    p.slots = c.plan->slots;
    p.adapters = c.plan->adapters;
    p.ks = lora_tile_splits(tiles, c.K, c.dev);
    // one CTA per SM takes all of the shared memory, a larger grid leaves room for three
    const int room = static_cast<int64_t>(tiles) * p.ks <= sms ? 227 * 1024 : 75 * 1024;
    p.stages = std::min(k13::kMaxStages, (room - k13::kSmemExtra) / k13::stage_bytes(jr));
    const int smem = p.stages * k13::stage_bytes(jr) + k13::kSmemExtra;
    p.N = c.N;
    p.up_chunks = (c.N + k14::kBN - 1) / k14::kBN;
    p.up_items = all * p.up_chunks;
    p.up_ctas = std::min(p.up_items, sms);
    p.up_ahead = std::min(k13::kYAhead, p.up_items / sms);
    CUtensorMap tX, tX128, tA, tYin128;
    if (!make_tmap(&tX, c.X, bf, 2, c.M, c.K, k13::kChunk, 32, CU_TENSOR_MAP_SWIZZLE_128B, c.ldx) ||
        !make_tmap(&tX128, c.X, bf, 2, c.M, c.K, k13::kChunk, 128, CU_TENSOR_MAP_SWIZZLE_128B, c.ldx) ||
        !make_tmap(&tYin128, c.Yin, bf, 2, c.M, c.N, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B, c.ldyin) ||
        !make_tmap(&tA, c.A, bf, 2, static_cast<uint64_t>(p.adapters) * c.rank, c.K, k13::kChunk, c.rank,
                   CU_TENSOR_MAP_SWIZZLE_128B) ||
        !set_smem_once<k13::lora_tile_down_kernel>(227 * 1024, c.dev))
      return SVDQ_ERR_CUDA;
    if (!launch_pdl(k13::lora_tile_down_kernel, dim3(tiles, p.ks), k13::kThreads, smem, c.stream, tX, tX128, tA,
                    tYin128, p))
      return SVDQ_ERR_CUDA;
  }
  k14::Params p;
  p.tiles = c.tiles;
  p.parts = static_cast<const float*>(c.ws);
  p.ks = lora_tile_splits(tiles, c.K, c.dev);
  p.Y = static_cast<__nv_bfloat16*>(c.Y);
  p.ldy = c.ldy;
  p.ntiles = tiles;
  p.N = c.N;
  p.chunks = (c.N + k14::kBN - 1) / k14::kBN;
  p.items = all * p.chunks;
  p.rank = c.rank;
  p.slots = c.plan->slots;
  p.adapters = c.plan->adapters;
  p.wb = c.rank % 64 == 0 ? 64 : c.rank % 32 == 0 ? 32 : 16;
  p.early = tiles > 0;
  p.stages = std::min(k14::kMaxStages, (227 * 1024 - k14::kSmemExtra) / k14::stage_bytes(jr));
  const int smem = p.stages * k14::stage_bytes(jr) + k14::kSmemExtra;
  auto swizzle = [](int w) {
    return w == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : w == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
  };
  CUtensorMap tB, tYin, tYin128, tY;
  if (!make_tmap(&tYin, c.Yin, bf, 2, c.M, c.N, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B, c.ldyin) ||
      !make_tmap(&tYin128, c.Yin, bf, 2, c.M, c.N, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B, c.ldyin) ||
      !make_tmap(&tY, c.Y, bf, 2, c.M, c.N, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B, c.ldy))
    return SVDQ_ERR_CUDA;
  tB = tY;                                          // not read when every tile is a copy
  if (tiles > 0 && !make_tmap(&tB, c.B, bf, 2, static_cast<uint64_t>(p.adapters) * c.N, c.rank, p.wb, k14::kBN, swizzle(p.wb)))
    return SVDQ_ERR_CUDA;
  if (!set_smem_once<k14::lora_tile_up_kernel>(227 * 1024, c.dev)) return SVDQ_ERR_CUDA;
  if (!launch_pdl(k14::lora_tile_up_kernel, dim3(std::min(p.items, sms)), k14::kThreads, smem, c.stream, tB, tYin,
                  tYin128, tY, p))
    return SVDQ_ERR_CUDA;
  return SVDQ_OK;
}

// Kernels 11 and 12: the groups of short requests, and (copy) of the rows to copy.
static int lora_groups_launch(const LoraCall& c, bool copy, float* part) {
  namespace k11 = svdq::k11;
  k11::Params p;
  p.X = static_cast<const __nv_bfloat16*>(c.X);
  p.A = static_cast<const __nv_bfloat16*>(c.A);
  p.B = static_cast<const __nv_bfloat16*>(c.B);
  p.Yin = static_cast<const __nv_bfloat16*>(c.Yin);
  p.Y = static_cast<__nv_bfloat16*>(c.Y);
  p.ldx = c.ldx;
  p.ldyin = c.ldyin;
  p.ldy = c.ldy;
  p.groups = c.groups;
  p.part = part;
  p.N = c.N;
  p.K = c.K;
  p.rank = c.rank;
  p.slots = c.plan->slots;
  p.ngroups = c.plan->groups;
  p.early = p.ngroups > 0;
  p.ks = 1;
  if (p.ngroups > 0) {
    p.ks = lora_short_splits(p.ngroups, c.K, c.jr, c.dev);
    if (!launch_pdl(k11::lora_short_down_kernel, dim3(p.ngroups, c.jr / 16, p.ks), k11::kThreads, 0, c.stream, p))
      return SVDQ_ERR_CUDA;
  }
  const int all = p.ngroups + (copy ? c.plan->copy_groups : 0);
  const int strips = (c.N / k11::kUpCols + k11::kUpWarps - 1) / k11::kUpWarps;
  const dim3 grid(all, std::max(1, std::min(strips, 4 * sm_count(c.dev) / all)));   // four CTAs per SM
  const int passes = (strips - 1) / static_cast<int>(grid.y) + 1;
  const int piece = k11::kUpWarps * k11::up_piece_bytes(c.jr);   // of all warps of a CTA
  p.depth = std::max(2, std::min({k11::kUpMaxDepth, k11::kUpRingBytes / piece, passes}));
  const int smem = p.depth * piece;
#define SVDQ_LORA_UP(WIDE_, STEPS_)                                                                                  \
  case STEPS_:                                                                                                       \
    return set_smem_once<k11::lora_short_up_kernel<WIDE_, STEPS_>>(                                                  \
               std::max(k11::kUpRingBytes, 2 * k11::kUpWarps * k11::up_piece_bytes(svdq::kLoraMaxRank)), c.dev) &&  \
                   launch_pdl(k11::lora_short_up_kernel<WIDE_, STEPS_>, grid, k11::kUpThreads, smem, c.stream, p) \
               ? SVDQ_OK                                                                                             \
               : SVDQ_ERR_CUDA
  if (c.rank % 32 == 0) {
    switch (c.jr / 32) {
      SVDQ_LORA_UP(true, 1);
      SVDQ_LORA_UP(true, 2);
      SVDQ_LORA_UP(true, 3);
      SVDQ_LORA_UP(true, 4);
    }
  } else {
    switch (c.jr / 16) {
      SVDQ_LORA_UP(false, 1);
      SVDQ_LORA_UP(false, 2);
      SVDQ_LORA_UP(false, 3);
      SVDQ_LORA_UP(false, 4);
      SVDQ_LORA_UP(false, 5);
      SVDQ_LORA_UP(false, 6);
      SVDQ_LORA_UP(false, 7);
      SVDQ_LORA_UP(false, 8);
    }
  }
#undef SVDQ_LORA_UP
  return SVDQ_ERR_UNSUPPORTED_SHAPE;
}

int svdq_lora_add(const void* X, int64_t ldx, const void* Yin, int64_t ldyin, const void* A, const void* B,
                  const svdq_lora_plan* plan, const void* plan_dev, size_t plan_bytes, int M, int N, int K, int rank,
                  void* workspace, size_t workspace_bytes, void* Y, int64_t ldy, void* stream) {
  if (M < 0 || N <= 0 || K <= 0 || rank <= 0 || !lora_plan_ok(plan) || plan->M != M) return SVDQ_ERR_INVALID_ARG;
  if (rank % 16 != 0 || plan->slots * static_cast<int64_t>(rank) > svdq::kLoraMaxRank || K % 64 != 0 || N % 64 != 0)
    return SVDQ_ERR_UNSUPPORTED_SHAPE;
  // tile coordinates and piece counts are 32-bit
  const int64_t all_tiles = static_cast<int64_t>(plan->tiles) + plan->copy_tiles;
  if (static_cast<int64_t>(plan->adapters) * N > INT32_MAX - N ||
      static_cast<int64_t>(plan->adapters) * rank > INT32_MAX - rank || all_tiles * (N / 64) > INT32_MAX ||
      all_tiles * svdq::kLoraTileRows > INT32_MAX)
    return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (M == 0) return SVDQ_OK;
  if (!Yin || !Y || !aligned16(Yin) || !aligned16(Y) || ldyin < N || ldy < N || ldyin % 8 != 0 || ldy % 8 != 0)
    return SVDQ_ERR_INVALID_ARG;
  const bool in_place = Y == Yin && (ldy == ldyin || M == 1);   // a single row's stride says nothing
  if (!in_place && rows_overlap(Yin, ldyin, N, Y, ldy, N, M)) return SVDQ_ERR_INVALID_ARG;
  if (!plan_dev || !aligned16(plan_dev) || plan_bytes < static_cast<size_t>(plan->bytes)) return SVDQ_ERR_INVALID_ARG;
  const bool work = plan->tiles > 0 || plan->groups > 0;
  if (work) {
    if (!X || !A || !B || !workspace || !aligned16(X) || !aligned16(A) || !aligned16(B) || !aligned16(workspace) ||
        ldx < K || ldx % 8 != 0)
      return SVDQ_ERR_INVALID_ARG;
    if (rows_overlap(X, ldx, K, Y, ldy, N, M)) return SVDQ_ERR_INVALID_ARG;
  }
  int dev;
  if (int st = current_device_ok(&dev)) return st;
  const LoraWorkspace ws = lora_workspace(plan, K, plan->slots * rank, dev);
  if (work && workspace_bytes < ws.total) return SVDQ_ERR_INVALID_ARG;

  const svdq::LoraLayout L = svdq::lora_layout(plan->slots, all_tiles, static_cast<size_t>(plan->groups) + plan->copy_groups);
  const int32_t* words = static_cast<const int32_t*>(plan_dev);
  const LoraCall c{X,    Yin, A, B, Y, workspace, stream, ldx, ldyin, ldy, plan, words + L.tiles, words + L.groups, M, N, K,
                   rank, plan->slots * rank, dev};
  if (plan->tiles > 0 || (plan->copy_tiles > 0 && !in_place))
    if (int st = lora_tiles_launch(c, !in_place)) return st;
  if (plan->groups > 0 || (plan->copy_groups > 0 && !in_place))
    if (int st = lora_groups_launch(c, !in_place, reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + ws.part)))
      return st;
  return launch_status();
}

}  // extern "C"
