// Kernels 13 and 14: the adapters of long requests, in tiles of up to 128 rows of one request.
//
// Mathematics.  out[m] = y[m] + sum_j B_j (w_j A_j x[m]).  Kernel 13 forms the tile's X [A_0; A_1; ...]^T (128 x
// slots rank, fp32), each CTA over a slice of K, and writes its part.  Kernel 14 adds a tile's parts in
// slice order, scales column block j by the request's w_j, splits the sum into a high and a low bf16 part
// (U = hi + lo to 2^-16 relative), forms [hi | lo] [B_0 B_1 ... | B_0 B_1 ...]^T for a 128 x 128 piece of the
// output, adds y and rounds once.
//
// What bounds them: memory.  With slots rank = 64 a row of X costs 2 K bytes and 2 K 64 flops, 64 flops per
// byte, and a value of Y 4 bytes and 256 flops -- against 265 flops per byte of the card.  So the MMAs only
// have to stay out of the way, and both kernels are streams: X through kernel 13, Y through kernel 14, each
// once; A, B and U come from L2.
//
// Kernel 13: grid of (tiles, slices of K).  The parts are small (512 slots rank bytes per row) and stay in L2; their
// layout [4 ranks][128 rows] makes a warp's stores and kernel 14's loads whole lines.  Summing them over
// distributed shared memory instead, in clusters along K, cost 4 to 5 us at the end of a 11 us kernel (4608 x 2560,
// 64 ranks): the clusters start late, wait for their slowest CTA, and their remote loads are slow.
// Kernel 14 is persistent: a CTA owns a run of (tile, 128 columns) pieces with the columns running first, so U
// is formed once per tile; it is the left operand and lives in tensor memory (two tiles of it), which leaves
// shared memory to the ring.  y and B arrive by TMA in a ring of stages, the sum overwrites y in its stage,
// and the stage is stored from there: 32-row slabs that the tile fills by TMA, a last partial slab row by
// row.  Rows of other requests in a partial tile are never stored; each row of an MMA's result depends on
// its own row of the left operand only.
//
// Every mbarrier wait is bounded (see ptx.cuh).
#pragma once

#include "lora_plan.h"
#include "lora_short.cuh"
#include "ptx.cuh"

namespace svdq {
namespace k13 {

constexpr int kRows = kLoraTileRows;
constexpr int kChunk = 64;
constexpr int kThreads = 192;                       // producer, MMA, four read-out warps
constexpr int kMaxStages = 6;                       // 8 and 12 gave nothing (4608 x 7680, 64 ranks: 35.8, 35.9, 36.5 us)
constexpr int kYAhead = 3;                          // pieces of y brought to L2 for kernel 14: 36.9 -> 35.7 us at 4608 x
                                                    // 7680, 64 ranks (1: 36.2, 2: 36.0, 4: 35.8, 6: 35.8)
constexpr int kXBytes = kRows * kChunk * 2;
constexpr int kTmemCols = 128;

struct Params {
  const int32_t* tiles;                             // the plan's tile records
  float* parts;                                     // [tiles][ks][slots rank / 4][128 rows][4]
  int K, rank, slots, adapters, ks, stages;
  int N, up_ctas, up_items, up_chunks;              // kernel 14's grid, its pieces, pieces per tile
  int up_ahead;                                     // how many pieces of y per CTA of it are brought to L2
};

// kind::f16 instruction descriptor: D f32, A and B bf16, K-major, M = 128.
__device__ __forceinline__ uint32_t idesc_bf16(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(128 >> 4) << 24);
}

__host__ __device__ constexpr int stage_bytes(int jr) { return kXBytes + jr * kChunk * 2; }
constexpr int kSmemExtra = 1024 + 8 * (2 * kMaxStages + 2) + 16 + 4 * kLoraMaxTileWords;

__global__ void __launch_bounds__(kThreads)
lora_tile_down_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmX128,
                      const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmYin128,
                      const Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const int jr = p.slots * p.rank;
  const int S = p.stages;
  const uint32_t off_bar = static_cast<uint32_t>(S * stage_bytes(jr));
  const uint32_t bars = base + off_bar;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kMaxStages + s); };
  const uint32_t acc_full = bars + 8u * (2 * kMaxStages);
  const uint32_t drain = acc_full + 8u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + off_bar + 8 * (2 * kMaxStages + 2));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* rec = reinterpret_cast<int32_t*>(tmem_slot + 4);   // the tile's record

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int32_t* rec_g = p.tiles + static_cast<size_t>(blockIdx.x) * lora_tile_words(p.slots);
  const int nck_all = p.K / kChunk;
  const int c0 = static_cast<int>(static_cast<long long>(nck_all) * blockIdx.y / p.ks);
  const int nck = static_cast<int>(static_cast<long long>(nck_all) * (blockIdx.y + 1) / p.ks) - c0;   // >= 1: ks <= K / 64

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < S; ++s) { mbar_init(full(s), 1); mbar_init(empty(s), 1); }
    mbar_init(acc_full, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmX);
    prefetch_tmap(&tmX128);
    prefetch_tmap(&tmA);
  }
  if (warp == 1) tmem_alloc<kTmemCols>(smem_addr(tmem_slot));
  if (warp == 2 && lane == 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(rec_g));   // a hint: L2 is coherent
  grid_dependency_wait();                           // X (or the plan, or an adapter) may come from the previous kernel
  if (warp == 2 && lane < 4 + p.slots) rec[lane] = __ldcg(rec_g + lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Kernel 14 counts on this coming after the wait.  After the allocation too, as in every kernel here that uses
  // tensor memory: what starts now may take the rest of it and wait for this grid.
  grid_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  const int row0 = rec[0], nrows = rec[1];
  const int32_t* ids = rec + 4;

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    const int slabs = (nrows + 31) / 32;
    for (int c = 0; c < nck; ++c) {
      const int s = c % S;
      const uint32_t sb = base + s * stage_bytes(jr);
      if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(empty(s), ((c / S) & 1u) ^ 1u, abort_flag, 71))) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(full(s), slabs * 4096 + jr * kChunk * 2);
        if (slabs == 4) tma_load_2d(sb, &tmX128, (c0 + c) * kChunk, row0, full(s));
        else
          for (int i = 0; i < slabs; ++i) tma_load_2d(sb + i * 4096, &tmX, (c0 + c) * kChunk, row0 + 32 * i, full(s));
        for (int j = 0; j < p.slots; ++j)           // an empty slot's rows lie past the pool: read as zeros
          tma_load_2d(sb + kXBytes + j * p.rank * kChunk * 2, &tmA, (c0 + c) * kChunk,
                      (ids[j] < 0 ? p.adapters : ids[j]) * p.rank, full(s));
      }
      __syncwarp();
    }
    // The memory is idle between the last of X and kernel 14: the first pieces of y of one of its CTAs come to L2
    // meanwhile (a hint), asked for when X has arrived, so that X does not wait for them.
    const int up = gridDim.x * gridDim.y - 1 - (blockIdx.x + blockIdx.y * gridDim.x);   // the last CTAs do it
    if (up < p.up_ctas && mbar_wait_bounded(full((nck - 1) % S), ((nck - 1) / S) & 1u, abort_flag, 75)) {
      const int i = static_cast<int>(static_cast<long long>(p.up_items) * up / p.up_ctas) + lane / 2;
      const int col = (i % p.up_chunks * 2 + lane % 2) * 64;   // lanes 2 k, 2 k + 1: the k-th piece's halves
      if (lane < 2 * p.up_ahead && col < p.N)
        tma_prefetch_l2_2d(&tmYin128, col, __ldcg(p.tiles + static_cast<size_t>(i / p.up_chunks) * lora_tile_words(p.slots)));
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issue (one elected lane)
    constexpr uint32_t kHiSw128 = smem_desc_hi(1024, 2);
    constexpr uint32_t kLbo = 1u << 16;
    const uint32_t idesc = idesc_bf16(jr);
    for (int c = 0; c < nck; ++c) {
      const int s = c % S;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(full(s), (c / S) & 1u, abort_flag, 72))) break;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t sb = base + s * stage_bytes(jr);
        const uint32_t a_lo = (sb >> 4) | kLbo, b_lo = ((sb + kXBytes) >> 4) | kLbo;
#pragma unroll
        for (int kk = 0; kk < kChunk / 16; ++kk)
          umma_bf16(tmem, make_desc(a_lo + kk * 2, kHiSw128), make_desc(b_lo + kk * 2, kHiSw128), idesc,
                    (c | kk) != 0 ? 1u : 0u);
        tc_commit(empty(s));
        if (c == nck - 1) tc_commit(acc_full);
      }
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------------- read-out: a row per thread
    const int q = warp & 3;
    if (__all_sync(0xFFFFFFFFu, mbar_wait_bounded(acc_full, 0, abort_flag, 73))) {
      tc_fence_after();
      float4* dst = reinterpret_cast<float4*>(p.parts) +
                    (static_cast<size_t>(blockIdx.x) * p.ks + blockIdx.y) * (jr / 4) * kRows + q * 32 + lane;
      for (int c = 0; c < jr; c += 32) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(q * 32) << 16) + c, v);
        tmem_wait_ld_regs(v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + 4 * j < jr)
            dst[(c / 4 + j) * kRows] = make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                                   __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
      }
      tc_fence_before();
    }
  }
  __syncthreads();
  if (*abort_flag) {
    // a wait ran out: let the MMAs and copies already issued finish before the memory goes away
    if (warp == 1) {
      if (elect_one()) tc_commit(drain);
      __syncwarp();
      mbar_wait_bounded(drain, 0, nullptr, 74);
    }
    if (warp == 0 && lane == 0) {
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 2000000ull) { }
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<kTmemCols>(tmem);
  }
}

}  // namespace k13

namespace k14 {

constexpr int kRows = kLoraTileRows;
constexpr int kGroups = 2;                          // epilogue groups of four warps, taking pieces in turn
constexpr int kUWarp0 = 2 + 4 * kGroups;
constexpr int kThreads = (kUWarp0 + 8) * 32;        // producer, MMA, epilogue, U makers
constexpr int kMaxStages = 6;
constexpr int kBN = 128;                            // output columns per piece
constexpr int kAhead = 4;                           // pieces of y brought to L2 behind the first ring: 38.6 -> 36.5 us at
                                                    // 4608 x 7680, 64 ranks (2: 37.1, 6: 36.9, 12: 37.9)
constexpr int kTmemU = kGroups * kBN;               // tensor memory: an accumulator per group, then two U
constexpr int kTmemCols = 512;
static_assert(kTmemU + 2 * kLoraMaxRank <= kTmemCols, "tensor memory");

struct Params {
  const int32_t* tiles;                             // the plan's tile records
  const float* parts;                               // kernel 13's
  int ks;
  __nv_bfloat16* Y;
  long long ldy;
  int ntiles;                                       // tiles with adapters; tiles after them are copied
  int items, chunks;                                // (tile, kBN columns) pieces; pieces per tile
  int N, rank, slots, adapters, stages;
  int wb;                                           // columns per box of B: 64, 32 or 16
  int early;                                        // y, B and the plan are complete before this grid's dependency
};

// Shared memory (1024-byte aligned): stages of (B, y) | barriers.
__host__ __device__ constexpr int b_bytes(int jr) { return kBN * jr * 2; }
__host__ __device__ constexpr int stage_bytes(int jr) { return b_bytes(jr) + kRows * kBN * 2; }
constexpr int kNumBars = 2 * kMaxStages + 5 + 2 * kGroups;   // full, empty; u_full[2], u_empty[2], drain; acc_full, acc_empty
constexpr int kSmemExtra = 1024 + 8 * kNumBars + 16;

// Descriptor words of a K-major tile stored as boxes of w columns (128-, 64- or 32-byte swizzle).  All by
// shifts: one thread issues the MMAs, and with divisions here (w is not known when compiling) 16 of them
// took 3000 cycles.
struct Boxes {
  uint32_t hi, box_bytes;
  int lw;                                           // log2 w
};
__device__ __forceinline__ Boxes boxes(int w, int rows) {
  Boxes b;
  b.lw = w == 64 ? 6 : w == 32 ? 5 : 4;
  b.box_bytes = static_cast<uint32_t>(rows * w * 2);
  b.hi = w == 64 ? smem_desc_hi(1024, 2) : w == 32 ? smem_desc_hi(512, 4) : smem_desc_hi(256, 6);
  return b;
}
__device__ __forceinline__ uint64_t box_desc(const Boxes& b, uint32_t at, uint32_t col) {
  return make_desc(((at + (col >> b.lw) * b.box_bytes + (col & ((1u << b.lw) - 1)) * 2) >> 4) | (1u << 16), b.hi);
}

__global__ void __launch_bounds__(kThreads)
lora_tile_up_kernel(const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmYin,
                    const __grid_constant__ CUtensorMap tmYin128, const __grid_constant__ CUtensorMap tmY,
                    const Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const int jr = p.slots * p.rank;
  const int S = p.stages;
  const int stage = stage_bytes(jr);
  const uint32_t bars = base + S * stage;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kMaxStages + s); };
  auto u_full = [&](int u) { return bars + 8u * (2 * kMaxStages + u); };
  auto u_empty = [&](int u) { return bars + 8u * (2 * kMaxStages + 2 + u); };
  auto acc_full = [&](int b) { return bars + 8u * (2 * kMaxStages + 4 + b); };
  auto acc_empty = [&](int b) { return bars + 8u * (2 * kMaxStages + 4 + kGroups + b); };
  const uint32_t drain = bars + 8u * (2 * kMaxStages + 4 + 2 * kGroups);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + S * stage + 8 * kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int i0 = static_cast<int>(static_cast<long long>(p.items) * blockIdx.x / gridDim.x);
  const int i1 = static_cast<int>(static_cast<long long>(p.items) * (blockIdx.x + 1) / gridDim.x);

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < S; ++s) { mbar_init(full(s), 1); mbar_init(empty(s), 5); }   // four epilogue warps, the MMAs
    for (int u = 0; u < 2; ++u) { mbar_init(u_full(u), 8); mbar_init(u_empty(u), 1); }
    for (int b = 0; b < kGroups; ++b) { mbar_init(acc_full(b), 1); mbar_init(acc_empty(b), 4); }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmB);
    prefetch_tmap(&tmYin);
    prefetch_tmap(&tmYin128);
    prefetch_tmap(&tmY);
  }
  if (warp == 1) tmem_alloc<kTmemCols>(smem_addr(tmem_slot));
  if (!p.early) grid_dependency_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int tile_words = lora_tile_words(p.slots);
  auto tile_of = [&](int t) { return __ldcg(reinterpret_cast<const int4*>(p.tiles + static_cast<size_t>(t) * tile_words)); };

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    // With early, y, B and the plan are older than kernel 13 (which let this grid start after its own
    // dependency wait): their loads go out at once, and only U waits for kernel 13.
    int last = -1, it = 0;
    int4 tile = make_int4(0, 0, 0, 0);
    int b_row = 0;                                  // lane j: first row of slot j's adapter in B
    for (int i = i0; i < i1; ++i, ++it) {
      const int t = i / p.chunks, n0 = i % p.chunks * kBN;
      const int s = it % S;
      const bool busy = t < p.ntiles;
      if (t != last) {                              // the plan is read once per tile, not per piece
        tile = tile_of(t);
        if (busy && lane < p.slots) {
          const int id = __ldcg(p.tiles + static_cast<size_t>(t) * tile_words + 4 + lane);
          b_row = id < 0 ? -1 : id * p.N;
        }
        last = t;
      }
      if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(empty(s), ((it / S) & 1u) ^ 1u, abort_flag, 81))) break;
      const int slabs = (tile.y + 31) / 32, halves = min(kBN, p.N - n0) / 64;
      const uint32_t sb = base + s * stage;
      if (elect_one()) {
        mbar_arrive_expect_tx(full(s), slabs * halves * 4096 + (busy ? b_bytes(jr) : 0));
        for (int h = 0; h < halves; ++h) {
          if (slabs == 4) {                         // one box of 128 rows
            tma_load_2d(sb + b_bytes(jr) + h * 16384, &tmYin128, n0 + 64 * h, tile.x, full(s));
            continue;
          }
          for (int q = 0; q < slabs; ++q)
            tma_load_2d(sb + b_bytes(jr) + (h * 4 + q) * 4096, &tmYin, n0 + 64 * h, tile.x + 32 * q, full(s));
        }
      }
      __syncwarp();
      for (int j = 0; busy && j < p.slots; ++j) {   // an empty slot's rows lie past the pool: read as zeros
        const int row = __shfl_sync(0xFFFFFFFFu, b_row, j);
        if (elect_one())
          for (int c = 0; c < p.rank; c += p.wb)
            tma_load_2d(sb + (j * p.rank + c) * kBN * 2, &tmB, c, row < 0 ? p.adapters * p.N : row + n0, full(s));
        __syncwarp();
      }
      if (p.early && it == S - 1) {
        // The ring is full until U is formed: the next pieces of y come to L2 meanwhile (lane k: the k-th).
        const int k = i + 1 + lane;
        if (lane < kAhead && k < i1) {
          const int4 ahead = tile_of(k / p.chunks);
          const int nk = k % p.chunks * kBN;
          for (int h = 0; h < min(kBN, p.N - nk); h += 64)
            for (int r = 0; r < ahead.y; r += 32) tma_prefetch_l2_2d(&tmYin, nk + h, ahead.x + r);
        }
        __syncwarp();
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issue (one elected lane)
    const uint32_t idesc = k13::idesc_bf16(kBN);
    const Boxes bb = boxes(p.wb, kBN);
    int last = -1, it = 0, nu = 0;                  // nu: tiles begun
    for (int i = i0; i < i1; ++i, ++it) {
      const int t = i / p.chunks;
      const int s = it % S;
      const int b = it % kGroups;
      if (t >= p.ntiles) {                          // a copied piece: handed on in its turn, without an MMA
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(full(s), (it / S) & 1u, abort_flag, 83) &&
                                         mbar_wait_bounded(acc_empty(b), ((it / kGroups) & 1u) ^ 1u, abort_flag, 90)))
          break;
        if (lane == 0) {
          mbar_arrive(acc_full(b));
          mbar_arrive(empty(s));
        }
        continue;
      }
      bool ok = true;
      if (t != last) {
        ok = mbar_wait_bounded(u_full(nu & 1), (nu >> 1) & 1u, abort_flag, 84);
        last = t;
        ++nu;
      }
      ok = ok && mbar_wait_bounded(full(s), (it / S) & 1u, abort_flag, 85);
      ok = ok && mbar_wait_bounded(acc_empty(b), ((it / kGroups) & 1u) ^ 1u, abort_flag, 86);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t sb = base + s * stage;
        const uint32_t d = tmem + static_cast<uint32_t>(b * kBN);
        const uint32_t u = tmem + static_cast<uint32_t>(kTmemU + ((nu - 1) & 1) * kLoraMaxRank);
#pragma unroll 2
        for (int c = 0; c < jr; c += 16) {          // hi and lo against the same columns of B
          const uint64_t db = box_desc(bb, sb, c);
          umma_bf16_ta(d, u + c / 2, db, idesc, c != 0 ? 1u : 0u);
          umma_bf16_ta(d, u + (jr + c) / 2, db, idesc, 1u);
        }
        tc_commit(acc_full(b));
        tc_commit(empty(s));
        if (i + 1 == i1 || (i + 1) / p.chunks != t) tc_commit(u_empty((nu - 1) & 1));
      }
      __syncwarp();
    }
  } else if (warp >= kUWarp0) {
    // ---------------------------------------------------------------- U: a row per thread, two warps per lane
    // quarter taking blocks of 16 ranks in turn.  (With the epilogue's warps helping at a CTA's first tile, which
    // everything waits for, 64 and 128 ranks stayed within 1 % and 32 ranks lost 1.5 us of 30 to spilled registers.)
    if (p.early) grid_dependency_wait();            // kernel 13 is done
    const int q = warp & 3;
    const uint32_t trow = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(kTmemU);
    const size_t part = static_cast<size_t>(jr / 4) * kRows;   // float4 per part
    int nu = 0;
    for (int t = i0 / p.chunks; t < p.ntiles && t * static_cast<long long>(p.chunks) < i1; ++t, ++nu) {
      const int32_t* rec = p.tiles + static_cast<size_t>(t) * tile_words + 4;
      const int my_id = lane < p.slots ? __ldcg(rec + lane) : -1;   // lane j: slot j's adapter and weight
      const float my_w = lane < p.slots ? __int_as_float(__ldcg(rec + p.slots + lane)) : 0.f;
      const float4* src = reinterpret_cast<const float4*>(p.parts) + t * p.ks * part + q * 32 + lane;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(u_empty(nu & 1), ((nu >> 1) & 1u) ^ 1u, abort_flag, 82))) break;
      tc_fence_after();
      const uint32_t tu = trow + static_cast<uint32_t>((nu & 1) * kLoraMaxRank);
      for (int c = (warp - kUWarp0) / 4 * 16; c < jr; c += 32) {
        float4 u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int z = 0; z < p.ks; z += 4) {           // 16 loads in flight; added in slice order
          float4 v[4][4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (z + k < p.ks) v[k][j] = __ldcg(src + (z + k) * part + (c / 4 + j) * kRows);
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (z + k < p.ks) {
                u[j].x += v[k][j].x;
                u[j].y += v[k][j].y;
                u[j].z += v[k][j].z;
                u[j].w += v[k][j].w;
              }
        }
        const int slot = c / p.rank;
        const bool has = __shfl_sync(0xFFFFFFFFu, my_id, slot) >= 0;   // an empty slot adds nothing, whatever is in X
        const float w = __shfl_sync(0xFFFFFFFFu, my_w, slot);
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float uu[4] = {has ? u[j].x * w : 0.f, has ? u[j].y * w : 0.f, has ? u[j].z * w : 0.f,
                               has ? u[j].w * w : 0.f};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float l0, l1;
            const uint32_t h0 = k11::split_hi_lo(uu[2 * k], l0), h1 = k11::split_hi_lo(uu[2 * k + 1], l1);
            hi[2 * j + k] = h0 | (h1 << 16);
            lo[2 * j + k] = pack_bf16x2(l0, l1);
          }
        }
        tmem_st_32x32b_x8(tu + static_cast<uint32_t>(c / 2), hi);
        tmem_st_32x32b_x8(tu + static_cast<uint32_t>((jr + c) / 2), lo);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(u_full(nu & 1));
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3;                         // tensor-memory lane quarter = 32-row slab of the tile
    const int b = (warp - 2) / 4;                   // group, and its accumulator
    const uint32_t trow = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(b * kBN);
    const uint32_t sw = static_cast<uint32_t>(lane & 7);
    int last = -1;
    int4 tile = make_int4(0, 0, 0, 0);
    for (int it = b; i0 + it < i1; it += kGroups) {
      const int i = i0 + it;
      const int t = i / p.chunks, n0 = i % p.chunks * kBN;
      const int s = it % S;
      if (t != last) tile = tile_of(t);
      last = t;
      const bool busy = t < p.ntiles;
      // The accumulator first: pieces are handed over in order, so this piece's stage is then in its own phase.
      // (The other order could take an earlier phase's end for this one's, where the stage was last used by
      // the other group.)
      const bool ok = mbar_wait_bounded(acc_full(b), (it / kGroups) & 1u, abort_flag, 87) &&
                      mbar_wait_bounded(full(s), (it / S) & 1u, abort_flag, 88);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      tc_fence_after();
      const int rows = min(32, tile.y - 32 * q);    // of this slab; none or fewer where the tile ends
      const int halves = min(kBN, p.N - n0) / 64;
      const uint32_t yq = base + s * stage + b_bytes(jr) + q * 4096;
      if (rows > 0 && busy) {
        for (int h = 0; h < 2 * halves; ++h) {      // 32 columns at a time
          uint32_t v[32];
          tmem_ld_32x32b_x32(trow + static_cast<uint32_t>(32 * h), v);
          const uint32_t yrow = yq + (h >> 1) * 16384 + lane * 128;
          uint4 y[4];
#pragma unroll
          for (int c = 0; c < 4; ++c)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(y[c].x), "=r"(y[c].y), "=r"(y[c].z), "=r"(y[c].w)
                         : "r"(yrow + (((4u * (h & 1) + c) ^ sw) << 4)));
          tmem_wait_ld_regs(v);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t* w = reinterpret_cast<uint32_t*>(&y[c]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              w[j] = pack_bf16x2(bf16lo_to_f32(w[j]) + __uint_as_float(v[8 * c + 2 * j]),
                                 bf16hi_to_f32(w[j]) + __uint_as_float(v[8 * c + 2 * j + 1]));
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                         ::"r"(yrow + (((4u * (h & 1) + c) ^ sw) << 4)), "r"(y[c].x), "r"(y[c].y), "r"(y[c].z),
                           "r"(y[c].w)
                         : "memory");
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty(b));     // the accumulator has been read
      if (rows == 32) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
          for (int h = 0; h < halves; ++h) tma_store_2d(&tmY, yq + h * 16384, n0 + 64 * h, tile.x + 32 * q);
      } else if (rows > 0) {
        __syncwarp();
        for (int h = 0; h < halves; ++h)
          for (int r = lane / 8; r < rows; r += 4) {   // eight lanes write a row's 128 bytes
            const uint32_t c = static_cast<uint32_t>(lane & 7);
            uint4 v;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(yq + h * 16384 + r * 128 + ((c ^ (static_cast<uint32_t>(r) & 7u)) << 4)) : "memory");
            *reinterpret_cast<uint4*>(p.Y + (tile.x + 32 * q + r) * p.ldy + n0 + 64 * h + 8 * c) = v;
          }
        // TMA refills the stage: the warp's writes of the sums are ordered before that (another proxy), and every
        // lane has read what it stores (lanes leave the loop at different rows) before lane 0 hands the stage back.
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (lane == 0) {                              // hand the stage back once its store has read it
        bulk_commit_group();
        bulk_wait_group_read<0>();
        mbar_arrive(empty(s));
      }
      __syncwarp();
    }
    if (lane == 0) bulk_wait_group<0>();
    __syncwarp();
  }
  grid_launch_dependents();

  __syncthreads();
  if (*abort_flag) {
    if (warp == 1) {
      if (elect_one()) tc_commit(drain);
      __syncwarp();
      mbar_wait_bounded(drain, 0, nullptr, 89);
    }
    if (warp == 0 && lane == 0) {
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 2000000ull) { }
    }
    __syncthreads();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<kTmemCols>(tmem);
  }
}

}  // namespace k14
}  // namespace svdq
