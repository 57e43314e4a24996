// Layout of the adapters' plan (svdq_lora_plan_pack), shared by the host packer and the kernels.
//
// 32-bit words, every section on a 16-byte boundary:
//   [0, 16)   header: "SVDQLORA", M, requests, slots, adapters, tiles, copy_tiles, groups
//   requests  [requests][2 slots]   the request's adapter ids, then its weights (float bits)
//   tiles     [tiles + copy_tiles][4]   {first row, rows (1..128), request, 0}; the copy tiles cover
//                                   the rows that no adapter touches (request -1)
//   groups    [groups][group words] rows of short requests with the same adapters, gathered:
//                                   {rows (1..16), 0, 0, 0}, ids [8], row indexes [16],
//                                   weights [16][slots]
#pragma once

#include <stddef.h>
#include <stdint.h>

#if !defined(__CUDACC__)
#define __host__
#define __device__
#endif

namespace svdq {

constexpr int kLoraMaxSlots = 8;
constexpr int kLoraMaxRank = 128;          // slots x rank
constexpr int kLoraGroupRows = 16;
constexpr int kLoraTileRows = 128;
constexpr int kLoraShortRows = 16;          // requests of at most this many rows are gathered into groups

struct LoraLayout {
  size_t requests, tiles, groups, words;   // word offsets; words in all
};

__host__ __device__ inline int lora_group_words(int slots) { return 4 + 8 + kLoraGroupRows + kLoraGroupRows * slots; }

__host__ __device__ inline LoraLayout lora_layout(size_t requests, int slots, size_t tiles, size_t groups) {
  LoraLayout L;
  L.requests = 16;
  L.tiles = (L.requests + requests * 2 * slots + 3) / 4 * 4;
  L.groups = L.tiles + tiles * 4;
  L.words = L.groups + groups * lora_group_words(slots);
  return L;
}

}  // namespace svdq
