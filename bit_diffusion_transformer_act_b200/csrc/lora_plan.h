// Layout of the adapters' plan (svdq_lora_plan_pack), shared by the host packer and the kernels.
//
// 32-bit words, every section on a 16-byte boundary:
//   [0, 16)   header: "SVDQLORA", M, requests, slots, adapters, tiles, copy_tiles, groups, copy_groups
//   tiles     [tiles + copy_tiles][tile words]   rows of one long request: {first row, rows (1..128),
//             request, 0}, its ids [slots] and its weights [slots] (float bits); the copy tiles cover
//             runs of rows that no adapter touches (request -1; no kernel reads the request, it says whose
//             rows they are to who looks at a plan)
//   groups    [groups + copy_groups][group words]   rows of short requests with the same adapters,
//             gathered: {rows (1..16), 0, 0, 0}, ids [8], row indexes [16], weights [16][slots]; the
//             copy groups hold the rows of short untouched runs (every id -1) of a plan without tiles
// What a kernel needs of a tile or a group lies together, so that one round trip to memory fetches it.
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
constexpr int kLoraShortRows = 16;         // requests (and untouched runs) of at most this many rows go into groups
constexpr int kLoraMaxTileWords = 4 + 2 * kLoraMaxSlots;

struct LoraLayout {
  size_t tiles, groups, words;             // word offsets; words in all
};

__host__ __device__ inline int lora_tile_words(int slots) { return (4 + 2 * slots + 3) / 4 * 4; }
__host__ __device__ inline int lora_group_words(int slots) { return 4 + 8 + kLoraGroupRows + kLoraGroupRows * slots; }

inline LoraLayout lora_layout(int slots, size_t tiles, size_t groups) {
  LoraLayout L;
  L.tiles = 16;
  L.groups = L.tiles + tiles * lora_tile_words(slots);
  L.words = L.groups + groups * lora_group_words(slots);
  return L;
}

}  // namespace svdq
