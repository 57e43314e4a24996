// Host side of the per-request adapters: packs a batch's plan (lora_plan.h).  No GPU work.

#include <string.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "../../include/svdq.h"
#include "lora_plan.h"

namespace {

using svdq::kLoraGroupRows;
using svdq::kLoraTileRows;

bool sizes_ok(int M, int requests, int slots) {
  return M >= 0 && requests >= 0 && requests <= (1 << 24) && slots >= 1 && slots <= svdq::kLoraMaxSlots;
}

size_t tiles_of(size_t rows) { return (rows + kLoraTileRows - 1) / kLoraTileRows; }

// What a plan holds.
struct Pack {
  const int32_t* off;
  const int32_t* ids;
  const float* w;
  int requests, slots, M;
  std::vector<int> shorts;                 // short requests, ordered by their adapter ids
  size_t tiles = 0, copy_tiles = 0, groups = 0, copy_groups = 0;

  const int32_t* ids_of(int r) const { return ids + static_cast<size_t>(r) * slots; }
  const float* w_of(int r) const { return w + static_cast<size_t>(r) * slots; }
  bool has_adapter(int r) const {
    for (int j = 0; j < slots; ++j)
      if (ids_of(r)[j] >= 0) return true;
    return false;
  }
  int rows(int r) const { return off[r + 1] - off[r]; }

  // runs of rows that no adapter touches: f(first row, rows)
  template <class F>
  void untouched(F f) const {
    int from = 0;                          // first row not yet accounted for
    for (int r = 0; r < requests; ++r) {
      if (rows(r) == 0 || !has_adapter(r)) continue;
      if (off[r] > from) f(from, off[r] - from);
      from = off[r + 1];
    }
    if (M > from) f(from, M - from);
  }

  // Untouched runs become copy tiles, or rows of copy groups where they are short and kernel 14 is not
  // launched for long requests anyway.
  bool copied_as_rows(int n) const { return tiles == 0 && n <= svdq::kLoraShortRows; }

  int compare_ids(int a, int b) const {
    for (int j = 0; j < slots; ++j)
      if (ids_of(a)[j] != ids_of(b)[j]) return ids_of(a)[j] < ids_of(b)[j] ? -1 : 1;
    return 0;
  }

  // rows of short requests, those with the same ids together, in groups of at most kLoraGroupRows:
  // f(request, row, first of its group)
  template <class F>
  void grouped(F f) const {
    int held = 0;
    for (size_t i = 0; i < shorts.size(); ++i) {
      const int r = shorts[i];
      if (i > 0 && compare_ids(shorts[i - 1], r) != 0) held = 0;
      for (int m = off[r]; m < off[r + 1]; ++m) {
        f(r, m, held == 0);
        held = (held + 1) % kLoraGroupRows;
      }
    }
  }

  void count() {
    for (int r = 0; r < requests; ++r) {
      if (rows(r) == 0 || !has_adapter(r)) continue;
      if (rows(r) <= svdq::kLoraShortRows) shorts.push_back(r);
      else tiles += tiles_of(rows(r));
    }
    std::stable_sort(shorts.begin(), shorts.end(), [&](int a, int b) { return compare_ids(a, b) < 0; });
    grouped([&](int, int, bool first) { groups += first; });
    size_t few = 0;
    untouched([&](int, int n) {
      if (copied_as_rows(n)) few += n;
      else copy_tiles += tiles_of(n);
    });
    copy_groups = (few + kLoraGroupRows - 1) / kLoraGroupRows;
  }

  void write(int32_t* out, int adapters) const {
    const svdq::LoraLayout L = svdq::lora_layout(slots, tiles + copy_tiles, groups + copy_groups);
    memset(out, 0, L.words * sizeof(int32_t));
    memcpy(out, "SVDQLORA", 8);
    const int32_t head[8] = {M, requests, slots, adapters, static_cast<int32_t>(tiles),
                             static_cast<int32_t>(copy_tiles), static_cast<int32_t>(groups),
                             static_cast<int32_t>(copy_groups)};
    memcpy(out + 2, head, sizeof(head));
    const std::vector<int32_t> none(slots, -1);
    int32_t* t = out + L.tiles;
    auto put_tiles = [&](int row, int n, int r) {
      for (; n > 0; row += kLoraTileRows, n -= kLoraTileRows, t += svdq::lora_tile_words(slots)) {
        t[0] = row;
        t[1] = std::min(n, kLoraTileRows);
        t[2] = r;
        memcpy(t + 4, r < 0 ? none.data() : ids_of(r), slots * sizeof(int32_t));
        if (r >= 0) memcpy(t + 4 + slots, w_of(r), slots * sizeof(float));
      }
    };
    for (int r = 0; r < requests; ++r)
      if (rows(r) > svdq::kLoraShortRows && has_adapter(r)) put_tiles(off[r], rows(r), r);
    int32_t* g = nullptr;
    int32_t* next = out + L.groups;
    auto put_row = [&](int m, int r, bool first) {
      if (first) {
        g = next;
        next += svdq::lora_group_words(slots);
        for (int j = 0; j < 8; ++j) g[4 + j] = j < slots && r >= 0 ? ids_of(r)[j] : -1;
      }
      const int i = g[0]++;
      g[12 + i] = m;
      if (r >= 0) memcpy(g + 12 + kLoraGroupRows + i * slots, w_of(r), slots * sizeof(float));
    };
    grouped([&](int r, int m, bool first) { put_row(m, r, first); });
    int held = 0;
    untouched([&](int row, int n) {
      if (!copied_as_rows(n)) return put_tiles(row, n, -1);
      for (int m = row; m < row + n; ++m, held = (held + 1) % kLoraGroupRows) put_row(m, -1, held == 0);
    });
  }
};

}  // namespace

extern "C" {

size_t svdq_lora_plan_bytes(int M, int requests, int slots) {
  if (!sizes_ok(M, requests, slots)) return 0;
  const size_t r = static_cast<size_t>(requests), m = static_cast<size_t>(M);
  // every request, and every run of rows between requests, ends in a tile or group that may not be full
  const size_t tiles = 2 * (m / kLoraTileRows + r + 1);
  const size_t groups = m / kLoraGroupRows + r + 1;
  return svdq::lora_layout(slots, tiles, groups).words * sizeof(int32_t);
}

int svdq_lora_plan_pack(const int32_t* row_offsets, const int32_t* adapter_ids, const float* weights, int requests,
                        int slots, int M, int adapters, void* out, size_t out_bytes, svdq_lora_plan* plan) {
  if (!sizes_ok(M, requests, slots) || adapters < 0 || !out || !plan) return SVDQ_ERR_INVALID_ARG;
  if (requests > 0 && (!row_offsets || !adapter_ids || !weights)) return SVDQ_ERR_INVALID_ARG;
  if (requests > 0 && row_offsets[0] < 0) return SVDQ_ERR_INVALID_ARG;
  for (int r = 0; r < requests; ++r)
    if (row_offsets[r + 1] < row_offsets[r]) return SVDQ_ERR_INVALID_ARG;
  if (requests > 0 && row_offsets[requests] > M) return SVDQ_ERR_INVALID_ARG;
  for (size_t i = 0; i < static_cast<size_t>(requests) * slots; ++i)
    if (adapter_ids[i] < -1 || adapter_ids[i] >= adapters || !std::isfinite(weights[i])) return SVDQ_ERR_INVALID_ARG;
  try {
    Pack p{row_offsets, adapter_ids, weights, requests, slots, M, {}};
    p.count();
    const svdq::LoraLayout L = svdq::lora_layout(slots, p.tiles + p.copy_tiles, p.groups + p.copy_groups);
    if (out_bytes < L.words * sizeof(int32_t)) return SVDQ_ERR_INVALID_ARG;
    p.write(static_cast<int32_t*>(out), adapters);
    *plan = svdq_lora_plan{M, requests, slots, adapters, static_cast<int32_t>(p.tiles),
                           static_cast<int32_t>(p.copy_tiles), static_cast<int32_t>(p.groups),
                           static_cast<int32_t>(p.copy_groups), static_cast<int64_t>(L.words * sizeof(int32_t))};
  } catch (...) {                          // no memory for the host's lists
    return SVDQ_ERR_INVALID_ARG;
  }
  return SVDQ_OK;
}

}  // extern "C"
