// Work items of the grouped expert GEMMs that need no tile list: every wave
// finds its output tile and rows from the experts' offsets.
#pragma once

#include "moe_internal.hpp"

namespace moe {

struct ItemArgs {
  const int32_t* offsets;
  int routed;                   // whether the routed experts are computed
  int per;                      // experts per lane in find_item, ceil(E / 64)
  int shared_rows;              // T, or 0 without the shared expert
  int ntn;                      // items per M-tile (max over groups)
  int E, K;
};

// This workgroup's output tile and rows.  Group g < E is routed expert g with
// rows [offsets[g], offsets[g + 1]), group E the shared expert with all T
// tokens; a group of n rows is cut into mt = ceil(n / kRows) M-tiles of equal
// height (+-1 row).  Items are numbered group by group, in a group N-tile by
// N-tile, so the M-tiles that share a weight tile run together, and dealt to
// the XCDs in chunks (as xcd_chunked).  Every wave finds its item itself from
// the offsets, a few experts a lane and a scan over the lanes: a list made by
// a kernel of its own costs that kernel's 4 us in every call.
__device__ __forceinline__ uint32_t wave_inclusive_scan(uint32_t v) {
  // Data-parallel moves: within each row of 16 lanes by 1, 2, 4, 8 (lanes
  // without a source add 0), then the last lane of row 0 / 2 to row 1 / 3 and
  // of row 1 to rows 2 and 3.
  v += __builtin_amdgcn_update_dpp(0u, v, 0x111, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0u, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0u, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0u, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0u, v, 0x142, 0xa, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0u, v, 0x143, 0xc, 0xf, false);
  return v;
}

struct Item {
  int g, row0, nrows, ntile;
  bool alone;   // the only M-tile of its group
};
template <int kRows>
__device__ __forceinline__ bool find_item(const ItemArgs& p, Item& it) {
  const int lane = threadIdx.x & 63;
  const uint32_t b = blockIdx.x, q = b / kNumXcd;
  const uint32_t w = ((q / kXcdChunk) * kNumXcd + b % kNumXcd) * kXcdChunk + q % kXcdChunk;
  const uint32_t i0 = w / (uint32_t)p.ntn;   // M-tile the item would be if each had ntn items
  auto tiles_of = [](int32_t n) { return (uint32_t)(n + kRows - 1) / kRows; };
  // M-tiles of this lane's experts, and the end of its range of M-tiles
  uint32_t mine = 0;
  int32_t from = 0;
  if (p.routed) {
    from = p.offsets[min(lane * p.per, p.E)];
    int32_t o = from;
    for (int j = 1; j <= p.per; ++j) {
      const int32_t next = p.offsets[min(lane * p.per + j, p.E)];
      mine += tiles_of(next - o);
      o = next;
    }
  }
  const uint32_t end = wave_inclusive_scan(mine);
  const uint32_t routed = __builtin_amdgcn_readlane(end, 63);
  int32_t g, n, r0;
  uint32_t L;
  if (i0 < routed) {
    const int src = __builtin_ctzll(__ballot(end > i0));
    // that lane's experts one by one, on the scalar unit
    g = src * p.per;
    L = __builtin_amdgcn_readlane(end - mine, src);
    r0 = __builtin_amdgcn_readlane(from, src);
    for (;; ++g) {
      const int32_t next = p.offsets[g + 1];
      n = next - r0;
      if (i0 < L + tiles_of(n) || g + 1 >= p.E) break;
      L += tiles_of(n);
      r0 = next;
    }
  } else {
    g = p.E;
    n = p.shared_rows;
    r0 = 0;
    L = routed;
    if (i0 >= routed + tiles_of(n)) return false;
  }
  const uint32_t mt = tiles_of(n), local = w - L * (uint32_t)p.ntn;
  if (mt == 1) {
    it = {g, r0, n, (int)local, true};
    return true;
  }
  const uint32_t m = local % mt;
  const int32_t first = (int32_t)((uint64_t)m * n / mt),
                last = (int32_t)((uint64_t)(m + 1) * n / mt);
  it = {g, r0 + first, last - first, (int)(local / mt), false};
  return true;
}

}  // namespace moe
