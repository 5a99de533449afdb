// Rows of several items packed one after the other: offsets [items + 1] int32
// on the device, ascending from 0; item b's rows are offsets[b] .. offsets[b +
// 1] - 1. Rows from offsets[items] on belong to no item; here they are the rows
// of one item more, number `items`, for which every operator writes zeros. A
// null pointer: one item of all rows.
//
// A launch knows the number of rows and of items, not their lengths, and
// nothing waits for those. Its workgroups are numbered slots: an item of L rows,
// `per` units a row, takes the slots from floor(start per / tile) + b on, at
// most floor(end per / tile) + b of them, which is never fewer than ceil(L per /
// tile). So total = floor(n per / tile) + items + 1 slots are enough for any
// lengths, an item's first slot follows from its offset alone, and a slot finds
// its item by a search that needs no prefix sums. Slots past an item's last tile
// have nothing to do.
//
// Offsets that descend or leave 0 .. n are cut to it: their results mean
// nothing, but no access leaves the tensors.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace submconv {

struct Items {
  const int32_t* offsets;  // or null
  int32_t items;
  int64_t n;
};
// (tiles of 2^shift units)
inline int64_t item_slots(const Items& it, int64_t per, int shift) {
  return (it.n * per >> shift) + it.items + 1;
}
inline int64_t chunk_slots(const Items& it, uint32_t chunk) { return it.n / chunk + it.items + 1; }

namespace {

// First row of item b, 0 <= b <= items + 1.
__device__ __forceinline__ int64_t item_start(const Items& it, int b) {
  if (b == 0) return 0;
  if (b > it.items || !it.offsets) return it.n;
  const int64_t v = it.offsets[b];
  return v < 0 ? 0 : v < it.n ? v : it.n;
}

struct ItemTile {
  int32_t item;
  int64_t row0, rows;  // of the item
  int64_t tile;        // of the item; below 0 or past its last where the slot has nothing to do
};

// The item of a slot, by the lanes of each wave: 64 items a probe. Up to 63 items
// one probe is all that is read. tile_of: row -> number of its tile, were there
// one item.
template <typename F>
__device__ __forceinline__ ItemTile find_item_by(const Items& it, int64_t slot, F&& tile_of) {
  const int lane = threadIdx.x & 63;
  ItemTile r;
  if (it.items < 64) {
    const int b = lane + 1;
    const int v = static_cast<int>(item_start(it, b));  // (n is below 2^31)
    const int c = __popcll(__ballot(b <= it.items && tile_of(v) + b <= slot));
    r.item = c;
    r.row0 = c > 0 ? __builtin_amdgcn_readlane(v, c - 1) : 0;
    const int64_t e = __builtin_amdgcn_readlane(v, c);
    r.rows = e > r.row0 ? e - r.row0 : 0;
  } else {
    int lo = 0, hi = it.items;
    while (lo < hi) {
      const int step = (hi - lo + 63) / 64;
      const int b = lo + (lane + 1) * step;
      const bool ok = b <= hi && tile_of(item_start(it, b)) + b <= slot;
      const int c = __popcll(__ballot(ok));  // at most (hi - lo) / step of them have b <= hi
      hi = min(hi, lo + (c + 1) * step - 1);
      lo += c * step;
    }
    r.item = __builtin_amdgcn_readfirstlane(lo);
    r.row0 = item_start(it, r.item);
    const int64_t e = item_start(it, r.item + 1);
    r.rows = e > r.row0 ? e - r.row0 : 0;
  }
  r.tile = slot - (tile_of(r.row0) + r.item);
  return r;
}
__device__ __forceinline__ ItemTile find_item(const Items& it, int64_t per, int shift, int64_t slot) {
  return find_item_by(it, slot, [&](int64_t v) { return v * per >> shift; });
}
// Tiles of `chunk` rows.
__device__ __forceinline__ ItemTile find_chunk(const Items& it, uint32_t chunk, int64_t slot) {
  return find_item_by(it, slot, [&](int64_t v) { return static_cast<int64_t>(static_cast<uint32_t>(v) / chunk); });
}

// The same tiles in the order of their place in their item, `from_end` counted
// from the last tile, furthest first: the order of work under a causal mask, so
// that the longest walks start first whatever the items' lengths. index: 0 ..;
// the rows of no item come last. Up to 64 items: one a lane.
constexpr int kOrderedItems = 64;
__device__ __forceinline__ ItemTile find_item_longest(const Items& it, int64_t per, int shift, int64_t index,
                                                      bool from_end) {
  const int lane = threadIdx.x & 63;
  int n = 0;  // tiles of item `lane`
  if (lane < it.items) {
    const int64_t s = item_start(it, lane), e = item_start(it, lane + 1);
    if (e > s) n = static_cast<int>(((e - s) * per + (int64_t{1} << shift) - 1) >> shift);
  }
  int most = 0, total = 0;
  for (int i = 0; i < it.items; ++i) {
    const int v = __builtin_amdgcn_readlane(n, i);
    most = max(most, v);
    total += v;
  }
  ItemTile r;
  if (index >= total) {
    r.item = it.items;
    r.tile = index - total;
  } else {
    // tiles whose place is past p; the smallest p with at most `index` of them
    auto past = [&](int p) {
      int sum = 0;
      for (int i = 0; i < it.items; ++i) sum += max(0, __builtin_amdgcn_readlane(n, i) - p);
      return sum;
    };
    int lo = 0, hi = most;  // past(lo) > index >= past(hi)
    while (hi - lo > 1) {
      const int step = (hi - lo + 63) / 64, p = lo + (lane + 1) * step;
      const int c = __popcll(__ballot(p < hi && past(p) > index));
      lo += c * step;
      hi = min(hi, lo + step);
    }
    uint64_t have = __ballot(n >= hi);  // (hi >= 1: lanes without an item have none)
    for (int k = static_cast<int>(index) - past(hi); k > 0; --k) have &= have - 1;
    r.item = __builtin_amdgcn_readfirstlane(__ffsll(static_cast<unsigned long long>(have)) - 1);
    r.tile = from_end ? __builtin_amdgcn_readlane(n, r.item) - hi : hi - 1;
  }
  const int64_t s = item_start(it, r.item), e = item_start(it, r.item + 1);
  r.row0 = s;
  r.rows = e > s ? e - s : 0;
  return r;
}

}  // namespace
}  // namespace submconv
