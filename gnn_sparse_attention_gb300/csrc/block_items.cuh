// block_items.cuh -- work items of the backward's key side: how many there can
// be, and how the units that chose a key tile become items.  Host and device
// code without CUDA types, so that the counting is tested without a GPU.
//
// Capacity.  A unit's list entry is a bit of one block, and with offsets in order
// a block belongs to one key tile, so the tiles' counts c add up to `entries` at
// most.  A tile of c > chunk units has ceil(c / chunk) <= 2 c / chunk items, each
// with a slot for its partial sums: 2 entries / chunk + 2 slots hold them all.
// Offsets that are not in order make tiles share blocks: a bit then counts in
// several of them and the items may want more than that.  A tile whose items do
// not all fit gets empty ones (its dK and dV are undefined then, as documented),
// and every item below the number that the kernels walk is written.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define GATTN_HD __host__ __device__ __forceinline__
#else
#define GATTN_HD inline
#endif

namespace gattn {

// Units of an item: about four items per SM when every unit lists topk blocks of
// other key tiles, at least 32 tiles of 128 rows each (fp32, whose products take
// twenty times as long: 1); more items than that cost partials (128 x 2D fp32
// each) without filling the GPU better.  At most 2^23 rows and 2^18 units, though: a
// warp that writes an item's results waits for all of it, and gives up after a
// second.  64 rows take 0.6 to 1 us (2^23: 0.13 s), a unit of few rows 0.3 us (2^18:
// 0.1 s), measured.
inline int item_units(int64_t entries, int rows, int sms, bool f32) {
  const int tile = rows > 128 ? rows : 128;
  const int64_t some = int64_t(f32 ? 1 : 32) * 128 / tile, least = some > 1 ? some : 1;
  const int64_t per = (entries + int64_t(sms) * 4 - 1) / (int64_t(sms) * 4);
  const int64_t most = (int64_t(1) << 23) / (rows > 32 ? rows : 32);
  return int(per < least ? least : per > most ? most : per);
}

// Item: x = key tile * Hkv + head, units [y, y + z) of those that chose the tile,
// w = slot of its partial sums or -1 (the tile's only item).
GATTN_HD int64_t item_slots(int64_t entries, int chunk) { return entries / chunk * 2 + 2; }

// items of a tile that c units chose (-1: a table row that is no tile)
GATTN_HD int tile_items(int c, int chunk) {
  return c < 0 ? 0 : c <= chunk ? 1 : int((int64_t(c) + chunk - 1) / chunk);
}

// Writes tile i's k items from number `item` on, with slots from `slot` on, and what
// the join reads of the tile: cnt[0] = units, cnt[1] = first slot or -1.
template <class Item>
GATTN_HD void put_items(int i, int k, int64_t item, int64_t slot, int chunk, int64_t slots,
                        int64_t max_items, int32_t* cnt, Item* items) {
  if (k <= 0) return;
  int c = cnt[0];
  if (item + k > max_items || (k > 1 && slot + k > slots)) cnt[0] = c = 0;
  const bool split = c > chunk;
  cnt[1] = split ? int32_t(slot) : -1;
  for (int j = 0; j < k && item + j < max_items; ++j) {
    Item x;
    x.x = i;
    x.y = split ? j * chunk : 0;
    x.z = split ? (c - x.y < chunk ? c - x.y : chunk) : c;
    x.w = split ? int32_t(slot + j) : -1;
    items[item + j] = x;
  }
}

}  // namespace gattn
