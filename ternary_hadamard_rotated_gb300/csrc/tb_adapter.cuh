// The adapters' plan, as its kernel writes it and the linear's kernels read it.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace tb {

constexpr int32_t kAdapterMagic = 0x41445054;
constexpr int kAdapterMaxB = 16384, kAdapterMaxN = 16384;
constexpr int kAdapterMaxR = 256;

// Tokens are grouped by adapter (within one in the order they come in; behind the last adapter those without
// one), and every adapter's group is cut into tiles of at most tile_rows(kind) tokens.
constexpr int kTileKinds = 2;
constexpr int tile_rows(int kind) { return kind == 0 ? 16 : 128; }

struct AdapterPlan {  // head of the plan; behind it order int32 [T], then the tiles of each kind
  int32_t magic, T, n;
  int32_t tiles[kTileKinds];
  int32_t bare;  // where the tokens without an adapter begin
  int32_t rows;  // tokens of all requests
  int32_t pad;
};

struct AdapterTile {
  int32_t adapter;
  int32_t first, count;  // in `order`
  int32_t pad;
};

inline int64_t adapter_max_tiles(int64_t T, int64_t n, int kind) {
  const int64_t m = T / tile_rows(kind) + n;  // a group's last tile may be a part of one
  return m < T ? m : T;
}
inline size_t adapter_order_at() { return sizeof(AdapterPlan); }
inline size_t adapter_tiles_at(int64_t T, int64_t n, int kind) {
  size_t at = adapter_order_at() + ((size_t)T * 4 + 15) / 16 * 16;
  for (int i = 0; i < kind; ++i) at += (size_t)adapter_max_tiles(T, n, i) * sizeof(AdapterTile);
  return at;
}

}  // namespace tb
