// Shared by the kernels of the gated block: the large tiles in turn, dispatch by type.
#pragma once
#include "ciera.h"
#include "ciera_act.h"
#include "ciera_big.h"
#include "ciera_mid.h"
#include "ciera_ops_internal.h"
#include "ciera_thin.h"
#include "ciera_tiles.h"

namespace ciera {
namespace {

// Column n0 of group g's matrix; rows of W are its columns where it is transposed.
template <bool TRANS>
__device__ __forceinline__ const uint16_t* weights(const void* w, int g, uint64_t gs, uint64_t ld, int n0) {
  return static_cast<const uint16_t*>(w) + (uint64_t)g * gs + (TRANS ? (uint64_t)n0 * ld : n0);
}

// The large tiles of a kernel in turn.  place(group tile, first row in it, rows left, column)
// asks for the first stages of a tile and says where its results go.
template <typename Tiles, typename Out, typename F>
__device__ __forceinline__ void big_tiles(const int32_t* offsets, int groups, int rows, int n, int k, Tiles& big, F place) {
  GroupTiles<256> tiles;
  tiles.init(offsets, groups, rows);
  const uint32_t nt = (n + Tiles::BN - 1) / Tiles::BN;
  TileList list;
  list.init((uint64_t)tiles.total * nt);
  Out out;
  int om, on, half = 0;
  // false: no more tiles, or a half without rows
  auto start = [&](uint32_t i) {
    uint64_t tile;
    int r0, many;
    if (!list.get(i, &tile, &r0, &many)) return false;
    const GroupTile t = tiles.find((uint32_t)(tile / nt));
    const int n0 = (int)(tile % nt) * Tiles::BN;
    om = min(t.count - t.m * 256 - r0, many);
    on = n - n0;
    if (om <= 0) return false;
    out = place(t.g, (uint64_t)t.begin + (uint64_t)t.m * 256 + r0, om, n0, on, half);
    return true;
  };
  if (!start(0)) return;
  for (uint32_t i = 1;; i++) {
    big.stages(om, k, &half);
    const Out done = out;
    const int dm = om, dn = on;
    const bool more = start(i);
    big.finish(done, dm, dn);
    if (!more) return;
  }
}

// Whether the large tiles take a call: more than 128 rows to a group (up to there tiles of that
// height have one to a group), half the card at least, and rows that can be read straight into
// LDS.  cols: columns of a tile.
template <bool TRANS>
bool big_enough(bool flat, int64_t rows, int64_t groups, int n, int k, int cols) {
  return flat && k && k % 8 == 0 && (TRANS || n % 8 == 0) && rows > 128 * groups &&
         max_row_tiles(rows, groups, 256) * ((n + cols - 1) / cols) >= kUnits / 2;
}

// f<operand type, transposed weights, output type>()
template <typename D, typename O, typename F>
hipError_t by_order(bool transpose_w, F f) {
  return transpose_w ? f.template run<D, true, O>() : f.template run<D, false, O>();
}
template <typename F>
hipError_t by_type(int dtype, bool out_f32, bool transpose_w, F f) {
  (void)hipGetLastError();
  if (dtype == CIERA_BF16)
    return out_f32 ? by_order<Bf16, float>(transpose_w, f) : by_order<Bf16, __bf16>(transpose_w, f);
  return out_f32 ? by_order<Fp16, float>(transpose_w, f) : by_order<Fp16, _Float16>(transpose_w, f);
}

}  // namespace
}  // namespace ciera
