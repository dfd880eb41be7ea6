// The experts' gated feed-forward block, h = act(x Wg) (x Wu) on the rows of every group,
// and its backward pass.
#include "ciera_glu.h"

namespace ciera {
namespace {

// Both products of a tile side by side: 64 columns of each, so that a lane has G and U of
// the same element.
template <typename D, bool TRANS, typename O, int BM, int TEAMS>
__global__ __launch_bounds__(256 * TEAMS, 2) void glu_mm_mid(GluMmArgs a) {
  GroupTile t;
  int tn;
  if (!find_group_tile<BM>(a.offsets, a.groups, a.rows, (a.n + 63) / 64, blockIdx.x, &t, &tn)) return;
  const uint64_t row = (uint64_t)t.begin + (uint64_t)t.m * BM;
  // the last tile ends with the matrix: it gives some columns a second time, the same values
  const int n0 = TRANS ? tn * 64 : max(min(tn * 64, a.n - 64), 0);
  const GluOut<O> out = {static_cast<O*>(a.out), static_cast<O*>(a.gate), static_cast<O*>(a.up), a.ldo, a.ldog, a.ldou, a.act};
  mid_tile<D, true, TRANS, BM, TEAMS, Mid::PAIR>(
      static_cast<const uint16_t*>(a.x) + row * a.ldx, a.ldx, t.count - t.m * BM,
      static_cast<const uint16_t*>(a.wg) + (uint64_t)t.g * a.gsg + (TRANS ? (uint64_t)n0 * a.ldg : n0), a.ldg, a.n - n0, a.k,
      out.at(row, n0), nullptr, nullptr, 0,
      static_cast<const uint16_t*>(a.wu) + (uint64_t)t.g * a.gsu + (TRANS ? (uint64_t)n0 * a.ldu : n0), a.ldu);
}

// Large tiles: 256 rows and 128 columns of both products, as much work as a plain 256 x 256 tile
// with a half or (G and U kept) one and a half times its results.  65536 rows over 64 experts of
// 2048 x 1024, all three kept: 565 us, 975 TFLOP/s; the plain kernel's two products alone take 560,
// and write as much without the activation.  Matrix instructions are busy 47 % of the time, the
// rest goes to the ends of tiles, where the next stages and the results pass L2 at once.
template <typename D, bool TRANS, typename O, bool KEEP>
__global__ __launch_bounds__(512) void glu_mm_big(GluMmArgs a) {
  typedef BigTiles<D, true, TRANS, GluOut<O>, Big::PAIR, WaveTilePair<D, true, TRANS, KEEP>> Tiles;
  __shared__ i32x4 lds[Tiles::kLds];
  Tiles big;
  big.init(lds);
  const GluOut<O> all = {static_cast<O*>(a.out), static_cast<O*>(a.gate), static_cast<O*>(a.up), a.ldo, a.ldog, a.ldou, a.act};
  big_tiles<Tiles, GluOut<O>>(a.offsets, a.groups, a.rows, a.n, a.k, big,
                              [&](int g, uint64_t row, int om, int n0, int on, int half) {
    big.start(static_cast<const uint16_t*>(a.x) + row * a.ldx, a.ldx, om, weights<TRANS>(a.wg, g, a.gsg, a.ldg, n0), a.ldg, on,
              a.k, half, weights<TRANS>(a.wu, g, a.gsu, a.ldu, n0), a.ldu);
    return all.at(row, n0);
  });
}

// Few rows to a group: 16 rows, and 16 * VEC columns ([N, K]: 16) of both products, so that x is
// read once for two weights.  1 token over 8 experts of 2048 x 1024: 15 us for 67 MB, most of it
// two latencies of memory (offsets, then weights) and the waves' 8 steps.
template <typename D, bool TRANS, typename O, int VEC>
__global__ __launch_bounds__(512) void glu_mm_thin(GluMmArgs a) {
  typedef typename ThinOf<D, TRANS, VEC, 2>::T Thin;
  constexpr int BN = Thin::BN;
  __shared__ ThinPart<BN, 2> part;
  GroupTile t;
  int tn;
  if (!find_group_tile<16>(a.offsets, a.groups, a.rows, (a.n + BN - 1) / BN, blockIdx.x, &t, &tn)) return;
  const int n0 = tn * BN, left = a.n - n0, rows = t.count - t.m * 16;
  const uint64_t row = (uint64_t)t.begin + (uint64_t)t.m * 16;
  Thin thin;
  thin.run(static_cast<const uint16_t*>(a.x) + row * a.ldx, a.ldx, rows, left, a.k,
           {weights<TRANS>(a.wg, t.g, a.gsg, a.ldg, n0), weights<TRANS>(a.wu, t.g, a.gsu, a.ldu, n0)}, {a.ldg, a.ldu});
  thin.put(part);
  const GluOut<O> all = {static_cast<O*>(a.out), static_cast<O*>(a.gate), static_cast<O*>(a.up), a.ldo, a.ldog, a.ldou, a.act};
  const GluOut<O> out = all.at(row, n0);
  part.join(rows, left, [&](int m, int c, const f32x4* v) { out.put4(m, c, left, v[0], v[1]); });
}

template <typename D, bool TRANS, typename O, int BM, int TEAMS>
hipError_t run_glu_mm_mid(const GluMmArgs& a, hipStream_t s) {
  
  dim3 grid;
  if (hipError_t e = tile_grid(max_row_tiles(a.rows, a.groups, BM) * ((a.n + 63) / 64), 256 * TEAMS, &grid)) return e;
  glu_mm_mid<D, TRANS, O, BM, TEAMS><<<grid, dim3(256 * TEAMS), 0, s>>>(a);
  return hipGetLastError();
}
template <typename D, bool TRANS, typename O, int VEC>
hipError_t run_glu_mm_thin(const GluMmArgs& a, hipStream_t s) {
  constexpr int BN = TRANS ? 16 : 16 * VEC;
  dim3 grid;
  if (hipError_t e = tile_grid(max_row_tiles(a.rows, a.groups, 16) * ((a.n + BN - 1) / BN), 512, &grid)) return e;
  glu_mm_thin<D, TRANS, O, VEC><<<grid, dim3(512), 0, s>>>(a);
  return hipGetLastError();
}

template <typename D, bool TRANS, typename O>
hipError_t run_glu_mm(bool flat, const GluMmArgs& a, hipStream_t s) {
  // By rows to a group on average; 64 experts of 2048 x 1024, bf16, us, inputs from call to call
  // in turn:
  //   rows                2    8   16   32   64  100  128  192  256
  //   [K, N] thin       99  100  102  143  254
  //          64 rows   105  105  107  110  116  151  154  214
  //          128 rows       103  106  111  119  126  129  184
  //          256 x 128                                      145
  //   [N, K] thin           117       239
  //          64 rows         90       102
  // The thin kernel takes [N, K], and more rows, only where tiles of 64 rows are too few for the
  // card (1 token over 8 of the experts, [N, K], 15 us for 17; one matrix 4096 x 1024, 200 rows, 27
  // for 32), with half the columns where even its workgroups are few (24 rows 20.9 for 23.5).  Two
  // teams to a tile where there is one tile to a unit at most (900 rows 32 for 36).
  if (big_enough<TRANS>(flat, a.rows, a.groups, a.n, a.k, 128) && short_stride(a.ldx) && short_stride(a.ldg) &&
      short_stride(a.ldu)) {
    if (a.gate) glu_mm_big<D, TRANS, O, true><<<dim3(kUnits), dim3(512), 0, s>>>(a);
    else glu_mm_big<D, TRANS, O, false><<<dim3(kUnits), dim3(512), 0, s>>>(a);
    return hipGetLastError();
  }
  const int64_t rows = a.rows, groups = a.groups;
  const uint64_t nt = (a.n + 63) / 64, mid = max_row_tiles(rows, groups, 64) * nt;
  if ((rows <= 16 * groups && (!TRANS || mid < kUnits)) || (rows <= 256 * groups && mid <= kUnits / 4)) {
    if (!TRANS && max_row_tiles(rows, groups, 16) * ((a.n + 63) / 64) < kUnits / 2)
      return run_glu_mm_thin<D, TRANS, O, TRANS ? 4 : 2>(a, s);
    return run_glu_mm_thin<D, TRANS, O, 4>(a, s);
  }
  if (mid < kUnits && a.k >= 1024) return run_glu_mm_mid<D, TRANS, O, 64, 2>(a, s);
  if (rows <= 64 * groups || max_row_tiles(rows, groups, 128) * nt < 2 * kUnits)
    return run_glu_mm_mid<D, TRANS, O, 64, 1>(a, s);
  return run_glu_mm_mid<D, TRANS, O, 128, 1>(a, s);
}

struct RunMm {
  bool flat;
  const GluMmArgs& a;
  hipStream_t s;
  template <typename D, bool TRANS, typename O>
  hipError_t run() {
    return run_glu_mm<D, TRANS, O>(flat, a, s);
  }
};
}  // namespace

hipError_t launch_glu_mm(int dtype, bool out_f32, bool transpose_w, bool flat, const GluMmArgs& a, hipStream_t s) {
  return by_type(dtype, out_f32, transpose_w, RunMm{flat, a, s});
}
}  // namespace ciera
