// The gated block's backward pass: the gradient of its input, the sum of two products.
#include "ciera_glu.h"

namespace ciera {
namespace {

// One product to each of two teams of waves, added up through LDS.
template <typename D, bool TRANS, typename O, int BM>
__global__ __launch_bounds__(512, 2) void glu_xgrad_mid(GluXgradArgs a) {
  GroupTile t;
  int tn;
  if (!find_group_tile<BM>(a.offsets, a.groups, a.rows, (a.n + 127) / 128, blockIdx.x, &t, &tn)) return;
  const uint64_t row = (uint64_t)t.begin + (uint64_t)t.m * BM;
  const int n0 = TRANS ? tn * 128 : max(min(tn * 128, a.n - 128), 0);
  mid_tile<D, true, TRANS, BM, 2, Mid::SUM>(
      static_cast<const uint16_t*>(a.xg) + row * a.ldxg, a.ldxg, t.count - t.m * BM,
      static_cast<const uint16_t*>(a.wg) + (uint64_t)t.g * a.gsg + (TRANS ? (uint64_t)n0 * a.ldg : n0), a.ldg, a.n - n0, a.k,
      MidStore<O>{static_cast<O*>(a.out) + row * a.ldo + n0, a.ldo}, nullptr, nullptr, 0,
      static_cast<const uint16_t*>(a.wu) + (uint64_t)t.g * a.gsu + (TRANS ? (uint64_t)n0 * a.ldu : n0), a.ldu,
      static_cast<const uint16_t*>(a.xu) + row * a.ldxu, a.ldxu);
}

// Large tiles over both contractions in turn: the result is written once, and a tile has twice the
// stages.  65536 rows, 64 experts of 2048 x 1024: 530-580 us, 950-1040 TFLOP/s (two products of
// ciera_group_mm and the addition would take 560 and 80).  Matrix instructions are busy 54 %.
// A contraction that is not a multiple of 64 is taken without the loop that interleaves loads and
// products, since a whole stage may follow on a part of one (1024 and 1032 steps: 467 and 547 us,
// [N, K] 484 and 617; ciera_group_mm, which keeps the loop, loses as much to its last stage: 258 and
// 302, 265 and 342).
template <typename D, bool TRANS, typename O>
__global__ __launch_bounds__(512) void glu_xgrad_big(GluXgradArgs a) {
  typedef BigTiles<D, true, TRANS, BigOut<O>, Big::SUM> Tiles;
  __shared__ i32x4 lds[Tiles::kLds];
  Tiles big;
  big.init(lds);
  const BigOut<O> all = {static_cast<O*>(a.out), a.ldo};
  big_tiles<Tiles, BigOut<O>>(a.offsets, a.groups, a.rows, a.n, a.k, big,
                              [&](int g, uint64_t row, int om, int n0, int on, int half) {
    big.start(static_cast<const uint16_t*>(a.xg) + row * a.ldxg, a.ldxg, om, weights<TRANS>(a.wg, g, a.gsg, a.ldg, n0), a.ldg, on,
              a.k, half, weights<TRANS>(a.wu, g, a.gsu, a.ldu, n0), a.ldu,
              static_cast<const uint16_t*>(a.xu) + row * a.ldxu);
    return all.at(row, n0);
  });
}

// Few rows to a group: one product after the other into the same sums.
template <typename D, bool TRANS, typename O, int VEC>
__global__ __launch_bounds__(512) void glu_xgrad_thin(GluXgradArgs a) {
  typedef typename ThinOf<D, TRANS, VEC, 1>::T Thin;
  constexpr int BN = Thin::BN;
  __shared__ ThinPart<BN, 1> part;
  GroupTile t;
  int tn;
  if (!find_group_tile<16>(a.offsets, a.groups, a.rows, (a.n + BN - 1) / BN, blockIdx.x, &t, &tn)) return;
  const int n0 = tn * BN, left = a.n - n0, rows = t.count - t.m * 16;
  const uint64_t row = (uint64_t)t.begin + (uint64_t)t.m * 16;
  Thin thin;
  thin.run(static_cast<const uint16_t*>(a.xg) + row * a.ldxg, a.ldxg, rows, left, a.k,
           {weights<TRANS>(a.wg, t.g, a.gsg, a.ldg, n0)}, {a.ldg});
  thin.run(static_cast<const uint16_t*>(a.xu) + row * a.ldxu, a.ldxu, rows, left, a.k,
           {weights<TRANS>(a.wu, t.g, a.gsu, a.ldu, n0)}, {a.ldu});
  thin.put(part);
  O* out = static_cast<O*>(a.out) + row * a.ldo + n0;
  part.join(rows, left, [&](int m, int c, const f32x4* v) { store4(out + (uint64_t)m * a.ldo, c, left, v[0]); });
}

template <typename D, bool TRANS, typename O, int BM>
hipError_t run_glu_xgrad_mid(const GluXgradArgs& a, hipStream_t s) {
  constexpr int TEAMS = 2;
  dim3 grid;
  if (hipError_t e = tile_grid(max_row_tiles(a.rows, a.groups, BM) * ((a.n + 127) / 128), 256 * TEAMS, &grid)) return e;
  glu_xgrad_mid<D, TRANS, O, BM><<<grid, dim3(256 * TEAMS), 0, s>>>(a);
  return hipGetLastError();
}
template <typename D, bool TRANS, typename O, int VEC>
hipError_t run_glu_xgrad_thin(const GluXgradArgs& a, hipStream_t s) {
  constexpr int BN = TRANS ? 16 : 16 * VEC;
  dim3 grid;
  if (hipError_t e = tile_grid(max_row_tiles(a.rows, a.groups, 16) * ((a.n + BN - 1) / BN), 512, &grid)) return e;
  glu_xgrad_thin<D, TRANS, O, VEC><<<grid, dim3(512), 0, s>>>(a);
  return hipGetLastError();
}

template <typename D, bool TRANS, typename O>
hipError_t run_glu_xgrad(bool flat, const GluXgradArgs& a, hipStream_t s) {
  // As in glu_mm; 64 experts of 2048 x 1024, bf16, us:
  //   rows                2    8   16   32   64  100  128  192  256
  //   [K, N] thin       94   99  106  143  236
  //          64 rows    97   96  100  104  112  150  160  211
  //          128 rows        99   99  104  114  122  127  193
  //          256 x 256                                      138
  //   [N, K] thin          107       238
  //          64 rows        90       112
  // Tiles of two teams take a unit each: 128 rows also where those of 64 would be more than one
  // round of the card (13 groups, 2234 rows, 1447 x 777, 46 for 57; 7 groups, 2006 rows, 515 x 777,
  // are one round: 17 for 21).  The large tiles address the second product's operands with the
  // first one's offsets, so both have to have the same strides.
  if (big_enough<TRANS>(flat, a.rows, a.groups, a.n, a.k, 256) && short_stride(a.ldxg) && short_stride(a.ldg) &&
      a.ldxg == a.ldxu && a.ldg == a.ldu) {
    glu_xgrad_big<D, TRANS, O><<<dim3(kUnits), dim3(512), 0, s>>>(a);
    return hipGetLastError();
  }
  const int64_t rows = a.rows, groups = a.groups;
  const uint64_t nt = (a.n + 127) / 128, mid = max_row_tiles(rows, groups, 64) * nt;
  if ((rows <= 16 * groups && (!TRANS || mid < kUnits)) || (rows <= 256 * groups && mid <= kUnits / 4)) {
    if (!TRANS && max_row_tiles(rows, groups, 16) * ((a.n + 63) / 64) < kUnits / 2)
      return run_glu_xgrad_thin<D, TRANS, O, TRANS ? 4 : 2>(a, s);
    return run_glu_xgrad_thin<D, TRANS, O, 4>(a, s);
  }
  const int64_t tiles = (rows / 64 + groups / 2 + 1) * (int64_t)nt;  // of groups that end anywhere
  if (rows <= 64 * groups || tiles <= (int64_t)kUnits) return run_glu_xgrad_mid<D, TRANS, O, 64>(a, s);
  return run_glu_xgrad_mid<D, TRANS, O, 128>(a, s);
}

struct RunXgrad {
  bool flat;
  const GluXgradArgs& a;
  hipStream_t s;
  template <typename D, bool TRANS, typename O>
  hipError_t run() {
    return run_glu_xgrad<D, TRANS, O>(flat, a, s);
  }
};

}  // namespace

hipError_t launch_glu_xgrad(int dtype, bool out_f32, bool transpose_w, bool flat, const GluXgradArgs& a, hipStream_t s) {
  return by_type(dtype, out_f32, transpose_w, RunXgrad{flat, a, s});
}

}  // namespace ciera
