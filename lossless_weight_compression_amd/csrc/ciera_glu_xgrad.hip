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

template <typename D, bool TRANS, typename O>
__global__ __launch_bounds__(512) void glu_xgrad_big(GluXgradArgs a) {
  typedef BigTiles<D, true, TRANS, BigOut<O>, Big::SUM> Tiles;
  __shared__ i32x4 lds[Tiles::kLds];
  Tiles big;
  big.init(lds);
  const BigOut<O> all = {static_cast<O*>(a.out), a.ldo};
  big_tiles<Tiles, BigOut<O>>(a.offsets, a.groups, a.rows, a.n, a.k, big, [&](int g, uint64_t row, int om, int n0, int on, int half) {
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

template <typename D, bool TRANS, typename O>
hipError_t run_glu_xgrad(bool flat, const GluXgradArgs& a, hipStream_t s) {
  // the second product's operands are addressed with the first one's offsets
  if (big_enough<TRANS>(flat, a.rows, a.groups, a.n, a.k, 256) && short_stride(a.ldxg) && short_stride(a.ldg) &&
      a.ldxg == a.ldxu && a.ldg == a.ldu) {
    glu_xgrad_big<D, TRANS, O><<<dim3(kUnits), dim3(512), 0, s>>>(a);
    return hipGetLastError();
  }
  const uint64_t thin = max_row_tiles(a.rows, a.groups, 16);
  if (a.rows <= 16 * (int64_t)a.groups) {
    constexpr int VEC = 4, BN = TRANS ? 16 : 16 * VEC;
    dim3 grid;
    if (hipError_t e = tile_grid(thin * ((a.n + BN - 1) / BN), 512, &grid)) return e;
    glu_xgrad_thin<D, TRANS, O, VEC><<<grid, dim3(512), 0, s>>>(a);
    return hipGetLastError();
  }
  dim3 grid;
  if (hipError_t e = tile_grid(max_row_tiles(a.rows, a.groups, 64) * ((a.n + 127) / 128), 512, &grid)) return e;
  glu_xgrad_mid<D, TRANS, O, 64><<<grid, dim3(512), 0, s>>>(a);
  return hipGetLastError();
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
