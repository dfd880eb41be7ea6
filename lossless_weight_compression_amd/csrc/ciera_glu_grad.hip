// The gated block's backward pass: the gradients of both projections.
#include "ciera_glu.h"

namespace ciera {
namespace {

template <typename D, bool TRANS, typename O, int BM, int TEAMS>
__global__ __launch_bounds__(256 * TEAMS, 2) void glu_grad_mid(GluGradArgs a) {
  GroupTile t;
  int tn;
  if (!find_group_tile<BM>(a.offsets, a.groups, a.rows, (a.n + 127) / 128, blockIdx.x, &t, &tn)) return;
  const uint64_t row = (uint64_t)t.begin + (uint64_t)t.m * BM;
  const int n0 = TRANS ? tn * 128 : max(min(tn * 128, a.n - 128), 0);
  const GradOut<O> out = {static_cast<const O*>(a.gate), static_cast<const O*>(a.up), static_cast<O*>(a.dgate),
                          static_cast<O*>(a.dup), a.ldg, a.ldu, a.lddg, a.lddu, a.act};
  mid_tile<D, true, TRANS, BM, TEAMS>(
      static_cast<const uint16_t*>(a.dy) + row * a.ldx, a.ldx, t.count - t.m * BM,
      static_cast<const uint16_t*>(a.w) + (uint64_t)t.g * a.gsw + (TRANS ? (uint64_t)n0 * a.ldw : n0), a.ldw, a.n - n0, a.k,
      out.at(row, n0));
}

// Large tiles, the gradients in their epilogue: D is neither written nor read again.  65536 rows,
// 64 experts of 1024 x 2048: 390-415 us; the product alone takes 290, the 540 MB that the epilogue
// reads and writes 80 at the memory's rate.  Each wave asks for G and U of the next 8 rows while
// it finishes 8 (four ahead took 50 registers more than there are), past the caches (1 %).
template <typename D, bool TRANS, typename O>
__global__ __launch_bounds__(512) void glu_grad_big(GluGradArgs a) {
  typedef BigTiles<D, true, TRANS, GradOut<O>, Big::PLAIN, WaveTileGrad<D, true, TRANS>> Tiles;
  __shared__ i32x4 lds[Tiles::kLds];
  Tiles big;
  big.init(lds);
  const GradOut<O> all = {static_cast<const O*>(a.gate), static_cast<const O*>(a.up), static_cast<O*>(a.dgate),
                          static_cast<O*>(a.dup), a.ldg, a.ldu, a.lddg, a.lddu, a.act};
  big_tiles<Tiles, GradOut<O>>(a.offsets, a.groups, a.rows, a.n, a.k, big,
                               [&](int g, uint64_t row, int om, int n0, int on, int half) {
    big.start(static_cast<const uint16_t*>(a.dy) + row * a.ldx, a.ldx, om, weights<TRANS>(a.w, g, a.gsw, a.ldw, n0), a.ldw, on,
              a.k, half);
    return all.at(row, n0);
  });
}

// Few rows to a group.
template <typename D, bool TRANS, typename O, int VEC>
__global__ __launch_bounds__(512) void glu_grad_thin(GluGradArgs a) {
  typedef typename ThinOf<D, TRANS, VEC, 1>::T Thin;
  constexpr int BN = Thin::BN;
  __shared__ ThinPart<BN, 1> part;
  GroupTile t;
  int tn;
  if (!find_group_tile<16>(a.offsets, a.groups, a.rows, (a.n + BN - 1) / BN, blockIdx.x, &t, &tn)) return;
  const int n0 = tn * BN, left = a.n - n0, rows = t.count - t.m * 16;
  const uint64_t row = (uint64_t)t.begin + (uint64_t)t.m * 16;
  Thin thin;
  thin.run(static_cast<const uint16_t*>(a.dy) + row * a.ldx, a.ldx, rows, left, a.k,
           {weights<TRANS>(a.w, t.g, a.gsw, a.ldw, n0)}, {a.ldw});
  thin.put(part);
  const GradOut<O> all = {static_cast<const O*>(a.gate), static_cast<const O*>(a.up), static_cast<O*>(a.dgate),
                          static_cast<O*>(a.dup), a.ldg, a.ldu, a.lddg, a.lddu, a.act};
  const GradOut<O> out = all.at(row, n0);
  part.join(rows, left, [&](int m, int c, const f32x4* v) { out.put(m, c, min(left - c, 4), v[0], f32x4{0, 0, 0, 0}); });
}

template <typename D, bool TRANS, typename O, int BM, int TEAMS>
hipError_t run_glu_grad_mid(const GluGradArgs& a, hipStream_t s) {
  
  dim3 grid;
  if (hipError_t e = tile_grid(max_row_tiles(a.rows, a.groups, BM) * ((a.n + 127) / 128), 256 * TEAMS, &grid)) return e;
  glu_grad_mid<D, TRANS, O, BM, TEAMS><<<grid, dim3(256 * TEAMS), 0, s>>>(a);
  return hipGetLastError();
}
template <typename D, bool TRANS, typename O, int VEC>
hipError_t run_glu_grad_thin(const GluGradArgs& a, hipStream_t s) {
  constexpr int BN = TRANS ? 16 : 16 * VEC;
  dim3 grid;
  if (hipError_t e = tile_grid(max_row_tiles(a.rows, a.groups, 16) * ((a.n + BN - 1) / BN), 512, &grid)) return e;
  glu_grad_thin<D, TRANS, O, VEC><<<grid, dim3(512), 0, s>>>(a);
  return hipGetLastError();
}

template <typename D, bool TRANS, typename O>
hipError_t run_glu_grad(bool flat, const GluGradArgs& a, hipStream_t s) {
  // As in glu_mm; 64 experts of 2048 x 1024, bf16, us:
  //   rows                2    8   16   32   64  100  128  192  256
  //   [K, N] thin       51   54   59   80  129
  //          64 rows    49   48   49   55   62   89   95  126
  //          128 rows        53   53   56   66   74   82  127
  //          256 x 256                                       94
  //   [N, K] thin           74       158
  //          64 rows        52        57
  // (One matrix 4096 x 1024, 200 rows, thin 17 for 40; 24 rows, half the columns, 9.9 for 14.9; 900
  // rows with two teams 33 for 41; but 777 x 515, 2006 rows over 7 groups, 21 for 20.)
  if (big_enough<TRANS>(flat, a.rows, a.groups, a.n, a.k, 256) && short_stride(a.ldx) && short_stride(a.ldw) &&
      short_stride(a.ldg) && short_stride(a.ldu) && short_stride(a.lddg) && short_stride(a.lddu)) {
    glu_grad_big<D, TRANS, O><<<dim3(kUnits), dim3(512), 0, s>>>(a);
    return hipGetLastError();
  }
  const int64_t rows = a.rows, groups = a.groups;
  const uint64_t nt = (a.n + 127) / 128, mid = max_row_tiles(rows, groups, 64) * nt;
  if ((rows <= 16 * groups && (!TRANS || mid < kUnits)) || (rows <= 256 * groups && mid <= kUnits / 4)) {
    if (!TRANS && max_row_tiles(rows, groups, 16) * ((a.n + 63) / 64) < kUnits / 2)
      return run_glu_grad_thin<D, TRANS, O, TRANS ? 4 : 2>(a, s);
    return run_glu_grad_thin<D, TRANS, O, 4>(a, s);
  }
  if (mid < kUnits && a.k >= 1024) return run_glu_grad_mid<D, TRANS, O, 64, 2>(a, s);
  if (rows <= 64 * groups || max_row_tiles(rows, groups, 128) * nt < 2 * kUnits)
    return run_glu_grad_mid<D, TRANS, O, 64, 1>(a, s);
  return run_glu_grad_mid<D, TRANS, O, 128, 1>(a, s);
}

struct RunGrad {
  bool flat;
  const GluGradArgs& a;
  hipStream_t s;
  template <typename D, bool TRANS, typename O>
  hipError_t run() {
    return run_glu_grad<D, TRANS, O>(flat, a, s);
  }
};

}  // namespace

hipError_t launch_glu_grad(int dtype, bool out_f32, bool transpose_w, bool flat, const GluGradArgs& a, hipStream_t s) {
  return by_type(dtype, out_f32, transpose_w, RunGrad{flat, a, s});
}

}  // namespace ciera
