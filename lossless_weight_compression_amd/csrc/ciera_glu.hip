// The experts' gated feed-forward block, h = act(x Wg) (x Wu) on the rows of every group,
// and its backward pass.
#include "ciera.h"
#include "ciera_act.h"
#include "ciera_mid.h"
#include "ciera_ops_internal.h"
#include "ciera_tiles.h"

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
hipError_t run_glu_mm(bool flat, const GluMmArgs& a, hipStream_t s) {
  dim3 grid;
  if (hipError_t e = tile_grid(max_row_tiles(a.rows, a.groups, 64) * ((a.n + 63) / 64), 256, &grid)) return e;
  glu_mm_mid<D, TRANS, O, 64, 1><<<grid, dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

template <typename D, bool TRANS, typename O>
hipError_t run_glu_grad(bool flat, const GluGradArgs& a, hipStream_t s) {
  dim3 grid;
  if (hipError_t e = tile_grid(max_row_tiles(a.rows, a.groups, 64) * ((a.n + 127) / 128), 256, &grid)) return e;
  glu_grad_mid<D, TRANS, O, 64, 1><<<grid, dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

template <typename D, bool TRANS, typename O>
hipError_t run_glu_xgrad(bool flat, const GluXgradArgs& a, hipStream_t s) {
  dim3 grid;
  if (hipError_t e = tile_grid(max_row_tiles(a.rows, a.groups, 64) * ((a.n + 127) / 128), 512, &grid)) return e;
  glu_xgrad_mid<D, TRANS, O, 64><<<grid, dim3(512), 0, s>>>(a);
  return hipGetLastError();
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
struct RunMm {
  bool flat;
  const GluMmArgs& a;
  hipStream_t s;
  template <typename D, bool TRANS, typename O>
  hipError_t run() {
    return run_glu_mm<D, TRANS, O>(flat, a, s);
  }
};
struct RunGrad {
  bool flat;
  const GluGradArgs& a;
  hipStream_t s;
  template <typename D, bool TRANS, typename O>
  hipError_t run() {
    return run_glu_grad<D, TRANS, O>(flat, a, s);
  }
};
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

hipError_t launch_glu_mm(int dtype, bool out_f32, bool transpose_w, bool flat, const GluMmArgs& a, hipStream_t s) {
  return by_type(dtype, out_f32, transpose_w, RunMm{flat, a, s});
}
hipError_t launch_glu_grad(int dtype, bool out_f32, bool transpose_w, bool flat, const GluGradArgs& a, hipStream_t s) {
  return by_type(dtype, out_f32, transpose_w, RunGrad{flat, a, s});
}
hipError_t launch_glu_xgrad(int dtype, bool out_f32, bool transpose_w, bool flat, const GluXgradArgs& a, hipStream_t s) {
  return by_type(dtype, out_f32, transpose_w, RunXgrad{flat, a, s});
}

}  // namespace ciera
