// Products grouped by expert: y = x W_g on the rows of every group, and the
// gradient of the weights, x_g^T dy_g.
#include "ciera.h"
#include "ciera_ops_internal.h"
#include "ciera_tiles.h"

namespace ciera {
namespace {

// One BM x BN tile of C = A B over `klen` contraction steps, 4 waves of
// (BM / 2) x (BN / 2).  A has `am` rows left, B `bn` columns; loads go through
// registers, so that rows may start at any element and end anywhere.
template <typename D, bool AKC, bool BKC, bool FLAT, typename O, int BM, int BN>
__device__ __forceinline__ void general_tile(const uint16_t* a, uint64_t lda, int am, const uint16_t* b, uint64_t ldb,
                                             int bn, int klen, O* out, uint64_t ldo, int om, int on) {
  constexpr int BK = 32;
  typedef LdsTile<AKC, BM, BK> TA;
  typedef LdsTile<BKC, BN, BK> TB;
  constexpr int NA = TA::kChunks / 256, NB = TB::kChunks / 256;
  constexpr int WM = BM / 2 / 16, WN = BN / 2 / 16;
  __shared__ i32x4 la[2][TA::kChunks];
  __shared__ i32x4 lb[2][TB::kChunks];
  const int tid = threadIdx.x, wave = tid >> 6;
  const int r0 = (wave >> 1) * (BM / 2), c0 = (wave & 1) * (BN / 2);

  i32x4 ra[NA], rb[NB];
  auto load = [&](int k0) {
#pragma unroll
    for (int i = 0; i < NA; i++) {
      const int p = i * 256 + tid, line = p / TA::kPerRow, c = p % TA::kPerRow;
      ra[i] = AKC ? load_chunk<FLAT>(a, lda, line, am, k0 + c * 8, klen)
                  : load_chunk<FLAT>(a, lda, k0 + line, klen, c * 8, am);
    }
#pragma unroll
    for (int i = 0; i < NB; i++) {
      const int p = i * 256 + tid, line = p / TB::kPerRow, c = p % TB::kPerRow;
      rb[i] = BKC ? load_chunk<FLAT>(b, ldb, line, bn, k0 + c * 8, klen)
                  : load_chunk<FLAT>(b, ldb, k0 + line, klen, c * 8, bn);
    }
  };
  auto put = [&](int s) {
#pragma unroll
    for (int i = 0; i < NA; i++) {
      const int p = i * 256 + tid;
      la[s][TA::pos(p / TA::kPerRow, p % TA::kPerRow)] = ra[i];
    }
#pragma unroll
    for (int i = 0; i < NB; i++) {
      const int p = i * 256 + tid;
      lb[s][TB::pos(p / TB::kPerRow, p % TB::kPerRow)] = rb[i];
    }
  };

  f32x4 acc[WM][WN];
#pragma unroll
  for (int i = 0; i < WM; i++)
#pragma unroll
    for (int j = 0; j < WN; j++) acc[i][j] = f32x4{0, 0, 0, 0};

  const int steps = (klen + BK - 1) / BK;
  if (steps) {
    load(0);
    put(0);
  }
  __syncthreads();
  for (int s = 0; s < steps; s++) {
    const bool more = s + 1 < steps;
    if (more) load((s + 1) * BK);
    const int cur = s & 1;
    typename D::V fa[WM], fb[WN];
#pragma unroll
    for (int i = 0; i < WM; i++) fa[i] = __builtin_bit_cast(typename D::V, TA::fragment(la[cur], r0 + i * 16, 0));
#pragma unroll
    for (int j = 0; j < WN; j++) fb[j] = __builtin_bit_cast(typename D::V, TB::fragment(lb[cur], c0 + j * 16, 0));
#pragma unroll
    for (int i = 0; i < WM; i++)
#pragma unroll
      for (int j = 0; j < WN; j++) acc[i][j] = mfma(fb[j], fa[i], acc[i][j]);
    if (more) put(cur ^ 1);
    __syncthreads();
  }
  // the operands are given in swapped order: a lane holds 4 consecutive columns of a row
  const int lane = tid & 63;
#pragma unroll
  for (int i = 0; i < WM; i++) {
    const int m = r0 + i * 16 + (lane & 15);
    if (m >= om) continue;
#pragma unroll
    for (int j = 0; j < WN; j++) store4(out + (uint64_t)m * ldo, c0 + j * 16 + (lane >> 4) * 4, on, acc[i][j]);
  }
}

template <typename D, bool TRANS, bool FLAT, typename O, int BM, int BN>
__global__ __launch_bounds__(256) void group_mm_general(GroupMmArgs a) {
  GroupTile t;
  if (!find_group_tile(a.offsets, a.groups, a.rows, BM, (a.n + BN - 1) / BN, blockIdx.x, &t)) return;
  const uint64_t row = (uint64_t)t.begin + (uint64_t)t.m * BM;
  const int mleft = t.count - t.m * BM, n0 = t.n * BN, nleft = a.n - n0;
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + row * a.ldx;
  const uint16_t* w = static_cast<const uint16_t*>(a.w) + (uint64_t)t.g * a.gsw + (TRANS ? (uint64_t)n0 * a.ldw : n0);
  O* out = static_cast<O*>(a.out) + row * a.ldo + n0;
  general_tile<D, true, TRANS, FLAT, O, BM, BN>(x, a.ldx, mleft, w, a.ldw, nleft, a.k, out, a.ldo, mleft, nleft);
}

template <typename D, bool FLAT, typename O, int BM, int BN>
__global__ __launch_bounds__(256) void group_wgrad_general(GroupWgradArgs a) {
  const uint32_t mt = (a.k + BM - 1) / BM, nt = (a.n + BN - 1) / BN;
  const uint64_t all = (uint64_t)mt * nt * a.groups, per = all / kXcds, rem = all % kXcds;
  const uint32_t x = blockIdx.x % kXcds, idx = blockIdx.x / kXcds;
  if (idx >= per + (x < rem ? 1 : 0)) return;
  const uint64_t tile = x * per + min((uint64_t)x, rem) + idx;
  const int g = tile / ((uint64_t)mt * nt);
  const int m0 = (tile / nt % mt) * BM, n0 = (tile % nt) * BN;
  int begin, count;
  group_range(a.offsets, g, a.rows, &begin, &count);
  const uint16_t* px = static_cast<const uint16_t*>(a.x) + (uint64_t)begin * a.ldx + m0;
  const uint16_t* pd = static_cast<const uint16_t*>(a.dy) + (uint64_t)begin * a.ldy + n0;
  O* out = static_cast<O*>(a.out) + (uint64_t)g * a.gso + (uint64_t)m0 * a.ldo + n0;
  general_tile<D, false, false, FLAT, O, BM, BN>(px, a.ldx, a.k - m0, pd, a.ldy, a.n - n0, count, out, a.ldo, a.k - m0,
                                                 a.n - n0);
}

// Most row tiles of height bm that ascending offsets can make of `rows` rows.
uint64_t max_row_tiles(const GroupMmArgs& a, uint64_t bm) {
  const uint64_t one = (a.rows + bm - 1) / bm;
  if (a.groups == 1) return one;
  const uint64_t full = a.rows / bm, groups = (uint64_t)a.groups;
  return full + (groups < (uint64_t)a.rows ? groups : (uint64_t)a.rows);
}

template <typename D, bool TRANS, bool FLAT, typename O>
hipError_t run_mm(const GroupMmArgs& a, hipStream_t s) {
  constexpr int BM = 128, BN = 128;
  const uint64_t tiles = max_row_tiles(a, BM) * ((a.n + BN - 1) / BN);
  const uint64_t grid = (tiles + kXcds - 1) / kXcds * kXcds;
  if (grid * 256 >> 32) return hipErrorInvalidConfiguration;
  group_mm_general<D, TRANS, FLAT, O, BM, BN><<<dim3((uint32_t)grid), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

template <typename D, bool FLAT, typename O>
hipError_t run_wgrad(const GroupWgradArgs& a, hipStream_t s) {
  constexpr int BM = 128, BN = 128;
  const uint64_t tiles = (uint64_t)a.groups * ((a.k + BM - 1) / BM) * ((a.n + BN - 1) / BN);
  const uint64_t grid = (tiles + kXcds - 1) / kXcds * kXcds;
  if (grid * 256 >> 32) return hipErrorInvalidConfiguration;
  group_wgrad_general<D, FLAT, O, BM, BN><<<dim3((uint32_t)grid), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

template <typename D, bool TRANS, typename O>
hipError_t pick_mm(bool flat, const GroupMmArgs& a, hipStream_t s) {
  return flat ? run_mm<D, TRANS, true, O>(a, s) : run_mm<D, TRANS, false, O>(a, s);
}
template <typename D, typename O>
hipError_t pick_mm(bool transpose_w, bool flat, const GroupMmArgs& a, hipStream_t s) {
  return transpose_w ? pick_mm<D, true, O>(flat, a, s) : pick_mm<D, false, O>(flat, a, s);
}
template <typename D, typename O>
hipError_t pick_wgrad(bool flat, const GroupWgradArgs& a, hipStream_t s) {
  return flat ? run_wgrad<D, true, O>(a, s) : run_wgrad<D, false, O>(a, s);
}

}  // namespace

hipError_t launch_group_mm(int dtype, bool out_f32, bool transpose_w, bool flat, const GroupMmArgs& a, hipStream_t s) {
  (void)hipGetLastError();
  if (dtype == CIERA_BF16)
    return out_f32 ? pick_mm<Bf16, float>(transpose_w, flat, a, s) : pick_mm<Bf16, __bf16>(transpose_w, flat, a, s);
  return out_f32 ? pick_mm<Fp16, float>(transpose_w, flat, a, s) : pick_mm<Fp16, _Float16>(transpose_w, flat, a, s);
}

hipError_t launch_group_wgrad(int dtype, bool out_f32, bool flat, const GroupWgradArgs& a, hipStream_t s) {
  (void)hipGetLastError();
  if (dtype == CIERA_BF16)
    return out_f32 ? pick_wgrad<Bf16, float>(flat, a, s) : pick_wgrad<Bf16, __bf16>(flat, a, s);
  return out_f32 ? pick_wgrad<Fp16, float>(flat, a, s) : pick_wgrad<Fp16, _Float16>(flat, a, s);
}

}  // namespace ciera
