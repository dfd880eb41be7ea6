// Products with few rows to a group.
// What counts then is how fast the weights are read, once for every 16 rows of a group
// (64 tokens over 8 of 256 experts each, 7168 x 2048, [K, N]: 959 us, 6.0 TB/s).  A
// workgroup takes 16 rows of a group and some columns; its 8 waves take the contraction steps in turn, so
// that all of them read at once, from memory into registers.  A wave asks for the next step's values
// before it multiplies one, but each load stands behind a branch (is there a next step, is it a whole
// one), behind which the compiler waits for all loads: of every two steps the second is multiplied
// without a wait, the first when the values of both are there, and what hides latency is the other
// waves.  The waves' sums are joined through LDS in their order.
#pragma once
#include "ciera_tiles.h"

namespace ciera {
namespace {

constexpr int kThinWaves = 8;

// Each wave's sums of 16 rows and COLS columns of M products, and their join.
template <int COLS, int M>
struct ThinPart {
  static constexpr int kLd = COLS + 4;
  __attribute__((aligned(16))) float v[M][kThinWaves * 16 * kLd];

  // where the lane's row's results of a wave go
  __device__ __forceinline__ float* mine(int p) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    return v[p] + (wave * 16 + (lane & 15)) * kLd;
  }
  // put(row, column, the M sums of 4 columns) for rows and columns that are there
  template <typename F>
  __device__ __forceinline__ void join(int rows, int cols, F put) {
    __syncthreads();
    for (int p = threadIdx.x; p < 16 * COLS / 4; p += kThinWaves * 64) {
      const int m = p / (COLS / 4), c = p % (COLS / 4) * 4;
      if (m >= rows || c >= cols) continue;
      f32x4 sum[M];
#pragma unroll
      for (int i = 0; i < M; i++) {
        sum[i] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kThinWaves; w++) sum[i] += *reinterpret_cast<const f32x4*>(v[i] + (w * 16 + m) * kLd + c);
      }
      put(m, c, sum);
    }
  }
};

template <int M>
struct Sources {
  const uint16_t* w[M];  // first column of each product's weights
};
template <int M>
struct Strides {
  uint64_t ld[M];
};

// M products of the same rows with W [K, N]: a lane holds 8 contraction steps of VEC columns
// (two-byte values, 2 * VEC bytes of 8 rows) and turns them around in registers; 16 lanes
// cover 16 * VEC columns.
template <typename D, int VEC, int M>
struct ThinN {
  static constexpr int BN = 16 * VEC, W = VEC / 2;  // words of a row's columns in a lane
  f32x4 acc[M][VEC];
  struct Step {
    uint32_t w[M][8][W];
    i32x4 x;
  };
  __device__ __forceinline__ ThinN() {
#pragma unroll
    for (int p = 0; p < M; p++)
#pragma unroll
      for (int j = 0; j < VEC; j++) acc[p][j] = f32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void multiply(const Step& s) {
#pragma unroll
    for (int p = 0; p < M; p++)
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        i32x4 v;
#pragma unroll
        for (int i = 0; i < 4; i++)
          v[i] = __builtin_amdgcn_perm(s.w[p][2 * i + 1][j / 2], s.w[p][2 * i][j / 2], j & 1 ? 0x07060302u : 0x05040100u);
        acc[p][j] = mfma(__builtin_bit_cast(typename D::V, v), __builtin_bit_cast(typename D::V, s.x), acc[p][j]);
      }
  }
  // adds the products of `rows` rows from x on and the `left` columns from w on
  __device__ __forceinline__ void run(const uint16_t* x, uint64_t ldx, int rows, int left, int klen, Sources<M> src,
                                      Strides<M> ldw) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = (lane & 15) * VEC, q = lane >> 4;
    x += (uint64_t)min(lane & 15, rows - 1) * ldx;
    auto load = [&](Step& s, int k0) {
      const int k = k0 + q * 8;
      if (k0 + 32 <= klen && left >= BN) {
#pragma unroll
        for (int m = 0; m < M; m++)
#pragma unroll
          for (int j = 0; j < 8; j++) {
            const uint16_t* p = src.w[m] + c + (uint64_t)(k + j) * ldw.ld[m];
            if constexpr (VEC == 8) {
              const i32x4 v = load16(p);
#pragma unroll
              for (int i = 0; i < 4; i++) s.w[m][j][i] = v[i];
            } else {
              const Pack<uint32_t, W> v = *reinterpret_cast<const Pack<uint32_t, W>*>(p);
#pragma unroll
              for (int i = 0; i < W; i++) s.w[m][j][i] = v.v[i];
            }
          }
        s.x = load16(x + k);
      } else {
        // All at once: outside the matrix its last row or column again, then zeros (100 rows
        // over 13 groups, 2048 x 1000: 21.1 us, 40.8 with a branch to each value).
#pragma unroll
        for (int m = 0; m < M; m++)
#pragma unroll
          for (int j = 0; j < 8; j++) {
            const uint16_t* p = src.w[m] + (uint64_t)min(k + j, klen - 1) * ldw.ld[m];
#pragma unroll
            for (int i = 0; i < W; i++) {
              const uint32_t lo = p[min(c + 2 * i, left - 1)], hi = p[min(c + 2 * i + 1, left - 1)];
              s.w[m][j][i] =
                  (k + j < klen && c + 2 * i < left ? lo : 0) | (k + j < klen && c + 2 * i + 1 < left ? hi << 16 : 0);
            }
          }
        s.x = load_some(x + k, klen - k);
      }
    };
    constexpr int STEP = 32 * kThinWaves;
    int k0 = wave * 32;
    Step s[2];
    if (k0 < klen) load(s[0], k0);
    while (k0 < klen) {
      if (k0 + STEP < klen) load(s[1], k0 + STEP);
      multiply(s[0]);
      k0 += STEP;
      if (k0 >= klen) break;
      if (k0 + STEP < klen) load(s[0], k0 + STEP);
      multiply(s[1]);
      k0 += STEP;
    }
  }
  // results of a lane: row lane % 16, columns (lane / 16 * 4 + i) * VEC + j
  __device__ __forceinline__ void put(ThinPart<BN, M>& part) {
#pragma unroll
    for (int p = 0; p < M; p++) {
      float* mine = part.mine(p) + ((threadIdx.x & 63) >> 4) * 4 * VEC;
      if constexpr (VEC >= 4) {
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
          for (int j = 0; j < VEC; j += 4)
            *reinterpret_cast<f32x4*>(mine + i * VEC + j) =
                f32x4{acc[p][j][i], acc[p][j + 1][i], acc[p][j + 2][i], acc[p][j + 3][i]};
      } else {
#pragma unroll
        for (int i = 0; i < 4; i += 2)
          *reinterpret_cast<f32x4*>(mine + i * VEC) = f32x4{acc[p][0][i], acc[p][1][i], acc[p][0][i + 1], acc[p][1][i + 1]};
      }
    }
  }
};

// W [N, K]: a lane reads 64 bytes of one of 16 rows of W (4 loads, so that 4 lanes cover 256
// bytes of a row).
template <typename D, int M>
struct ThinT {
  static constexpr int BN = 16;
  f32x4 acc[M];
  struct Step {
    i32x4 w[M][4], x[4];
  };
  __device__ __forceinline__ ThinT() {
#pragma unroll
    for (int p = 0; p < M; p++) acc[p] = f32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void multiply(const Step& s) {
#pragma unroll
    for (int u = 0; u < 4; u++)
#pragma unroll
      for (int p = 0; p < M; p++)
        acc[p] = mfma(__builtin_bit_cast(typename D::V, s.w[p][u]), __builtin_bit_cast(typename D::V, s.x[u]), acc[p]);
  }
  __device__ __forceinline__ void run(const uint16_t* x, uint64_t ldx, int rows, int left, int klen, Sources<M> src,
                                      Strides<M> ldw) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane >> 4;
    const uint16_t* w[M];
#pragma unroll
    for (int p = 0; p < M; p++) w[p] = src.w[p] + (uint64_t)min(lane & 15, left - 1) * ldw.ld[p];
    x += (uint64_t)min(lane & 15, rows - 1) * ldx;
    auto load = [&](Step& s, int k0) {
      const int k = k0 + q * 32;
      if (k0 + 128 <= klen) {
#pragma unroll
        for (int u = 0; u < 4; u++) {
#pragma unroll
          for (int p = 0; p < M; p++) s.w[p][u] = load16(w[p] + k + u * 8);
          s.x[u] = load16(x + k + u * 8);
        }
      } else {
#pragma unroll
        for (int u = 0; u < 4; u++) {
#pragma unroll
          for (int p = 0; p < M; p++) s.w[p][u] = load_some(w[p] + k + u * 8, klen - k - u * 8);
          s.x[u] = load_some(x + k + u * 8, klen - k - u * 8);
        }
      }
    };
    constexpr int STEP = 128 * kThinWaves;
    int k0 = wave * 128;
    Step s[2];
    if (k0 < klen) load(s[0], k0);
    while (k0 < klen) {
      if (k0 + STEP < klen) load(s[1], k0 + STEP);
      multiply(s[0]);
      k0 += STEP;
      if (k0 >= klen) break;
      if (k0 + STEP < klen) load(s[0], k0 + STEP);
      multiply(s[1]);
      k0 += STEP;
    }
  }
  // results of a lane: row lane % 16, columns lane / 16 * 4 + i
  __device__ __forceinline__ void put(ThinPart<BN, M>& part) {
#pragma unroll
    for (int p = 0; p < M; p++) *reinterpret_cast<f32x4*>(part.mine(p) + ((threadIdx.x & 63) >> 4) * 4) = acc[p];
  }
};

// The thin form of weights [K, N] (VEC columns to a lane) or [N, K].
template <typename D, bool TRANS, int VEC, int M>
struct ThinOf {
  typedef ThinN<D, VEC, M> T;
};
template <typename D, int VEC, int M>
struct ThinOf<D, true, VEC, M> {
  typedef ThinT<D, M> T;
};

}  // namespace
}  // namespace ciera
