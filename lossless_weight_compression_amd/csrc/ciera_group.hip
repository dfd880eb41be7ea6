// Products grouped by expert: y = x W_g on the rows of every group, and the
// gradient of the weights, x_g^T dy_g.
#include "ciera.h"
#include "ciera_big.h"
#include "ciera_mid.h"
#include "ciera_ops_internal.h"
#include "ciera_tiles.h"

namespace ciera {
namespace {

template <typename D, bool TRANS, typename O, int BM, int TEAMS>
__global__ __launch_bounds__(256 * TEAMS, 2) void group_mm_mid(GroupMmArgs a) {
  GroupTile t;
  int tn;
  if (!find_group_tile<BM>(a.offsets, a.groups, a.rows, (a.n + 127) / 128, blockIdx.x, &t, &tn)) return;
  const uint64_t row = (uint64_t)t.begin + (uint64_t)t.m * BM;
  // the last tile ends with the matrix: it gives some columns a second time, the same values
  const int n0 = TRANS ? tn * 128 : max(min(tn * 128, a.n - 128), 0);
  mid_tile<D, true, TRANS, O, BM, TEAMS>(
      static_cast<const uint16_t*>(a.x) + row * a.ldx, a.ldx, t.count - t.m * BM,
      static_cast<const uint16_t*>(a.w) + (uint64_t)t.g * a.gsw + (TRANS ? (uint64_t)n0 * a.ldw : n0), a.ldw, a.n - n0, a.k,
      static_cast<O*>(a.out) + row * a.ldo + n0, a.ldo);
}

template <typename D, typename O, int BM, int TEAMS>
__global__ __launch_bounds__(256 * TEAMS, 2) void group_wgrad_mid(GroupWgradArgs a) {
  const uint32_t mt = (a.k + BM - 1) / BM, nt = (a.n + 127) / 128;
  uint64_t first;
  uint32_t many;
  die_run((uint64_t)mt * nt * a.groups, blockIdx.x % kXcds, &first, &many);
  if (blockIdx.x / kXcds >= many) return;
  const uint64_t tile = first + blockIdx.x / kXcds;
  const int g = tile / ((uint64_t)mt * nt);
  const int m0 = max(min((int)(tile / nt % mt) * BM, a.k - BM), 0), n0 = max(min((int)(tile % nt) * 128, a.n - 128), 0);
  int begin, count;
  group_range(a.offsets, g, a.rows, &begin, &count);
  begin = __builtin_amdgcn_readfirstlane(begin);
  count = __builtin_amdgcn_readfirstlane(count);
  mid_tile<D, false, false, O, BM, TEAMS>(static_cast<const uint16_t*>(a.x) + (uint64_t)begin * a.ldx + m0, a.ldx, a.k - m0,
                                   static_cast<const uint16_t*>(a.dy) + (uint64_t)begin * a.ldy + n0, a.ldy, a.n - n0, count,
                                   static_cast<O*>(a.out) + (uint64_t)g * a.gso + (uint64_t)m0 * a.ldo + n0, a.ldo);
}

template <typename D, bool TRANS, typename O>
__global__ __launch_bounds__(512) void group_mm_big(GroupMmArgs a) {
  __shared__ i32x4 lds[BigTiles<D, true, TRANS, O>::kLds];
  GroupTiles<256> tiles;
  tiles.init(a.offsets, a.groups, a.rows);
  const uint32_t nt = (a.n + 255) / 256;
  TileList list;
  list.init((uint64_t)tiles.total * nt);
  BigTiles<D, true, TRANS, O> big;
  big.init(lds);
  O* out;
  int om, on, half = 0;
  // false: no more tiles, or a half without rows
  auto start = [&](uint32_t i) {
    uint64_t tile;
    int r0, rows;
    if (!list.get(i, &tile, &r0, &rows)) return false;
    const GroupTile t = tiles.find((uint32_t)(tile / nt));
    const int n0 = (int)(tile % nt) * 256;
    const uint64_t row = (uint64_t)t.begin + (uint64_t)t.m * 256 + r0;
    om = min(t.count - t.m * 256 - r0, rows);
    on = a.n - n0;
    if (om <= 0) return false;
    out = static_cast<O*>(a.out) + row * a.ldo + n0;
    big.start(static_cast<const uint16_t*>(a.x) + row * a.ldx, a.ldx, om,
              static_cast<const uint16_t*>(a.w) + (uint64_t)t.g * a.gsw + (TRANS ? (uint64_t)n0 * a.ldw : n0), a.ldw, on,
              a.k, half);
    return true;
  };
  if (!start(0)) return;
  for (uint32_t i = 1;; i++) {
    big.stages(om, a.k, &half);
    O* done = out;
    const int dm = om, dn = on;
    const bool more = start(i);
    big.finish(done, a.ldo, dm, dn);
    if (!more) return;
  }
}

// The tiles of the groups' gradients, `per` to a group, shared out to the dies.  A tile
// takes as long as its group has rows.  Up to 64 groups: each is cut into equal units
// of consecutive tiles, 64 units at most, which are given out one by one, the most work
// first, to the die with the least so far; a lane keeps one unit.  (64 groups whose
// sizes spread by a factor of 10: the busiest die has 2 % more than its share, against
// 33 % if each took 8 groups in order.)  More groups: each die takes one run of tiles of
// equal work.
struct GradTiles {
  const int32_t* off;
  int groups, rows;
  uint32_t per, die;
  int begin, count;           // of the lane's group
  uint32_t unit, parts;       // tiles of a unit, units of a group
  uint32_t own, before;       // the lane's unit: its tiles, if on this die, and those of the die before it
  uint64_t first;             // more than 64 groups: the die's first tile
  uint64_t many;              // tiles of the die

  static __device__ __forceinline__ int cost(int c) { return (c + 63) / 64 + 4; }  // in stages; 4: start and stores
  __device__ __forceinline__ int chunk(int c) {
    const int g = c + (threadIdx.x & 63);
    begin = count = 0;
    if (g < groups) group_range(off, g, rows, &begin, &count);
    return wave_inclusive_sum(g < groups ? cost(count) : 0);
  }
  // more than 64 groups: the first tile that begins at work w or later
  __device__ __forceinline__ uint64_t tile_at(uint64_t w) {
    uint64_t sum = 0;
    for (int c = 0; c < groups; c += 64) {
      const int incl = chunk(c);
      const uint64_t hit = __ballot((sum + (uint32_t)incl) * per > w);
      if (hit && c + __builtin_ctzll(hit) < groups) {
        const int l = __builtin_ctzll(hit);
        const uint32_t one = cost(__builtin_amdgcn_readlane(count, l));
        const uint64_t pre = (sum + (uint32_t)__builtin_amdgcn_readlane(incl, l) - one) * per;
        return (uint64_t)(c + l) * per + (w - pre + one - 1) / one;
      }
      sum += (uint32_t)__builtin_amdgcn_readlane(incl, 63);
    }
    return (uint64_t)groups * per;
  }
  __device__ __forceinline__ void share_runs() {
    uint64_t total = 0;
    for (int c = 0; c < groups; c += 64) total += (uint32_t)__builtin_amdgcn_readlane(chunk(c), 63);
    const uint64_t part = total * per / kXcds;
    first = tile_at(part * die);
    many = (die + 1 == kXcds ? (uint64_t)groups * per : tile_at(part * (die + 1))) - first;
  }
  __device__ __forceinline__ void share_units() {
    const uint32_t lane = threadIdx.x & 63;
    parts = min(64u / (uint32_t)groups, per);
    unit = (per + parts - 1) / parts;
    const uint32_t g = lane / parts, part = lane % parts;
    const uint32_t tiles = g < (uint32_t)groups && part * unit < per ? min(unit, per - part * unit) : 0;
    begin = count = 0;
    if (tiles) group_range(off, g, rows, &begin, &count);
    const float work = tiles ? (float)cost(count) * (float)tiles : -1.f;
    int rank = 0;
    for (int l = 0; l < 64; l++) {
      const float w = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, work), l));
      rank += w > work || (w == work && l < (int)lane);
    }
    // the first 8 units go to the dies in order
    own = before = 0;
    uint32_t dealt = 0;
    const uint64_t mine = __ballot(rank == (int)die && tiles);
    if (mine) dealt = __builtin_amdgcn_readlane(tiles, __builtin_ctzll(mine));
    if (rank == (int)die) own = tiles;
    float load = __builtin_bit_cast(float, __builtin_amdgcn_ds_permute((rank & 63) * 4, __builtin_bit_cast(int, work)));
    if (lane >= kXcds) load = 3e38f;  // lane x < 8: work of die x
    for (int r = kXcds; r < 64; r++) {
      const int l = __builtin_ctzll(__ballot(rank == r));
      const float w = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, work), l));
      if (w < 0.f) break;
      float m = load;
      m = fminf(m, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, m), 0xb1, 0xf, 0xf, false)));   // lane ^ 1
      m = fminf(m, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, m), 0x4e, 0xf, 0xf, false)));   // lane ^ 2
      m = fminf(m, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, m), 0x141, 0xf, 0xf, false)));  // 7 - lane
      const uint32_t d = __builtin_ctzll(__ballot(load == m));
      if (lane == d) load += w;
      if (d == die) {
        if (lane == (uint32_t)l) {
          own = tiles;
          before = dealt;
        }
        dealt += __builtin_amdgcn_readlane(tiles, l);
      }
    }
    many = dealt;
  }
  __device__ __forceinline__ void share(const GroupWgradArgs& a, uint32_t tiles, uint32_t d) {
    off = a.offsets;
    groups = a.groups;
    rows = a.rows;
    per = tiles;
    die = d;
    if (groups <= 64) share_units();
    else share_runs();
  }
  // tile t < many of the die: its group, the tile in the group, the group's rows
  __device__ __forceinline__ void find(uint64_t t, int* g, uint32_t* in, int* b, int* n) {
    if (groups <= 64) {
      const int l = __builtin_ctzll(__ballot((uint32_t)t - before < own));
      *g = l / (int)parts;
      *in = l % parts * unit + (uint32_t)t - (uint32_t)__builtin_amdgcn_readlane(before, l);
      *b = __builtin_amdgcn_readlane(begin, l);
      *n = __builtin_amdgcn_readlane(count, l);
    } else {
      *g = (int)((first + t) / per);
      *in = (uint32_t)((first + t) % per);
      group_range(off, *g, rows, b, n);
      *b = __builtin_amdgcn_readfirstlane(*b);
      *n = __builtin_amdgcn_readfirstlane(*n);
    }
  }
};

template <typename D, typename O>
__global__ __launch_bounds__(512) void group_wgrad_big(GroupWgradArgs a) {
  __shared__ i32x4 lds[BigTiles<D, false, false, O>::kLds];
  const uint32_t nt = (a.n + 255) / 256, stride = gridDim.x / kXcds, me = blockIdx.x / kXcds;
  GradTiles tiles;
  tiles.share(a, (uint32_t)((a.k + 255) / 256) * nt, blockIdx.x % kXcds);
  // the die's tiles are dealt to its workgroups forth and back: the first have most work
  uint64_t round = 0, tile = me;
  if (tile >= tiles.many) return;
  BigTiles<D, false, false, O> big;
  big.init(lds);
  O* out;
  int om, on, count, half = 0;
  auto start = [&]() {
    int g, begin;
    uint32_t in;
    tiles.find(tile, &g, &in, &begin, &count);
    const int m0 = (int)(in / nt) * 256, n0 = (int)(in % nt) * 256;
    om = a.k - m0;
    on = a.n - n0;
    out = static_cast<O*>(a.out) + (uint64_t)g * a.gso + (uint64_t)m0 * a.ldo + n0;
    big.start(static_cast<const uint16_t*>(a.x) + (uint64_t)begin * a.ldx + m0, a.ldx, om,
              static_cast<const uint16_t*>(a.dy) + (uint64_t)begin * a.ldy + n0, a.ldy, on, count, half);
  };
  start();
  for (;;) {
    big.stages(om, count, &half);
    O* done = out;
    const int dm = om, dn = on;
    round++;
    tile = round * stride + (round & 1 ? stride - 1 - me : me);
    const bool more = tile < tiles.many;
    if (more) start();
    big.finish(done, a.ldo, dm, dn);
    if (!more) return;
  }
}

// ------------------------------------------------------- few rows to a group
// What counts then is how fast the weights are read, once for every 16 rows of a group
// (64 tokens over 8 of 256 experts each, 7168 x 2048, [K, N]: 959 us, 6.0 TB/s).  A
// workgroup takes 16 rows of a group and some columns; its 8 waves take the contraction steps in turn, so
// that all of them read at once, from memory into registers, the next step's values
// under way while this one's are multiplied; their sums are joined through LDS in the
// order of the waves.
constexpr int kThinWaves = 8;

// The joined sums: cols columns of 16 rows, of which `rows` are stored.  part: each
// wave's [16][kLd] floats.
template <typename O, int COLS>
struct ThinJoin {
  static constexpr int kLd = COLS + 4;
  static __device__ __forceinline__ void store(const float* part, O* out, uint64_t ldo, int rows, int cols) {
    for (int p = threadIdx.x; p < 16 * COLS / 4; p += kThinWaves * 64) {
      const int m = p / (COLS / 4), c = p % (COLS / 4) * 4;
      if (m >= rows || c >= cols) continue;
      f32x4 v = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kThinWaves; w++) v += *reinterpret_cast<const f32x4*>(part + (w * 16 + m) * kLd + c);
      store4(out + (uint64_t)m * ldo, c, cols, v);
    }
  }
};

// W [K, N]: a lane holds 8 contraction steps of VEC columns (two-byte values, 2 * VEC
// bytes of 8 rows) and turns them around in registers; 16 lanes cover 16 * VEC columns.
template <typename D, typename O, int VEC>
__global__ __launch_bounds__(512) void group_mm_thin(GroupMmArgs a) {
  constexpr int BN = 16 * VEC, W = VEC / 2;  // words of a row's columns in a lane
  typedef ThinJoin<O, BN> Join;
  __shared__ __attribute__((aligned(16))) float part[kThinWaves * 16 * Join::kLd];
  GroupTile t;
  int tn;
  if (!find_group_tile<16>(a.offsets, a.groups, a.rows, (a.n + BN - 1) / BN, blockIdx.x, &t, &tn)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = tn * BN, left = a.n - n0, rows = t.count - t.m * 16;
  const uint64_t row = (uint64_t)t.begin + (uint64_t)t.m * 16;
  const int c = (lane & 15) * VEC, q = lane >> 4;
  const uint16_t* w = static_cast<const uint16_t*>(a.w) + (uint64_t)t.g * a.gsw + n0 + c;
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + (row + min(lane & 15, rows - 1)) * a.ldx;

  struct Step {
    uint32_t w[8][W];
    i32x4 x;
  };
  auto load = [&](Step& s, int k0) {
    const int k = k0 + q * 8;
    if (k0 + 32 <= a.k && left >= BN) {
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const uint16_t* p = w + (uint64_t)(k + j) * a.ldw;
        if constexpr (VEC == 8) {
          const i32x4 v = load16(p);
#pragma unroll
          for (int i = 0; i < 4; i++) s.w[j][i] = v[i];
        } else {
          const Pack<uint32_t, 2> v = *reinterpret_cast<const Pack<uint32_t, 2>*>(p);
          s.w[j][0] = v.v[0];
          s.w[j][1] = v.v[1];
        }
      }
      s.x = load16(x + k);
    } else {
      // All at once: outside the matrix its last row or column again, then zeros (100 rows
      // over 13 groups, 2048 x 1000: 21.1 us, 40.8 with a branch to each value).
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const uint16_t* p = w + (uint64_t)min(k + j, a.k - 1) * a.ldw - c;
#pragma unroll
        for (int i = 0; i < W; i++) {
          const uint32_t lo = p[min(c + 2 * i, left - 1)], hi = p[min(c + 2 * i + 1, left - 1)];
          s.w[j][i] = (k + j < a.k && c + 2 * i < left ? lo : 0) | (k + j < a.k && c + 2 * i + 1 < left ? hi << 16 : 0);
        }
      }
      s.x = load_some(x + k, a.k - k);
    }
  };
  f32x4 acc[VEC];
#pragma unroll
  for (int j = 0; j < VEC; j++) acc[j] = f32x4{0, 0, 0, 0};
  auto multiply = [&](const Step& s) {
#pragma unroll
    for (int j = 0; j < VEC; j++) {
      i32x4 v;
#pragma unroll
      for (int i = 0; i < 4; i++)
        v[i] = __builtin_amdgcn_perm(s.w[2 * i + 1][j / 2], s.w[2 * i][j / 2], j & 1 ? 0x07060302u : 0x05040100u);
      acc[j] = mfma(__builtin_bit_cast(typename D::V, v), __builtin_bit_cast(typename D::V, s.x), acc[j]);
    }
  };
  constexpr int STEP = 32 * kThinWaves;
  int k0 = wave * 32;
  Step s[2];
  if (k0 < a.k) load(s[0], k0);
  while (k0 < a.k) {
    if (k0 + STEP < a.k) load(s[1], k0 + STEP);
    multiply(s[0]);
    k0 += STEP;
    if (k0 >= a.k) break;
    if (k0 + STEP < a.k) load(s[0], k0 + STEP);
    multiply(s[1]);
    k0 += STEP;
  }
  // results of a lane: row lane % 16, columns (lane / 16 * 4 + i) * VEC + j
  float* mine = part + (wave * 16 + (lane & 15)) * Join::kLd + (lane >> 4) * 4 * VEC;
#pragma unroll
  for (int i = 0; i < 4; i++)
#pragma unroll
    for (int j = 0; j < VEC; j += 4)
      *reinterpret_cast<f32x4*>(mine + i * VEC + j) = f32x4{acc[j][i], acc[j + 1][i], acc[j + 2][i], acc[j + 3][i]};
  __syncthreads();
  Join::store(part, static_cast<O*>(a.out) + row * a.ldo + n0, a.ldo, rows, left);
}

// W [N, K]: a lane reads 64 bytes of one of 16 rows of W (4 loads, so that 4 lanes cover 256
// bytes of a row).
template <typename D, typename O>
__global__ __launch_bounds__(512) void group_mm_thin_t(GroupMmArgs a) {
  constexpr int BN = 16;
  typedef ThinJoin<O, BN> Join;
  __shared__ __attribute__((aligned(16))) float part[kThinWaves * 16 * Join::kLd];
  GroupTile t;
  int tn;
  if (!find_group_tile<16>(a.offsets, a.groups, a.rows, (a.n + BN - 1) / BN, blockIdx.x, &t, &tn)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = tn * BN, left = a.n - n0, rows = t.count - t.m * 16;
  const uint64_t row = (uint64_t)t.begin + (uint64_t)t.m * 16;
  const int q = lane >> 4;
  const uint16_t* w =
      static_cast<const uint16_t*>(a.w) + (uint64_t)t.g * a.gsw + (uint64_t)(n0 + min(lane & 15, left - 1)) * a.ldw;
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + (row + min(lane & 15, rows - 1)) * a.ldx;
  struct Step {
    i32x4 w[4], x[4];
  };
  auto load = [&](Step& s, int k0) {
    const int k = k0 + q * 32;
    if (k0 + 128 <= a.k) {
#pragma unroll
      for (int u = 0; u < 4; u++) {
        s.w[u] = load16(w + k + u * 8);
        s.x[u] = load16(x + k + u * 8);
      }
    } else {
#pragma unroll
      for (int u = 0; u < 4; u++) {
        s.w[u] = load_some(w + k + u * 8, a.k - k - u * 8);
        s.x[u] = load_some(x + k + u * 8, a.k - k - u * 8);
      }
    }
  };
  f32x4 acc = {0, 0, 0, 0};
  auto multiply = [&](const Step& s) {
#pragma unroll
    for (int u = 0; u < 4; u++)
      acc = mfma(__builtin_bit_cast(typename D::V, s.w[u]), __builtin_bit_cast(typename D::V, s.x[u]), acc);
  };
  constexpr int STEP = 128 * kThinWaves;
  int k0 = wave * 128;
  Step s[2];
  if (k0 < a.k) load(s[0], k0);
  while (k0 < a.k) {
    if (k0 + STEP < a.k) load(s[1], k0 + STEP);
    multiply(s[0]);
    k0 += STEP;
    if (k0 >= a.k) break;
    if (k0 + STEP < a.k) load(s[0], k0 + STEP);
    multiply(s[1]);
    k0 += STEP;
  }
  // results of a lane: row lane % 16, columns lane / 16 * 4 + i
  float* mine = part + (wave * 16 + (lane & 15)) * Join::kLd + (lane >> 4) * 4;
  *reinterpret_cast<f32x4*>(mine) = acc;
  __syncthreads();
  Join::store(part, static_cast<O*>(a.out) + row * a.ldo + n0, a.ldo, rows, left);
}

// Narrow columns to a workgroup where wide ones would not make enough workgroups for the
// card.
template <typename D, bool TRANS, typename O>
hipError_t run_thin(const GroupMmArgs& a, hipStream_t s) {
  constexpr int WIDE = 128, NARROW = TRANS ? 16 : 64;
  const uint64_t mt = max_row_tiles(a.rows, a.groups, 16);
  const bool wide = !TRANS && mt * ((a.n + WIDE - 1) / WIDE) >= 4 * kUnits;
  const int bn = wide ? WIDE : NARROW;
  dim3 grid;
  if (hipError_t e = tile_grid(mt * ((a.n + bn - 1) / bn), 512, &grid)) return e;
  if constexpr (TRANS) {
    group_mm_thin_t<D, O><<<grid, dim3(512), 0, s>>>(a);
  } else {
    if (wide) group_mm_thin<D, O, 8><<<grid, dim3(512), 0, s>>>(a);
    else group_mm_thin<D, O, 4><<<grid, dim3(512), 0, s>>>(a);
  }
  return hipGetLastError();
}

template <typename D, bool TRANS, typename O, int BM, int TEAMS>
hipError_t run_mid(const GroupMmArgs& a, hipStream_t s) {
  dim3 grid;
  if (hipError_t e = tile_grid(max_row_tiles(a.rows, a.groups, BM) * ((a.n + 127) / 128), 256 * TEAMS, &grid)) return e;
  group_mm_mid<D, TRANS, O, BM, TEAMS><<<grid, dim3(256 * TEAMS), 0, s>>>(a);
  return hipGetLastError();
}

template <typename D, bool TRANS, typename O>
hipError_t run_mm(bool flat, const GroupMmArgs& a, hipStream_t s) {
  // By rows to a group on average; 64 experts of 2048 x 1024, bf16, us, the same operands
  // from call to call:
  //   rows             2    8   16   24   32   64  100  128  160  200  256
  //   [K, N] thin     29   44   50
  //          64 rows  32   44   55   55   55   56   70   83   89  107  115
  //          256 x 256                                 110  107  112  116
  //   [N, K] thin     32   53   66
  //          64 rows  29   41   52   50   51   53   71   83   89  106  113
  // The thin kernel takes [N, K], and more rows, only where tiles of 64 x 128 are too few
  // for the card (1 token over 8 of the experts 10.9 us for 15.3; one matrix 2048 x 7168,
  // 24 rows 15.6 for 36.7, 64 rows 27.9 for 39.6).  Two teams to a tile where there is one
  // tile to a unit at most (512 rows, 4096 x 1024: 27.4 us for 30.7).  The 256 x 256 kernel
  // takes what gives it half the card, the 128 x 128 one what is large but cannot be read
  // straight into LDS (13 groups, 40000 rows, 1447 x 777, fp16: 177 us for 213).  The host
  // knows the average only: 4096 rows over 256 experts of which one has 4033 read that one's
  // weights 253 times in the thin kernel, 172 us where the same call on [N, K] weights, in
  // tiles of 64 rows, takes 69.
  const int64_t rows = a.rows, groups = a.groups;
  const uint64_t nt = (a.n + 127) / 128;
  const uint64_t mid = max_row_tiles(rows, groups, 64) * nt;
  if ((rows <= 16 * groups && (!TRANS || mid < kUnits)) || (rows <= 64 * groups && mid < kUnits / 4))
    return run_thin<D, TRANS, O>(a, s);
  const uint64_t big = max_row_tiles(rows, groups, 256) * ((a.n + 255) / 256);
  if (flat && a.k && a.k % 8 == 0 && (TRANS || a.n % 8 == 0) && rows >= 256 * groups && big >= kUnits / 2 &&
      short_stride(a.ldx) && short_stride(a.ldw)) {
    group_mm_big<D, TRANS, O><<<dim3(kUnits), dim3(512), 0, s>>>(a);
    return hipGetLastError();
  }
  if (mid < kUnits && a.k >= 512) return run_mid<D, TRANS, O, 64, 2>(a, s);
  if (rows <= 96 * groups || max_row_tiles(rows, groups, 128) * nt < 2 * kUnits) return run_mid<D, TRANS, O, 64, 1>(a, s);
  return run_mid<D, TRANS, O, 128, 1>(a, s);
}

template <typename D, typename O>
hipError_t run_wgrad(bool flat, const GroupWgradArgs& a, hipStream_t s) {
  const uint64_t big = (uint64_t)a.groups * ((a.k + 255) / 256) * ((a.n + 255) / 256);
  if (flat && a.k % 8 == 0 && a.n % 8 == 0 && a.k >= 256 && a.n >= 256 && big >= kUnits / 2 && short_stride(a.ldx) &&
      short_stride(a.ldy)) {
    group_wgrad_big<D, O><<<dim3(kUnits), dim3(512), 0, s>>>(a);
    return hipGetLastError();
  }
  dim3 grid;
  const uint64_t wide = (uint64_t)a.groups * ((a.k + 127) / 128) * ((a.n + 127) / 128);
  if (wide < 2 * kUnits) {
    const uint64_t tiles = (uint64_t)a.groups * ((a.k + 63) / 64) * ((a.n + 127) / 128);
    const bool teams = tiles < kUnits && a.rows >= 256 * (int64_t)a.groups;
    if (hipError_t e = tile_grid(tiles, teams ? 512 : 256, &grid)) return e;
    if (teams) group_wgrad_mid<D, O, 64, 2><<<grid, dim3(512), 0, s>>>(a);
    else group_wgrad_mid<D, O, 64, 1><<<grid, dim3(256), 0, s>>>(a);
  } else {
    if (hipError_t e = tile_grid(wide, 256, &grid)) return e;
    group_wgrad_mid<D, O, 128, 1><<<grid, dim3(256), 0, s>>>(a);
  }
  return hipGetLastError();
}

template <typename D, typename O>
hipError_t pick_mm(bool transpose_w, bool flat, const GroupMmArgs& a, hipStream_t s) {
  return transpose_w ? run_mm<D, true, O>(flat, a, s) : run_mm<D, false, O>(flat, a, s);
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
    return out_f32 ? run_wgrad<Bf16, float>(flat, a, s) : run_wgrad<Bf16, __bf16>(flat, a, s);
  return out_f32 ? run_wgrad<Fp16, float>(flat, a, s) : run_wgrad<Fp16, _Float16>(flat, a, s);
}

}  // namespace ciera
