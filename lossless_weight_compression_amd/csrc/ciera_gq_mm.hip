// Products of two-byte activations with 4-bit integer weights that have group scales.
//
// y[m, n] = sum over blocks b of s[n, b] (sum_k x[m, k] q[n, k] - z[n, b] sum_k x[m, k]):
// codes are exact in two bytes, both sums over a block come from matrix instructions (the
// second one with ones for codes), and are scaled in fp32: no weight is rounded.  x is the
// instruction's first operand, so that a lane holds results of one column, whose scale and
// zero it needs, for 4 rows.
#include "ciera.h"
#include "ciera_act.h"
#include "ciera_big.h"
#include "ciera_gq.h"
#include "ciera_mid.h"
#include "ciera_ops_internal.h"
#include "ciera_tiles.h"

namespace ciera {
namespace {

// acc += s (sum - z xsum)
__device__ __forceinline__ void add_block(f32x4& acc, f32x4 sum, f32x4 xsum, float s, float z) {
#pragma unroll
  for (int e = 0; e < 4; e++) acc[e] = __builtin_fmaf(s, __builtin_fmaf(-z, xsum[e], sum[e]), acc[e]);
}

// Keeps the order of what comes before, up to v, and of what uses v afterwards: the sums of
// one block at a time take registers.
template <typename V>
__device__ __forceinline__ void in_order(V& v) {
  asm volatile("" : "+v"(v));
}

// N bytes at any address.
template <int N>
struct __attribute__((packed, aligned(1))) Raw {
  uint32_t v[N / 4];
};
template <>
struct __attribute__((packed, aligned(1))) Raw<2> {
  uint16_t v[1];
};

// The zeros of a stack, from memory where it has some: else the scales' bytes are read in
// their place (a branch would end the counting of loads under way), and 8 taken.
struct Zeros {
  const uint8_t* p;
  uint32_t kept;  // all ones: zeros come from memory
  __device__ __forceinline__ Zeros(const GqStack& w)
      : p(w.zeros ? w.zeros : reinterpret_cast<const uint8_t*>(w.scales)), kept(w.zeros ? ~0u : 0u) {}
  __device__ __forceinline__ float value(uint32_t word, int i) const {
    return (float)(((word & kept) | (0x08080808u & ~kept)) >> 8 * i & 255u);
  }
};

// N scales and zeros of a row.
template <int N>
struct Scales {
  Raw<2 * N> s;
  Raw<N> z;
  __device__ __forceinline__ void load(const GqStack& w, const Zeros& zeros, uint64_t at) {
    s = *reinterpret_cast<const Raw<2 * N>*>(w.scales + at);
    z = *reinterpret_cast<const Raw<N>*>(zeros.p + at);
  }
  // not taken apart before this
  __device__ __forceinline__ void wait() {
#pragma unroll
    for (auto& v : s.v) in_order(v);
#pragma unroll
    for (auto& v : z.v) in_order(v);
  }
  __device__ __forceinline__ float scale(int i, uint32_t half) const {
    return scale_of(s.v[i / 2] >> (i & 1 ? 16 : 0) & 0xffffu, half);
  }
  __device__ __forceinline__ float zero(const Zeros& zeros, int i) const { return zeros.value(z.v[i / 4], i & 3); }
};

// ------------------------------------------------------------------ few rows to a group
// What counts is how fast the codes are read, once for every 16 rows of a group.  A workgroup
// takes 16 rows and 16 columns (GLU: of each matrix); its waves take 256 contraction steps in
// turn, from memory into registers, the next ones' values under way while these are
// multiplied: of every column 2 x 16 bytes of codes to a lane, which hold 4 words of 32 steps
// each, and the scales of those steps in one load.  The waves' sums are joined through LDS in
// order.  (1 token over 8 experts of 2048 x 1024: 6 us, gated 8.7; 8 waves, one step each, 10 and
// 10.)
constexpr int kGqWaves = 4;

template <typename D, int BLOCK, bool GLU>
__global__ __launch_bounds__(64 * kGqWaves) void gq_mm_thin(GqMmArgs a) {
  constexpr int BN = 16, LD = BN + 4, M = GLU ? 2 : 1, S = 256 / BLOCK;
  __shared__ __attribute__((aligned(16))) float part[M][kGqWaves * 16 * LD];
  GroupTile t;
  int tn;
  if (!find_group_tile<16>(a.offsets, a.groups, a.rows, (a.n + BN - 1) / BN, blockIdx.x, &t, &tn)) return;
  typedef typename D::V V;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = tn * BN, left = a.n - n0, rows = t.count - t.m * 16, q = lane >> 4;
  const uint64_t row = (uint64_t)t.begin + (uint64_t)t.m * 16;
  const int blocks = (a.k + 127) / 128;  // of 128 steps
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + (row + min(lane & 15, rows - 1)) * a.ldx + q * 8;
  const Zeros zeros[2] = {a.w[0], a.w[M - 1]};
  const uint64_t wb = ((uint64_t)t.g * a.n + n0 + min(lane & 15, left - 1)) * blocks;  // the lane's row's first block
  struct Step {
    i32x4 w[M][2], x[8];
    Scales<S> s[M];
  };
  auto load = [&](Step& s, int b) {
#pragma unroll
    for (int f = 0; f < M; f++) {
      const i32x4* p = reinterpret_cast<const i32x4*>(a.w[f].codes) + (wb + b) * 4 + q;
      s.w[f][0] = p[0];
      s.w[f][1] = p[4];
      s.s[f].load(a.w[f], zeros[f], (wb + b) * (S / 2));
    }
#pragma unroll
    for (int u = 0; u < 8; u++) s.x[u] = load16(x + b * 128 + u * 32);
  };
  // the last one or two blocks, up to the end of x; zeros behind them
  auto load_last = [&](Step& s, int b) {
#pragma unroll
    for (int f = 0; f < M; f++) {
#pragma unroll
      for (auto& v : s.s[f].s.v) v = 0;
#pragma unroll
      for (auto& v : s.s[f].z.v) v = 0;
#pragma unroll
      for (int h = 0; h < 2; h++) {
        s.w[f][h] = i32x4{0, 0, 0, 0};
        if (b + h >= blocks) continue;
        const uint64_t at = wb + b + h;
        s.w[f][h] = (reinterpret_cast<const i32x4*>(a.w[f].codes) + at * 4)[q];
#pragma unroll
        for (int i = 0; i < S / 2; i++) {
          const int o = h * (S / 2) + i;
          s.s[f].s.v[o / 2] |= (uint32_t)a.w[f].scales[at * (S / 2) + i] << (o & 1 ? 16 : 0);
          s.s[f].z.v[o / 4] |= (uint32_t)zeros[f].p[at * (S / 2) + i] << 8 * (o & 3);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 8; u++) s.x[u] = load_some(x + b * 128 + u * 32, a.k - b * 128 - u * 32 - q * 8);
  };
  const V one = ones(D());
  f32x4 acc[M];
#pragma unroll
  for (int f = 0; f < M; f++) acc[f] = f32x4{0, 0, 0, 0};
  auto multiply = [&](Step& s) {
#pragma unroll
    for (int f = 0; f < M; f++) s.s[f].wait();
    f32x4 sum[M], xsum = {0, 0, 0, 0};
#pragma unroll
    for (int f = 0; f < M; f++) sum[f] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < 8; u++) {
      V xu = __builtin_bit_cast(V, s.x[u]);
      if (u * 32 % BLOCK == 0) in_order(xu);
#pragma unroll
      for (int f = 0; f < M; f++) sum[f] = mfma(xu, expand(s.w[f][u / 4][u % 4], D()), sum[f]);
      xsum = mfma(xu, one, xsum);
      if ((u + 1) * 32 % BLOCK == 0) {
        const int i = u * 32 / BLOCK;
#pragma unroll
        for (int f = 0; f < M; f++) {
          add_block(acc[f], sum[f], xsum, s.s[f].scale(i, a.half), s.s[f].zero(zeros[f], i));
          in_order(acc[f]);
          sum[f] = f32x4{0, 0, 0, 0};
        }
        xsum = f32x4{0, 0, 0, 0};
      }
    }
  };
  // this wave's whole steps of 256: no branch on the way, so that the loads of the next one stay
  // under way while one is multiplied
  const int whole = a.k / 256, many = whole > wave ? (whole - wave + kGqWaves - 1) / kGqWaves : 0;
  Step s[2];
  int i = 0;
  if (many) load(s[0], wave * 2);
  for (; i + 2 < many; i += 2) {
    load(s[1], (wave + (i + 1) * kGqWaves) * 2);
    multiply(s[0]);
    load(s[0], (wave + (i + 2) * kGqWaves) * 2);
    multiply(s[1]);
  }
  if (i + 1 < many) {
    load(s[1], (wave + (i + 1) * kGqWaves) * 2);
    multiply(s[0]);
    multiply(s[1]);
  } else if (i < many) {
    multiply(s[0]);
  }
  if (whole * 2 < blocks && whole % kGqWaves == wave) {
    load_last(s[0], whole * 2);
    multiply(s[0]);
  }
  // a lane: column lane % 16 of each 16, rows lane / 16 * 4 + e
#pragma unroll
  for (int f = 0; f < M; f++)
#pragma unroll
    for (int e = 0; e < 4; e++) part[f][(wave * 16 + q * 4 + e) * LD + (lane & 15)] = acc[f][e];
  __syncthreads();
  const int r = threadIdx.x >> 2, c = (threadIdx.x & 3) * 4;
  if (threadIdx.x >= 64 || r >= rows || c >= left) return;
  f32x4 v[M];
#pragma unroll
  for (int m = 0; m < M; m++) {
    v[m] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kGqWaves; i++) v[m] += *reinterpret_cast<const f32x4*>(part[m] + (i * 16 + r) * LD + c);
  }
  if (GLU) v[0] = gated(v[0], v[M - 1], a.act);
  const uint64_t at = (row + r) * a.ldo + n0;
  if (a.out_f32) store4(static_cast<float*>(a.out) + at, c, left, v[0]);
  else store4(static_cast<typename D::T*>(a.out) + at, c, left, v[0]);
}

// The same where there are enough columns for the card: every wave has all of the steps of
// 32 columns of its own (GLU: 16 of each matrix), and x, which the waves share, goes through LDS,
// 2048 steps at a time.  What bounds this is the lines that loads touch, 16 rows each, more than
// the bytes: so the scales are loaded 8 at a time (64 tokens over 8 of 256 experts, 7168 x 2048,
// both forms: 790 us, 5.5 TB/s; with x read by each wave and scales by each step 1220, of which x
// took 170 and the scales 210, the expansion of the codes nothing that could be seen).
constexpr int kSideWaves = 8;

template <typename D, int BLOCK, bool GLU>
__global__ __launch_bounds__(64 * kSideWaves) void gq_mm_side(GqMmArgs a) {
  constexpr int NF = GLU ? 1 : 2, BN = 16 * NF, M = GLU ? 2 : 1, F = M * NF;
  constexpr int GS = 8 * BLOCK / 256;  // steps of 256 to a group of scales
  constexpr int CHUNK = 2048, ROW = CHUNK / 8, LD = BN + 4;  // contraction steps in LDS; 16-byte pieces of a row
  __shared__ i32x4 xs[16 * ROW];
  static_assert(sizeof(xs) >= M * kSideWaves * 16 * LD * 4, "the results pass through x's memory");
  GroupTile t;
  int tn;
  if (!find_group_tile<16>(a.offsets, a.groups, a.rows, (a.n + kSideWaves * BN - 1) / (kSideWaves * BN), blockIdx.x, &t, &tn))
    return;
  typedef typename D::V V;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane >> 4;
  const int n0 = (tn * kSideWaves + wave) * BN, left = a.n - n0, rows = min(t.count - t.m * 16, 16);
  const uint64_t row = (uint64_t)t.begin + (uint64_t)t.m * 16;
  const int blocks = (a.k + 127) / 128, many = blocks * (128 / BLOCK);  // of 128 steps; scales of a row
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + row * a.ldx;
  const Zeros zeros[2] = {a.w[0], a.w[M - 1]};
  uint64_t wr[NF];  // the lane's rows; a wave without columns reads the last row
#pragma unroll
  for (int j = 0; j < NF; j++) wr[j] = (uint64_t)t.g * a.n + min(n0 + (lane & 15) + j * 16, a.n - 1);
  struct Codes {
    i32x4 w[F][2];
  };
  auto load = [&](Codes& c, int b) {
#pragma unroll
    for (int f = 0; f < F; f++) {
      const i32x4* p = reinterpret_cast<const i32x4*>(a.w[f / NF].codes) + (wr[f % NF] * blocks + b) * 4 + q;
      c.w[f][0] = p[0];
      c.w[f][1] = p[4];
    }
  };
  auto load_last = [&](Codes& c, int b) {
#pragma unroll
    for (int f = 0; f < F; f++)
#pragma unroll
      for (int h = 0; h < 2; h++) {
        c.w[f][h] = i32x4{0, 0, 0, 0};
        if (b + h < blocks)
          c.w[f][h] = (reinterpret_cast<const i32x4*>(a.w[f / NF].codes) + (wr[f % NF] * blocks + b + h) * 4)[q];
      }
  };
  // scales of 8 blocks, or of one step
  struct Group {
    Scales<8> s[F];
  };
  constexpr int S = 256 / BLOCK;
  struct Single {
    Scales<S> s[F];
  };
  auto load_scales = [&](auto& g, int at) {
#pragma unroll
    for (int f = 0; f < F; f++) g.s[f].load(a.w[f / NF], zeros[f / NF], wr[f % NF] * many + at);
  };
  auto load_scales_last = [&](Single& g, int at) {
#pragma unroll
    for (int f = 0; f < F; f++) {
#pragma unroll
      for (auto& v : g.s[f].s.v) v = 0;
#pragma unroll
      for (auto& v : g.s[f].z.v) v = 0;
#pragma unroll
      for (int i = 0; i < S; i++) {
        if (at + i >= many) continue;
        g.s[f].s.v[i / 2] |= (uint32_t)a.w[f / NF].scales[wr[f % NF] * many + at + i] << (i & 1 ? 16 : 0);
        g.s[f].z.v[i / 4] |= (uint32_t)zeros[f / NF].p[wr[f % NF] * many + at + i] << 8 * (i & 3);
      }
    }
  };
  // x from step k0 on, zeros behind its end; the pieces of a row are permuted by the row, so that
  // 16 rows lie in different banks
  auto stage = [&](int k0) {
    __syncthreads();
    for (int p = threadIdx.x; p < rows * ROW; p += 64 * kSideWaves) {
      const int r = p / ROW, c = p % ROW, k = k0 + c * 8;
      xs[r * ROW + (c ^ r)] = load_some(x + (uint64_t)r * a.ldx + k, a.k - k);
    }
    __syncthreads();
  };
  const int r = min(lane & 15, rows - 1);
  const V one = ones(D());
  f32x4 acc[F];
#pragma unroll
  for (int f = 0; f < F; f++) acc[f] = f32x4{0, 0, 0, 0};
  // step `st` of 256, the i-th of its group of scales
  auto multiply = [&](const Codes& c, const auto& g, int st, auto i) {
    const int piece = (st * 32 & (ROW - 1)) + q;
    f32x4 sum[F], xsum = {0, 0, 0, 0};
#pragma unroll
    for (int f = 0; f < F; f++) sum[f] = f32x4{0, 0, 0, 0};
    each<8>([&](auto u) {
      V xu = __builtin_bit_cast(V, xs[r * ROW + ((piece + u.v * 4) ^ r)]);
      if (u.v * 32 % BLOCK == 0) in_order(xu);
#pragma unroll
      for (int f = 0; f < F; f++) sum[f] = mfma(xu, expand(c.w[f][u.v / 4][u.v % 4], D()), sum[f]);
      xsum = mfma(xu, one, xsum);
      if constexpr ((u.v + 1) * 32 % BLOCK == 0) {
        constexpr int B = (i.v * 256 + u.v * 32) / BLOCK;
#pragma unroll
        for (int f = 0; f < F; f++) {
          add_block(acc[f], sum[f], xsum, g.s[f].scale(B, a.half), g.s[f].zero(zeros[f / NF], B));
          in_order(acc[f]);
          sum[f] = f32x4{0, 0, 0, 0};
        }
        xsum = f32x4{0, 0, 0, 0};
      }
    });
  };
  const int whole = a.k / (8 * BLOCK);  // groups of 8 scales
  int st = 0;
  Codes c[2];
  Group g[2];
  if (whole) {
    load(c[0], 0);
    load_scales(g[0], 0);
  }
  // The next group's scales and the next step's codes are under way while a step is
  // multiplied, without a branch on the way.
  auto group = [&](int i, auto last) {
    if (st * 256 % CHUNK == 0) stage(st * 256);
    if constexpr (!last.v) load_scales(g[1], (i + 1) * 8);
    each<GS>([&](auto s) {
      if constexpr (!last.v || s.v + 1 < GS) load(c[1], st * 2 + 2);
      multiply(c[0], g[0], st, s);
      c[0] = c[1];
      st++;
    });
    g[0] = g[1];
  };
  for (int i = 0; i + 1 < whole; i++) group(i, Int<0>());
  if (whole) group(whole - 1, Int<1>());
  // The whole steps that are left, less than a group, in the same way with their own scales, and
  // what is left then.
  const int steps = a.k / 256;
  if (st < steps) {
    Single one_step[2];
    load(c[0], st * 2);
    load_scales(one_step[0], st * S);
    for (; st + 1 < steps; st++) {
      if (st * 256 % CHUNK == 0) stage(st * 256);
      load(c[1], st * 2 + 2);
      load_scales(one_step[1], (st + 1) * S);
      multiply(c[0], one_step[0], st, Int<0>());
      c[0] = c[1];
      one_step[0] = one_step[1];
    }
    if (st * 256 % CHUNK == 0) stage(st * 256);
    multiply(c[0], one_step[0], st++, Int<0>());
  }
  if (st * 256 < a.k) {
    Single last;
    load_last(c[0], st * 2);
    load_scales_last(last, st * S);
    if (st * 256 % CHUNK == 0) stage(st * 256);
    multiply(c[0], last, st, Int<0>());
  }
  // a lane: column lane % 16 of each 16, rows lane / 16 * 4 + e
  __syncthreads();
  float* part = reinterpret_cast<float*>(xs) + wave * M * 16 * LD;
#pragma unroll
  for (int f = 0; f < F; f++)
#pragma unroll
    for (int e = 0; e < 4; e++) part[(f / NF * 16 + q * 4 + e) * LD + f % NF * 16 + (lane & 15)] = acc[f][e];
  wave_order();
  for (int p = lane; p < 4 * BN; p += 64) {
    const int m = p / (BN / 4), col = p % (BN / 4) * 4;
    if (m >= rows || col >= left) continue;
    f32x4 v = *reinterpret_cast<const f32x4*>(part + m * LD + col);
    if (GLU) v = gated(v, *reinterpret_cast<const f32x4*>(part + ((M - 1) * 16 + m) * LD + col), a.act);
    const uint64_t at = (row + m) * a.ldo + n0;
    if (a.out_f32) store4(static_cast<float*>(a.out) + at, col, left, v);
    else store4(static_cast<typename D::T*>(a.out) + at, col, left, v);
  }
}

// ------------------------------------------------------------------------ more rows
// BM x 128 tiles (GLU: 64 columns of each matrix), 4 waves of BM / 2 x 64.  x goes through
// LDS, 64 steps at a time, codes and scales of 128 steps too, and are expanded by the waves that
// multiply them.  (16384 rows over 64 experts of 2048 x 1024, both forms: codes read from
// memory by each of these waves 531 us, once to a workgroup 491, x and codes straight into LDS
// 437, codes read from there 16 bytes at a time 394.)  A block's sums are kept apart from the
// tile's: as many registers again.  Matrix instructions are under way 35 to 40 % of the time, as
// many vector instructions (expansion, scales) beside them.
template <typename D, int BLOCK, bool GLU, int BM>
struct GqTile {
  static constexpr int WM = BM / 32, WN = 4, COLUMNS = GLU ? 64 : 128, S = 128 / BLOCK, LD = 68;
  typedef StageTile<true, false, 16, BM> TA;
  typedef typename D::V V;
  static constexpr int kTurn = 4 * 16 * LD / 4;  // chunks that the results pass through
  int lane, wave, q, r0, c0;
  f32x4 acc[WM][WN], sum[WM][WN], xsum[WM];
  i32x4 w[WN];  // the block's codes

  __device__ __forceinline__ GqTile() {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    q = lane >> 4;
    r0 = (wave >> 1) * (BM / 2);
    c0 = (wave & 1) * (COLUMNS / 2);
#pragma unroll
    for (int i = 0; i < WM; i++)
#pragma unroll
      for (int j = 0; j < WN; j++) acc[i][j] = f32x4{0, 0, 0, 0};
  }
  // fragment j: 16 columns of the matrix j / 2 (GLU) or the only one, from this one of the tile's
  __device__ __forceinline__ int column(int j) const { return (GLU ? j / 2 * 64 + c0 + j % 2 * 16 : c0 + j * 16) + (lane & 15); }
  // Half H of a block of 128 steps: 64 steps of x, the block's codes [column][quarter] and its
  // scales, with the zeros in their upper halves.
  template <int H>
  __device__ __forceinline__ void multiply(const i32x4* x, const i32x4* codes, const uint32_t (*scales)[128], uint32_t half) {
    const uint32_t pa = TA::place(x, r0);
    if (H == 0) {
      // all 16 bytes at once: 8 for each half would use half of the banks
#pragma unroll
      for (int j = 0; j < WN; j++) w[j] = codes[column(j) * 4 + q];
    }
    each<2>([&](auto part) {
      constexpr int U = H * 2 + part.v;
      constexpr bool FIRST = U * 32 % BLOCK == 0;  // of a block: its sums begin with the instruction's constant 0
      constexpr f32x4 zero = {0, 0, 0, 0};
      V fx[WM];
      each<WM>([&](auto i) { fx[i.v] = __builtin_bit_cast(V, TA::template fragment<i.v, part.v>(pa)); });
      const V one = ones(D());
#pragma unroll
      for (int i = 0; i < WM; i++) xsum[i] = mfma(fx[i], one, FIRST ? zero : xsum[i]);
#pragma unroll
      for (int j = 0; j < WN; j++) {
        V fw = expand(w[j][U], D());
        in_order(fw);
#pragma unroll
        for (int i = 0; i < WM; i++) sum[i][j] = mfma(fx[i], fw, FIRST ? zero : sum[i][j]);
      }
      if constexpr ((U + 1) * 32 % BLOCK == 0) {
#pragma unroll
        for (int j = 0; j < WN; j++) {
          const uint32_t v = scales[U * 32 / BLOCK][column(j)];
          const float sc = scale_of(v & 0xffffu, half), ze = (float)(v >> 16);
#pragma unroll
          for (int i = 0; i < WM; i++) {
            add_block(acc[i][j], sum[i][j], xsum[i], sc, ze);
            in_order(acc[i][j]);
          }
        }
      }
    });
  }
  // A lane has column lane % 16 of each fragment, rows lane / 16 * 4 + e: turned around in LDS,
  // 16 rows at a time, to 16 (GLU: 8) consecutive columns of a row.
  __device__ __forceinline__ void store(const GqMmArgs& a, uint64_t row, int rows, int n0, i32x4* lds) {
    float* turn = reinterpret_cast<float*>(lds) + wave * 16 * LD;
    const int left = a.n - n0;
#pragma unroll
    for (int i = 0; i < WM; i++) {
      constexpr int N = GLU ? 2 : 4;
#pragma unroll
      for (int j = 0; j < N; j++) {
        const f32x4 v = GLU ? gated(acc[i][j], acc[i][(j + 2) % WN], a.act) : acc[i][j];
#pragma unroll
        for (int e = 0; e < 4; e++) turn[(q * 4 + e) * LD + j * 16 + (lane & 15)] = v[e];
      }
      wave_order();
      const int r = r0 + i * 16 + (lane >> 2), c = (lane & 3) * 4 * N;
#pragma unroll
      for (int h = 0; h < N / 2; h++) {
        const f32x4 lo = *reinterpret_cast<const f32x4*>(turn + (lane >> 2) * LD + c + h * 8);
        const f32x4 hi = *reinterpret_cast<const f32x4*>(turn + (lane >> 2) * LD + c + h * 8 + 4);
        const uint64_t at = (row + r) * a.ldo + n0 + c0 + c + h * 8;
        const int more = left - c0 - c - h * 8;
        if (r < rows) {
          if (a.out_f32) store_row8(static_cast<float*>(a.out) + at, more, lo, hi);
          else store_row8(static_cast<typename D::T*>(a.out) + at, more, lo, hi);
        }
      }
      wave_order();
    }
  }
};

// The scales and zeros of one column for N blocks from memory, packed as the tiles take them.
template <int N>
struct ColumnScales {
  Scales<N> s;
  __device__ __forceinline__ uint32_t packed(int i, uint32_t kept) const {
    const uint32_t z = ((uint32_t)s.z.v[i / 4] & kept) | (0x08080808u & ~kept);
    return (s.s.v[i / 2] >> (i & 1 ? 16 : 0) & 0xffffu) | (z >> 8 * (i & 3) & 255u) << 16;
  }
};

// Rows of x that start anywhere: x, codes and scales come through registers, the next ones
// under way while half a block is multiplied.  The sums of a block that is longer than 32 stay in
// registers from one part to the next, and with what is under way beside them there are not enough:
// 12 to 33 spill (blocks of 32: none), some of them in the loop; blocks of 64, which have most of
// these, take 1.4 to 1.5 times as long as those of 32.
template <typename D, int BLOCK, bool GLU, int BM>
__global__ __launch_bounds__(256, 2) void gq_mm_mid(GqMmArgs a) {
  typedef GqTile<D, BLOCK, GLU, BM> Tile;
  typedef typename Tile::TA TA;
  typedef StageLoad<true, BM> LA;
  constexpr int COLUMNS = Tile::COLUMNS, S = Tile::S;
  __shared__ i32x4 lds[2 * TA::kChunks > Tile::kTurn ? 2 * TA::kChunks : Tile::kTurn];  // or the results
  __shared__ i32x4 codes[2][128 * 4];      // [block][column][quarter]
  __shared__ uint32_t scales[2][S][128];
  GroupTile t;
  int tn;
  if (!find_group_tile<BM>(a.offsets, a.groups, a.rows, (a.n + COLUMNS - 1) / COLUMNS, blockIdx.x, &t, &tn)) return;
  const int tid = threadIdx.x, n0 = tn * COLUMNS, left = a.n - n0, rows = t.count - t.m * BM;
  const int blocks = (a.k + 127) / 128;
  const uint64_t row = (uint64_t)t.begin + (uint64_t)t.m * BM;
  LA ga;
  ga.init(static_cast<const uint16_t*>(a.x) + row * a.ldx, a.ldx, rows);
  // What a thread loads of a block: a quarter of two columns' codes, 64 columns apart, and the
  // scales of one column.  Blocks are counted from that of column n0.
  const uint64_t first = ((uint64_t)t.g * a.n + n0) * blocks;
  const uint32_t c1 = (uint32_t)min(tid >> 2, left - 1) * blocks;
  const uint32_t c2 = (uint32_t)min((tid >> 2) + (GLU ? 0 : 64), left - 1) * blocks;
  const uint32_t cs = (uint32_t)min(tid & (COLUMNS - 1), left - 1) * blocks;
  const GqStack &wa = a.w[0], &wb = a.w[GLU ? 1 : 0];
  const Zeros za(wa), zb(wb);
  const bool up = GLU && (tid & 64);
  const char* ps = reinterpret_cast<const char*>((up ? wb : wa).scales + first * S);
  const uint8_t* pz = (up ? zb : za).p + first * S;
  struct Next {
    i32x4 w[2];
    Raw<2 * S> s;
    uint32_t z;
  };
  auto load_codes = [&](Next& n, int b) {
    n.w[0] = *reinterpret_cast<const i32x4*>(wa.codes + first * 64 + ((c1 + b) * 64 + (tid & 3) * 16));
    n.w[1] = *reinterpret_cast<const i32x4*>(wb.codes + first * 64 + ((c2 + b) * 64 + (tid & 3) * 16));
    n.s = *reinterpret_cast<const Raw<2 * S>*>(ps + (cs + b) * (2 * S));
    if constexpr (S == 4) n.z = reinterpret_cast<const Raw<4>*>(pz + (cs + b) * S)->v[0];
    else if constexpr (S == 2) n.z = reinterpret_cast<const Raw<2>*>(pz + (cs + b) * S)->v[0];
    else n.z = pz[cs + b];
  };
  auto put_codes = [&](const Next& n, int h) {
    codes[h][tid] = n.w[0];
    codes[h][256 + tid] = n.w[1];
    if (tid < 128) {
      const uint32_t z = (n.z & za.kept) | (0x08080808u & ~za.kept);
#pragma unroll
      for (int i = 0; i < S; i++)
        scales[h][i][tid] = ((uint32_t)n.s.v[i / 2] >> (i & 1 ? 16 : 0) & 0xffffu) | (z >> 8 * i & 255u) << 16;
    }
  };
  i32x4 xr[LA::N];
  auto load_x = [&](int stage) {
    if (stage * 64 + 64 <= a.k) ga.load(xr, stage * 64);
    else ga.load(xr, stage * 64, a.k);
  };
  auto put = [&](int h) {
#pragma unroll
    for (int i = 0; i < LA::N; i++) lds[h * TA::kChunks + TA::pos(ga.line + i * (256 / TA::kPerRow), ga.col / 8)] = xr[i];
  };
  Tile tile;
  Next next;
  if (blocks > 0) {
    load_x(0);
    load_codes(next, 0);
    put(0);
    put_codes(next, 0);
  }
  __syncthreads();
  // A block's codes and the first half of its x are here.  Blocks that another whole one
  // follows are taken without a branch, so that loads stay under way.
  int b = 0;
  for (; b + 1 < a.k / 128; b++) {
    ga.load(xr, b * 128 + 64);
    load_codes(next, b + 1);
    __builtin_amdgcn_sched_barrier(0);
    tile.template multiply<0>(lds, codes[b & 1], scales[b & 1], a.half);
    put(1);
    __syncthreads();
    ga.load(xr, b * 128 + 128);
    __builtin_amdgcn_sched_barrier(0);
    tile.template multiply<1>(lds + TA::kChunks, codes[b & 1], scales[b & 1], a.half);
    put(0);
    put_codes(next, (b + 1) & 1);
    __syncthreads();
  }
  for (; b < blocks; b++) {
    load_x(2 * b + 1);
    tile.template multiply<0>(lds, codes[b & 1], scales[b & 1], a.half);
    put(1);
    __syncthreads();
    if (b + 1 < blocks) {
      load_x(2 * b + 2);
      load_codes(next, b + 1);
    }
    tile.template multiply<1>(lds + TA::kChunks, codes[b & 1], scales[b & 1], a.half);
    if (b + 1 < blocks) {
      put(0);
      put_codes(next, (b + 1) & 1);
    }
    __syncthreads();
  }
  tile.store(a, row, rows, n0, lds);
}

// Rows of x that start at multiples of 16 bytes and hold multiples of 8 values: x and codes go
// straight into LDS, two stages of 64 steps ahead (three of x, two blocks of codes in LDS), with
// counted waits; scales 8 or 16 blocks at a time.
template <typename D, int BLOCK, bool GLU, int BM>
__global__ __launch_bounds__(256, 2) void gq_mm_flat(GqMmArgs a) {
  typedef GqTile<D, BLOCK, GLU, BM> Tile;
  typedef typename Tile::TA TA;
  constexpr int COLUMNS = Tile::COLUMNS, S = Tile::S, PARTS = TA::kChunks / 256;
  constexpr int SN = S == 1 ? 8 : 16, CB = SN / S;  // scales at a time; blocks of 128 that they are for
  __shared__ i32x4 lds[3 * TA::kChunks > Tile::kTurn ? 3 * TA::kChunks : Tile::kTurn];  // or the results
  __shared__ i32x4 codes[2][128 * 4];  // [block][column][quarter]
  __shared__ uint32_t scales[2][SN][128];
  GroupTile t;
  int tn;
  if (!find_group_tile<BM>(a.offsets, a.groups, a.rows, (a.n + COLUMNS - 1) / COLUMNS, blockIdx.x, &t, &tn)) return;
  const int tid = threadIdx.x, n0 = tn * COLUMNS, left = a.n - n0, rows = t.count - t.m * BM;
  const int blocks = (a.k + 127) / 128;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), many = blocks * S;
  const uint64_t row = (uint64_t)t.begin + (uint64_t)t.m * BM;
  const uint64_t first = ((uint64_t)t.g * a.n + n0) * blocks;
  const GqStack &wa = a.w[0], &wb = a.w[GLU ? 1 : 0];
  const Zeros za(wa), zb(wb);
  // this lane's chunks: of x, bytes from the stage's first value, and of codes, from the block
  const char* const px = scalar(reinterpret_cast<const char*>(static_cast<const uint16_t*>(a.x) + row * a.ldx));
  const char* const pa = scalar(reinterpret_cast<const char*>(wa.codes + first * 64));
  const char* const pb = scalar(reinterpret_cast<const char*>(wb.codes + first * 64));
  uint32_t ox[PARTS];
#pragma unroll
  for (int i = 0; i < PARTS; i++) {
    const int p = i * 256 + tid, line = p / TA::kPerRow;
    ox[i] = 2 * ((uint32_t)min(line, rows - 1) * (uint32_t)a.ldx + TA::swizzle(line, p % TA::kPerRow) * 8);
  }
  const uint32_t oa = (uint32_t)min(tid >> 2, left - 1) * blocks * 64 + (tid & 3) * 16;
  const uint32_t ob = (uint32_t)min((tid >> 2) + (GLU ? 0 : 64), left - 1) * blocks * 64 + (tid & 3) * 16;
  // stage s of x into its third of LDS; behind the end zeros
  auto load_x = [&](int s, int buf) {
    i32x4* at = lds + buf * TA::kChunks + wave * 64;
    const char* from = scalar(px + (uint64_t)s * 128);
    if (s * 64 + 64 <= a.k) {
#pragma unroll
      for (int i = 0; i < PARTS; i++) load_lds16(from, ox[i], at + i * 256);
    } else {
#pragma unroll
      for (int i = 0; i < PARTS; i++) {
        const int p = i * 256 + tid, k = s * 64 + TA::swizzle(p / TA::kPerRow, p % TA::kPerRow) * 8;
        load_lds16(k < a.k ? from + ox[i] : reinterpret_cast<const char*>(&kZeros), at + i * 256);
      }
    }
  };
  auto load_codes = [&](int b) {
    load_lds16(scalar(pa + (uint64_t)b * 64), oa, codes[b & 1] + wave * 64);
    load_lds16(scalar(pb + (uint64_t)b * 64), ob, codes[b & 1] + 256 + wave * 64);
  };
  // the scales of CB blocks from b on
  const bool up = GLU && (tid & 64);
  const uint64_t cs = first * S + (uint64_t)min(tid & (COLUMNS - 1), left - 1) * many;
  auto fetch_scales = [&](int b) {
    if (tid >= 128) return;
    ColumnScales<SN> c;
    const GqStack& w = up ? wb : wa;
    const Zeros& z = up ? zb : za;
    if (b * S + SN <= many) {
      c.s.load(w, z, cs + b * S);
    } else {
#pragma unroll
      for (auto& v : c.s.s.v) v = 0;
#pragma unroll
      for (auto& v : c.s.z.v) v = 0;
#pragma unroll
      for (int i = 0; i < SN; i++) {
        if (b * S + i >= many) continue;
        c.s.s.v[i / 2] |= (uint32_t)w.scales[cs + b * S + i] << (i & 1 ? 16 : 0);
        c.s.z.v[i / 4] |= (uint32_t)z.p[cs + b * S + i] << 8 * (i & 3);
      }
    }
#pragma unroll
    for (int i = 0; i < SN; i++) scales[b / CB & 1][i][tid] = c.packed(i, za.kept);
  };
  // all but the last N of the wave's loads are there, and its LDS accesses done; then every wave's
  auto arrive = [&](auto n) {
    __builtin_amdgcn_s_waitcnt((n.v & 15) | (n.v >> 4 << 14) | 0x0070);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  Tile tile;
  if (blocks > 0) {
    load_codes(0);
    load_x(0, 0);
    load_x(1, 1);
    fetch_scales(0);
  }
  arrive(Int<0>());
  int buf = 0;  // of x, of the stage that is multiplied
  for (int b = 0; b < blocks; b++) {
    const bool more = b + 1 < blocks;
    const uint32_t(*sc)[128] = scales[b / CB & 1] + b % CB * S;
    if (more) {
      load_codes(b + 1);
      load_x(2 * b + 2, buf == 0 ? 2 : buf - 1);
    }
    tile.template multiply<0>(lds + buf * TA::kChunks, codes[b & 1], sc, a.half);
    if (more) arrive(Int<2 + PARTS>());
    else arrive(Int<0>());
    buf = buf == 2 ? 0 : buf + 1;
    if (more) load_x(2 * b + 3, buf == 0 ? 2 : buf - 1);
    tile.template multiply<1>(lds + buf * TA::kChunks, codes[b & 1], sc, a.half);
    if (more && (b + 1) % CB == 0) fetch_scales(b + 1);
    arrive(Int<PARTS>());
    buf = buf == 2 ? 0 : buf + 1;
  }
  tile.store(a, row, rows, n0, lds);
}

template <typename D, int BLOCK, bool GLU>
hipError_t run_thin(uint64_t row_tiles, const GqMmArgs& a, hipStream_t s) {
  dim3 grid;
  if (hipError_t e = tile_grid(row_tiles * ((a.n + 15) / 16), 64 * kGqWaves, &grid)) return e;
  gq_mm_thin<D, BLOCK, GLU><<<grid, dim3(64 * kGqWaves), 0, s>>>(a);
  return hipGetLastError();
}
constexpr int side_columns(bool glu) { return (glu ? 16 : 32) * kSideWaves; }
template <typename D, int BLOCK, bool GLU>
hipError_t run_side(uint64_t row_tiles, const GqMmArgs& a, hipStream_t s) {
  constexpr int WIDE = side_columns(GLU);
  dim3 grid;
  if (hipError_t e = tile_grid(row_tiles * ((a.n + WIDE - 1) / WIDE), 64 * kSideWaves, &grid)) return e;
  gq_mm_side<D, BLOCK, GLU><<<grid, dim3(64 * kSideWaves), 0, s>>>(a);
  return hipGetLastError();
}
template <typename D, int BLOCK, bool GLU, int BM>
hipError_t run_mid(bool straight, const GqMmArgs& a, hipStream_t s) {
  constexpr int COLUMNS = GLU ? 64 : 128;
  dim3 grid;
  if (hipError_t e = tile_grid(max_row_tiles(a.rows, a.groups, BM) * ((a.n + COLUMNS - 1) / COLUMNS), 256, &grid)) return e;
  if (straight) gq_mm_flat<D, BLOCK, GLU, BM><<<grid, dim3(256), 0, s>>>(a);
  else gq_mm_mid<D, BLOCK, GLU, BM><<<grid, dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

template <typename D, int BLOCK, bool GLU>
hipError_t run_gq_mm(bool flat, const GqMmArgs& a, hipStream_t s) {
  // By rows to a group on average; 64 experts of 2048 x 1024, as many rows to each, blocks of 128,
  // bf16, us, one product and (GLU) both; tiles with x straight into LDS (where groups end anywhere
  // 64 rows take side workgroups 53 and 95, tiles 42 and 83, 48 rows 42 and 76, 42 and 81).
  //   rows                2        8       16       32       64      100      128      256
  //   thin           32  58   43  68   49  72   90 132  171 254
  //   side           15  26   17  28   17  27   26  46   45  85   74 137   85 158  162 304
  //   tiles                                                       47  88   50  89   93 169
  // The thin kernel is for calls with few columns to the card (1 token over 8 of the experts 6.0 and
  // 8.3 for 12 and 12; one matrix 4096 x 1024, 64 rows, 8.8 and 11 for 24 and 22; 200 rows 24 and 32
  // for 24 and 24), tiles only for what fills the card with them (900 rows 77 and 83 for 25 and 39).
  // With x through registers tiles win later, with blocks of 64 hardly at all: those of 64 and 128
  // spill.  The same experts, rows of x 2 bytes off, groups that end anywhere, side and tiles:
  //   rows                  64          96         160         256         512        1024
  //   block  32, one   79   77    109   79    167  146    255  181    494  326    960  602
  //              both 148  145    200  147    320  276    497  339    966  623   1913 1165
  //   block 128, one   57   65     75   65    114  120    174  168    340  283    662  510
  //              both 100  134    135  133    216  252    333  312    658  561   1298 1021
  //   block  64, one   62  107     84  112    130  197    198  271    383  465    756  846
  //              both 113  214    151  223    246  409    380  530    759  968   1485 1784
  // (24 experts 1447 x 1515, blocks of 128 at 192 rows 75 and 76, both 137 and 126; of 64 at 384
  // rows 158 and 136, 306 and 289; one matrix 2047 x 2048, blocks of 64, 8192 rows, 240 and 171.)
  const int64_t rows = a.rows, groups = a.groups;
  const uint64_t thin = max_row_tiles(rows, groups, 16), wide = side_columns(GLU);
  const uint64_t mid = max_row_tiles(rows, groups, 128) * ((a.n + (GLU ? 63 : 127)) / (GLU ? 64 : 128));
  // (the tiles count blocks of 128 rows in 32 bits)
  const bool straight = flat && a.k % 8 == 0 && short_stride(a.ldx);
  constexpr int kThroughRegisters = BLOCK == 32 ? 80 : BLOCK == 64 ? 1024 : 192;
  if (rows > (straight ? 80 : kThroughRegisters) * groups && mid >= 2 * kUnits && a.k <= 1 << 25)
    return run_mid<D, BLOCK, GLU, 128>(straight, a, s);
  if (thin * ((a.n + wide - 1) / wide) >= 3 * kUnits / 8) return run_side<D, BLOCK, GLU>(thin, a, s);
  return run_thin<D, BLOCK, GLU>(thin, a, s);
}
template <typename D, bool GLU>
hipError_t by_block(int block, bool flat, const GqMmArgs& a, hipStream_t s) {
  if (block == 32) return run_gq_mm<D, 32, GLU>(flat, a, s);
  if (block == 64) return run_gq_mm<D, 64, GLU>(flat, a, s);
  return run_gq_mm<D, 128, GLU>(flat, a, s);
}
template <typename D>
hipError_t by_form(bool glu, int block, bool flat, const GqMmArgs& a, hipStream_t s) {
  return glu ? by_block<D, true>(block, flat, a, s) : by_block<D, false>(block, flat, a, s);
}

}  // namespace

hipError_t launch_gq_mm(int dtype, bool glu, int block, bool flat, const GqMmArgs& a, hipStream_t s) {
  (void)hipGetLastError();
  return dtype == CIERA_BF16 ? by_form<Bf16>(glu, block, flat, a, s) : by_form<Fp16>(glu, block, flat, a, s);
}

}  // namespace ciera
