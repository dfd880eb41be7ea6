// The products that the large-tile engine does not take: rows that start at any
// element and end anywhere, and matrices or groups too small to fill its tiles.
#pragma once
#include "ciera_tiles.h"

namespace ciera {
namespace {

// What one thread loads of one operand's stage: chunks of 8 values (or 32 codes), into
// registers.  `lines` rows (KC) or columns of the operand are left; rows past the last
// repeat it.
template <bool KC, int R>
struct StageLoad {
  typedef StageTile<KC, false, 16, R> Any;  // chunk counts do not depend on the order in a tile
  static constexpr int N = Any::kChunks / 256;
  const uint16_t* p[N];
  uint64_t ld;
  int line, col, left;  // of the first chunk; columns left from there (not KC)

  // PAIR: the first half of the rows (KC) or columns from `base`, the other one from `base2`.
  template <bool PAIR = false>
  __device__ __forceinline__ void init(const uint16_t* base, uint64_t l, int lines, const uint16_t* base2 = nullptr,
                                       uint64_t l2 = 0) {
    const int tid = threadIdx.x & 255;
    if constexpr (PAIR) {
      constexpr int H = R / 2;
      line = tid / Any::kPerRow;
      col = tid % Any::kPerRow * 8;
      const bool second = !KC && col >= H;
      ld = second ? l2 : l;
      left = lines - (col & (H - 1));
#pragma unroll
      for (int i = 0; i < N; i++) {
        const int k = line + i * (256 / Any::kPerRow);
        if (KC) p[i] = (i < N / 2 ? base + (uint64_t)min(k, lines - 1) * l : base2 + (uint64_t)min(k - H, lines - 1) * l2) + col;
        else p[i] = (second ? base2 - H : base) + (uint64_t)k * ld + col;
      }
      return;
    }
    ld = l;
    line = tid / Any::kPerRow;
    col = tid % Any::kPerRow * 8;
    left = lines - col;
#pragma unroll
    for (int i = 0; i < N; i++) {
      const int k = line + i * (256 / Any::kPerRow);
      p[i] = base + (uint64_t)(KC ? min(k, lines - 1) : k) * l + col;
    }
  }
  // the stage at contraction step k0, all of it
  __device__ __forceinline__ void load(i32x4* to, int k0) const {
#pragma unroll
    for (int i = 0; i < N; i++) to[i] = load16(p[i] + (KC ? (uint64_t)k0 : (uint64_t)k0 * ld));
  }
  // up to step klen, zeros behind; columns past the last as zeros
  __device__ __forceinline__ void load(i32x4* to, int k0, int klen) const {
#pragma unroll
    for (int i = 0; i < N; i++) {
      to[i] = i32x4{0, 0, 0, 0};
      if (KC) to[i] = load_some(p[i] + k0, klen - k0 - col);
      else if (k0 + line + i * (256 / Any::kPerRow) < klen) to[i] = load_some(p[i] + (uint64_t)k0 * ld, left);
    }
  }
};

// What becomes of a tile's results: put(row, column, columns left from there, values of 8
// columns), for rows of the tile only.
template <typename O>
struct MidStore {
  O* out;
  uint64_t ldo;
  __device__ __forceinline__ void put(int r, int c, int left, f32x4 lo, f32x4 hi) const {
    store_row8(out + (uint64_t)r * ldo + c, left, lo, hi);
  }
};

// PLAIN: C = A B.  PAIR: A B and A B2, 64 columns of each in the place of the tile's 128;
// put() gets both products' values.  SUM: A B + A2 B2, one product to each of two teams.
enum class Mid { PLAIN, PAIR, SUM };

// One BM x 128 tile of C = A B, 4 waves of BM / 2 x 64.  Stages of 64 contraction steps
// (256 codes) go from memory into registers, DEPTH of them under way (4 are no faster than
// 2), from there into one half of LDS while the other is multiplied.  A has `am` rows left, B `bn` columns.  The
// loop over whole stages has no branches, so that the compiler can wait for the older
// stage alone: operands whose contiguous side is not the contraction have to fill the
// tile for that (the callers move the last tile back to end with the matrix).
// Scaled operands: sa, sb, `srow` bytes of scales a row.
//
// TEAMS 2: two teams of 4 waves, each with half of the stages; the second one's sums are
// added to the first's through LDS.  For two-byte tiles that are too few to fill the card
// otherwise.
template <typename D, bool AKC, bool BKC, int BM, int TEAMS, Mid KIND = Mid::PLAIN, typename Out>
__device__ __forceinline__ void mid_tile(const uint16_t* a, uint64_t lda, int am, const uint16_t* b, uint64_t ldb, int bn,
                                         int klen, Out out, const uint8_t* sa = nullptr, const uint8_t* sb = nullptr,
                                         uint32_t srow = 0, const uint16_t* b2 = nullptr, uint64_t ldb2 = 0,
                                         const uint16_t* a2 = nullptr, uint64_t lda2 = 0) {
  constexpr bool PAIR = KIND == Mid::PAIR, SUM = KIND == Mid::SUM;
  constexpr int BN = 128, BK = 64, WM = BM / 32, WN = 4, ROWS = BM + BN, DEPTH = 2, COLUMNS = PAIR ? BN / 2 : BN;
  typedef StageTile<AKC, false, 16, BM> TA;
  typedef StageTile<BKC, true, 16, BN> TB;
  typedef StageLoad<AKC, BM> LA;
  typedef StageLoad<BKC, BN> LB;
  typedef typename D::V V;
  static_assert((TEAMS == 1 && KIND == Mid::PLAIN) || !D::kScaled, "one team and one product for scaled operands");
  static_assert(TEAMS == 2 || !SUM, "a team to each product");
  constexpr int HALF = TA::kChunks + TB::kChunks;
  static_assert(2 * HALF >= BM * BN / 4, "the joined sums take the place of a team's stages");
  __shared__ i32x4 lds[TEAMS * 2 * HALF];
  __shared__ uint32_t scales[TEAMS * 2][D::kScaled ? 2 * ROWS : 1];  // scale words: [half of the stage][row]
  const int tid = threadIdx.x & 255, lane = tid & 63, team = TEAMS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  i32x4* const la[2] = {lds + team * 2 * HALF, lds + team * 2 * HALF + HALF};
  i32x4* const lb[2] = {la[0] + TA::kChunks, la[1] + TA::kChunks};
  uint32_t* const ls[2] = {scales[team * 2], scales[team * 2 + 1]};
  // the team's stages; the second one's may be one less, and then end with zeros
  const int steps = SUM ? (klen + BK - 1) / BK : ((klen + BK - 1) / BK + TEAMS - 1) / TEAMS;
  const int whole = TEAMS == 1 || SUM ? klen / BK : max(klen / BK - steps, 0);  // that every team has
  if (SUM) {
    if (team) {
      a = a2;
      lda = lda2;
      b = b2;
      ldb = ldb2;
    }
  } else if (TEAMS > 1 && team) {
    const uint64_t k = (uint64_t)steps * BK;
    a += AKC ? k : k * lda;
    b += BKC ? k : k * ldb;
    if (PAIR) b2 += BKC ? k : k * ldb2;
    klen = max(klen - steps * BK, 0);
  } else if (TEAMS > 1) {
    klen = min(klen, steps * BK);
  }
  const int r0 = (wave >> 1) * (BM / 2), c0 = (wave & 1) * (COLUMNS / 2);
  LA ga;
  LB gb;
  ga.init(a, lda, am);
  gb.template init<PAIR>(b, ldb, bn, b2, ldb2);
  const uint8_t* ps = nullptr;
  if constexpr (D::kScaled)
    ps = tid < BM ? sa + (uint64_t)min(tid, am - 1) * srow : sb + (uint64_t)min(tid - BM, bn - 1) * srow;  // all in range
  struct Regs {
    i32x4 a[LA::N], b[LB::N];
    uint32_t s[2];
  };
  auto load_whole = [&](Regs& r, int s) {
    ga.load(r.a, s * BK);
    gb.load(r.b, s * BK);
    if constexpr (D::kScaled) {
      r.s[0] = *reinterpret_cast<const uint32_t*>(ps + s * 8);
      r.s[1] = *reinterpret_cast<const uint32_t*>(ps + s * 8 + 4);
    }
  };
  auto load = [&](Regs& r, int s) {
    ga.load(r.a, s * BK, klen);
    gb.load(r.b, s * BK, klen);
    if constexpr (D::kScaled) {
      r.s[0] = s * BK < klen ? *reinterpret_cast<const uint32_t*>(ps + s * 8) : 0;
      r.s[1] = s * BK + 32 < klen ? *reinterpret_cast<const uint32_t*>(ps + s * 8 + 4) : 0;
    }
  };
  auto put = [&](const Regs& r, int h) {
#pragma unroll
    for (int i = 0; i < LA::N; i++) la[h][TA::pos(ga.line + i * (256 / TA::kPerRow), ga.col / 8)] = r.a[i];
#pragma unroll
    for (int i = 0; i < LB::N; i++) lb[h][TB::pos(gb.line + i * (256 / TB::kPerRow), gb.col / 8)] = r.b[i];
    if constexpr (D::kScaled) {
      if (tid < ROWS) {
        ls[h][tid] = r.s[0];
        ls[h][ROWS + tid] = r.s[1];
      }
    }
  };
  f32x4 acc[WM][WN];
#pragma unroll
  for (int i = 0; i < WM; i++)
#pragma unroll
    for (int j = 0; j < WN; j++) acc[i][j] = f32x4{0, 0, 0, 0};
  auto multiply = [&](int h) {
    const uint32_t pa = TA::place(la[h], r0), pb = TB::place(lb[h], c0);
    each<2>([&](auto part) {
      V fa[WM], fb[WN];
      int xa[WM], xb[WN];
      each<WN>([&](auto j) {
        fb[j.v] = __builtin_bit_cast(V, TB::template fragment<j.v, part.v, PAIR ? 64 : 32>(pb));
        if constexpr (D::kScaled)
          xb[j.v] = reinterpret_cast<const uint8_t*>(
              ls[h])[(part.v * ROWS + BM + c0 + TB::first_row() + (j.v >> 1) * 32 + (j.v & 1) * 4) * 4 + (lane >> 4)];
      });
      each<WM>([&](auto i) {
        fa[i.v] = __builtin_bit_cast(V, TA::template fragment<i.v, part.v>(pa));
        if constexpr (D::kScaled)
          xa[i.v] = reinterpret_cast<const uint8_t*>(ls[h])[(part.v * ROWS + r0 + TA::first_row() + i.v * 16) * 4 + (lane >> 4)];
      });
#pragma unroll
      for (int i = 0; i < WM; i++)
#pragma unroll
        for (int j = 0; j < WN; j++) {
          if constexpr (D::kScaled) acc[i][j] = mfma(fb[j], xb[j], fa[i], xa[i], acc[i][j]);
          else acc[i][j] = mfma(fb[j], fa[i], acc[i][j]);
        }
    });
  };
  Regs r[DEPTH];  // stage s in r[s % DEPTH], then in half s % 2 of LDS
  int s = 0;
  const int full = (AKC || am >= BM) && (BKC || bn >= COLUMNS) ? whole : 0;
  each<DEPTH>([&](auto i) {
    if (full >= DEPTH) load_whole(r[i.v], i.v);
    else if (i.v < steps) load(r[i.v], i.v);
  });
  if (steps > 0) put(r[0], 0);
  __syncthreads();
  for (; s + 2 * DEPTH - 1 < full; s += DEPTH) {
    each<DEPTH>([&](auto i) {
      load_whole(r[i.v], s + i.v + DEPTH);
      multiply(i.v & 1);
      put(r[(i.v + 1) % DEPTH], (i.v + 1) & 1);
      __syncthreads();
    });
  }
  for (; s < steps; s += DEPTH) {
    each<DEPTH>([&](auto i) {
      if (s + i.v >= steps) return;
      if (s + i.v + DEPTH < steps) load(r[i.v], s + i.v + DEPTH);
      multiply(i.v & 1);
      if (s + i.v + 1 < steps) put(r[(i.v + 1) % DEPTH], (i.v + 1) & 1);
      __syncthreads();
    });
  }
  if constexpr (TEAMS > 1) {
    // every wave is past its last read of the stages
    i32x4* sums = lds + wave * (WM * WN * 64) + lane;
    if (team) {
      each<WM * WN>([&](auto i) { sums[i.v * 64] = __builtin_bit_cast(i32x4, acc[i.v / WN][i.v % WN]); });
    }
    __syncthreads();
    if (team) return;
    each<WM * WN>([&](auto i) { acc[i.v / WN][i.v % WN] += __builtin_bit_cast(f32x4, sums[i.v * 64]); });
  }
  // a lane: row lane % 16 of each fragment, of its columns 8 * (lane / 16) ... in each 32
  const int c = c0 + (lane >> 4) * 8;
#pragma unroll
  for (int i = 0; i < WM; i++) {
    const int r = r0 + i * 16 + (lane & 15);
    if (r < am) {
      if constexpr (PAIR) {
        out.put(r, c, bn - c, acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
      } else {
        out.put(r, c, bn - c, acc[i][0], acc[i][1]);
        out.put(r, c + 32, bn - c - 32, acc[i][2], acc[i][3]);
      }
    }
  }
}

}  // namespace
}  // namespace ciera
