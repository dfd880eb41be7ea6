// The engine of the large products: 256 x 256 tiles fed straight into LDS.
#pragma once
#include "ciera_act.h"
#include "ciera_tiles.h"

namespace ciera {
namespace {

// 16 zero bytes: what is loaded in place of contraction steps past the end.
__device__ const i32x4 kZeros = {0, 0, 0, 0};

// 16 bytes per lane from memory straight into LDS, lane l's at `lds` + l.  Written in
// assembly because the compiler, where it sees such a load, waits for it before the
// next LDS read of any address; the kernels here wait themselves (arrive).  It has no
// result register; the clobber keeps LDS reads from moving across it.  m0, which holds
// the address in LDS, is the compiler's scratch register too, set anew at each use.
__device__ __forceinline__ void load_lds16(const void* p, i32x4* lds) {
  const uint32_t at = lds_address(lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(p) : "memory");
}
__device__ __forceinline__ void load_lds16(const char* base, uint32_t offset, i32x4* lds) {
  const uint32_t at = lds_address(lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(at), "v"(offset), "s"(base)
               : "memory");
}

// A pointer that all lanes agree on, in scalar registers, where the compiler does not see that.
__device__ __forceinline__ const char* scalar(const char* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  return reinterpret_cast<const char*>((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)v) |
                                       (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32)) << 32);
}
// 4 bytes per lane.
__device__ __forceinline__ void load_lds4(const void* p, void* lds) {
  const uint32_t at = lds_address(lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(at), "v"(p) : "memory");
}

__device__ __forceinline__ void load_lds4(const char* base, uint32_t offset, void* lds) {
  const uint32_t at = lds_address(lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(at), "v"(offset), "s"(base)
               : "memory");
}

// 16 bytes that are not read again soon: kept from displacing operands in L2 (64 experts of
// 2048 x 1024, 4-bit product 121 -> 94 us; one group 8192^3, [N, K], 951 -> 796 us).
typedef int i32x4_any __attribute__((ext_vector_type(4), aligned(2)));
template <typename O, typename P>
__device__ __forceinline__ void store_past(O* at, const P& p) {
  __builtin_nontemporal_store(__builtin_bit_cast(i32x4, p), reinterpret_cast<i32x4_any*>(at));
}

template <typename P>
__device__ __forceinline__ P load_past(const char* at) {
  return __builtin_bit_cast(P, (i32x4)__builtin_nontemporal_load(reinterpret_cast<const i32x4_any*>(at)));
}

// Where a tile's results go.
template <typename O>
struct BigOut {
  typedef O T;
  O* out;
  uint64_t ldo;
  __device__ __forceinline__ BigOut at(uint64_t row, int col) const { return BigOut{out + row * ldo + col, ldo}; }
};

// What a wave does with a stage in LDS: 128 x 64 results, by quarters of 4 parts.
// read<U, I> fetches what part I of quarter U needs new, multiply<U, I> multiplies it; the
// parts of a quarter may be read while the quarter before is multiplied.
//
// Two-byte operands: 16 x 16 x 32 instructions (32 x 32 x 16 ones read and write twice as
// many sums for a product and were 5 % slower here); a quarter is 64 of the 128 rows in half
// of the stage.
template <typename D, bool AKC, bool BKC>
struct WaveTile16 {
  typedef StageTile<AKC, false, 16> TA;
  typedef StageTile<BKC, false, 16> TB;
  typedef typename D::V V;
  static constexpr int kCols = 256, kRows = 128;  // of a tile, of a wave
  static constexpr bool kReads = false;  // the results' store reads other operands
  template <typename O>
  static constexpr int stores() {  // store instructions of a whole tile
    return 8 * (int)sizeof(O);
  }
  static __device__ __forceinline__ int row0(int wave) { return (wave >> 2) * 128; }
  static __device__ __forceinline__ int col0(int wave) { return (wave & 3) * 64; }
  f32x4 acc[8][4];
  V fa[2][4], fb[2][4];
  uint32_t pa, pb;

  __device__ __forceinline__ void init(const i32x4* lds, int r0, int c0) {
    pa = TA::place(lds, r0);
    pb = TB::place(lds + TA::kChunks, c0);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; i++)
#pragma unroll
      for (int j = 0; j < 4; j++) acc[i][j] = f32x4{0, 0, 0, 0};
  }
  template <int U, int I>
  __device__ __forceinline__ void read(uint32_t half) {
    fa[U & 1][I] = __builtin_bit_cast(V, TA::template fragment<(U & 1) * 4 + I, U / 2>(pa + half));
    if constexpr (U % 2 == 0) fb[U / 2][I] = __builtin_bit_cast(V, TB::template fragment<I, U / 2>(pb + half));
  }
  template <int U, int I>
  __device__ __forceinline__ void multiply() {
#pragma unroll
    for (int j = 0; j < 4; j++) {
      f32x4& c = acc[(U & 1) * 4 + I][j];
      c = mfma(fb[U / 2][j], fa[U & 1][I], c);
    }
  }
  __device__ __forceinline__ void next_stage() {}

  // Results to `out`, where the wave's first one belongs: `om` rows and `on` columns
  // (WHOLE: all).  A lane has row lane % 16 of each fragment and of its columns
  // 4 * (lane / 16) ... in each 16.  Through LDS (kTurn chunks of the wave's own) rows of 128
  // bytes, 64 columns or 32 in fp32, are made of them, 16 at a time, so that 8 lanes
  // store a whole line (stored directly, 64 bytes of a row to an instruction, 64 experts
  // of 2048 x 1024 took 294 us for 285, the input gradient 310 for 291).
  static constexpr int kTurn = 128;
  template <bool WHOLE, typename O>
  __device__ __forceinline__ void store(const BigOut<O>& o, int om, int on, i32x4* turn) {
    O* const out = o.out;
    const uint64_t ldo = o.ldo;
    constexpr int PER = 16 / sizeof(O), SPLIT = sizeof(O) / 2;
    const int l = afresh(threadIdx.x & 63), row = l & 15, q = l >> 4, chunk = l & 7;
    each<8 * SPLIT>([&](auto step) {
      constexpr int I = step.v / SPLIT, J = step.v % SPLIT * 2;
#pragma unroll
      for (int j = 0; j < 4 / SPLIT; j++) {
        const int at = SPLIT == 1 ? j * 2 + (q >> 1) : j * 4 + q;
        Pack<O, 4> p;
#pragma unroll
        for (int e = 0; e < 4; e++) p.v[e] = (O)acc[I][J + j][e];
        char* to = reinterpret_cast<char*>(turn + row * 8 + (at ^ (row >> 1)));
        __builtin_memcpy(__builtin_assume_aligned(to + (SPLIT == 1 ? (q & 1) * 8 : 0), 8 * SPLIT), &p, sizeof(p));
      }
      wave_order();
#pragma unroll
      for (int t = 0; t < 2; t++) {
        const int r = t * 8 + (l >> 3), m = I * 16 + r, n = J * 16 + chunk * PER;
        const Pack<O, PER> p = __builtin_bit_cast(Pack<O, PER>, turn[r * 8 + (chunk ^ (r >> 1))]);
        O* at = out + (uint64_t)m * ldo + n;
        if (WHOLE || (m < om && n + PER <= on)) {
          store_past(at, p);
        } else if (m < om) {
#pragma unroll
          for (int e = 0; e < PER; e++)
            if (n + e < on) at[e] = p.v[e];
        }
      }
      wave_order();
    });
  }
};

// 4-bit operands: 32 x 32 x 64 instructions.  A chunk holds one block of 32 codes; behind
// the codes of a stage lie the two scale words of every row, [operand][half][row], one
// for each half of the wave, whose byte u belongs to quarter u: the instruction picks it.
// A part is one of the four 32 rows.
struct WaveTile32 {
  typedef StageTile<true, false, 32> TA;
  typedef StageTile<true, true, 32> TB;
  static constexpr int kCols = 256, kRows = 128;  // of a tile, of a wave
  static constexpr bool kReads = false;  // the results' store reads other operands
  template <typename O>
  static constexpr int stores() {
    return 8 * (int)sizeof(O);
  }
  static __device__ __forceinline__ int row0(int wave) { return (wave >> 2) * 128; }
  static __device__ __forceinline__ int col0(int wave) { return (wave & 3) * 64; }
  f32x16 acc[4][2];
  i32x4 fa[2][4], fb[2][2];
  int xa[4], xb[2], yb[2];  // scale words; yb: of the next stage
  uint32_t pa, pb, sa, sb;

  __device__ __forceinline__ void init(const i32x4* lds, int r0, int c0) {
    const int half = (threadIdx.x >> 5) & 1;
    pa = TA::place(lds, r0);
    pb = TB::place(lds + TA::kChunks, c0);
    sa = lds_address(lds + TA::kChunks + TB::kChunks) + half * 1024 + (r0 + TA::first_row()) * 4;
    sb = lds_address(lds + TA::kChunks + TB::kChunks) + 2048 + half * 1024 + (c0 + TB::first_row()) * 4;
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int j = 0; j < 2; j++) acc[i][j] = f32x16{};
  }
  template <int U, int I>
  __device__ __forceinline__ void read(uint32_t half) {
    fa[U & 1][I] = __builtin_bit_cast(i32x4, TA::fragment<I, U>(pa + half));
    if constexpr (U == 0) xa[I] = read_lds<int>(sa + half + I * 128);
    if constexpr (I < 2) fb[U & 1][I] = __builtin_bit_cast(i32x4, TB::fragment<I, U>(pb + half));
    if constexpr (I < 2 && U == 0) yb[I] = read_lds<int>(sb + half + I * 128);
  }
  template <int U, int I>
  __device__ __forceinline__ void multiply() {
#pragma unroll
    for (int j = 0; j < 2; j++) acc[I][j] = mfma<U>(fb[U & 1][j], xb[j], fa[U & 1][I], xa[I], acc[I][j]);
  }
  __device__ __forceinline__ void next_stage() {
    xb[0] = yb[0];
    xb[1] = yb[1];
  }
  // As above; a lane has row lane % 32 of each fragment and of its columns
  // 8 * (lane / 32) ... in each 16.  (Stored as they lie, 32 bytes of 32 rows to an
  // instruction, a tile of every unit took 7 us longer.)
  static constexpr int kTurn = 128;
  template <bool WHOLE, typename O>
  __device__ __forceinline__ void store(const BigOut<O>& o, int om, int on, i32x4* turn) {
    O* const out = o.out;
    const uint64_t ldo = o.ldo;
    constexpr int PER = 16 / sizeof(O), SPLIT = sizeof(O) / 2;
    const int l = afresh(threadIdx.x & 63), row = l & 15, h = l >> 5, chunk = l & 7;
    each<8 * SPLIT>([&](auto step) {
      constexpr int I = step.v / (2 * SPLIT), UP = step.v / SPLIT % 2, J = step.v % SPLIT;
      if (((l >> 4) & 1) == UP) {
#pragma unroll
        for (int c = 0; c < 4; c++) {
          Pack<O, PER> p;
#pragma unroll
          for (int e = 0; e < PER; e++) p.v[e] = (O)(SPLIT == 1 ? acc[I][c >> 1][(c & 1) * 8 + e] : acc[I][J][c * 4 + e]);
          const int at = SPLIT == 1 ? c * 2 + h : (c >> 1) * 4 + h * 2 + (c & 1);
          turn[row * 8 + (at ^ (row & 7))] = __builtin_bit_cast(i32x4, p);
        }
      }
      wave_order();
#pragma unroll
      for (int t = 0; t < 2; t++) {
        const int r = t * 8 + (l >> 3), m = I * 32 + UP * 16 + r, n = J * 32 + chunk * PER;
        const Pack<O, PER> p = __builtin_bit_cast(Pack<O, PER>, turn[r * 8 + (chunk ^ (r & 7))]);
        O* at = out + (uint64_t)m * ldo + n;
        if (WHOLE || (m < om && n + PER <= on)) {
          store_past(at, p);
        } else if (m < om) {
#pragma unroll
          for (int e = 0; e < PER; e++)
            if (n + e < on) at[e] = p.v[e];
        }
      }
      wave_order();
    });
  }
};
// 16 rows of results and 64 / SPLIT columns to `out` through LDS, as WaveTile16::store: part
// j of the columns is val(j), 4 columns of a row in a lane.
template <bool WHOLE, typename O, typename F>
__device__ __forceinline__ void store_rows16(F val, O* out, uint64_t ldo, int om, int on, i32x4* turn) {
  constexpr int PER = 16 / sizeof(O), SPLIT = sizeof(O) / 2;
  const int l = afresh(threadIdx.x & 63), row = l & 15, q = l >> 4, chunk = l & 7;
#pragma unroll
  for (int j = 0; j < 4 / SPLIT; j++) {
    const f32x4 v = val(j);
    const int at = SPLIT == 1 ? j * 2 + (q >> 1) : j * 4 + q;
    Pack<O, 4> p;
#pragma unroll
    for (int e = 0; e < 4; e++) p.v[e] = (O)v[e];
    char* to = reinterpret_cast<char*>(turn + row * 8 + (at ^ (row >> 1)));
    __builtin_memcpy(__builtin_assume_aligned(to + (SPLIT == 1 ? (q & 1) * 8 : 0), 8 * SPLIT), &p, sizeof(p));
  }
  wave_order();
#pragma unroll
  for (int t = 0; t < 2; t++) {
    const int r = t * 8 + (l >> 3), n = chunk * PER;
    const Pack<O, PER> p = __builtin_bit_cast(Pack<O, PER>, turn[r * 8 + (chunk ^ (r >> 1))]);
    O* at = out + (uint64_t)r * ldo + n;
    if (WHOLE || (r < om && n + PER <= on)) {
      store_past(at, p);
    } else if (r < om) {
#pragma unroll
      for (int e = 0; e < PER; e++)
        if (n + e < on) at[e] = p.v[e];
    }
  }
  wave_order();
}

// Two products of the same rows: 64 rows and 64 columns of each to a wave.  The second
// operands' halves of a stage lie behind each other, and a quarter is one product in half of
// the stage.  So a lane holds both products of an element, and rows of 128 bytes of act(G) U
// come out of one wave.
template <typename D, bool AKC, bool BKC, bool KEEP>
struct WaveTilePair {
  typedef StageTile<AKC, false, 16> TA;
  typedef StageTile<BKC, false, 16, 128> TB;
  typedef typename D::V V;
  static constexpr int kCols = 128, kRows = 64, kTurn = 128;
  static constexpr bool kReads = false;
  template <typename O>
  static constexpr int stores() {
    return 4 * (int)sizeof(O) * (KEEP ? 3 : 1);
  }
  static __device__ __forceinline__ int row0(int wave) { return (wave >> 1) * 64; }
  static __device__ __forceinline__ int col0(int wave) { return (wave & 1) * 64; }
  f32x4 acc[4][8];
  V fa[2][4], fb[2][4];
  uint32_t pa, pb;

  __device__ __forceinline__ void init(const i32x4* lds, int r0, int c0) {
    pa = TA::place(lds, r0);
    pb = TB::place(lds + TA::kChunks, c0);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int j = 0; j < 8; j++) acc[i][j] = f32x4{0, 0, 0, 0};
  }
  template <int U, int I>
  __device__ __forceinline__ void read(uint32_t half) {
    fb[U & 1][I] = __builtin_bit_cast(V, TB::template fragment<I, U / 2>(pb + half + (U & 1) * TB::kChunks * 16));
    if constexpr (U % 2 == 0) fa[U / 2][I] = __builtin_bit_cast(V, TA::template fragment<I, U / 2>(pa + half));
  }
  template <int U, int I>
  __device__ __forceinline__ void multiply() {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      f32x4& c = acc[i][(U & 1) * 4 + I];
      c = mfma(fb[U & 1][I], fa[U / 2][i], c);
    }
  }
  __device__ __forceinline__ void next_stage() {}
  template <bool WHOLE, typename O>
  __device__ __forceinline__ void store(const GluOut<O>& o, int om, int on, i32x4* turn) {
    constexpr int SPLIT = sizeof(O) / 2;
    each<4 * SPLIT>([&](auto step) {
      constexpr int I = step.v / SPLIT, J = step.v % SPLIT * 2, C = J * 16;
      const int m = om - I * 16, n = on - C;
      store_rows16<WHOLE>([&](int j) { return gated(acc[I][J + j], acc[I][4 + J + j], o.act); },
                          o.out + (uint64_t)(I * 16) * o.ldo + C, o.ldo, m, n, turn);
      if constexpr (KEEP) {
        store_rows16<WHOLE>([&](int j) { return acc[I][J + j]; }, o.gate + (uint64_t)(I * 16) * o.ldog + C, o.ldog, m, n, turn);
        store_rows16<WHOLE>([&](int j) { return acc[I][4 + J + j]; }, o.up + (uint64_t)(I * 16) * o.ldou + C, o.ldou, m, n,
                            turn);
      }
    });
  }
};

// A product D that is not written itself: dG = D U act'(G) and dU = D act(G).  8 rows at a
// time go through LDS in fp32, so that a lane has 8 consecutive columns for whole-line reads
// of G and U and writes of dG and dU, and D is not rounded.
template <typename D, bool AKC, bool BKC>
struct WaveTileGrad : WaveTile16<D, AKC, BKC> {
  static constexpr bool kReads = true;
  template <typename O>
  static constexpr int stores() {
    return 16 * (int)sizeof(O);
  }
  template <typename O>
  struct Eight {
    Pack<O, 16 / sizeof(O)> v[sizeof(O) / 2];
    __device__ __forceinline__ float operator[](int i) const { return (float)v[i * sizeof(O) / 16].v[i % (16 / sizeof(O))]; }
  };
  template <bool WHOLE, typename O>
  __device__ __forceinline__ void store(const GradOut<O>& o, int om, int on, i32x4* turn) {
    constexpr int AHEAD = 2, PER = 16 / sizeof(O);  // rows' operands under way; values of 16 bytes
    const int l = afresh(threadIdx.x & 63), row = l & 15, q = l >> 4, r = l >> 3, c = (l & 7) * 8;
    // a lane's place from the first of 8 rows (their strides are short), which all lanes agree on
    const char *pg = scalar(reinterpret_cast<const char*>(o.gate)), *pu = scalar(reinterpret_cast<const char*>(o.up));
    char* pdg = const_cast<char*>(scalar(reinterpret_cast<const char*>(o.dgate)));
    char* pdu = const_cast<char*>(scalar(reinterpret_cast<const char*>(o.dup)));
    const uint32_t og = (r * (uint32_t)o.ldg + c) * sizeof(O), ou = (r * (uint32_t)o.ldu + c) * sizeof(O);
    const uint32_t odg = (r * (uint32_t)o.lddg + c) * sizeof(O), odu = (r * (uint32_t)o.lddu + c) * sizeof(O);
    Eight<O> g[AHEAD], u[AHEAD];
    auto load = [&](int s) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(O) / 2; i++) {
        g[s % AHEAD].v[i] = load_past<Pack<O, PER>>(pg + og + i * 16);
        u[s % AHEAD].v[i] = load_past<Pack<O, PER>>(pu + ou + i * 16);
      }
      pg += 8 * o.ldg * sizeof(O);
      pu += 8 * o.ldu * sizeof(O);
    };
    if (WHOLE) each<AHEAD - 1>([&](auto s) { load(s.v); });
    each<16>([&](auto s) {
      constexpr int I = s.v / 2, UP = s.v % 2;
      if (WHOLE && s.v + AHEAD - 1 < 16) load(s.v + AHEAD - 1);
      if ((row >> 3) == UP) {
#pragma unroll
        for (int j = 0; j < 4; j++)
          turn[(row & 7) * 16 + ((j * 4 + q) ^ ((row & 7) * 2))] = __builtin_bit_cast(i32x4, this->acc[I][j]);
      }
      wave_order();
      const f32x4 lo = __builtin_bit_cast(f32x4, turn[r * 16 + ((l & 7) ^ r) * 2]);
      const f32x4 hi = __builtin_bit_cast(f32x4, turn[r * 16 + ((l & 7) ^ r) * 2 + 1]);
      if constexpr (WHOLE) {
        Eight<O> dg, du;
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const float d = i < 4 ? lo[i & 3] : hi[i & 3];
          float value, slope;
          act_grad(g[s.v % AHEAD][i], o.act, &value, &slope);
          dg.v[i / PER].v[i % PER] = (O)product(d, u[s.v % AHEAD][i] * slope);
          du.v[i / PER].v[i % PER] = (O)product(d, value);
        }
#pragma unroll
        for (int i = 0; i < (int)sizeof(O) / 2; i++) {
          store_past(reinterpret_cast<O*>(pdg + odg) + i * PER, dg.v[i]);
          store_past(reinterpret_cast<O*>(pdu + odu) + i * PER, du.v[i]);
        }
        pdg += 8 * o.lddg * sizeof(O);
        pdu += 8 * o.lddu * sizeof(O);
      } else {
        if (s.v * 8 + r < om) o.put(s.v * 8 + r, c, on - c, lo, hi);
      }
      wave_order();
    });
  }
};

template <typename D, bool AKC, bool BKC>
struct WaveTileOf {
  typedef WaveTile16<D, AKC, BKC> T;
};
template <>
struct WaveTileOf<Mx4, true, true> {
  typedef WaveTile32 T;
};

// 256 x 256 tiles of C = A B, one after another by the same workgroup: 8 waves of
// 128 x 64 of a tile each.  Rows start at multiples of 16 bytes and hold multiples of
// 8 values along their contiguous side.  64 contraction steps at a time (a stage)
// go from memory into one half of LDS, not passing registers, while the other half
// is multiplied; fragments are read a quarter stage ahead of their use, across the
// one barrier of a stage too.  The first two stages of the next tile are on their way
// before this one's results are stored, and do not wait for these stores.
//
// Scaled (4-bit) operands have the same shape in bytes.
//
// Big::PAIR: two second operands, 128 columns of each.  Big::SUM: a second pair of operands with
// the strides of the first, whose stages follow on those of the first.
enum class Big { PLAIN, PAIR, SUM };
template <typename D, bool AKC, bool BKC, typename Out, Big KIND = Big::PLAIN,
          typename Wave = typename WaveTileOf<D, AKC, BKC>::T>
struct BigTiles {
  typedef typename Out::T O;
  static constexpr bool PAIR = KIND == Big::PAIR, SUM = KIND == Big::SUM;
  static constexpr int BM = 256, BN = Wave::kCols, BK = 64, T = 512;
  typedef typename Wave::TA TA;
  typedef typename Wave::TB TB;
  static constexpr int kParts = TA::kChunks / T;  // of a stage's loads of one operand
  static constexpr int kCodes = 2 * TA::kChunks;
  static constexpr int kStage = kCodes + (D::kScaled ? 256 : 0);  // chunks; scales: [operand][half][row] words
  static constexpr int kLds = 2 * kStage + 8 * Wave::kTurn;
  static constexpr int kLoads = 2 * kParts + (D::kScaled ? 2 : 0);  // a wave's load instructions for a stage
  static constexpr int kStores = Wave::template stores<O>();        // and its store instructions, where its part of the tile is whole

  i32x4* lds;
  int wave, lane, r0, c0;
  bool ahead;                  // the stores of all the wave's part of a tile may still be under way
  // the tile being loaded
  const char *pa, *pb;         // its operands at the next stage
  const char *pa2, *pb2;       // PAIR: the other second operand; SUM: the second pair
  uint64_t da, db, db2;        // bytes from stage to stage
  int again;                   // SUM: steps of the second pair, not begun yet
  uint32_t oa[kParts], ob[kParts];  // this lane's chunks of a stage, bytes from there
  int left;                    // contraction steps not loaded yet
  const char *sa, *sb;         // scaled: its scales at the next stage
  uint32_t osa, osb;
  // the tile being multiplied
  Wave tile;

  __device__ __forceinline__ void init(i32x4* l) {
    lds = l;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    lane = threadIdx.x & 63;
    r0 = Wave::row0(wave);
    c0 = Wave::col0(wave);
    ahead = false;
    tile.init(lds, r0, c0);
  }
  // A lane's chunk has a fixed place in LDS, so it fetches what the permutation puts
  // there; rows and columns past the tile's end repeat the last one.  Asks for the
  // first stage into half `buf` and the second, if there is one, into the other.
  __device__ __forceinline__ void start(const uint16_t* a, uint64_t lda, int am, const uint16_t* b, uint64_t ldb, int bn,
                                        int klen, int buf, const uint16_t* b2 = nullptr, uint64_t ldb2 = 0,
                                        const uint16_t* a2 = nullptr) {
    pa = reinterpret_cast<const char*>(a);
    pb = reinterpret_cast<const char*>(b);
    da = AKC ? BK * 2 : BK * 2 * lda;
    db = BKC ? BK * 2 : BK * 2 * ldb;
    left = klen;
    if constexpr (PAIR) db2 = BKC ? BK * 2 : BK * 2 * ldb2;
    if constexpr (PAIR || SUM) pb2 = reinterpret_cast<const char*>(b2);
    if constexpr (SUM) {
      pa2 = reinterpret_cast<const char*>(a2);
      again = klen;
    }
    const int tid = afresh(threadIdx.x);
#pragma unroll
    for (int i = 0; i < kParts; i++) {
      const int p = i * T + tid, line = p / TA::kPerRow, c = TA::swizzle(line, p % TA::kPerRow) * 8;
      oa[i] = 2 * (AKC ? (uint32_t)min(line, am - 1) * (uint32_t)lda + c : line * (uint32_t)lda + min(c, am - 8));
    }
#pragma unroll
    for (int i = 0; i < kParts; i++) {
      const int p = b_chunk(i, tid), line = p / TB::kPerRow, c = TB::swizzle(line, p % TB::kPerRow) * 8;
      const uint32_t ld = PAIR && i >= kParts / 2 ? (uint32_t)ldb2 : (uint32_t)ldb;
      ob[i] = 2 * (BKC ? (uint32_t)min(line, bn - 1) * ld + c : line * ld + min(c, bn - 8));
    }
    keep_scalar();
    load(buf);
    if (klen > BK || SUM) load(buf ^ 1);
  }
  // (all lanes agree on the operands' addresses, which the compiler loses sight of in these
  // forms)
  __device__ __forceinline__ void keep_scalar() {
    if constexpr (SUM || Wave::kReads) {
      pa = scalar(pa);
      pb = scalar(pb);
    }
  }
  // This lane's chunk of part i of the second operand (PAIR: of its operand)
  static __device__ __forceinline__ int b_chunk(int i, int tid) { return (PAIR ? i % (kParts / 2) : i) * T + tid; }
  // The same for scaled operands of `row` bytes of scales a row; to be called before start.
  __device__ __forceinline__ void scales(const uint8_t* a, int am, const uint8_t* b, int bn, uint32_t row) {
    const int tid = afresh(threadIdx.x), r = tid & 255, h = tid >> 8;
    sa = reinterpret_cast<const char*>(a);
    sb = reinterpret_cast<const char*>(b);
    osa = (uint32_t)min(r, am - 1) * row + h * 4;
    osb = (uint32_t)min(r, bn - 1) * row + h * 4;
  }
  // Part i of the next stage into half `buf`.  FULL: the stage has 64 steps; else
  // steps past the end arrive as zeros.
  template <bool FULL>
  __device__ __forceinline__ void load_a(int buf, int i) {
    i32x4* at = lds + buf * kStage + wave * 64 + i * T;
    if (FULL) return load_lds16(pa, oa[i], at);
    const int p = i * T + afresh(threadIdx.x), line = p / TA::kPerRow;
    const int k = AKC ? TA::swizzle(line, p % TA::kPerRow) * 8 : line;
    load_lds16(k < left ? pa + oa[i] : reinterpret_cast<const char*>(&kZeros), at);
  }
  template <bool FULL>
  __device__ __forceinline__ void load_b(int buf, int i) {
    i32x4* at = lds + buf * kStage + TA::kChunks + wave * 64 + i * T;
    const char* from = PAIR && i >= kParts / 2 ? pb2 : pb;
    if (FULL) return load_lds16(from, ob[i], at);
    const int p = b_chunk(i, afresh(threadIdx.x)), line = p / TB::kPerRow;
    const int k = BKC ? TB::swizzle(line, p % TB::kPerRow) * 8 : line;
    load_lds16(k < left ? from + ob[i] : reinterpret_cast<const char*>(&kZeros), at);
  }
  template <bool FULL>
  __device__ __forceinline__ void load_scales(int buf) {
    if constexpr (D::kScaled) {
      char* at = reinterpret_cast<char*>(lds + buf * kStage + kCodes) + wave * 256;
      if (FULL) {
        load_lds4(sa, osa, at);
        load_lds4(sb, osb, at + 2048);
      } else {
        const bool in = (int)(threadIdx.x >> 8) * 32 < left;
        load_lds4(in ? sa + osa : reinterpret_cast<const char*>(&kZeros), at);
        load_lds4(in ? sb + osb : reinterpret_cast<const char*>(&kZeros), at + 2048);
      }
    }
  }
  __device__ __forceinline__ void loaded() {
    pa += da;
    pb += db;
    if constexpr (PAIR) pb2 += db2;
    if constexpr (D::kScaled) {
      sa += 8;
      sb += 8;
    }
    left -= BK;
    if constexpr (SUM) {
      if (left <= 0 && again) {
        pa = pa2;
        pb = pb2;
        left = again;
        again = 0;
      }
    }
    keep_scalar();
  }
  __device__ __forceinline__ void load(int buf) {
    if (left >= BK) {
#pragma unroll
      for (int i = 0; i < kParts; i++) load_a<true>(buf, i);
#pragma unroll
      for (int i = 0; i < kParts; i++) load_b<true>(buf, i);
      load_scales<true>(buf);
    } else {
#pragma unroll
      for (int i = 0; i < kParts; i++) load_a<false>(buf, i);
#pragma unroll
      for (int i = 0; i < kParts; i++) load_b<false>(buf, i);
      load_scales<false>(buf);
    }
    loaded();
  }
  // All but the last N of this wave's loads and stores are done (they end in order),
  // as are its LDS reads; then the same for every wave.  The counter has six bits: with more
  // stores than that under way it waits for some of them too.
  template <int MANY>
  static __device__ __forceinline__ void arrive() {
    constexpr int N = MANY < 63 ? MANY : 63;
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4 << 14) | 0x0070);  // vmcnt N, lgkmcnt 0
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  }
  // One part of the loads of a whole stage: 3 of the 4 go out in a stage's last quarter,
  // the others in the quarter after it.
  template <bool FOURTH, int I>
  __device__ __forceinline__ void load_part(int buf) {
    if constexpr ((I == 3) == FOURTH) {
      load_a<true>(buf, I);
      load_b<true>(buf, I);
      if (FOURTH) {
        load_scales<true>(buf);
        loaded();
      }
    }
  }
  // The last quarter of the stage in half `buf` ^ 1 (not if FIRST) and the first three
  // of the one in `buf`: the matrix instructions of a part each and between them, in a
  // fixed order, the reads of the next quarter's fragments and (LOAD) the loads of the
  // stage after these two, into the half that the first of them leaves.
  template <bool FIRST, bool LOAD>
  __device__ __forceinline__ void stage(int buf) {
    const uint32_t half = buf * (kStage * 16);
    each<4>([&](auto i) {
      if (LOAD) load_part<false, i.v>(buf ^ 1);
      if (!FIRST) tile.template multiply<3, i.v>();
      tile.template read<0, i.v>(half);
      __builtin_amdgcn_sched_barrier(0);
    });
    tile.next_stage();
    each<3>([&](auto u) {
      each<4>([&](auto i) {
        if (LOAD && u.v == 0) load_part<true, i.v>(buf ^ 1);
        tile.template multiply<u.v, i.v>();
        tile.template read<u.v + 1, i.v>(half);
        __builtin_amdgcn_sched_barrier(0);
      });
    });
  }
  // WORK: not for a wave without rows of the tile, which only loads.
  template <bool WORK>
  __device__ __forceinline__ void run(int klen, int* half) {
    // (SUM: a whole stage may follow on one that is not)
    const int steps = SUM ? 2 * ((klen + BK - 1) / BK) : max((klen + BK - 1) / BK, 1);
    const int full = !SUM ? klen / BK : klen % BK ? 0 : steps;
    int buf = *half;
    // stage 0 is here; the second stage's loads and the last tile's stores may not be
    if (!ahead) arrive<0>();
    else if (steps > 1) arrive<kStores + kLoads>();
    else arrive<kStores>();
    if (WORK) stage<true, false>(buf);
    if (ahead) arrive<kStores>();
    else arrive<0>();
    int s = 0;
    for (; s + 2 < full; s++) {
      buf ^= 1;
      if (WORK) stage<false, true>(buf);
      else load(buf ^ 1);
      arrive<0>();
    }
    for (; s + 1 < steps; s++) {
      buf ^= 1;
      if (s + 2 < steps) load(buf ^ 1);
      if (WORK) stage<false, false>(buf);
      arrive<0>();
    }
    *half = buf ^ 1;
  }
  // All but the last quarter of the tile that was started in half *half, of `om` rows
  // and `klen` contraction steps; then both halves are free, *half the one for the next.
  __device__ __forceinline__ void stages(int om, int klen, int* half) {
    tile.clear();
    if (r0 < om) run<true>(klen, half);
    else run<false>(klen, half);
  }
  // The last quarter, and the results.
  __device__ __forceinline__ void finish(const Out& out, int om, int on) {
    ahead = om - r0 >= Wave::kRows && on - c0 >= 64;
    if (r0 >= om) return;
    each<4>([&](auto i) { tile.template multiply<3, i.v>(); });
    i32x4* turn = lds + 2 * kStage + wave * Wave::kTurn;
    if (ahead) tile.template store<true>(out.at(r0, c0), om - r0, on - c0, turn);
    else tile.template store<false>(out.at(r0, c0), om - r0, on - c0, turn);
  }
};

// The tiles of one workgroup: those of its die in turn, and where what is left in the
// end is at most half as many as there are workgroups, one half (128 rows) of one each.
struct TileList {
  uint64_t first;
  uint32_t stride, me, rounds, rest;
  __device__ __forceinline__ void init(uint64_t all) {
    uint32_t many;
    die_run(all, blockIdx.x % kXcds, &first, &many);
    stride = gridDim.x / kXcds;
    me = blockIdx.x / kXcds;
    rounds = many / stride;
    rest = many % stride;
  }
  // the i-th: rows from `row` on of the tile, `rows` of them; false: no more
  __device__ __forceinline__ bool get(uint32_t i, uint64_t* tile, int* row, int* rows) const {
    const bool split = i == rounds && 2 * rest <= stride;
    *tile = first + (uint64_t)i * stride + (split ? me / 2 : me);
    *row = split ? (me & 1) * 128 : 0;
    *rows = split ? 128 : 256;
    return i < rounds || (i == rounds && me < (split ? 2 * rest : rest));
  }
};

// Whether a tile's operands can be addressed with 32-bit byte offsets from their
// first element: 256 rows, or 64 contraction steps, of `ld` two-byte values.
inline bool short_stride(uint64_t ld) { return ld < (1u << 22); }

}  // namespace
}  // namespace ciera
