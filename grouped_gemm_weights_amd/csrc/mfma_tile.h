// A bf16 product of one workgroup: C[m][n] = sum_k A(m, k) B(k, n) into fp32 accumulators, for
// operands whose rows run along the depth ("row" operands) or across it ("column" operands, read
// transposed).  Used by the gradients of the grouped SwiGLU and of the products by expert, which need both;
// row_tile.h builds its loop for row operands on the shapes, copies and epilogues here.
//
// Two tile sizes, four waves each:
//   256 x 256  one wave per SIMD with a 128 x 128 quarter in 256 accumulators (4 x 4 MFMAs of
//              32x32x16 per 16 of depth): every operand read from LDS feeds four MFMAs.  A tile
//              with fewer rows gives every wave all of them and 64 columns.
//   64 x 64    (64 x 128 with DUAL) a wave a 32 x 32 block (or two): for products too small to give
//              every CU a large tile.  A stage is a few MFMAs, so its time is latency; eight
//              stages are in flight.
// Depth goes in stages of 32:
//
// * Global memory to LDS by buffer_load ... lds, 16 bytes a lane, without passing registers: the
//   accumulators leave none for a staging ring.  A lane outside the operand gets an offset past
//   the descriptor's range, for which the hardware writes zeros, so rows, columns and depth of any
//   size need no other code.  With S stage buffers, stage s + S is issued when the last reads of
//   stage s are done: the large tile's four cover about three stages of MFMA work (3000 cycles).
// * LDS to registers: a row operand is stored as [row][32 k], 64 bytes a row, its 16-byte chunks
//   permuted by (row / 4) % 4, so that the 16 rows a quarter wave reads lie in different banks.  A
//   column operand is stored as it comes, [k][columns], and read by ds_read_b64_tr_b16, which hands
//   each lane four consecutive k of its column; its 32-byte granules are permuted by k % 4, so
//   that the four k rows of one transposed read lie in different banks.  The copy writes LDS
//   linearly, so both permutations are applied to the global address of each lane.
// * The operands of the next 16 k are read while the MFMAs of the current 16 issue, one read or
//   copy per MFMA.  One barrier a stage.  With one wave per SIMD every instruction between two
//   MFMAs counts: stage offsets are immediates, bounds leave the loop (Operand::bound).
// * The MFMAs compute the transposed block (B's columns as their rows), so a lane ends with four
//   consecutive columns of one row: 16 bytes of an fp32 output, 8 of a bf16 one.  bf16 blocks go
//   through LDS once more (store_block) and leave as 16-byte stores of whole row segments.
//
// Measured on 65536 rows of 7168 x 2048 (random bf16): 1.1-1.2 PFLOP/s, the MFMA pipes 70-75 % busy
// at the 1.5-1.7 GHz that the power limit leaves; with fewer instructions per MFMA the pipes get
// busier and the clock lower.
#pragma once

#include <type_traits>

#include "common.h"

namespace moe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;

constexpr int kStageK = 32;
// Of a tile of TR rows (256 or 64): columns of its B operand, stages in flight, and LDS bytes (128 KB;
// 64 KB, 96 KB with DUAL).
constexpr int tile_columns(int tr, bool dual) { return tr == 256 ? 256 : dual ? 128 : 64; }
constexpr int tile_stages(int tr) { return tr == 256 ? 4 : 8; }
constexpr int operand_bytes(int rows) { return rows * kStageK * 2; }  // one operand's stage
constexpr int stage_bytes(int tr, bool dual) { return operand_bytes(tr) + operand_bytes(tile_columns(tr, dual)); }
constexpr int tile_lds(int tr, bool dual) { return tile_stages(tr) * stage_bytes(tr, dual); }
// Granule permutation of depth k of a column operand (its rows must keep their granules).
constexpr int granule_swap(int columns, int k) { return columns >= 128 ? 2 * (k & 3) : k & 2; }
constexpr uint32_t kOutside = 0x80000000u;              // lane offsets from here on read zeros

// 16 bytes per lane from buffer r + voff to LDS at `lds` + OFF + 16 lane (lds wave-uniform).  The
// scalar write of m0 needs one wait state before the copy reads it.
template <int OFF>
__device__ __forceinline__ void copy_to_lds(u32x4 r, uint32_t voff, uint32_t lds) {
  asm volatile(
      "s_add_u32 m0, %0, %3\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(voff), "s"(r), "n"(OFF)
      : "memory", "scc");
}

template <int N>
__device__ __forceinline__ void wait_copies_and_sync() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// One operand: how its stages are copied.  COLS: a column operand.  ROWS: rows (or, for a column
// operand, columns) of the tile that are staged.
template <bool COLS, int ROWS>
struct Operand {
  static constexpr int N = ROWS / 64;                      // copies per wave and stage
  static constexpr int CHUNKS = ROWS / 8;                  // column operand: 16-byte chunks of a depth
  static constexpr int DEPTHS = COLS ? kWave / CHUNKS : 0;  // and depths of a copy
  static constexpr int WAVE_STEP = COLS ? N * 1024 : 1024;  // LDS bytes from a wave's copy to the next wave's
  static constexpr int COPY_STEP = COLS ? 1024 : 4096;     // and from a wave's copy to its next
  uint64_t base;       // wave-uniform: where the stage to issue next starts
  uint32_t step;       // bytes from a stage to the next
  int left;            // steps of depth from there on
  uint32_t voff[N];    // this lane's offset in each copy, kOutside for what does not exist
  int k_at;            // depth of this lane's copy 0 within a stage

  // Row operand: tile row r is at p + src(r) * ld elements, src(r) < 0 for none.
  // Column operand: depth k is at p + k * ld, tile column c at src(c), 8 columns at a time.
  template <typename Src>
  __device__ __forceinline__ void init(const uint16_t* p, int64_t ld, int K, Src src) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const uint64_t at = reinterpret_cast<uint64_t>(p);
    base = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at))) |
           static_cast<uint64_t>(static_cast<uint32_t>(
               __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at >> 32)))) << 32;
    left = K;
    if constexpr (COLS) {
      step = static_cast<uint32_t>(kStageK * ld * 2);
      k_at = wave * 8 + lane / CHUNKS;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int k = k_at + DEPTHS * i, q = lane % CHUNKS;
        const int col = ((((q >> 1) ^ granule_swap(ROWS, k)) << 1) | (q & 1)) * 8;
        const int c = src(col);
        voff[i] = c < 0 ? kOutside : static_cast<uint32_t>(k * ld + c) * 2u;
      }
    } else {
      step = kStageK * 2;
      k_at = ((lane & 3) ^ (lane >> 4)) * 8;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int r = src((i * 4 + wave) * 16 + (lane >> 2));
        voff[i] = r < 0 ? kOutside : static_cast<uint32_t>(r * ld + k_at) * 2u;
      }
    }
    bound();
  }

  // The last stage may be short and the ones after it are empty: lanes past the depth copy zeros
  // from there on.
  __device__ __forceinline__ void bound() {
    if (left < kStageK) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (k_at + (COLS ? DEPTHS * i : 0) >= left) voff[i] = kOutside;
    }
  }
  __device__ __forceinline__ void next_stage() {
    base += step;
    left -= kStageK;
    bound();
  }

  // Copy I of the stage at `base` to LDS offset OFF (the operand's stage buffer); lds is this
  // wave's place: the tile's LDS + wave * WAVE_STEP.
  template <int I, int OFF>
  __device__ __forceinline__ void copy(uint32_t lds) const {
    const u32x4 r = {static_cast<uint32_t>(base), static_cast<uint32_t>(base >> 32), kOutside, 0x00020000u};
    copy_to_lds<OFF + I * COPY_STEP>(r, voff[I], lds);
  }
};

// Fragment reads of one operand: 32 rows (columns) by 16 k, lane l holding row l % 32, k
// 8 (l / 32) .. +8.
template <bool COLS, int BLOCKS, int ROWS, int STAGES, int STAGE>
struct Fragments {
  static constexpr int N = COLS ? BLOCKS : 2;
  static constexpr int BASES = STAGES * STAGE > 65536 ? 2 : 1;  // an LDS read's own offset reaches 64 KB
  static constexpr int PER = STAGES / BASES;
  int at[BASES][N];

  // first(b): tile row (column) of block b, a multiple of 32; for rows, first(b) - first(0) is
  // a compile-time constant.  lds: the operand's buffer of stage 0.
  template <typename First>
  __device__ __forceinline__ void init(int lds, First first) {
    const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (COLS) {
        const int k = (lane >> 5) * 8 + ((lane & 15) >> 2);
        at[0][i] = lds + k * ROWS * 2 + (((first(i) >> 4) + ((lane >> 4) & 1)) ^ granule_swap(ROWS, k)) * 32 + (lane & 3) * 8;
      } else {
        at[0][i] = lds + (first(0) + (lane & 31)) * 64 + ((i * 2 + (lane >> 5)) ^ ((lane >> 2) & 3)) * 16;
      }
      if (BASES > 1) at[BASES - 1][i] = at[0][i] + PER * STAGE;
    }
  }

  // Block b (delta rows from block 0) of the 16 k at half s of stage buffer `buf`.
  __device__ __forceinline__ bf16x8 read(int buf, int b, int delta, int s) const {
    const int base = buf / PER, off = buf % PER * STAGE;
    if constexpr (COLS) {
      typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
      const lds_char* p = reinterpret_cast<const lds_char*>(at[base][b]) + off + s * 16 * ROWS * 2;
      union {
        i16x4 h[2];
        bf16x8 v;
      } u;
      u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          reinterpret_cast<lds_i16x4*>(const_cast<lds_char*>(p)));
      u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          reinterpret_cast<lds_i16x4*>(const_cast<lds_char*>(p + 4 * ROWS * 2)));
      return u.v;
    } else {
      typedef const __attribute__((address_space(3))) bf16x8 lds_bf16x8;
      return *reinterpret_cast<lds_bf16x8*>(reinterpret_cast<const lds_char*>(at[base][s]) + off + delta * 64);
    }
  }
};

// A tile of at most TR rows.  MI = 0: a full tile, two by two waves; MI > 0 (TR = 256): at most 32 MI
// rows, every wave all of them and a quarter of the columns.  DUAL: the first half of B's tile
// columns are columns of one matrix and the second half the same columns of another, and a
// wave's accumulators [.][j] and [.][j + NJ / 2] hold matching columns of the two.
template <int TR, int MI, bool DUAL>
struct TileShape {
  static constexpr int TN = tile_columns(TR, DUAL);
  static constexpr int MW = MI ? MI : TR / 64;                    // 32-row blocks per wave
  static constexpr int NJ = MI ? 2 : TN / 64;                     // 32-column blocks per wave
  static constexpr int ROWS = MI ? (MI < 2 ? 64 : MI * 32) : TR;  // staged rows of A
  static constexpr int SPAN = DUAL ? NJ * 16 : NJ * 32;           // columns of a matrix per wave
  static __device__ __forceinline__ int wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x / kWave); }
  static __device__ __forceinline__ int first_row() { return MI ? 0 : (wave() >> 1) * (TR / 2); }
  // first tile column of the wave's block j = first_col() + col(j)
  static __device__ __forceinline__ int first_col() { return (MI ? wave() : wave() & 1) * SPAN; }
  static constexpr int col(int j) {
    return !DUAL || j < NJ / 2 ? j * 32 : TN / 2 + (j - NJ / 2) * 32;
  }
};

// Calls f(integral_constant<int, I>) for I in [LO, HI).
template <int LO, int HI, typename F>
__device__ __forceinline__ void each(F f) {
  if constexpr (LO < HI) {
    f(std::integral_constant<int, LO>{});
    each<LO + 1, HI>(f);
  }
}

template <int TR, int MI, bool DUAL, bool A_COLS, bool B_COLS>
struct TileProduct {
  using S = TileShape<TR, MI, DUAL>;
  using OA = Operand<A_COLS, S::ROWS>;
  using OB = Operand<B_COLS, S::TN>;
  static constexpr int MW = S::MW, NJ = S::NJ, STAGES = tile_stages(TR), STAGE = stage_bytes(TR, DUAL);
  static constexpr int NA = OA::N, NL = NA + OB::N;   // copies per wave and stage
  static constexpr int NF = NL / 2;                   // of these, issued in a stage's second half
  static constexpr int NMF = MW * NJ, NRD = MW + NJ;  // MFMAs and fragments per 16 k
  static constexpr int NS = NMF > NRD ? NMF : NRD;
  OA& A;
  OB& B;
  floatx16 (&acc)[MW][NJ];
  Fragments<A_COLS, MW, S::ROWS, STAGES, STAGE> fa;
  Fragments<B_COLS, NJ, S::TN, STAGES, STAGE> fb;
  uint32_t lds_a, lds_b;
  bf16x8 pa[MW], pb[NJ], qa[MW], qb[NJ];

  template <int C, int BUF>
  __device__ __forceinline__ void copy() {
    if constexpr (C < NA) A.template copy<C, BUF * STAGE>(lds_a);
    else B.template copy<C - NA, BUF * STAGE + operand_bytes(TR)>(lds_b);
  }
  __device__ __forceinline__ void next_stage() {
    A.next_stage();
    B.next_stage();
  }
  __device__ __forceinline__ void read(bf16x8 (&ra)[MW], bf16x8 (&rb)[NJ], int t, int buf, int s) {
    if (t < MW) ra[t % MW] = fa.read(buf, t % MW, t % MW * 32, s);
    else rb[(t - MW) % NJ] = fb.read(buf, (t - MW) % NJ, S::col((t - MW) % NJ), s);
  }

  // The 16 k held in (ra, rb): one MFMA per slot; beside them the reads of the 16 k at half s of
  // stage buffer RBUF into (na, nb), and copies LO .. HI - 1 of the stage to issue into CBUF.
  template <int RBUF, int RS, int CBUF, int LO, int HI>
  __device__ __forceinline__ void half(bf16x8 (&ra)[MW], bf16x8 (&rb)[NJ], bf16x8 (&na)[MW],
                                       bf16x8 (&nb)[NJ]) {
    each<0, NS>([&](auto slot) {
      constexpr int t = decltype(slot)::value;
      if constexpr (t < NMF)
        acc[t / NJ][t % NJ] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(rb[t % NJ], ra[t / NJ],
                                                                     acc[t / NJ][t % NJ], 0, 0, 0);
      if constexpr (t < NRD) read(na, nb, t, RBUF, RS);
      each<LO, HI>([&](auto c) {
        if constexpr ((decltype(c)::value - LO) * NS / (HI - LO) == t) copy<decltype(c)::value, CBUF>();
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  }

  // One stage, in buffer BUF.  Its first half also issues the second part of the copies of the last
  // stage in flight (STAGES - 1 ahead).  Then this wave's copies of the next stage are there and
  // its reads of this one done; past the barrier that holds for every wave, and this buffer
  // takes the stage STAGES ahead.
  template <int BUF>
  __device__ __forceinline__ void stage() {
    half<BUF, 1, (BUF + STAGES - 1) % STAGES, NF, NL>(pa, pb, qa, qb);
    next_stage();
    wait_copies_and_sync<(STAGES - 2) * NL>();
    half<(BUF + 1) % STAGES, 0, BUF, 0, NF>(qa, qb, pa, pb);
  }

  __device__ __forceinline__ void run(int K, lds_char* smem) {
#pragma unroll
    for (int i = 0; i < MW; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;
    if (K <= 0) return;
    const int lds = static_cast<int>(reinterpret_cast<uintptr_t>(smem));
    fa.init(lds, [](int b) { return S::first_row() + b * 32; });
    fb.init(lds + operand_bytes(TR), [](int b) { return S::first_col() + S::col(b); });
    lds_a = lds + S::wave() * OA::WAVE_STEP;
    lds_b = lds + S::wave() * OB::WAVE_STEP;
    // the stages past the last are copied too, as zeros: the copies in flight stay countable
    each<0, STAGES>([&](auto s) {
      constexpr int BUF = decltype(s)::value;
      each<0, (BUF < STAGES - 1 ? NL : NF)>([&](auto c) { copy<decltype(c)::value, BUF>(); });
      if constexpr (BUF < STAGES - 1) next_stage();
    });
    wait_copies_and_sync<(STAGES - 2) * NL + NF>();
#pragma unroll
    for (int t = 0; t < NRD; ++t) read(pa, pb, t, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
    int stages = static_cast<int>((static_cast<uint32_t>(K) + kStageK - 1) / kStageK);
    for (; stages >= STAGES; stages -= STAGES) {
      stage<0>();
      stage<1>();
      stage<2>();
      stage<3>();
      if constexpr (STAGES == 8) {
        stage<4>();
        stage<5>();
        stage<6>();
        stage<7>();
      }
    }
    if (stages > 0) stage<0>();
    if (stages > 1) stage<1>();
    if (stages > 2) stage<2>();
    if constexpr (STAGES == 8) {
      if (stages > 3) stage<3>();
      if (stages > 4) stage<4>();
      if (stages > 5) stage<5>();
      if (stages > 6) stage<6>();
    }
    // the epilogue writes LDS: every wave's copies have landed and its reads are done
    wait_copies_and_sync<0>();
  }
};

template <int TR, int MI, bool DUAL, bool A_COLS, bool B_COLS>
__device__ __forceinline__ void tile_product(
    Operand<A_COLS, TileShape<TR, MI, DUAL>::ROWS>& A, Operand<B_COLS, TileShape<TR, MI, DUAL>::TN>& B,
    int K, lds_char* smem,
    floatx16 (&acc)[TileShape<TR, MI, DUAL>::MW][TileShape<TR, MI, DUAL>::NJ]) {
  TileProduct<TR, MI, DUAL, A_COLS, B_COLS> p{A, B, acc};
  p.run(K, smem);
}

// Row within the tile that this lane holds of accumulator block i, and the first of the four
// consecutive columns, within block j, of its elements 4 v .. 4 v + 3.
template <int TR, int MI, bool DUAL>
__device__ __forceinline__ int lane_row(int i) {
  return TileShape<TR, MI, DUAL>::first_row() + i * 32 + (threadIdx.x & 31);
}
__device__ __forceinline__ int lane_col(int v) {
  return v * 8 + ((threadIdx.x & 63) >> 5) * 4;
}

// 32 rows x COLS columns of bf16 from this wave's accumulators to memory.  put(j, v) gives the
// four values of column block j, elements 4 v .. 4 v + 3, as packed bf16.  The LDS rows are padded
// by 16 bytes, which spreads the 16 rows of a write over all banks.  The stores are non-temporal: a
// round of tiles writes as much as all of L2 holds, and would push out the panels that the next
// reads (weight gradients of 384 rows an expert: 450 -> 420 us).  out: the block's first row and
// column; rows, cols: how many exist (cols a multiple of 8).
template <int COLS, typename Put>
__device__ __forceinline__ void store_block(lds_char* smem, uint16_t* out, int64_t ld, int rows,
                                            int cols, Put put) {
  constexpr int PITCH = COLS * 2 + 16, LANES = COLS / 8, PER = kWave / LANES;
  typedef __attribute__((address_space(3))) u32x2 lds_u32x2;
  typedef __attribute__((address_space(3))) const u32x4 lds_u32x4;
  const int lane = threadIdx.x & (kWave - 1);
  lds_char* mine = smem + (threadIdx.x / kWave) * 16384;
#pragma unroll
  for (int j = 0; j < COLS / 32; ++j)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      *reinterpret_cast<lds_u32x2*>(mine + (lane & 31) * PITCH + (j * 32 + lane_col(v)) * 2) = put(j, v);
    }
  wave_lds_sync();
  const int c = (lane % LANES) * 8;
#pragma unroll
  for (int i = 0; i < 32 / PER; ++i) {
    const int r = i * PER + lane / LANES;
    const u32x4 d = *reinterpret_cast<lds_u32x4*>(mine + r * PITCH + c * 2);
    if (r < rows && c < cols) __builtin_nontemporal_store(d, reinterpret_cast<u32x4*>(out + r * ld + c));
  }
  wave_lds_sync();
}

__device__ __forceinline__ u32x2 pack4(float a, float b, float c, float d) {
  return u32x2{f32_to_bf16(a) | (static_cast<uint32_t>(f32_to_bf16(b)) << 16),
               f32_to_bf16(c) | (static_cast<uint32_t>(f32_to_bf16(d)) << 16)};
}

}  // namespace moe
