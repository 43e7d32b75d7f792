// A bf16 product of one workgroup: C[m][n] = sum_k A(m, k) B(k, n) into fp32 accumulators, for
// operands whose rows run along the depth ("row" operands) or across it ("column" operands, read
// transposed).  Used by the grouped SwiGLU's gradient, whose products need both.
//
// Four waves, one per SIMD.  A full tile is 256 x 256, each wave a 128 x 128 quarter in 256
// accumulators (4 x 4 MFMAs of 32x32x16 per 16 steps of depth); a tile with fewer rows gives every
// wave all of them and 64 columns.  Depth goes in stages of 32:
//
// * Global memory to LDS by buffer_load ... lds, 16 bytes a lane, without passing registers: the
//   accumulators leave none for a staging ring.  A lane outside the operand gets an offset past
//   the descriptor's range, for which the hardware writes zeros, so rows, columns and depth of any
//   size need no other code.  Four stage buffers: stage s + 4 is issued when the last reads of
//   stage s are done, so about three stages of MFMA work (3000 cycles) cover the latency.
// * LDS to registers: a row operand is stored as [row][32 k], 64 bytes a row, its 16-byte chunks
//   permuted by (row / 4) % 4, so that the 16 rows a quarter wave reads lie in different banks.  A
//   column operand is stored as it comes, [k][256], and read by ds_read_b64_tr_b16, which hands
//   each lane four consecutive k of its column; its 32-byte granules are permuted by 2 (k % 4), so
//   that the four k rows of one transposed read lie in different banks.  The copy writes LDS
//   linearly, so both permutations are applied to the global address of each lane.
// * The operands of the next 16 k are read while the MFMAs of the current 16 issue, one read or
//   copy per MFMA.  One barrier a stage.
// * The MFMAs compute the transposed block (B's columns as their rows), so a lane ends with four
//   consecutive columns of one row: 16 bytes of an fp32 output, 8 of a bf16 one.  bf16 blocks go
//   through LDS once more (store_block) and leave as 16-byte stores of whole row segments.
#pragma once

#include "common.h"

namespace moe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;

constexpr int kStageK = 32, kStages = 4, kTileN = 256;
constexpr int kOperandBytes = 256 * kStageK * 2;        // 16 KB: one operand's stage
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kTileLds = kStages * kStageBytes;         // 128 KB
constexpr uint32_t kOutside = 0x80000000u;              // lane offsets from here on read zeros

// 16 bytes per lane from base + voff to LDS at `lds` + 16 lane (wave-uniform).  The scalar move of
// m0 needs one wait state before the copy reads it.
__device__ __forceinline__ void copy_to_lds(const void* base, uint32_t voff, uint32_t lds) {
  __amdgpu_buffer_rsrc_t r =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, kOutside, 0x00020000);
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(voff), "s"(r)
      : "memory");
}

template <int N>
__device__ __forceinline__ void wait_copies_and_sync() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// One operand: how its stages are copied and its fragments read.  COLS: a column operand.
// ROWS: rows (or, for a column operand, columns) of the tile that are staged.
template <bool COLS, int ROWS>
struct Operand {
  static constexpr int N = COLS ? 4 : ROWS / 64;  // copies per wave and stage
  const char* base;    // wave-uniform: where the stage to issue next starts
  int64_t step;        // bytes from a stage to the next
  uint32_t voff[N];    // this lane's offset in each copy, kOutside for a row it does not have
  int k_at;            // depth of this lane's copy 0 within a stage

  // Row operand: tile row r is at base + src(r) * ld elements, src(r) < 0 for none.
  // Column operand: depth k is at base + k * ld, tile column c at src(c), 8 columns at a time.
  template <typename Src>
  __device__ __forceinline__ void init(const uint16_t* p, int64_t ld, Src src) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    base = reinterpret_cast<const char*>(p);
    if constexpr (COLS) {
      step = kStageK * ld * 2;
      k_at = wave * 8 + (lane >> 5);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int k = k_at + 2 * i, q = lane & 31;
        const int col = ((((q >> 1) ^ (2 * (k & 3))) << 1) | (q & 1)) * 8;
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
  }

  // Copy i of the stage at `base`, of which `left` steps of depth exist.
  __device__ __forceinline__ void copy(int i, int left, uint32_t lds) const {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const bool in = k_at + (COLS ? 2 * i : 0) < left;
    copy_to_lds(base, in ? voff[i] : kOutside,
                lds + (COLS ? (wave * 4 + i) * 1024 : (i * 4 + wave) * 1024));
  }
};

// Fragment reads of one operand: 32 rows (columns) by 16 k, lane l holding row l % 32, k
// 8 (l / 32) .. +8.
template <bool COLS, int BLOCKS>
struct Fragments {
  static constexpr int N = COLS ? BLOCKS : 2;
  int at[N];

  // first(b): tile row (column) of block b, a multiple of 32; for rows, first(b) - first(0) is
  // a compile-time constant.
  template <typename First>
  __device__ __forceinline__ void init(First first) {
    const int lane = threadIdx.x & (kWave - 1);
    if constexpr (COLS) {
      const int k = (lane >> 5) * 8 + ((lane & 15) >> 2);
#pragma unroll
      for (int b = 0; b < BLOCKS; ++b)
        at[b] = k * 512 + (((first(b) >> 4) + ((lane >> 4) & 1)) ^ (2 * (k & 3))) * 32 + (lane & 3) * 8;
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s)
        at[s] = (first(0) + (lane & 31)) * 64 + ((s * 2 + (lane >> 5)) ^ ((lane >> 2) & 3)) * 16;
    }
  }

  // Block b (delta rows from block 0) of the 16 k at half s of the stage at `lds`.
  __device__ __forceinline__ bf16x8 read(const lds_char* lds, int b, int delta, int s) const {
    if constexpr (COLS) {
      typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
      const lds_char* p = lds + at[b] + s * 16 * 512;
      union {
        i16x4 h[2];
        bf16x8 v;
      } u;
      u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          reinterpret_cast<lds_i16x4*>(const_cast<lds_char*>(p)));
      u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          reinterpret_cast<lds_i16x4*>(const_cast<lds_char*>(p + 4 * 512)));
      return u.v;
    } else {
      typedef const __attribute__((address_space(3))) bf16x8 lds_bf16x8;
      return *reinterpret_cast<lds_bf16x8*>(lds + at[s] + delta * 64);
    }
  }
};

// MI = 0: a full tile; MI > 0: at most 32 MI rows.  DUAL: B's 256 tile columns are 128 columns of
// one matrix and the same 128 of another, and a wave's accumulators [.][j] and [.][j + NJ / 2]
// hold matching columns of the two.
template <int MI, bool DUAL>
struct TileShape {
  static constexpr int MW = MI ? MI : 4;          // 32-row blocks per wave
  static constexpr int NJ = MI ? 2 : 4;           // 32-column blocks per wave
  static constexpr int ROWS = MI ? (MI < 2 ? 64 : MI * 32) : 256;  // staged rows of A
  static __device__ __forceinline__ int wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x / kWave); }
  static __device__ __forceinline__ int first_row() { return MI ? 0 : (wave() >> 1) * 128; }
  // first tile column of the wave's block j = first_col() + col(j)
  static __device__ __forceinline__ int first_col() {
    return MI ? wave() * (DUAL ? 32 : 64) : (wave() & 1) * (DUAL ? 64 : 128);
  }
  static constexpr int col(int j) {
    return !DUAL ? j * 32 : (j < NJ / 2 ? j * 32 : 128 + (j - NJ / 2) * 32);
  }
};

template <int MI, bool DUAL, bool A_COLS, bool B_COLS>
__device__ __forceinline__ void tile_product(
    Operand<A_COLS, TileShape<MI, DUAL>::ROWS>& A, Operand<B_COLS, 256>& B, int K, lds_char* smem,
    floatx16 (&acc)[TileShape<MI, DUAL>::MW][TileShape<MI, DUAL>::NJ]) {
  using S = TileShape<MI, DUAL>;
  constexpr int MW = S::MW, NJ = S::NJ;
  constexpr int NA = Operand<A_COLS, S::ROWS>::N, NL = NA + Operand<B_COLS, 256>::N;
  constexpr int NMF = MW * NJ, NRD = MW + NJ;
  constexpr int NS = NMF > NRD ? NMF : NRD;
  Fragments<A_COLS, MW> fa;
  Fragments<B_COLS, NJ> fb;
  fa.init([](int b) { return S::first_row() + b * 32; });
  fb.init([](int b) { return S::first_col() + S::col(b); });
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(smem));

#pragma unroll
  for (int i = 0; i < MW; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;
  const int nk = (K + kStageK - 1) / kStageK;
  if (nk == 0) return;

  // the stages past the last are copied too, as zeros: the copies in flight stay countable
  int left = K;
#define COPY(c, buf)                                                                     \
  do {                                                                                   \
    if ((c) < NA) A.copy((c) % NA, left, lds0 + (buf) * kStageBytes);                    \
    else B.copy(((c) - NA) % (NL - NA), left, lds0 + (buf) * kStageBytes + kOperandBytes); \
  } while (0)
#define NEXT_STAGE()   \
  do {                 \
    A.base += A.step;  \
    B.base += B.step;  \
    left -= kStageK;   \
  } while (0)
#pragma unroll
  for (int s = 0; s < kStages; ++s) {
#pragma unroll
    for (int c = 0; c < NL; ++c) COPY(c, s);
    NEXT_STAGE();
  }
  bf16x8 pa[MW], pb[NJ], qa[MW], qb[NJ];
#define READ(RA, RB, t, stage, s)                                                        \
  do {                                                                                   \
    if ((t) < MW) RA[(t) % MW] = fa.read(stage, (t) % MW, ((t) % MW) * 32, s);           \
    else RB[((t) - MW) % NJ] = fb.read((stage) + kOperandBytes, ((t) - MW) % NJ,         \
                                       S::col(((t) - MW) % NJ), s);                      \
  } while (0)
  wait_copies_and_sync<3 * NL>();
#pragma unroll
  for (int t = 0; t < NRD; ++t) READ(pa, pb, t, smem, 0);
  __builtin_amdgcn_sched_barrier(0);

  int buf = 0;
  for (int kt = 0; kt < nk; ++kt) {
    const lds_char* cur = smem + buf * kStageBytes;
    const int nbuf = (buf + 1) % kStages;
    const lds_char* next = smem + nbuf * kStageBytes;
#pragma unroll
    for (int t = 0; t < NS; ++t) {
      if (t < NMF)
        acc[t / NJ % MW][t % NJ] =
            __builtin_amdgcn_mfma_f32_32x32x16_bf16(pb[t % NJ], pa[t / NJ % MW], acc[t / NJ % MW][t % NJ], 0, 0, 0);
      if (t < NRD) READ(qa, qb, t, cur, 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    // this wave's copies of stage kt + 1 are there and its reads of stage kt done; past the
    // barrier that holds for every wave, and stage kt's buffer takes stage kt + 4
    wait_copies_and_sync<2 * NL>();
#pragma unroll
    for (int t = 0; t < NS; ++t) {
      if (t < NMF)
        acc[t / NJ % MW][t % NJ] =
            __builtin_amdgcn_mfma_f32_32x32x16_bf16(qb[t % NJ], qa[t / NJ % MW], acc[t / NJ % MW][t % NJ], 0, 0, 0);
      if (t < NRD) READ(pa, pb, t, next, 0);
#pragma unroll
      for (int c = 0; c < NL; ++c)
        if (c * NS / NL == t) COPY(c, buf);
      __builtin_amdgcn_sched_barrier(0);
    }
    NEXT_STAGE();
    buf = nbuf;
  }
#undef COPY
#undef NEXT_STAGE
#undef READ
  // the epilogue writes LDS: every wave's copies have landed and its reads are done
  wait_copies_and_sync<0>();
}

// Row within the tile that this lane holds of accumulator block i, and the first of the four
// consecutive columns, within block j, of its elements 4 v .. 4 v + 3.
template <int MI, bool DUAL>
__device__ __forceinline__ int lane_row(int i) {
  return TileShape<MI, DUAL>::first_row() + i * 32 + (threadIdx.x & 31);
}
__device__ __forceinline__ int lane_col(int v) {
  return v * 8 + ((threadIdx.x & 63) >> 5) * 4;
}

// 32 rows x COLS columns of bf16 from this wave's accumulators to memory.  put(j, v) gives the
// four values of column block j, elements 4 v .. 4 v + 3, as packed bf16.  The LDS rows are padded
// by 16 bytes, which spreads the 16 rows of a write over all banks.  out: the block's first row
// and column; rows, cols: how many exist (cols a multiple of 8).
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
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  const int c = (lane % LANES) * 8;
#pragma unroll
  for (int i = 0; i < 32 / PER; ++i) {
    const int r = i * PER + lane / LANES;
    const u32x4 d = *reinterpret_cast<lds_u32x4*>(mine + r * PITCH + c * 2);
    if (r < rows && c < cols) *reinterpret_cast<u32x4*>(out + r * ld + c) = d;
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ u32x2 pack4(float a, float b, float c, float d) {
  return u32x2{f32_to_bf16(a) | (static_cast<uint32_t>(f32_to_bf16(b)) << 16),
               f32_to_bf16(c) | (static_cast<uint32_t>(f32_to_bf16(d)) << 16)};
}

}  // namespace moe
