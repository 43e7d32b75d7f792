// A product of one workgroup, C[m][n] = sum_k A(m, k) B(n, k) into fp32 accumulators, for operands whose
// rows both run along the depth: bf16 values, or e4m3 values with a scale for each 32 of them (mx.h).
// 256 x 256 tiles of four waves in the shapes of mfma_tile.h; depth is counted in bytes of a row.
//
// * Stages of 128 bytes, two in LDS (64 KB each).  A copy instruction takes 128 bytes of 8 rows: a
//   whole cache line a row.  Measured on copies alone, lines in L2: 23.6 TB/s over the chip, against
//   13.8 where a stage takes half a line of 16 rows (the other half is evicted from L1 before its stage).
// * Half a stage is 64 bytes of depth, four chunks of 16.  A lane l holds row l % 32 and, with h = l / 32,
//   chunks h and 2 + h.  bf16: each chunk is eight values of one of two MFMAs (32x32x16).  8 bits: both
//   go into one (32x32x64), which takes the scale of chunks 0 and 1 from the lanes with h = 0 and that
//   of chunks 2 and 3 from the others.  Exact 8 bits: each chunk is expanded to two bf16 operands.
// * LDS holds a row's eight chunks permuted by (row / 2) % 8, so that the 16 rows that a quarter wave
//   reads lie in different banks.
// * The fragments of the next half are read from LDS while the MFMAs of this one issue.  A first half
//   begins with the reads of the second half's fragments; past a barrier everybody has read the whole
//   stage, and the copies of the stage after next into its buffer begin.  They are spread over 32 slots
//   of an MFMA: a copy's issue takes the time of several instructions, and where two come together
//   the MFMA pipe runs dry.  In the second half a barrier waits for the next stage's copies; behind it
//   come the reads of that stage's first half.  (8 bits, 65536 rows of 7168 x 4096: copies over 7
//   slots 1.81 ms, 12 1.75, 17 1.66, 26 and more 1.57.)
// * Scales go to LDS 16 bytes a row (four stages) at a time, four stages ahead, and to registers
//   eight bytes (two stages) at a time.  A lane shifts its block's byte to a word's bytes 0 and 2, one
//   for each half of the stage, and the MFMA picks one.
//
// Measured on random values, 65536 rows of 32 experts of 7168 x 4096, 8 bits: 1.57 ms, 2450 TFLOP/s (all
// zeros, which cost less power, 1.34 ms); a large library product reaches 3000 with one scale a matrix
// and 1200 with scales like these.
#pragma once

#include "mfma_tile.h"
#include "mx.h"

namespace moe {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

// kMx: the 8-bit MFMA, whose sums of eight products are cut below 2^-13 of the largest of them, for outputs
// that bf16 rounds 60 times as much; kMxExact: f32 sums of exact products, for f32 outputs, at half the rate
// (65536 rows of 32 experts of 2048 x 7168 907 / 1694 us).
enum class Kind { kBf16, kMx, kMxExact };
constexpr int value_bytes(Kind k) { return k == Kind::kBf16 ? 2 : 1; }

constexpr int kRowBytes = 128;                     // of a row and stage
constexpr int kRowOperand = 256 * kRowBytes;       // of an operand's stage
constexpr int kRowStage = 2 * kRowOperand;
constexpr int kScaleBytes = 256 * 16;              // of an operand's scales, four stages
constexpr int kScaleAt = 2 * kRowStage;            // behind two stages: two buffers of two operands
// 128 KB; 8 bits, with the scales and a place for nothing, 152 KB
constexpr int row_tile_lds(Kind k) { return kScaleAt + (k == Kind::kBf16 ? 0 : 3 * 2 * kScaleBytes); }

// acc += A B^T for 32 rows of each: 64 e4m3 values with scales in bytes OP of sa and sb, or 16 bf16 ones.
// In assembly: with the builtins the compiler of this loop keeps more than it has registers for (132 of
// them go to memory).  The wait states: two after a vector write of an operand.  The addend may be
// the result of the MFMA before (the same registers need no wait).
template <int OP>
__device__ __forceinline__ void mfma(floatx16& acc, const i32x8& a, int sa, const i32x8& b, int sb) {
  static_assert(OP == 0 || OP == 2, "the byte is named in the instruction");
  if constexpr (OP == 0)
    asm volatile("s_nop 1\n\tv_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0]"
                 : "+a"(acc) : "v"(a), "v"(b), "v"(sa), "v"(sb));
  else
    asm volatile("s_nop 1\n\tv_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[1,1,0]"
                 : "+a"(acc) : "v"(a), "v"(b), "v"(sa), "v"(sb));
}
__device__ __forceinline__ void mfma(floatx16& acc, const i32x4& a, const i32x4& b) {
  asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}
// Between the last of these and a read of their results other than as an addend: 32 wait states, where
// the longest MFMA asks for 19.
__device__ __forceinline__ void mfma_done(floatx16& acc) {
  asm volatile("s_nop 15\n\ts_nop 15" : "+a"(acc));
}

// Sixteen e4m3 values times 2^(byte - 127) as bf16, which holds them exactly (from byte 3 on: an element has
// steps of 2^-9, and bf16's subnormals steps of 2^-133): two MFMA operands.
__device__ __forceinline__ void expand(const i32x4& v, uint32_t byte, i32x4 (&out)[2]) {
  const float scale = __uint_as_float(byte << 23);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    out[i / 2][i % 2 * 2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], scale, false));
    out[i / 2][i % 2 * 2 + 1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], scale, true));
  }
}

__device__ __forceinline__ uint64_t uniform(const void* p) {
  const uint64_t at = reinterpret_cast<uint64_t>(p);
  return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at))) |
         static_cast<uint64_t>(static_cast<uint32_t>(
             __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at >> 32)))) << 32;
}

// Four bytes per lane from buffer r + voff to LDS at `lds` + OFF + 4 lane.
template <int OFF>
__device__ __forceinline__ void copy_word_to_lds(u32x4 r, uint32_t voff, uint32_t lds) {
  asm volatile(
      "s_add_u32 m0, %0, %3\n\t"
      "s_nop 0\n\t"
      "buffer_load_dword %1, %2, 0 offen lds" ::"s"(lds), "v"(voff), "s"(r), "n"(OFF)
      : "memory", "scc");
}

// Where a product is in its depth: pieces of STEP bytes of a row, from `start` on and around its end.
template <int STEP>
struct Depth {
  int bytes, at, todo;  // of a row; the piece to issue next; pieces still to be issued
  __device__ __forceinline__ void init(int row, int start) {
    bytes = row;
    at = start;
    todo = (row + STEP - 1) / STEP;
  }
  // Bytes of a row from the piece on: what lies past them is not there.
  __device__ __forceinline__ int left() const { return todo > 0 ? bytes - at : 0; }
  __device__ __forceinline__ void next() {
    at = at + STEP >= bytes ? 0 : at + STEP;
    --todo;
  }
};

// How an operand's scales are copied: a lane a row.
struct ScaleRows {
  uint64_t base;   // wave-uniform
  Depth<16> depth;
  uint32_t voff;   // this lane's row, kOutside for none

  template <typename Src>
  __device__ __forceinline__ void init(const uint8_t* p, int64_t pitch, int start, Src src) {
    base = uniform(p);
    depth.init(static_cast<int>(pitch), start);
    const int r = src(threadIdx.x);
    voff = r < 0 ? kOutside : static_cast<uint32_t>(r * pitch);
  }
  template <int OFF>
  __device__ __forceinline__ void copy(uint32_t lds, bool live) {
    const uint64_t at = base + depth.at;
    const u32x4 r = {static_cast<uint32_t>(at), static_cast<uint32_t>(at >> 32), kOutside, 0x00020000u};
    copy_to_lds<OFF>(r, live && depth.left() > 0 ? voff : kOutside, lds);
    const Depth<16> now = depth;
    depth.next();
    depth.at = live ? depth.at : now.at;
    depth.todo = live ? depth.todo : now.todo;
  }
};

// One operand: how its stages are copied.
template <int ROWS>
struct RowOperand {
  static constexpr int N = ROWS / 32;  // copies per wave and stage, of 8 rows each
  uint64_t base;     // wave-uniform
  Depth<kRowBytes> depth;
  uint32_t voff[N];  // this lane's offset in each copy, kOutside for what does not exist
  int k_at;          // this lane's byte of a stage

  // Tile row r is at p + src(r) * bytes, src(r) < 0 for none.
  template <typename Src>
  __device__ __forceinline__ void init(const char* p, int bytes, int start, Src src) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    base = uniform(p);
    depth.init(bytes, start);
    k_at = ((lane & 7) ^ ((wave & 1) * 4 + (lane >> 4))) * 16;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = src((i * 4 + wave) * 8 + (lane >> 3));
      voff[i] = r < 0 ? kOutside : static_cast<uint32_t>(static_cast<int64_t>(r) * bytes + k_at);
    }
  }
  // Copy I of the next stage to LDS offset OFF (the operand's stage buffer); lds is this wave's place:
  // the tile's LDS + wave * 1024.  Past the depth it copies zeros.
  template <int I, int OFF>
  __device__ __forceinline__ void copy(uint32_t lds) const {
    const uint64_t at = base + depth.at;
    const u32x4 r = {static_cast<uint32_t>(at), static_cast<uint32_t>(at >> 32), kOutside, 0x00020000u};
    copy_to_lds<OFF + I * 4096>(r, k_at < depth.left() ? voff[I] : kOutside, lds);
  }
};

template <Kind KIND, int MI>
struct RowProduct {
  static constexpr bool SCALES = KIND != Kind::kBf16;
  using S = TileShape<256, MI, false>;
  using OA = RowOperand<S::ROWS>;
  using OB = RowOperand<S::TN>;
  static constexpr int MW = S::MW, NJ = S::NJ;
  static constexpr int NA = OA::N, NL = NA + OB::N;   // copies per wave and stage
  static constexpr int NMF = MW * NJ, NF = MW + NJ;   // MFMAs and fragments of half a stage
  static constexpr int NS = NMF > NF ? NMF : NF;      // slots
  static constexpr int FREE = NS >= 8 ? NS * 5 / 16 + 1 : NS - 1;            // slots of the first half up to its barrier
  static constexpr int READ = NS >= 8 ? FREE - 1 : FREE;                    // and of its reads
  static constexpr int LAND = NS >= 8 ? NS * 9 / 16 : 1;                    // slots of the second half up to its barrier
  static constexpr int BEFORE = NS - FREE;                                  // and of the first behind its own
  static constexpr int SPREAD = BEFORE + NS + (NS >= 8 ? FREE : 0);         // slots over which a stage's copies go
  static constexpr int slot_of(int copy) { return copy * SPREAD / NL; }
  static constexpr int issued(int slots) {
    int n = 0;
    for (int c = 0; c < NL; ++c) n += slot_of(c) < slots ? 1 : 0;
    return n;
  }
  static constexpr int ISSUED = issued(BEFORE + LAND);  // of a stage's copies, where the one before it has to be there
  static constexpr int EARLY = issued(BEFORE + NS);     // and before the first half of the stage before it
  OA& A;
  OB& B;
  ScaleRows& SA;
  ScaleRows& SB;
  floatx16 (&acc)[MW][NJ];
  uint32_t lds_c, lds_s;  // where this wave's copies go: data, scales
  int at_a[2][2][2], at_b[2][2][2];  // where this lane's rows are: stage buffer, half of the stage, chunk of the two
  int at_sa, at_sb;  // where this lane's rows' scales are in the first buffer
  int next_word;     // bytes from there to the words of the next two stages
  int shift;
  i32x8 p[NF], q[NF];
  i32x2 words[NF];  // scales of two stages
  int sc[NF];       // and of one, from this lane's block on, or (kMxExact) of half a one
  i32x4 xa[2][4], xb[NJ][4];  // kMxExact: expanded fragments, A's of this row of MFMAs and of the next

  template <int C, int BUF>
  __device__ __forceinline__ void copy() {
    if constexpr (C < NA) A.template copy<C, BUF * kRowStage>(lds_c);
    else B.template copy<C - NA, BUF * kRowStage + kRowOperand>(lds_c);
  }
  __device__ __forceinline__ void next_stage() {
    A.depth.next();
    B.depth.next();
  }
  // The next group's scales to `to` bytes from the first buffer; live: otherwise zeros, and it stays the next.
  __device__ __forceinline__ void copy_scales(uint32_t to, bool live) {
    SA.template copy<0>(lds_s + to, live);
    SB.template copy<kScaleBytes>(lds_s + to, live);
  }
  // Fragment f (A's first) of half h of stage buffer buf.
  __device__ __forceinline__ i32x8 fragment(int f, int buf, int h) const {
    typedef const __attribute__((address_space(3))) i32x4 lds_i32x4;
    i32x4 c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = f < MW ? at_a[buf][h][i] + f * 32 * kRowBytes : at_b[buf][h][i] + (f - MW) * 32 * kRowBytes;
      c[i] = *reinterpret_cast<lds_i32x4*>(static_cast<uintptr_t>(at));
    }
    return __builtin_shufflevector(c[0], c[1], 0, 1, 2, 3, 4, 5, 6, 7);
  }
  // The words of two stages' scales of fragment f.
  __device__ __forceinline__ i32x2 scales(int f, int at) const {
    typedef const __attribute__((address_space(3))) i32x2 lds_i32x2;
    return *reinterpret_cast<lds_i32x2*>(static_cast<uintptr_t>((f < MW ? at_sa + f * 512 : at_sb + (f - MW) * 512) + at));
  }

  // kMxExact: chunk c of fragment f expanded.
  __device__ __forceinline__ void expand_chunk(const i32x8 (&cur)[NF], int f, int c, i32x4 (&to)[4]) const {
    const i32x4 v = c == 0 ? __builtin_shufflevector(cur[f], cur[f], 0, 1, 2, 3)
                           : __builtin_shufflevector(cur[f], cur[f], 4, 5, 6, 7);
    i32x4 two[2];
    expand(v, static_cast<uint32_t>(sc[f]) >> c * 8 & 0xff, two);
    to[2 * c] = two[0];
    to[2 * c + 1] = two[1];
  }

  // Half J % 2 of stage J / 2 of two, MFMA by MFMA: beside each the reads, copies and barriers that the
  // head of this file tells of.
  template <int J>
  __device__ __forceinline__ void half(i32x8 (&cur)[NF], i32x8 (&nxt)[NF]) {
    constexpr bool SECOND = J % 2;
    constexpr int BUF = J / 2, OP = SECOND ? 2 : 0;
    constexpr int FROM = SECOND ? LAND : 0, TO = SECOND ? NS : READ;  // slots of the reads
    constexpr int READS = SCALES && J == 3 ? 2 * NF : NF;  // fragments, then the next two stages' scales
    if constexpr (KIND == Kind::kMx && !SECOND) {
#pragma unroll
      for (int f = 0; f < NF; ++f) sc[f] = static_cast<uint32_t>(words[f][BUF]) >> shift;
    }
    if constexpr (KIND == Kind::kMxExact) {
#pragma unroll
      for (int f = 0; f < NF; ++f) sc[f] = static_cast<uint32_t>(words[f][BUF]) >> J % 2 * 16;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        expand_chunk(cur, 0, c, xa[0]);
#pragma unroll
        for (int j = 0; j < NJ; ++j) expand_chunk(cur, MW + j, c, xb[j]);
      }
    }
    each<0, NS>([&](auto slot) {
      constexpr int t = decltype(slot)::value;
      if constexpr (SECOND && t == LAND) {
        wait_copies_and_sync<ISSUED>();  // newer than the next stage's copies: some of the stage after it
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (!SECOND && t == FREE) {
        wait_copies_and_sync<63>();
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (t < NMF) {
        constexpr int i = t / NJ, j = t % NJ;
        // the transposed block
        if constexpr (KIND == Kind::kMx) {
          mfma<OP>(acc[i][j], cur[MW + j], sc[MW + j], cur[i], sc[i]);
        } else if constexpr (KIND == Kind::kBf16) {
          mfma(acc[i][j], __builtin_shufflevector(cur[MW + j], cur[MW + j], 0, 1, 2, 3),
               __builtin_shufflevector(cur[i], cur[i], 0, 1, 2, 3));
          mfma(acc[i][j], __builtin_shufflevector(cur[MW + j], cur[MW + j], 4, 5, 6, 7),
               __builtin_shufflevector(cur[i], cur[i], 4, 5, 6, 7));
        } else {
          each<0, 4>([&](auto c) { mfma(acc[i][j], xb[j][decltype(c)::value], xa[i % 2][decltype(c)::value]); });
          // the next row's A beside the first two columns of this one
          if constexpr (i + 1 < MW && j < 2) expand_chunk(cur, i + 1, j, xa[(i + 1) % 2]);
        }
      }
      each<0, READS>([&](auto r) {
        constexpr int R = decltype(r)::value;
        if constexpr (FROM + R * (TO - FROM) / READS == t) {
          if constexpr (R < NF) nxt[R] = fragment(R, SECOND ? 1 - BUF : BUF, SECOND ? 0 : 1);
          else words[R - NF] = scales(R - NF, next_word);
        }
      });
      // slots since the buffer that is being filled was free: this stage's, or before that the other
      constexpr bool OTHER = !SECOND && t < FREE;
      constexpr int u = OTHER ? BEFORE + NS + t : SECOND ? BEFORE + t : t - FREE;
      each<0, NL>([&](auto c) {
        if constexpr (slot_of(decltype(c)::value) == u) copy<decltype(c)::value, OTHER ? 1 - BUF : BUF>();
      });
      if constexpr (OTHER && t == FREE - 1) next_stage();
      __builtin_amdgcn_sched_barrier(0);
    });
  }
  template <int J>
  __device__ __forceinline__ void turn() {
    if constexpr (J % 2 == 0) half<J>(p, q);
    else half<J>(q, p);
  }

  // bytes: of a row's depth
  __device__ __forceinline__ void run(int bytes, lds_char* smem) {
#pragma unroll
    for (int i = 0; i < MW; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    const int lds = static_cast<int>(reinterpret_cast<uintptr_t>(smem));
    const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int chunk = ((4 * h + 2 * i + (lane >> 5)) ^ ((lane >> 1) & 7)) * 16;
          at_a[b][h][i] = lds + b * kRowStage + (S::first_row() + (lane & 31)) * kRowBytes + chunk;
          at_b[b][h][i] = lds + b * kRowStage + kRowOperand + (S::first_col() + (lane & 31)) * kRowBytes + chunk;
        }
    lds_c = lds + S::wave() * 1024;
    lds_s = lds + kScaleAt + S::wave() * 1024;
    at_sa = lds + kScaleAt + (S::first_row() + (lane & 31)) * 16;
    at_sb = lds + kScaleAt + kScaleBytes + (S::first_col() + (lane & 31)) * 16;
    shift = (lane >> 5) * 8;
    if constexpr (SCALES) copy_scales(0, true);
    // the stages past the last are copied too, as zeros: the copies in flight stay countable
    each<0, NL>([&](auto c) { copy<decltype(c)::value, 0>(); });
    next_stage();
    each<0, EARLY>([&](auto c) { copy<decltype(c)::value, 1>(); });
    wait_copies_and_sync<EARLY>();
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      p[f] = fragment(f, 0, 0);
      if constexpr (SCALES) words[f] = scales(f, 0);
    }
    int halves = (bytes + 63) / 64;
    // The words of two stages are the first or second half of a row's 16 bytes.  With the first, the
    // other buffer's last words were read a stage ago and its next are three away: it takes the next
    // group.  With the second, zeros go to a place that nobody reads, as a branch around the copies
    // would cost the compiler a second set of accumulators.
    int word = 0;
    next_word = 8;
    for (; halves >= 4; halves -= 4) {
      if constexpr (SCALES) {
        const bool first = !(word & 8);
        copy_scales(first ? (word ? 0 : 2 * kScaleBytes) : 4 * kScaleBytes, first);
      }
      each<0, 4>([&](auto j) { turn<decltype(j)::value>(); });
      word = next_word;
      next_word = (word & 8) ? (word ^ 2 * kScaleBytes) - 8 : word + 8;
    }
    each<0, 3>([&](auto j) {
      if (halves > decltype(j)::value) turn<decltype(j)::value>();
    });
#pragma unroll
    for (int i = 0; i < MW; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) mfma_done(acc[i][j]);
    // the epilogue writes LDS: every wave's copies have landed and its reads are done
    wait_copies_and_sync<0>();
  }
};

// A tile of 32 MW rows (MW = 1 or 2) by 64 columns for products that have too few of the tiles above to
// fill the CUs: what bounds them is latency, so each of the four waves has the whole tile, every
// fourth stage of its depth and two stages of its own in LDS, and waits for nobody until the four sums
// are added in wave order.
template <Kind KIND, int MW>
struct SplitProduct {
  static constexpr bool SCALES = KIND != Kind::kBf16;
  static constexpr int NJ = 2, NA = MW * 4, NB = NJ * 4, NL = NA + NB + (SCALES ? 2 : 0);  // copies of a stage
  static constexpr int STAGE = 2 * 64 * kRowBytes, SCALE_STAGE = 2 * 256;
  static constexpr int WAVE = 2 * STAGE;                                  // LDS of a wave, 32 KB
  static constexpr int LDS = 4 * WAVE + (SCALES ? 4 * 2 * SCALE_STAGE : 0);
  uint64_t a, b, as, bs;       // wave-uniform: where a row's next stage of this wave starts, and its scales
  int left;                    // bytes of a row from there on
  uint32_t va[NA], vb[NB], vas, vbs;
  int k_at;

  // As for RowOperand; tile rows and columns below 64.
  template <typename Row, typename Col>
  __device__ __forceinline__ void init(const char* A, const char* B, const uint8_t* SA, const uint8_t* SB, int bytes,
                                       int64_t pitch, Row row, Col col) {
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    a = uniform(A) + wave * kRowBytes;
    b = uniform(B) + wave * kRowBytes;
    as = uniform(SA) + wave * 4;
    bs = uniform(SB) + wave * 4;
    left = bytes - wave * kRowBytes;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      // copy i takes rows 8 i .. +7, chunks permuted by (row / 2) % 8
      const int r = i * 8 + (lane >> 3);
      if (i == 0) k_at = ((lane & 7) ^ (lane >> 4)) * 16;
      const int k = k_at ^ (i & 1) * 64;
      const int c = col(r);
      vb[i] = c < 0 ? kOutside : static_cast<uint32_t>(static_cast<int64_t>(c) * bytes + k);
      if (i < NA) {
        const int s = row(r);
        va[i % NA] = s < 0 ? kOutside : static_cast<uint32_t>(static_cast<int64_t>(s) * bytes + k);
      }
    }
    if constexpr (SCALES) {
      const int s = lane < MW * 32 ? row(lane) : -1, c = col(lane);
      vas = s < 0 ? kOutside : static_cast<uint32_t>(s * pitch);
      vbs = c < 0 ? kOutside : static_cast<uint32_t>(c * pitch);
    }
  }

  static __device__ __forceinline__ u32x4 buffer(uint64_t at) {
    return u32x4{static_cast<uint32_t>(at), static_cast<uint32_t>(at >> 32), kOutside, 0x00020000u};
  }
  // This wave's next stage to its buffer BUF; past the depth zeros.
  template <int BUF>
  __device__ __forceinline__ void copy(uint32_t lds, uint32_t lds_s) {
    const bool even = k_at < left, odd = (k_at ^ 64) < left;  // the two orders of chunks
    each<0, NB>([&](auto i) {
      constexpr int I = decltype(i)::value;
      const bool in = I % 2 ? odd : even;
      if constexpr (I < NA) copy_to_lds<BUF * STAGE + I * 1024>(buffer(a), in ? va[I % NA] : kOutside, lds);
      copy_to_lds<BUF * STAGE + 64 * kRowBytes + I * 1024>(buffer(b), in ? vb[I] : kOutside, lds);
    });
    if constexpr (SCALES) {
      copy_word_to_lds<BUF * SCALE_STAGE>(buffer(as), left > 0 ? vas : kOutside, lds_s);
      copy_word_to_lds<BUF * SCALE_STAGE + 256>(buffer(bs), left > 0 ? vbs : kOutside, lds_s);
    }
    a += 4 * kRowBytes;
    b += 4 * kRowBytes;
    as += 16;
    bs += 16;
    left -= 4 * kRowBytes;
  }

  template <int BUF>
  __device__ __forceinline__ void stage(floatx16 (&acc)[MW][NJ], int mine, int mine_s) {
    typedef const __attribute__((address_space(3))) i32x4 lds_i32x4;
    typedef const __attribute__((address_space(3))) uint32_t lds_u32;
    const int lane = threadIdx.x & (kWave - 1);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(NL) : "memory");
    i32x4 f[MW + NJ][4];
    uint32_t sc[MW + NJ];
#pragma unroll
    for (int q = 0; q < MW + NJ; ++q) {
      const int at = mine + BUF * STAGE + (q < MW ? q * 32 : 64 + (q - MW) * 32) * kRowBytes + (lane & 31) * kRowBytes;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        f[q][c] = *reinterpret_cast<lds_i32x4*>(
            static_cast<uintptr_t>(at + ((2 * c + (lane >> 5)) ^ ((lane >> 1) & 7)) * 16));
      if constexpr (SCALES)
        sc[q] = *reinterpret_cast<lds_u32*>(static_cast<uintptr_t>(
            mine_s + BUF * SCALE_STAGE + (q < MW ? q * 32 : 64 + (q - MW) * 32) * 4 + (lane & 31) * 4));
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    copy<BUF>(lds_d, lds_sc);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (KIND == Kind::kMx) {
#pragma unroll
        for (int i = 0; i < MW; ++i)
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const i32x8 x = __builtin_shufflevector(f[i][2 * h], f[i][2 * h + 1], 0, 1, 2, 3, 4, 5, 6, 7);
            const i32x8 w = __builtin_shufflevector(f[MW + j][2 * h], f[MW + j][2 * h + 1], 0, 1, 2, 3, 4, 5, 6, 7);
            const int own = (lane >> 5) * 8 + 16 * h;  // this lane's block's byte
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                w, x, acc[i][j], 0, 0, 0, static_cast<int>(sc[MW + j] >> own), 0, static_cast<int>(sc[i] >> own));
          }
      } else {
        constexpr int N = KIND == Kind::kBf16 ? 1 : 2;  // MFMAs a chunk
        i32x4 x[MW + NJ][2 * N];
#pragma unroll
        for (int q = 0; q < MW + NJ; ++q)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if constexpr (N == 1) {
              x[q][c] = f[q][2 * h + c];
            } else {
              i32x4 two[2];
              expand(f[q][2 * h + c], sc[q] >> (16 * h + 8 * c) & 0xff, two);
              x[q][2 * c % (2 * N)] = two[0];
              x[q][(2 * c + 1) % (2 * N)] = two[1];
            }
          }
#pragma unroll
        for (int c = 0; c < 2 * N; ++c)
#pragma unroll
          for (int i = 0; i < MW; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x[MW + j][c]),
                                                                 __builtin_bit_cast(bf16x8, x[i][c]), acc[i][j], 0, 0, 0);
      }
    }
  }

  uint32_t lds_d, lds_sc;  // this wave's places

  // bytes: of a row's depth.  put(row, column, sums): four consecutive columns of a row of the tile.
  template <typename Put>
  __device__ __forceinline__ void run(int bytes, lds_char* smem, Put put) {
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    floatx16 acc[MW][NJ];
#pragma unroll
    for (int i = 0; i < MW; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    const int lds = static_cast<int>(reinterpret_cast<uintptr_t>(smem));
    lds_d = lds + wave * WAVE;
    lds_sc = lds + 4 * WAVE + wave * 2 * SCALE_STAGE;
    const int mine = static_cast<int>(lds_d), mine_s = static_cast<int>(lds_sc);
    copy<0>(lds_d, lds_sc);
    copy<1>(lds_d, lds_sc);
    // every wave makes the same number of turns; stages past the depth add zeros
    const int stages = (bytes + 4 * kRowBytes - 1) / (4 * kRowBytes);
    for (int s = 0; s < stages; s += 2) {
      stage<0>(acc, mine, mine_s);
      stage<1>(acc, mine, mine_s);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    typedef __attribute__((address_space(3))) floatx4 lds_floatx4;
    lds_floatx4* sums = reinterpret_cast<lds_floatx4*>(smem);  // [wave][block][quarter][lane]: own buffers first
#pragma unroll
    for (int i = 0; i < MW; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          sums[wave * (WAVE / 16) + ((i * NJ + j) * 4 + v) * kWave + lane] =
              floatx4{acc[i][j][v * 4], acc[i][j][v * 4 + 1], acc[i][j][v * 4 + 2], acc[i][j][v * 4 + 3]};
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MW; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const lds_floatx4* p = sums + ((i * NJ + j) * 4 + wave) * kWave + lane;
        const floatx4 s = (p[0] + p[WAVE / 16]) + (p[2 * (WAVE / 16)] + p[3 * (WAVE / 16)]);
        put(i * 32 + (lane & 31), j * 32 + lane_col(wave), s);
      }
  }
};

}  // namespace moe
