// An 8-bit product of one workgroup: C[m][n] = sum_k A(m, k) B(n, k) into fp32 accumulators, for rows of
// e4m3 values with a scale for each 32 of them (mx.h), by the MFMA that takes such scales
// (32x32x64).  The 256 x 256 tile of mfma_tile.h, its shapes, operands and LDS layout: 64 values are
// the 64 bytes that 32 bf16 values are there, so a stage is 64 deep and one MFMA takes all of it.
//
// * An MFMA's lane l holds row l % 32 and, with h = l / 32, the values 16 h .. +16 of each of the stage's
//   two blocks of 32: chunks h and 2 + h of the row's four, as a bf16 stage's two halves are read.
//   The scale of block b is taken from the lanes with h = b.
// * The fragments of stage s + 1 are read from LDS while the MFMAs of stage s issue; past the barrier
//   that opens stage s everybody has read stage s, so its buffer takes stage s + 4.
// * Scales go to LDS 16 bytes a row (eight stages) at a time, eight stages ahead, and to registers a
//   word (two stages) at a time.  A lane shifts its block's byte to the word's bytes 0 and 2, one
//   for each of the two stages, and the MFMA picks one.
#pragma once

#include "mfma_tile.h"
#include "mx.h"

namespace moe {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kMxScaleBytes = 256 * 16;                           // of an operand, eight stages
constexpr int kMxScaleAt = tile_lds(256, false);                  // two buffers of two operands
constexpr int kMxTileLds = kMxScaleAt + 3 * 2 * kMxScaleBytes;    // and a place for nothing: 152 KB

// acc += A B^T for 32 rows of each by 64 values, scales in bytes OP of sa and sb.  In assembly because the
// compiler gives the builtin's result other registers than its addend's, and a tile of 256
// accumulators has no others.  The wait states: two after a vector write of an operand.
// The addend may be the result of the MFMA before (the same registers need no wait).
template <int OP>
__device__ __forceinline__ void mx_mfma(floatx16& acc, const i32x8& a, int sa, const i32x8& b, int sb) {
  static_assert(OP == 0 || OP == 2, "the byte is named in the instruction");
  if constexpr (OP == 0)
    asm volatile("s_nop 1\n\tv_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0]"
                 : "+a"(acc) : "v"(a), "v"(b), "v"(sa), "v"(sb));
  else
    asm volatile("s_nop 1\n\tv_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[1,1,0]"
                 : "+a"(acc) : "v"(a), "v"(b), "v"(sa), "v"(sb));
}
// Between the last of these and a read of their results other than as an addend: 32 wait states, where
// the longest MFMA asks for 19.
__device__ __forceinline__ void mx_mfma_done(floatx16& acc) {
  asm volatile("s_nop 15\n\ts_nop 15" : "+a"(acc));
}

// How an operand's scales are copied: a lane a row.
struct ScaleRows {
  uint64_t base;   // wave-uniform: where the group to issue next starts
  int left;        // bytes of a row from there on
  uint32_t voff;   // this lane's row, kOutside for none

  template <typename Src>
  __device__ __forceinline__ void init(const uint8_t* p, int64_t pitch, Src src) {
    const uint64_t at = reinterpret_cast<uint64_t>(p);
    base = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at))) |
           static_cast<uint64_t>(static_cast<uint32_t>(
               __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at >> 32)))) << 32;
    left = static_cast<int>(pitch);
    const int r = src(threadIdx.x);
    voff = r < 0 ? kOutside : static_cast<uint32_t>(r * pitch);
  }
  template <int OFF>
  __device__ __forceinline__ void copy(uint32_t lds, bool live) {
    const u32x4 r = {static_cast<uint32_t>(base), static_cast<uint32_t>(base >> 32), kOutside, 0x00020000u};
    copy_to_lds<OFF>(r, live && left > 0 ? voff : kOutside, lds);
    base += live ? 16 : 0;
    left -= live ? 16 : 0;
  }
};

template <int MI>
struct MxProduct {
  using S = TileShape<256, MI, false>;
  using OA = Operand<false, S::ROWS>;
  using OB = Operand<false, S::TN>;
  static constexpr int MW = S::MW, NJ = S::NJ, STAGES = tile_stages(256), STAGE = stage_bytes(256, false);
  static constexpr int NA = OA::N, NL = NA + OB::N;   // copies per wave and stage
  static constexpr int NMF = MW * NJ, NF = MW + NJ;   // MFMAs and fragments of a stage
  static constexpr int NRD = 2 * NF;                  // reads of a stage: fragments, then scale words
  static constexpr int NS = NMF > NF ? NMF : NF;      // slots
  OA& A;
  OB& B;
  ScaleRows& SA;
  ScaleRows& SB;
  floatx16 (&acc)[MW][NJ];
  Fragments<false, MW, S::ROWS, STAGES, STAGE> fa;
  Fragments<false, NJ, S::TN, STAGES, STAGE> fb;
  uint32_t lds_a, lds_b, lds_s;
  int at_sa, at_sb;  // where this lane's rows' scales are in the first buffer
  int word, next_word;  // bytes from there to the word of stages 0 and 1 of these four, and of the next four
  int shift;
  i32x8 p[NF], q[NF];
  int sc[NF], next_sc[NF];

  template <int C, int BUF>
  __device__ __forceinline__ void copy() {
    if constexpr (C < NA) A.template copy<C, BUF * STAGE>(lds_a);
    else B.template copy<C - NA, BUF * STAGE + operand_bytes(256)>(lds_b);
  }
  // The next group's scales to `to` bytes from the first buffer; live: otherwise zeros, and it stays the next.
  __device__ __forceinline__ void copy_scales(uint32_t to, bool live) {
    SA.template copy<0>(lds_s + to, live);
    SB.template copy<kMxScaleBytes>(lds_s + to, live);
  }
  // Fragment f (A's first) of stage buffer buf.
  __device__ __forceinline__ i32x8 fragment(int f, int buf) const {
    i32x4 h[2];
#pragma unroll
    for (int s = 0; s < 2; ++s)
      h[s] = __builtin_bit_cast(i32x4, f < MW ? fa.read(buf, f, f * 32, s) : fb.read(buf, f - MW, (f - MW) * 32, s));
    return __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7);
  }
  // The word of two stages' scales of fragment f.
  __device__ __forceinline__ int scales(int f, int word) const {
    typedef const __attribute__((address_space(3))) int lds_int;
    const int at = f < MW ? at_sa + f * 512 : at_sb + (f - MW) * 512;
    return *reinterpret_cast<lds_int*>(static_cast<uintptr_t>(at + word));
  }
  // Stage J of four.
  template <int J>
  __device__ __forceinline__ void stage(i32x8 (&cur)[NF], i32x8 (&nxt)[NF]) {
    constexpr int BUF = J % STAGES, OP = J % 2 * 2;
    constexpr int READS = J % 2 ? NRD : NF;  // the second stage of a pair reads the next one's scales
    wait_copies_and_sync<(STAGES - 2) * NL>();
    if constexpr (J % 2 == 0) {
#pragma unroll
      for (int f = 0; f < NF; ++f) sc[f] = static_cast<uint32_t>(next_sc[f]) >> shift;
    }
    each<0, NS>([&](auto slot) {
      constexpr int t = decltype(slot)::value;
      if constexpr (t < NMF) {
        constexpr int i = t / NJ, j = t % NJ;
        mx_mfma<OP>(acc[i][j], cur[MW + j], sc[MW + j], cur[i], sc[i]);  // the transposed block
      }
      each<0, READS>([&](auto r) {
        constexpr int R = decltype(r)::value;
        if constexpr (R * (NS - NS / 4) / READS == t) {
          if constexpr (R < NF) nxt[R] = fragment(R, (J + 1) % STAGES);
          else next_sc[R - NF] = scales(R - NF, J == 1 ? word + 4 : next_word);
        }
      });
      each<0, NL>([&](auto c) {
        if constexpr (decltype(c)::value * NS / NL == t) copy<decltype(c)::value, BUF>();
      });
      __builtin_amdgcn_sched_barrier(0);
    });
    A.next_stage();
    B.next_stage();
  }
  template <int J>
  __device__ __forceinline__ void turn() {
    if constexpr (J % 2 == 0) stage<J>(p, q);
    else stage<J>(q, p);
  }

  __device__ __forceinline__ void run(int K, lds_char* smem) {
#pragma unroll
    for (int i = 0; i < MW; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    const int lds = static_cast<int>(reinterpret_cast<uintptr_t>(smem));
    const int lane = threadIdx.x & (kWave - 1);
    fa.init(lds, [](int b) { return S::first_row() + b * 32; });
    fb.init(lds + operand_bytes(256), [](int b) { return S::first_col() + b * 32; });
    lds_a = lds + S::wave() * OA::WAVE_STEP;
    lds_b = lds + S::wave() * OB::WAVE_STEP;
    lds_s = lds + kMxScaleAt + S::wave() * 1024;
    at_sa = lds + kMxScaleAt + (S::first_row() + (lane & 31)) * 16;
    at_sb = lds + kMxScaleAt + kMxScaleBytes + (S::first_col() + (lane & 31)) * 16;
    shift = (lane >> 5) * 8;
    copy_scales(0, true);
    // the stages past the last are copied too, as zeros: the copies in flight stay countable
    each<0, STAGES>([&](auto s) {
      constexpr int BUF = decltype(s)::value;
      each<0, NL>([&](auto c) { copy<decltype(c)::value, BUF>(); });
      A.next_stage();
      B.next_stage();
    });
    wait_copies_and_sync<(STAGES - 1) * NL>();
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      p[f] = fragment(f, 0);
      next_sc[f] = scales(f, 0);
    }
    int stages = (K + 63) / 64;
    // The words of four stages are the first or second half of a row's 16 bytes.  With the first, the
    // other buffer's last words were read two stages ago and its next are seven away: it takes the next
    // group.  With the second, zeros go to a place that nobody reads, as a branch around the copies
    // would cost the compiler a second set of accumulators.
    word = 0;
    next_word = 8;
    for (; stages >= 4; stages -= 4) {
      const bool first = !(word & 8);
      copy_scales(first ? (word ? 0 : 2 * kMxScaleBytes) : 4 * kMxScaleBytes, first);
      each<0, 4>([&](auto j) { turn<decltype(j)::value>(); });
      word = next_word;
      next_word = (word & 8) ? (word ^ 2 * kMxScaleBytes) - 8 : word + 8;
    }
    each<0, 3>([&](auto j) {
      if (stages > decltype(j)::value) turn<decltype(j)::value>();
    });
#pragma unroll
    for (int i = 0; i < MW; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) mx_mfma_done(acc[i][j]);
    // the epilogue writes LDS: every wave's copies have landed and its reads are done
    wait_copies_and_sync<0>();
  }
};

}  // namespace moe
