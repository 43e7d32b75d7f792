// 8-bit rows with block scales (the OCP microscaling format MXFP8, e4m3): 32 consecutive values of a
// row share a scale 2^s, kept as the byte s + 127, and are held as e4m3(v / 2^s).  s is the smallest
// whole number with max |v| <= 448 * 2^s, 448 = 1.75 * 2^8 being the largest e4m3 value, so that no
// value saturates; a block of zeros has scale byte 0.  A value that is not finite becomes NaN and the
// block's scale is that of its finite values.
#pragma once

#include "common.h"

namespace moe {

constexpr int kMxBlock = 32;
constexpr int kMxUnit = 512;  // values of a row whose scales are 16 bytes: what a wave handles at once

inline bool is_dtype(moe_dtype dt) { return dt == MOE_F32 || dt == MOE_BF16; }

// Bytes of a row's scales.
__host__ __device__ __forceinline__ int64_t mx_pitch(int64_t cols) { return (cols + kMxUnit - 1) / kMxUnit * 16; }

#define MX_DPP(v, CTRL) static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, true))

// The lane's eight values v (a quarter of a block: lanes 4 i .. 4 i + 3 hold one) as eight e4m3 bytes.
// *word: the scale bytes of the 16 lanes' four blocks, the same in each of them.  All lanes of the
// wave call this.  The exchanges stay on the data path between lanes.
__device__ __forceinline__ void mx_pack(const float (&v)[8], uint32_t (&bytes)[2], uint32_t* word) {
  constexpr uint32_t kInf = 0x7f800000u;
  float f[8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[i] = v[i];
    top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);  // as whole numbers, floats keep their order
  }
  top = max(top, MX_DPP(top, 0xb1));  // lanes 1 0 3 2
  top = max(top, MX_DPP(top, 0x4e));  // lanes 2 3 0 1
  if (__any(top >= kInf)) {
    top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t a = __float_as_uint(v[i]) & 0x7fffffffu;
      if (a < kInf) top = max(top, a);
      else f[i] = __uint_as_float(0x7fc00000u);
    }
    top = max(top, MX_DPP(top, 0xb1));
    top = max(top, MX_DPP(top, 0x4e));
  }
  // top = 1.m * 2^(e - 127); one more where 1.m > 1.75
  const int byte = max(static_cast<int>(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0), 0);
  // 2^(127 - byte): byte is 247 at most, so this is a normal number
  const float inv = __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);
  int b = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    b = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h] * inv, f[4 * h + 1] * inv, b, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h + 2] * inv, f[4 * h + 3] * inv, b, true);
    bytes[h] = static_cast<uint32_t>(b);
  }
  uint32_t w = static_cast<uint32_t>(byte) << (threadIdx.x & 12) * 2;  // 8 (lane / 4 % 4)
  w |= MX_DPP(w, 0x124);  // the row of 16 lanes turned by 4
  w |= MX_DPP(w, 0x128);  // and by 8
  *word = w;
}

// The same for eight columns at `at` (a multiple of 8) of a row of `cols`, stored: q the row's values,
// scales its mx_pitch(cols) bytes.  Consecutive lanes hold consecutive eights, and a wave starts at a
// multiple of 512; lanes past the row hold zeros.  A wave that starts past the row stores nothing.
__device__ __forceinline__ void mx_store(const float (&v)[8], int64_t at, int cols, uint8_t* q,
                                         uint8_t* scales) {
  typedef uint32_t u32x2_a8 __attribute__((ext_vector_type(2), aligned(8)));
  uint32_t bytes[2], word;
  mx_pack(v, bytes, &word);
  if (at < cols) __builtin_nontemporal_store(u32x2_a8{bytes[0], bytes[1]}, reinterpret_cast<u32x2_a8*>(q + at));
  const int lane = threadIdx.x & (kWave - 1);
  if ((lane & 15) == 0 && at - lane * 8 < cols)
    *reinterpret_cast<uint32_t*>(scales + at / (4 * kMxBlock) * 4) = word;
}

#undef MX_DPP

}  // namespace moe
