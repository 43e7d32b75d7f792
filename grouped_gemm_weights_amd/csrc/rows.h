// Row access shared by the bandwidth-bound kernels (layer norm, combine and permute
// gradients): eight consecutive elements of a row per lane, converted to fp32, at whatever
// alignment the row has.
#pragma once

#include "common.h"

namespace moe {

// Rows start at any element (H need not be a multiple of anything), so the vector types claim
// the alignment of one element only.  gfx950 loads and stores 16 bytes at any such address in
// one instruction.
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

constexpr int kVec = 8;             // elements per lane and step
constexpr int kMaxRow = 1 << 28;    // longest row: column indices stay in 31 bits

// Eight elements as they lie in memory: a row's loads can be in flight before they are unpacked.
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  uint32_t w[4];
};
template <>
struct Raw8<float> {
  float w[8];
};

// Elements [8 v, 8 v + 8) of a row of n elements; elements past n read as zero.  NT: a
// non-temporal load, for rows that are read exactly once.
template <bool NT>
__device__ __forceinline__ void load_raw(const uint16_t* row, int64_t v, int n, Raw8<uint16_t>& out) {
  const int64_t at = v * kVec;
  if (at + kVec <= n) {
    const u32x4_a2* p = reinterpret_cast<const u32x4_a2*>(row + at);
    const u32x4_a2 b = NT ? __builtin_nontemporal_load(p) : *p;
#pragma unroll
    for (int i = 0; i < 4; ++i) out.w[i] = b[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = at + 2 * i < n ? row[at + 2 * i] : 0;
      const uint32_t hi = at + 2 * i + 1 < n ? row[at + 2 * i + 1] : 0;
      out.w[i] = lo | hi << 16;
    }
  }
}

template <bool NT>
__device__ __forceinline__ void load_raw(const float* row, int64_t v, int n, Raw8<float>& out) {
  const int64_t at = v * kVec;
  if (at + kVec <= n) {
    const f32x4_a4* p = reinterpret_cast<const f32x4_a4*>(row + at);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4_a4 b = NT ? __builtin_nontemporal_load(p + h) : p[h];
#pragma unroll
      for (int i = 0; i < 4; ++i) out.w[4 * h + i] = b[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) out.w[i] = at + i < n ? row[at + i] : 0.f;
  }
}

__device__ __forceinline__ void unpack(const Raw8<uint16_t>& r, float* out) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    out[2 * i] = __uint_as_float(r.w[i] << 16);
    out[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ void unpack(const Raw8<float>& r, float* out) {
#pragma unroll
  for (int i = 0; i < kVec; ++i) out[i] = r.w[i];
}

template <bool NT, typename T>
__device__ __forceinline__ void load8(const T* row, int64_t v, int n, float* out) {
  Raw8<T> r;
  load_raw<NT>(row, v, n, r);
  unpack(r, out);
}

template <bool NT>
__device__ __forceinline__ void store8(uint16_t* row, int64_t v, int n, const float* in) {
  const int64_t at = v * kVec;
  if (at + kVec <= n) {
    u32x4_a2 b;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      b[i] = f32_to_bf16(in[2 * i]) | (static_cast<uint32_t>(f32_to_bf16(in[2 * i + 1])) << 16);
    u32x4_a2* p = reinterpret_cast<u32x4_a2*>(row + at);
    if (NT) __builtin_nontemporal_store(b, p);
    else *p = b;
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (at + i < n) row[at + i] = f32_to_bf16(in[i]);
  }
}

template <bool NT>
__device__ __forceinline__ void store8(float* row, int64_t v, int n, const float* in) {
  const int64_t at = v * kVec;
  if (at + kVec <= n) {
    f32x4_a4* p = reinterpret_cast<f32x4_a4*>(row + at);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4_a4 b = {in[4 * h], in[4 * h + 1], in[4 * h + 2], in[4 * h + 3]};
      if (NT) __builtin_nontemporal_store(b, p + h);
      else p[h] = b;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (at + i < n) row[at + i] = in[i];
  }
}

// Sum over the wave, the same in every lane: four adds of lanes 1, 2, 4 and 8 to the left within
// rows of 16 lanes, then row 0's (2's) total into row 1 (3) and the lower half's into the upper, on
// the data path between lanes (a sixth of the latency of six LDS permutes).
__device__ __forceinline__ float wave_sum(float v) {
#define ADD(CTRL, ROWS)                                                                       \
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xf, true))
  ADD(0x111, 0xf);
  ADD(0x112, 0xf);
  ADD(0x114, 0xf);
  ADD(0x118, 0xf);
  ADD(0x142, 0xa);
  ADD(0x143, 0xc);
#undef ADD
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

}  // namespace moe
