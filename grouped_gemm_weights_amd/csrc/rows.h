// Row access shared by the bandwidth-bound kernels (layer norm, combine and permute
// gradients): eight consecutive elements of a row per lane, converted to fp32, at whatever
// alignment the row has.
#pragma once

#include "common.h"

namespace moe {

// Whether a grid of `blocks` workgroups of `threads` is more than one launch takes (2^32 threads).
inline bool too_many(int64_t blocks, int threads) { return blocks * threads > UINT32_MAX; }

// Rows start at any element (H need not be a multiple of anything), so the vector types claim
// the alignment of one element only.  gfx950 loads and stores 16 bytes at any such address in
// one instruction.
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

constexpr int kCus = 256;
constexpr int kVec = 8;             // elements per lane and step
constexpr int kMaxRow = 1 << 26;    // longest row: grids and column indices stay in range

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

// Elements [8 v, 8 v + 8) of a row of n elements, to be unpacked with the same v and n.  A piece
// that ends past the row is loaded 8 - n % 8 elements early, as one whole vector, and shifted when
// it is unpacked, so that no load waits for another's value.  TAIL = false: n is a multiple of 8,
// and none of that is needed.  NT: a non-temporal load, for rows that are read exactly once.
template <bool NT, bool TAIL>
__device__ __forceinline__ void load_raw(const uint16_t* row, int64_t v, int n, Raw8<uint16_t>& out) {
  const int64_t at = v * kVec;
#pragma unroll
  for (int i = 0; i < 4; ++i) out.w[i] = 0;
  if (!TAIL || n >= kVec) {
    if (at < n) {
      const u32x4_a2* p = reinterpret_cast<const u32x4_a2*>(row + (!TAIL || at + kVec <= n ? at : n - kVec));
      const u32x4_a2 b = NT ? __builtin_nontemporal_load(p) : *p;
#pragma unroll
      for (int i = 0; i < 4; ++i) out.w[i] = b[i];
    }
  } else if (at == 0) {  // a row of fewer than 8: its last element last, as the shift expects
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (i >= kVec - n) out.w[i / 2] |= static_cast<uint32_t>(row[i - (kVec - n)]) << (i % 2 * 16);
  }
}

template <bool NT, bool TAIL>
__device__ __forceinline__ void load_raw(const float* row, int64_t v, int n, Raw8<float>& out) {
  const int64_t at = v * kVec;
#pragma unroll
  for (int i = 0; i < kVec; ++i) out.w[i] = 0.f;
  if (!TAIL || n >= kVec) {
    if (at < n) {
      const f32x4_a4* p = reinterpret_cast<const f32x4_a4*>(row + (!TAIL || at + kVec <= n ? at : n - kVec));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4_a4 b = NT ? __builtin_nontemporal_load(p + h) : p[h];
#pragma unroll
        for (int i = 0; i < 4; ++i) out.w[4 * h + i] = b[i];
      }
    }
  } else if (at == 0) {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (i >= kVec - n) out.w[i] = row[i - (kVec - n)];
  }
}

// Whole waves branch over the shift (one wave of a row has a piece to shift), lanes select.
template <bool TAIL>
__device__ __forceinline__ void unpack(const Raw8<uint16_t>& r, int64_t v, int n, float* out) {
  uint32_t w[4] = {r.w[0], r.w[1], r.w[2], r.w[3]};
  const int64_t over = v * kVec + kVec - n;
  if (TAIL && __any(over > 0)) {
    const int sh = over > 0 ? static_cast<int>(over) : 0;
    const bool four = sh & 4, two = sh & 2, one = sh & 1;
    w[0] = four ? w[2] : w[0];
    w[1] = four ? w[3] : w[1];
    w[2] = four ? 0 : w[2];
    w[3] = four ? 0 : w[3];
    w[0] = two ? w[1] : w[0];
    w[1] = two ? w[2] : w[1];
    w[2] = two ? w[3] : w[2];
    w[3] = two ? 0 : w[3];
    w[0] = one ? w[0] >> 16 | w[1] << 16 : w[0];
    w[1] = one ? w[1] >> 16 | w[2] << 16 : w[1];
    w[2] = one ? w[2] >> 16 | w[3] << 16 : w[2];
    w[3] = one ? w[3] >> 16 : w[3];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    out[2 * i] = __uint_as_float(w[i] << 16);
    out[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

template <bool TAIL>
__device__ __forceinline__ void unpack(const Raw8<float>& r, int64_t v, int n, float* out) {
#pragma unroll
  for (int i = 0; i < kVec; ++i) out[i] = r.w[i];
  const int64_t over = v * kVec + kVec - n;
  if (TAIL && __any(over > 0)) {
    const int sh = over > 0 ? static_cast<int>(over) : 0;
#pragma unroll
    for (int step = 4; step >= 1; step /= 2) {
      const bool take = sh & step;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const float next = i + step < kVec ? out[i + step] : 0.f;
        out[i] = take ? next : out[i];
      }
    }
  }
}

template <bool NT, bool TAIL, typename T>
__device__ __forceinline__ void load8(const T* row, int64_t v, int n, float* out) {
  Raw8<T> r;
  load_raw<NT, TAIL>(row, v, n, r);
  unpack<TAIL>(r, v, n, out);
}

template <bool NT, bool TAIL>
__device__ __forceinline__ void store8(uint16_t* row, int64_t v, int n, const float* in) {
  const int64_t at = v * kVec;
  if (TAIL ? at + kVec <= n : at < n) {
    u32x4_a2 b;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      b[i] = f32_to_bf16(in[2 * i]) | (static_cast<uint32_t>(f32_to_bf16(in[2 * i + 1])) << 16);
    u32x4_a2* p = reinterpret_cast<u32x4_a2*>(row + at);
    if (NT) __builtin_nontemporal_store(b, p);
    else *p = b;
  } else if (TAIL && at < n) {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (at + i < n) row[at + i] = f32_to_bf16(in[i]);
  }
}

template <bool NT, bool TAIL>
__device__ __forceinline__ void store8(float* row, int64_t v, int n, const float* in) {
  const int64_t at = v * kVec;
  if (TAIL ? at + kVec <= n : at < n) {
    f32x4_a4* p = reinterpret_cast<f32x4_a4*>(row + at);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4_a4 b = {in[4 * h], in[4 * h + 1], in[4 * h + 2], in[4 * h + 3]};
      if (NT) __builtin_nontemporal_store(b, p + h);
      else p[h] = b;
    }
  } else if (TAIL && at < n) {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (at + i < n) row[at + i] = in[i];
  }
}

// Inclusive prefix sum over the wave: four adds of lanes 1, 2, 4 and 8 to the left within rows of 16
// lanes, then row 0's (2's) total into row 1 (3) and the lower half's into the upper, all on the data
// path between lanes and not through LDS.
#define DPP(v, CTRL, ROWS) __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, true)
__device__ __forceinline__ int wave_scan(int v) {
  v += DPP(v, 0x111, 0xf);
  v += DPP(v, 0x112, 0xf);
  v += DPP(v, 0x114, 0xf);
  v += DPP(v, 0x118, 0xf);
  v += DPP(v, 0x142, 0xa);
  v += DPP(v, 0x143, 0xc);
  return v;
}

// Sum over the wave, the same in every lane: the scan's last lane.
__device__ __forceinline__ float wave_sum(float v) {
#define ADD(CTRL, ROWS) v += __int_as_float(DPP(__float_as_int(v), CTRL, ROWS))
  ADD(0x111, 0xf);
  ADD(0x112, 0xf);
  ADD(0x114, 0xf);
  ADD(0x118, 0xf);
  ADD(0x142, 0xa);
  ADD(0x143, 0xc);
#undef ADD
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
#undef DPP

}  // namespace moe
