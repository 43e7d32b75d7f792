// moe_mx_quantize: rows to 8 bits with block scales (mx.h), as they are or as the SwiGLU of their two
// halves, silu(gate) up.
//
// Bound by HBM.  A wave takes 512 columns of a row at a time: eight values a lane, one 16-byte load of
// bf16 (two with SwiGLU), eight bytes and, for every 16 lanes, a word of four scales out.  Measured, bf16:
// SwiGLU of 65536 rows of 2 x 2048 107 us (6.3 TB/s), 4096 x 7168 weights 16 us (5.6 TB/s).
#include "mx.h"
#include "rows.h"

namespace moe {
namespace {

// silu(g) u, with e^-g as 2^(-g log2 e) and the quotient from the hardware's exp2 and reciprocal
// (about 1 ulp each).  A sigmoid that saturates gives 0 or g exactly.
__device__ __forceinline__ float swiglu(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.4426950408889634f)) * u;
}

// `units` of 512 columns a row; wave w of the grid takes units w, w + all, ...
template <typename T, bool SWIGLU>
__global__ __launch_bounds__(256) void quantize_kernel(const T* __restrict__ x, uint32_t rows, int cols,
                                                       uint32_t units, uint8_t* __restrict__ q,
                                                       uint8_t* __restrict__ scales) {
  const int lane = threadIdx.x & (kWave - 1);
  // n is below 2^26 where a wave takes more than one: no sum here passes 32 bits
  const uint32_t all = gridDim.x * 4, n = rows * units;
  const int64_t pitch = mx_pitch(cols);
  for (uint32_t u = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave); u < n; u += all) {
    const int64_t row = u / units;
    const int64_t v = static_cast<int64_t>(u % units) * kWave + lane;  // of the row's eights
    const T* xr = x + row * cols * (SWIGLU ? 2 : 1);
    float f[kVec];
    load8<true, false>(xr, v, cols, f);
    if constexpr (SWIGLU) {
      float up[kVec];
      load8<true, false>(xr + cols, v, cols, up);
#pragma unroll
      for (int i = 0; i < kVec; ++i) f[i] = swiglu(f[i], up[i]);
    }
    mx_store(f, v * kVec, cols, q + row * cols, scales + row * pitch);
  }
}

template <typename T>
void launch(const void* x, int rows, int cols, bool swiglu, uint8_t* q, uint8_t* scales, hipStream_t s) {
  const int units = ceil_div(cols, kMxUnit);
  // A unit a wave, or, where that is at most 64 blocks a CU, 16 of them that take turns.  Measured, turns
  // against none: bf16 4096 x 7168 16.0 / 17.5 us, SwiGLU of 8192 x 1408 10.2 / 11.6 us; of 65536 x 2048 117 /
  // 107 us.
  const int64_t all = ceil_div64(static_cast<int64_t>(rows) * units, 4);
  const int64_t blocks = all <= kCus * 64 ? std::min<int64_t>(all, kCus * 16) : all;
  hipLaunchKernelGGL((swiglu ? quantize_kernel<T, true> : quantize_kernel<T, false>),
                     dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, static_cast<const T*>(x),
                     static_cast<uint32_t>(rows), cols, static_cast<uint32_t>(units), q, scales);
}

}  // namespace
}  // namespace moe

extern "C" int moe_mx_scale_pitch(int cols, size_t* bytes) {
  using namespace moe;
  if (!bytes || cols < 1) return fail(MOE_ERR_ARG, "moe_mx_scale_pitch: bad arguments");
  *bytes = static_cast<size_t>(mx_pitch(cols));
  return MOE_OK;
}

extern "C" int moe_mx_quantize(const void* x, int rows, int cols, moe_dtype dtype, int swiglu, uint8_t* q,
                               uint8_t* scales, moe_stream_t stream) {
  using namespace moe;
  const char* who = "moe_mx_quantize";
  if (rows < 0 || cols < 1 || !is_dtype(dtype) || (swiglu != 0 && swiglu != 1))
    return fail(MOE_ERR_ARG, "%s: bad sizes rows=%d cols=%d, dtype or swiglu", who, rows, cols);
  if (cols % kMxBlock != 0 || cols > kMaxRow)
    return fail(MOE_ERR_UNSUPPORTED, "%s: cols=%d is not a multiple of %d, or above %d", who, cols, kMxBlock, kMaxRow);
  if (too_many(ceil_div64(static_cast<int64_t>(rows) * ceil_div(cols, kMxUnit), 4), 256))
    return fail(MOE_ERR_UNSUPPORTED, "%s: rows=%d too many at cols=%d", who, rows, cols);
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(scales)) % 16 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "%s: q or scales is not aligned to 16 bytes", who);
  if (rows == 0) return MOE_OK;
  if (!x || !q || !scales) return fail(MOE_ERR_ARG, "%s: null pointer", who);
  hipStream_t s = as_stream(stream);
  if (dtype == MOE_F32) launch<float>(x, rows, cols, swiglu, q, scales, s);
  else launch<uint16_t>(x, rows, cols, swiglu, q, scales, s);
  MOE_LAUNCH_CHECK("moe_mx_quantize: launch");
  return debug_check(MOE_OK, who, s, nullptr);
}
