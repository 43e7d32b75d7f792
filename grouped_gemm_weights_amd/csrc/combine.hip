// moe_combine: weighted un-permute of the expert outputs, its gradient
// (moe_combine_backward), and the residual add used between pipeline layers.
//
// One 256-thread block per token: the k routing weights and row indices are
// read once, then each thread sweeps float4 columns of the k expert rows
// (k independent 16-byte loads in flight per step) and accumulates in j order
// with fused multiply-adds.  Every y_perm row is read exactly once, so its loads
// are non-temporal (9 % faster on prefill-sized layers than cached loads).
#include <algorithm>

#include "rows.h"

namespace moe {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));

template <bool VEC>
__global__ __launch_bounds__(256) void combine_kernel(const float* __restrict__ y_perm,
                                                      const int32_t* __restrict__ row_of,
                                                      const float* __restrict__ topk_w, int T,
                                                      int k, int H, float* __restrict__ y) {
  __shared__ int32_t rows[MOE_MAX_K];
  __shared__ float ws[MOE_MAX_K];
  const int t = blockIdx.x;
  if (threadIdx.x < k) {
    const int32_t r = row_of[static_cast<int64_t>(t) * k + threadIdx.x];
    // an unwritten row index (after an out-of-range expert id) must not fault
    const bool ok = r >= 0 && static_cast<int64_t>(r) < static_cast<int64_t>(T) * k;
    rows[threadIdx.x] = ok ? r : 0;
    ws[threadIdx.x] = ok ? topk_w[static_cast<int64_t>(t) * k + threadIdx.x] : 0.f;
  }
  __syncthreads();
  float* out = y + static_cast<int64_t>(t) * H;
  if (VEC) {
    const int H4 = H / 4;
    for (int c = threadIdx.x; c < H4; c += blockDim.x) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int j = 0; j < k; ++j) {
        const f32x4_t v = __builtin_nontemporal_load(
            reinterpret_cast<const f32x4_t*>(y_perm + static_cast<int64_t>(rows[j]) * H) + c);
        const float wj = ws[j];
        acc.x = fmaf(wj, v.x, acc.x);
        acc.y = fmaf(wj, v.y, acc.y);
        acc.z = fmaf(wj, v.z, acc.z);
        acc.w = fmaf(wj, v.w, acc.w);
      }
      reinterpret_cast<float4*>(out)[c] = acc;
    }
  } else {
    for (int c = threadIdx.x; c < H; c += blockDim.x) {
      float acc = 0.f;
      for (int j = 0; j < k; ++j) acc = fmaf(ws[j], y_perm[static_cast<int64_t>(rows[j]) * H + c], acc);
      out[c] = acc;
    }
  }
}

// out may alias x (each element is read before it is written by the same thread)
__global__ __launch_bounds__(256) void residual_kernel(const uint16_t* x, const float* __restrict__ y,
                                                       int64_t n, uint16_t* out) {
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += stride)
    out[i] = f32_to_bf16(bf16_to_f32(x[i]) + y[i]);
}

// Gradient of y[t] = sum_j w[t][j] y_perm[row_of[t k + j]]:
//   dy_perm[row] = w[t][j] dy[t],   dw[t][j] = <dy[t], y_perm[row]>.
// Bound by HBM: y_perm is read once (4 R H bytes) and dy_perm written once, so both bypass the
// caches; dy[t] stays in registers for the token's k rows.  A token has one to four waves, each
// lane NV vectors of 8 columns and sweep; a wave's share of a dot product goes to its own LDS
// slot, so the k sums cost one barrier, and the slots are added in wave order (the same bits
// every run).  Tokens of one wave go four to a block.  TAIL: H is not a multiple of 8.
// Measured: 8192 tokens x 8 of H = 7168, bf16 dy and dy_perm: 600 us, 4.9 TB/s.
template <typename D, typename O, int NV, int WAVES, bool TAIL>
__global__ __launch_bounds__(WAVES == 1 ? 256 : WAVES * kWave) void combine_backward_kernel(
    const D* __restrict__ dy, const float* __restrict__ y_perm, const int32_t* __restrict__ row_of,
    const float* __restrict__ topk_w, int T, int k, int H, O* __restrict__ dy_perm,
    float* __restrict__ dtopk_w) {
  __shared__ float dot[MOE_MAX_K][4];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int t = WAVES == 1 ? blockIdx.x * 4 + wave : blockIdx.x;
  if (t >= T) return;
  constexpr int threads = WAVES * kWave;
  const int tid = WAVES == 1 ? lane : threadIdx.x;
  const int64_t R = static_cast<int64_t>(T) * k;
  const int32_t* rows = row_of + static_cast<int64_t>(t) * k;
  const float* ws = topk_w + static_cast<int64_t>(t) * k;
  const D* dr = dy + static_cast<int64_t>(t) * H;
  const int pieces = (H + kVec - 1) / kVec;
  for (int c0 = 0; c0 < pieces; c0 += NV * threads) {
    float d[NV][kVec];
#pragma unroll
    for (int i = 0; i < NV; ++i) load8<true, TAIL>(dr, c0 + tid + i * threads, H, d[i]);
    for (int j = 0; j < k; ++j) {
      const int r = rows[j];
      const float w = ws[j];
      // an unwritten row index (after an out-of-range expert id) must not fault
      const bool ok = r >= 0 && r < R;
      float s = 0.f;
      if (ok) {
        O* out = dy_perm + static_cast<int64_t>(r) * H;
        if (dtopk_w) {
          const float* yr = y_perm + static_cast<int64_t>(r) * H;
          Raw8<float> y[NV];
#pragma unroll
          for (int i = 0; i < NV; ++i) load_raw<true, TAIL>(yr, c0 + tid + i * threads, H, y[i]);
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            float f[kVec];
            unpack<TAIL>(y[i], c0 + tid + i * threads, H, f);
#pragma unroll
            for (int q = 0; q < kVec; ++q) s = fmaf(d[i][q], f[q], s);
          }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float v[kVec];
#pragma unroll
          for (int q = 0; q < kVec; ++q) v[q] = w * d[i][q];
          store8<true, TAIL>(out, c0 + tid + i * threads, H, v);
        }
      }
      if (dtopk_w) {
        s = wave_sum(s);
        if (lane == 0) {
          if (WAVES == 1) dtopk_w[static_cast<int64_t>(t) * k + j] = s;  // one sweep: the whole sum
          else dot[j][wave] = c0 ? dot[j][wave] + s : s;
        }
      }
    }
  }
  if (dtopk_w && WAVES > 1) {
    __syncthreads();
    const int j = threadIdx.x;
    if (j < k) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < WAVES; ++i) s += dot[j][i];
      dtopk_w[static_cast<int64_t>(t) * k + j] = s;
    }
  }
}

template <typename D, typename O, bool TAIL>
void launch_combine_backward(const void* dy, const float* y_perm, const int32_t* row_of,
                             const float* topk_w, int T, int k, int H, void* dy_perm, float* dtopk_w,
                             hipStream_t s) {
  const int pieces = ceil_div(H, kVec);
  // one vector a lane up to 4 waves, then two and four; rows over 8192 columns are swept
  auto kernel = pieces <= 64    ? combine_backward_kernel<D, O, 1, 1, TAIL>
                : pieces <= 128 ? combine_backward_kernel<D, O, 1, 2, TAIL>
                : pieces <= 192 ? combine_backward_kernel<D, O, 1, 3, TAIL>
                : pieces <= 256 ? combine_backward_kernel<D, O, 1, 4, TAIL>
                : pieces <= 512 ? combine_backward_kernel<D, O, 2, 4, TAIL>
                                : combine_backward_kernel<D, O, 4, 4, TAIL>;
  const int waves = std::min(ceil_div(pieces, kWave), 4);
  hipLaunchKernelGGL(kernel, dim3(waves == 1 ? ceil_div(T, 4) : T),
                     dim3(waves == 1 ? 256 : waves * kWave), 0, s, static_cast<const D*>(dy), y_perm,
                     row_of, topk_w, T, k, H, static_cast<O*>(dy_perm), dtopk_w);
}

}  // namespace
}  // namespace moe

extern "C" int moe_combine(const float* y_perm, const int32_t* row_of, const float* topk_w, int T,
                           int k, int H, float* y, moe_stream_t stream) {
  using namespace moe;
  if (T < 0 || k < 1 || H < 1) return fail(MOE_ERR_ARG, "moe_combine: bad sizes T=%d k=%d H=%d", T, k, H);
  if (k > MOE_MAX_K) return fail(MOE_ERR_UNSUPPORTED, "moe_combine: k=%d above %d", k, MOE_MAX_K);
  if (T == 0) return MOE_OK;
  if (!y_perm || !row_of || !topk_w || !y) return fail(MOE_ERR_ARG, "moe_combine: null pointer");
  hipStream_t s = as_stream(stream);
  const bool vec = (H % 4 == 0) && ((reinterpret_cast<uintptr_t>(y_perm) | reinterpret_cast<uintptr_t>(y)) % 16 == 0);
  if (vec)
    hipLaunchKernelGGL(combine_kernel<true>, dim3(T), dim3(256), 0, s, y_perm, row_of, topk_w, T, k, H, y);
  else
    hipLaunchKernelGGL(combine_kernel<false>, dim3(T), dim3(256), 0, s, y_perm, row_of, topk_w, T, k, H, y);
  MOE_LAUNCH_CHECK("moe_combine: launch");
  return debug_check(MOE_OK, "moe_combine", s, nullptr);
}

extern "C" int moe_combine_backward(const void* dy, moe_dtype dy_dtype, const float* y_perm,
                                    const int32_t* row_of, const float* topk_w, int T, int k, int H,
                                    moe_dtype dtype, void* dy_perm, float* dtopk_w,
                                    moe_stream_t stream) {
  using namespace moe;
  if (T < 0 || k < 1 || H < 1 || (dy_dtype != MOE_F32 && dy_dtype != MOE_BF16) ||
      (dtype != MOE_F32 && dtype != MOE_BF16))
    return fail(MOE_ERR_ARG, "moe_combine_backward: bad sizes T=%d k=%d H=%d or dtype", T, k, H);
  if (k > MOE_MAX_K)
    return fail(MOE_ERR_UNSUPPORTED, "moe_combine_backward: k=%d above %d", k, MOE_MAX_K);
  if (static_cast<int64_t>(T) * k > INT32_MAX || H > kMaxRow || too_many(T, 256))
    return fail(MOE_ERR_UNSUPPORTED, "moe_combine_backward: T=%d, T*k or H=%d too large", T, H);
  if (T == 0) return MOE_OK;
  if (!dy || !row_of || !topk_w || !dy_perm || (dtopk_w && !y_perm))
    return fail(MOE_ERR_ARG, "moe_combine_backward: null pointer");
  hipStream_t s = as_stream(stream);
  auto launch = H % kVec == 0 ? launch_combine_backward<uint16_t, uint16_t, false>
                              : launch_combine_backward<uint16_t, uint16_t, true>;
  if (dy_dtype == MOE_F32 && dtype == MOE_F32)
    launch = H % kVec == 0 ? launch_combine_backward<float, float, false> : launch_combine_backward<float, float, true>;
  else if (dy_dtype == MOE_F32)
    launch = H % kVec == 0 ? launch_combine_backward<float, uint16_t, false>
                           : launch_combine_backward<float, uint16_t, true>;
  else if (dtype == MOE_F32)
    launch = H % kVec == 0 ? launch_combine_backward<uint16_t, float, false>
                           : launch_combine_backward<uint16_t, float, true>;
  launch(dy, y_perm, row_of, topk_w, T, k, H, dy_perm, dtopk_w, s);
  MOE_LAUNCH_CHECK("moe_combine_backward: launch");
  return debug_check(MOE_OK, "moe_combine_backward", s, nullptr);
}

extern "C" int moe_residual_add(const void* x, const float* y, int64_t n, void* out,
                                moe_stream_t stream) {
  using namespace moe;
  if (n < 0) return fail(MOE_ERR_ARG, "moe_residual_add: n < 0");
  if (n == 0) return MOE_OK;
  if (!x || !y || !out) return fail(MOE_ERR_ARG, "moe_residual_add: null pointer");
  const int64_t blocks64 = ceil_div64(n, 256);
  const int blocks = static_cast<int>(blocks64 < 65536 ? blocks64 : 65536);
  hipLaunchKernelGGL(residual_kernel, dim3(blocks), dim3(256), 0, as_stream(stream),
                     static_cast<const uint16_t*>(x), y, n, static_cast<uint16_t*>(out));
  MOE_LAUNCH_CHECK("moe_residual_add: launch");
  return debug_check(MOE_OK, "moe_residual_add", as_stream(stream), nullptr);
}
