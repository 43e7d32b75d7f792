// moe_layer_norm and moe_layer_norm_backward: the norm in front of the router and the experts.
//
//   forward   mu = mean x,  r = 1 / sqrt(mean (x - mu)^2 + eps),  y = (x - mu) r gamma + beta
//   backward  xh = (x - mu) r,  a = dy gamma,
//             dx = r (a - mean a - xh mean(a xh)),  dgamma = sum_t dy xh,  dbeta = sum_t dy
//
// Both are bound by HBM: a row is read once, held in registers as fp32, and every statistic is an
// fp32 sum over it (the variance from the centred values, not from a difference of two sums, so
// a row far from zero loses nothing).
#include "rows.h"

namespace moe {
namespace {

// Sum of one value over the WPR waves that share a row.  `part` is a buffer of WPR floats that
// no other sum of the same barrier interval uses.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* part) {
  v = wave_sum(v);
  if (WPR == 1) return v;
  if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < WPR; ++w) s += part[w];
  return s;
}

// WPR waves per row, each lane NV vectors of 8 elements: H <= WPR * 64 * NV * 8.
template <typename T, int WPR, int NV>
__global__ __launch_bounds__(WPR == 1 ? 256 : WPR * kWave) void norm_kernel(
    const T* __restrict__ x, const float* __restrict__ gamma, const float* __restrict__ beta,
    int rows, int H, float eps, T* __restrict__ y, float* __restrict__ mean,
    float* __restrict__ rstd) {
  __shared__ float part[2][WPR];
  const int row = WPR == 1 ? blockIdx.x * 4 + threadIdx.x / kWave : blockIdx.x;
  if (row >= rows) return;
  const int tid = WPR == 1 ? threadIdx.x & (kWave - 1) : threadIdx.x;
  const T* xr = x + static_cast<int64_t>(row) * H;
  float v[NV][kVec];
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load8<true>(xr, tid + i * WPR * kWave, H, v[i]);
#pragma unroll
    for (int j = 0; j < kVec; ++j) s += v[i][j];
  }
  const float mu = row_sum<WPR>(s, part[0]) / H;
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int at = (tid + i * WPR * kWave) * kVec + j;
      v[i][j] = at < H ? v[i][j] - mu : 0.f;
      q = fmaf(v[i][j], v[i][j], q);
    }
  const float r = 1.f / sqrtf(row_sum<WPR>(q, part[1]) / H + eps);
  T* yr = y + static_cast<int64_t>(row) * H;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = tid + i * WPR * kWave;
    float g[kVec], b[kVec];
    load8<false>(gamma, at, H, g);
#pragma unroll
    for (int j = 0; j < kVec; ++j) b[j] = 0.f;
    if (beta) load8<false>(beta, at, H, b);
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[i][j] = fmaf(v[i][j] * r, g[j], b[j]);
    store8<true>(yr, at, H, v[i]);
  }
  if (tid == 0) {
    if (mean) mean[row] = mu;
    if (rstd) rstd[row] = r;
  }
}

// Rows too long for registers (H > 32768): the row is read three times, the later two from L2.
template <typename T>
__global__ __launch_bounds__(1024) void norm_long_kernel(
    const T* __restrict__ x, const float* __restrict__ gamma, const float* __restrict__ beta, int H,
    float eps, T* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd) {
  __shared__ float part[2][16];
  const int row = blockIdx.x;
  const T* xr = x + static_cast<int64_t>(row) * H;
  const int64_t n_vec = (static_cast<int64_t>(H) + kVec - 1) / kVec;
  float v[kVec];
  float s = 0.f;
  for (int64_t at = threadIdx.x; at < n_vec; at += 1024) {
    load8<false>(xr, at, H, v);
#pragma unroll
    for (int j = 0; j < kVec; ++j) s += v[j];
  }
  const float mu = row_sum<16>(s, part[0]) / H;
  float q = 0.f;
  for (int64_t at = threadIdx.x; at < n_vec; at += 1024) {
    load8<false>(xr, at, H, v);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const float c = at * kVec + j < H ? v[j] - mu : 0.f;
      q = fmaf(c, c, q);
    }
  }
  const float r = 1.f / sqrtf(row_sum<16>(q, part[1]) / H + eps);
  T* yr = y + static_cast<int64_t>(row) * H;
  for (int64_t at = threadIdx.x; at < n_vec; at += 1024) {
    float g[kVec], b[kVec];
    load8<false>(xr, at, H, v);
    load8<false>(gamma, at, H, g);
#pragma unroll
    for (int j = 0; j < kVec; ++j) b[j] = 0.f;
    if (beta) load8<false>(beta, at, H, b);
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = fmaf((v[j] - mu) * r, g[j], b[j]);
    store8<true>(yr, at, H, v);
  }
  if (threadIdx.x == 0) {
    if (mean) mean[row] = mu;
    if (rstd) rstd[row] = r;
  }
}

// Backward.  WPR waves share a row; a group of WPR waves takes rows `group`, `group` + groups, ...
// and its lanes own fixed columns, so the sums over its rows for dgamma and dbeta stay in
// registers; a block's groups (WPR = 1: four) are joined in LDS and leave as one partial row of
// 2 H floats (partial != nullptr).  The next row's loads are issued before this row's sums, so
// they are in flight while the waves wait for one another.
template <typename T, int WPR, int NV>
__global__ __launch_bounds__(WPR == 1 ? 256 : WPR * kWave) void norm_backward_kernel(
    const T* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ gamma,
    const float* __restrict__ mean, const float* __restrict__ rstd, int rows, int H,
    T* __restrict__ dx, float* __restrict__ partial) {
  constexpr int GROUPS = WPR == 1 ? 4 : 1, LANES = WPR * kWave;
  __shared__ float part[2][2][WPR];
  __shared__ float joined[GROUPS > 1 ? 2 * LANES * NV * kVec : 1];
  const int tid = threadIdx.x % LANES;
  const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / LANES);
  const int step = gridDim.x * GROUPS;
  float sg[NV][kVec], sb[NV][kVec], g[NV][kVec];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load8<false>(gamma, tid + i * LANES, H, g[i]);
#pragma unroll
    for (int j = 0; j < kVec; ++j) sg[i][j] = sb[i][j] = 0.f;
  }
  int row = blockIdx.x * GROUPS + group;
  Raw8<T> xn[NV], dn[NV];
  float mu_n = 0.f, r_n = 0.f;
  auto fetch = [&](int r) {
    mu_n = mean[r];
    r_n = rstd[r];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      load_raw<true>(x + static_cast<int64_t>(r) * H, tid + i * LANES, H, xn[i]);
      load_raw<true>(dy + static_cast<int64_t>(r) * H, tid + i * LANES, H, dn[i]);
    }
  };
  if (row < rows) fetch(row);
  for (int turn = 0; row < rows; row += step, turn ^= 1) {
    const float mu = mu_n, r = r_n;
    float a[NV][kVec], xh[NV][kVec];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unpack(xn[i], xh[i]);
      unpack(dn[i], a[i]);
    }
    if (row + step < rows) fetch(row + step);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        // past the row a is zero, so what xh holds there does not count
        xh[i][j] = (xh[i][j] - mu) * r;
        sg[i][j] = fmaf(a[i][j], xh[i][j], sg[i][j]);
        sb[i][j] += a[i][j];
        a[i][j] *= g[i][j];
        s1 += a[i][j];
        s2 = fmaf(a[i][j], xh[i][j], s2);
      }
    s1 = wave_sum(s1);
    s2 = wave_sum(s2);
    if (WPR > 1) {
      // the buffers alternate from row to row, so one barrier a row is enough
      if ((tid & (kWave - 1)) == 0) {
        part[turn][0][tid / kWave] = s1;
        part[turn][1][tid / kWave] = s2;
      }
      __syncthreads();
      s1 = s2 = 0.f;
#pragma unroll
      for (int w = 0; w < WPR; ++w) {
        s1 += part[turn][0][w];
        s2 += part[turn][1][w];
      }
    }
    s1 /= H;
    s2 /= H;
    T* out = dx + static_cast<int64_t>(row) * H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) a[i][j] = r * (a[i][j] - s1 - xh[i][j] * s2);
      store8<true>(out, tid + i * LANES, H, a[i]);
    }
  }
  if (!partial) return;
  if (GROUPS > 1) {
    // the groups add their sums in group order
    for (int k = 0; k < GROUPS; ++k) {
      if (group == k)
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < kVec; ++j) {
            float* at = joined + ((i * kVec + j) * 2) * LANES + tid;
            if (k > 0) {
              sg[i][j] += at[0];
              sb[i][j] += at[LANES];
            }
            at[0] = sg[i][j];
            at[LANES] = sb[i][j];
          }
      __syncthreads();
    }
    if (group != GROUPS - 1) return;
  }
  float* p = partial + static_cast<int64_t>(blockIdx.x) * 2 * H;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    store8<false>(p, tid + i * LANES, H, sg[i]);
    store8<false>(p + H, tid + i * LANES, H, sb[i]);
  }
}

// Rows too long for registers: dx alone, the row read twice.
template <typename T>
__global__ __launch_bounds__(1024) void norm_backward_long_kernel(
    const T* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ gamma,
    const float* __restrict__ mean, const float* __restrict__ rstd, int H, T* __restrict__ dx) {
  __shared__ float part[2][16];
  const int row = blockIdx.x;
  const T* xr = x + static_cast<int64_t>(row) * H;
  const T* dr = dy + static_cast<int64_t>(row) * H;
  const float mu = mean[row], r = rstd[row];
  const int64_t n_vec = (static_cast<int64_t>(H) + kVec - 1) / kVec;
  float a[kVec], xh[kVec], g[kVec];
  float s1 = 0.f, s2 = 0.f;
  for (int64_t at = threadIdx.x; at < n_vec; at += 1024) {
    load8<false>(xr, at, H, xh);
    load8<false>(dr, at, H, a);
    load8<false>(gamma, at, H, g);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      s1 = fmaf(a[j], g[j], s1);
      s2 = fmaf(a[j] * g[j], (xh[j] - mu) * r, s2);
    }
  }
  s1 = row_sum<16>(s1, part[0]) / H;
  s2 = row_sum<16>(s2, part[1]) / H;
  T* out = dx + static_cast<int64_t>(row) * H;
  for (int64_t at = threadIdx.x; at < n_vec; at += 1024) {
    load8<false>(xr, at, H, xh);
    load8<false>(dr, at, H, a);
    load8<false>(gamma, at, H, g);
#pragma unroll
    for (int j = 0; j < kVec; ++j) a[j] = r * (a[j] * g[j] - s1 - (xh[j] - mu) * r * s2);
    store8<true>(out, at, H, a);
  }
}

// Its column sums: one thread per column and block of rows, straight from x and dy.
template <typename T>
__global__ __launch_bounds__(256) void norm_columns_kernel(
    const T* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ mean,
    const float* __restrict__ rstd, int rows, int H, float* __restrict__ partial) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= H) return;
  float sg = 0.f, sb = 0.f;
  for (int row = blockIdx.y; row < rows; row += gridDim.y) {
    const int64_t at = static_cast<int64_t>(row) * H + c;
    float d, v;
    if constexpr (sizeof(T) == 2) {
      d = bf16_to_f32(dy[at]);
      v = bf16_to_f32(x[at]);
    } else {
      d = dy[at];
      v = x[at];
    }
    sg = fmaf(d, (v - mean[row]) * rstd[row], sg);
    sb += d;
  }
  float* p = partial + static_cast<int64_t>(blockIdx.y) * 2 * H;
  p[c] = sg;
  p[H + c] = sb;
}

// dgamma and dbeta from n partial rows of 2 H floats: 64 columns per block, 16 waves that each
// take every 16th row, joined in LDS in wave order.
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(kSumWaves* kWave) void norm_sum_kernel(
    const float* __restrict__ partial, int n, int H, float* __restrict__ dgamma,
    float* __restrict__ dbeta) {
  __shared__ float s[kSumWaves][kWave];
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kWave + lane;
  const int64_t H2 = 2 * static_cast<int64_t>(H);
  float v = 0.f;
  if (c < H2) {
#pragma unroll 8
    for (int i = w; i < n; i += kSumWaves) v += partial[i * H2 + c];
  }
  s[w][lane] = v;
  __syncthreads();
  if (w == 0 && c < H2) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kSumWaves; ++i) v += s[i][lane];
    if (c < H) {
      if (dgamma) dgamma[c] = v;
    } else if (dbeta) {
      dbeta[c - H] = v;
    }
  }
}

constexpr int kMaxH = 16 * kWave * 4 * kVec;  // 32768: the longest row that stays in registers
constexpr int kPartials = 512;                // blocks of the backward pass, two a CU

int norm_partials(int T) { return T < kPartials ? T : kPartials; }

template <typename E, int WPR, int NV>
int launch_norm(const void* x, const float* gamma, const float* beta, int T, int H, float eps, void* y,
                float* mean, float* rstd, hipStream_t s) {
  const int blocks = WPR == 1 ? ceil_div(T, 4) : T;
  hipLaunchKernelGGL((norm_kernel<E, WPR, NV>), dim3(blocks), dim3(WPR == 1 ? 256 : WPR * kWave), 0, s,
                     static_cast<const E*>(x), gamma, beta, T, H, eps, static_cast<E*>(y), mean, rstd);
  MOE_LAUNCH_CHECK("moe_layer_norm: launch");
  return MOE_OK;
}

template <typename E>
int norm(const void* x, const float* gamma, const float* beta, int T, int H, float eps, void* y,
         float* mean, float* rstd, hipStream_t s) {
#define NORM(WPR, NV) return launch_norm<E, WPR, NV>(x, gamma, beta, T, H, eps, y, mean, rstd, s)
  if (H <= 512) NORM(1, 1);
  if (H <= 1024) NORM(1, 2);
  if (H <= 2048) NORM(4, 1);
  if (H <= 4096) NORM(4, 2);
  if (H <= 8192) NORM(4, 4);
  if (H <= 16384) NORM(16, 2);
  if (H <= kMaxH) NORM(16, 4);
#undef NORM
  hipLaunchKernelGGL(norm_long_kernel<E>, dim3(T), dim3(1024), 0, s, static_cast<const E*>(x), gamma,
                     beta, H, eps, static_cast<E*>(y), mean, rstd);
  MOE_LAUNCH_CHECK("moe_layer_norm: launch");
  return MOE_OK;
}

template <typename E, int WPR, int NV>
int launch_norm_backward(const void* dy, const void* x, const float* gamma, const float* mean,
                         const float* rstd, int T, int H, void* dx, float* partial, hipStream_t s) {
  hipLaunchKernelGGL((norm_backward_kernel<E, WPR, NV>), dim3(norm_partials(T)), dim3(WPR == 1 ? 256 : WPR * kWave), 0, s,
                     static_cast<const E*>(dy), static_cast<const E*>(x), gamma, mean, rstd, T, H,
                     static_cast<E*>(dx), partial);
  MOE_LAUNCH_CHECK("moe_layer_norm_backward: launch");
  return MOE_OK;
}

template <typename E>
int norm_backward(const void* dy, const void* x, const float* gamma, const float* mean, const float* rstd,
                  int T, int H, void* dx, float* partial, hipStream_t s) {
#define NORM(WPR, NV) return launch_norm_backward<E, WPR, NV>(dy, x, gamma, mean, rstd, T, H, dx, partial, s)
  if (H <= 512) NORM(1, 1);
  if (H <= 1024) NORM(1, 2);
  if (H <= 2048) NORM(4, 1);
  if (H <= 4096) NORM(8, 1);
  if (H <= 8192) NORM(16, 1);
  if (H <= 16384) NORM(16, 2);
#undef NORM
  hipLaunchKernelGGL(norm_backward_long_kernel<E>, dim3(T), dim3(1024), 0, s, static_cast<const E*>(dy),
                     static_cast<const E*>(x), gamma, mean, rstd, H, static_cast<E*>(dx));
  MOE_LAUNCH_CHECK("moe_layer_norm_backward: launch");
  if (partial) {
    hipLaunchKernelGGL(norm_columns_kernel<E>, dim3(ceil_div(H, 256), norm_partials(T)), dim3(256), 0, s,
                       static_cast<const E*>(dy), static_cast<const E*>(x), mean, rstd, T, H, partial);
    MOE_LAUNCH_CHECK("moe_layer_norm_backward: columns launch");
  }
  return MOE_OK;
}

size_t norm_backward_ws(int T, int H) {
  return align_up(static_cast<size_t>(norm_partials(T)) * 2 * H * sizeof(float), 256);
}

}  // namespace
}  // namespace moe

extern "C" int moe_layer_norm(const void* x, const float* gamma, const float* beta, int T, int H,
                              float eps, moe_dtype dtype, void* y, float* mean, float* rstd,
                              moe_stream_t stream) {
  using namespace moe;
  if (T < 0 || H < 1 || !(eps >= 0.f) || (dtype != MOE_F32 && dtype != MOE_BF16))
    return fail(MOE_ERR_ARG, "moe_layer_norm: bad sizes T=%d H=%d, eps or dtype", T, H);
  if (H > kMaxRow) return fail(MOE_ERR_UNSUPPORTED, "moe_layer_norm: H=%d above %d", H, kMaxRow);
  if (T == 0) return MOE_OK;
  if (!x || !gamma || !y) return fail(MOE_ERR_ARG, "moe_layer_norm: null pointer");
  hipStream_t s = as_stream(stream);
  const int rc = dtype == MOE_F32 ? norm<float>(x, gamma, beta, T, H, eps, y, mean, rstd, s)
                                  : norm<uint16_t>(x, gamma, beta, T, H, eps, y, mean, rstd, s);
  return debug_check(rc, "moe_layer_norm", s, nullptr);
}

extern "C" int moe_layer_norm_backward_workspace_size(int T, int H, size_t* bytes) {
  using namespace moe;
  if (!bytes || T < 0 || H < 1)
    return fail(MOE_ERR_ARG, "moe_layer_norm_backward_workspace_size: bad arguments");
  *bytes = norm_backward_ws(T, H);
  return MOE_OK;
}

extern "C" int moe_layer_norm_backward(const void* dy, const void* x, const float* gamma,
                                       const float* mean, const float* rstd, int T, int H,
                                       moe_dtype dtype, void* dx, float* dgamma, float* dbeta, void* ws,
                                       size_t ws_bytes, moe_stream_t stream) {
  using namespace moe;
  if (T < 0 || H < 1 || (dtype != MOE_F32 && dtype != MOE_BF16))
    return fail(MOE_ERR_ARG, "moe_layer_norm_backward: bad sizes T=%d H=%d or dtype", T, H);
  if (H > kMaxRow)
    return fail(MOE_ERR_UNSUPPORTED, "moe_layer_norm_backward: H=%d above %d", H, kMaxRow);
  const bool sums = dgamma || dbeta;
  if (T > 0 && (!dy || !x || !gamma || !mean || !rstd || !dx))
    return fail(MOE_ERR_ARG, "moe_layer_norm_backward: null pointer");
  const size_t need = norm_backward_ws(T, H);
  if (sums && need > 0 && (!ws || ws_bytes < need))
    return fail(MOE_ERR_WORKSPACE, "moe_layer_norm_backward: workspace %zu < %zu bytes", ws_bytes, need);
  if (T == 0 && !sums) return MOE_OK;
  hipStream_t s = as_stream(stream);
  float* partial = sums ? static_cast<float*>(ws) : nullptr;
  if (T > 0) {
    const int rc = dtype == MOE_F32
                       ? norm_backward<float>(dy, x, gamma, mean, rstd, T, H, dx, partial, s)
                       : norm_backward<uint16_t>(dy, x, gamma, mean, rstd, T, H, dx, partial, s);
    if (rc) return rc;
  }
  if (sums) {
    // no rows: zero sums
    hipLaunchKernelGGL(norm_sum_kernel,
                       dim3(static_cast<unsigned>(ceil_div64(2 * static_cast<int64_t>(H), kWave))),
                       dim3(kSumWaves * kWave), 0, s, partial, norm_partials(T), H, dgamma, dbeta);
    MOE_LAUNCH_CHECK("moe_layer_norm_backward: sum launch");
  }
  return debug_check(MOE_OK, "moe_layer_norm_backward", s, nullptr);
}
