// moe_layer_norm and moe_layer_norm_backward: the norm in front of the router and the experts.
//
//   forward   mu = mean x,  r = 1 / sqrt(mean (x - mu)^2 + eps),  y = (x - mu) r gamma + beta
//   backward  xh = (x - mu) r,  a = dy gamma,
//             dx = r (a - mean a - xh mean(a xh)),  dgamma = sum_t dy xh,  dbeta = sum_t dy
//
// Both are bound by HBM: a row is read once, held in registers as fp32, and every statistic is an
// fp32 sum over it (the variance from the centred values, not from a difference of two sums, so
// a row far from zero loses nothing).  Measured, bf16, 16384 rows of 7168: forward 93-105 us
// (4.5-5.1 TB/s), backward with all three gradients 149 us (4.7 TB/s); a copy kernel with as many loads
// in flight as it can use reaches 6.0.  One row 3.3 us.
#include <algorithm>

#include "rows.h"

namespace moe {
namespace {

constexpr int kMaxWaves = 16;

// The sum of 16 floats of LDS, in order: an entry per wave, zeros where there are fewer.
__device__ __forceinline__ float sum16(const float* part) {
  typedef float f32x4 __attribute__((ext_vector_type(4)));
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxWaves / 4; ++i) {
    const f32x4 v = reinterpret_cast<const f32x4*>(part)[i];
    s += (v[0] + v[1]) + (v[2] + v[3]);
  }
  return s;
}

// Sum of one value over the waves of a block that share a row.  `part` is 16 floats of LDS that no
// other sum of the same barrier interval uses, zero past the block's waves.
__device__ __forceinline__ float row_sum(float v, int waves, float* part) {
  v = wave_sum(v);
  if (waves == 1) return v;
  if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = v;
  __syncthreads();
  return sum16(part);
}

// `waves` waves per row, each lane NV vectors of 8 elements: H <= waves * 64 * NV * 8.  Rows of one
// wave go four to a block, each wave on its own.  A block (wave) takes every `step`-th row.  KEEP:
// gamma and beta stay in registers from row to row (as fp32 they are twice a bf16 row and would
// come from L2 again for each) and the next row's loads are issued before this row's sums.
// TAIL: H is not a multiple of 8.
template <typename T, int NV, bool KEEP, bool TAIL>
__global__ __launch_bounds__(1024) void norm_kernel(
    const T* __restrict__ x, const float* __restrict__ gamma, const float* __restrict__ beta,
    int rows, int H, int waves, float eps, T* __restrict__ y, float* __restrict__ mean,
    float* __restrict__ rstd) {
  __shared__ __attribute__((aligned(16))) float part[2][2][kMaxWaves];
  // entries without a wave: nobody else writes them, and a barrier comes before the first read
  if (waves > 1 && threadIdx.x < 4 * kMaxWaves && threadIdx.x % kMaxWaves >= waves)
    (&part[0][0][0])[threadIdx.x] = 0.f;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int tid = waves == 1 ? threadIdx.x & (kWave - 1) : threadIdx.x, lanes = waves * kWave;
  const int64_t step = waves == 1 ? static_cast<int64_t>(gridDim.x) * 4 : gridDim.x;
  int64_t row = waves == 1 ? static_cast<int64_t>(blockIdx.x) * 4 + wave : blockIdx.x;
  Raw8<T> raw[NV];
  float g[NV][kVec], b[NV][kVec];
  auto fetch = [&]() {
    const int n = row < rows ? H : 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) load_raw<true, TAIL>(x + (n ? row * H : 0), tid + i * lanes, n, raw[i]);
  };
  auto scale = [&](int i) {
    load8<false, TAIL>(gamma, tid + i * lanes, H, g[i]);
    load8<false, TAIL>(beta, tid + i * lanes, beta ? H : 0, b[i]);
  };
  fetch();
  if (KEEP)
#pragma unroll
    for (int i = 0; i < NV; ++i) scale(i);
  for (int turn = 0; row < rows; turn ^= 1) {
    const int64_t at_row = row;
    float v[NV][kVec];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unpack<TAIL>(raw[i], tid + i * lanes, H, v[i]);
#pragma unroll
      for (int j = 0; j < kVec; ++j) s += v[i][j];
    }
    row += step;
    if (KEEP) fetch();
    // the sums' buffers alternate from row to row
    const float mu = row_sum(s, waves, part[turn][0]) / H;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const int at = (tid + i * lanes) * kVec + j;
        v[i][j] = at < H ? v[i][j] - mu : 0.f;
        q = fmaf(v[i][j], v[i][j], q);
      }
    const float r = 1.f / sqrtf(row_sum(q, waves, part[turn][1]) / H + eps);
    T* yr = y + at_row * H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!KEEP) scale(i);
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[i][j] = fmaf(v[i][j] * r, g[i][j], b[i][j]);
      store8<true, TAIL>(yr, tid + i * lanes, H, v[i]);
    }
    if (tid == 0) {
      if (mean) mean[at_row] = mu;
      if (rstd) rstd[at_row] = r;
    }
    if (!KEEP) fetch();
  }
}

// Rows too long for registers (H > 32768): the row is read three times, the later two from L2.
template <typename T>
__global__ __launch_bounds__(1024) void norm_long_kernel(
    const T* __restrict__ x, const float* __restrict__ gamma, const float* __restrict__ beta, int H,
    float eps, T* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd) {
  constexpr bool TAIL = true;
  __shared__ __attribute__((aligned(16))) float part[2][kMaxWaves];
  const int row = blockIdx.x;
  const T* xr = x + static_cast<int64_t>(row) * H;
  const int64_t n_vec = (static_cast<int64_t>(H) + kVec - 1) / kVec;
  float v[kVec];
  float s = 0.f;
  for (int64_t at = threadIdx.x; at < n_vec; at += 1024) {
    load8<false, TAIL>(xr, at, H, v);
#pragma unroll
    for (int j = 0; j < kVec; ++j) s += v[j];
  }
  const float mu = row_sum(s, kMaxWaves, part[0]) / H;
  float q = 0.f;
  for (int64_t at = threadIdx.x; at < n_vec; at += 1024) {
    load8<false, TAIL>(xr, at, H, v);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const float c = at * kVec + j < H ? v[j] - mu : 0.f;
      q = fmaf(c, c, q);
    }
  }
  const float r = 1.f / sqrtf(row_sum(q, kMaxWaves, part[1]) / H + eps);
  T* yr = y + static_cast<int64_t>(row) * H;
  for (int64_t at = threadIdx.x; at < n_vec; at += 1024) {
    float g[kVec], b[kVec];
    load8<false, TAIL>(xr, at, H, v);
    load8<false, TAIL>(gamma, at, H, g);
#pragma unroll
    for (int j = 0; j < kVec; ++j) b[j] = 0.f;
    if (beta) load8<false, TAIL>(beta, at, H, b);
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = fmaf((v[j] - mu) * r, g[j], b[j]);
    store8<true, TAIL>(yr, at, H, v);
  }
  if (threadIdx.x == 0) {
    if (mean) mean[row] = mu;
    if (rstd) rstd[row] = r;
  }
}

// Backward.  `waves` waves share a row and the block has groups = blockDim / (64 waves) such
// teams; team g takes rows blockIdx * groups + g, then gridDim * groups further on.  Its lanes own
// fixed columns, so the sums over its rows for dgamma and dbeta stay in registers; the block's
// teams are joined in LDS in team order and leave as one partial row of 2 H floats
// (partial != nullptr).  Every team makes the same number of turns, so all waves meet at the
// barriers.  AHEAD: the next row's loads are issued before this row's sums, so they are in
// flight while the waves wait for one another, and gamma stays in registers (one vector a lane;
// with two, the registers go to the sums and gamma comes from L2).
template <typename T, int NV, bool AHEAD, bool TAIL>
__global__ __launch_bounds__(1024) void norm_backward_kernel(
    const T* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ gamma,
    const float* __restrict__ mean, const float* __restrict__ rstd, int rows, int H, int waves,
    int groups, T* __restrict__ dx, float* __restrict__ partial) {
  extern __shared__ __attribute__((aligned(16))) float joined[];  // [groups][2 H]
  __shared__ __attribute__((aligned(16))) float part[2][2][kMaxWaves][kMaxWaves];  // [team][wave]
  const int lanes = waves * kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int group = wave / waves, tid = threadIdx.x - group * lanes;
  const int step = gridDim.x * groups;
  const int in_team = wave - group * waves;
  // entries past a team's waves: nobody else writes them, and a barrier comes before the first read
  if (waves > 1)
    for (int i = threadIdx.x; i < 4 * kMaxWaves * kMaxWaves; i += blockDim.x)
      if (i % kMaxWaves >= waves) (&part[0][0][0][0])[i] = 0.f;
  float sg[NV][kVec], sb[NV][kVec], g[NV][kVec];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (AHEAD) load8<false, TAIL>(gamma, tid + i * lanes, H, g[i]);
#pragma unroll
    for (int j = 0; j < kVec; ++j) sg[i][j] = sb[i][j] = 0.f;
  }
  Raw8<T> xn[NV], dn[NV];
  float mu_n = 0.f, r_n = 0.f;
  auto fetch = [&](int64_t r) {
    const int n = r < rows ? H : 0;  // a turn without a row: zeros
    const int64_t at = r < rows ? r : 0;
    mu_n = n ? mean[at] : 0.f;
    r_n = n ? rstd[at] : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      load_raw<true, TAIL>(x + at * H, tid + i * lanes, n, xn[i]);
      load_raw<true, TAIL>(dy + at * H, tid + i * lanes, n, dn[i]);
    }
  };
  int64_t first = static_cast<int64_t>(blockIdx.x) * groups, row = first + group;
  if (AHEAD) fetch(row);
  for (int turn = 0; first < rows; first += step, row += step, turn ^= 1) {
    if (!AHEAD) fetch(row);
    const float mu = mu_n, r = r_n;
    float a[NV][kVec], xh[NV][kVec];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unpack<TAIL>(xn[i], tid + i * lanes, H, xh[i]);
      unpack<TAIL>(dn[i], tid + i * lanes, H, a[i]);
    }
    if (AHEAD) fetch(row + step);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!AHEAD) load8<false, TAIL>(gamma, tid + i * lanes, H, g[i]);
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
    }
    s1 = wave_sum(s1);
    s2 = wave_sum(s2);
    if (waves > 1) {
      // the buffers alternate from row to row, so one barrier a row is enough
      if ((threadIdx.x & (kWave - 1)) == 0) {
        part[turn][0][group][in_team] = s1;
        part[turn][1][group][in_team] = s2;
      }
      __syncthreads();
      s1 = sum16(part[turn][0][group]);
      s2 = sum16(part[turn][1][group]);
    }
    s1 /= H;
    s2 /= H;
    if (row >= rows) continue;
    T* out = dx + row * H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) a[i][j] = r * (a[i][j] - s1 - xh[i][j] * s2);
      store8<true, TAIL>(out, tid + i * lanes, H, a[i]);
    }
  }
  if (!partial) return;
  float* p = partial + static_cast<int64_t>(blockIdx.x) * 2 * H;
  if (groups == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      store8<false, TAIL>(p, tid + i * lanes, H, sg[i]);
      store8<false, TAIL>(p + H, tid + i * lanes, H, sb[i]);
    }
    return;
  }
  float* mine = joined + group * 2 * H;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    store8<false, TAIL>(mine, tid + i * lanes, H, sg[i]);
    store8<false, TAIL>(mine + H, tid + i * lanes, H, sb[i]);
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * H; c += blockDim.x) {
    float s = 0.f;
    for (int k = 0; k < groups; ++k) s += joined[k * 2 * H + c];
    p[c] = s;
  }
}

// Rows too long for registers: dx alone, the row read twice.
template <typename T>
__global__ __launch_bounds__(1024) void norm_backward_long_kernel(
    const T* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ gamma,
    const float* __restrict__ mean, const float* __restrict__ rstd, int H, T* __restrict__ dx) {
  constexpr bool TAIL = true;
  __shared__ __attribute__((aligned(16))) float part[2][kMaxWaves];
  const int row = blockIdx.x;
  const T* xr = x + static_cast<int64_t>(row) * H;
  const T* dr = dy + static_cast<int64_t>(row) * H;
  const float mu = mean[row], r = rstd[row];
  const int64_t n_vec = (static_cast<int64_t>(H) + kVec - 1) / kVec;
  float a[kVec], xh[kVec], g[kVec];
  float s1 = 0.f, s2 = 0.f;
  for (int64_t at = threadIdx.x; at < n_vec; at += 1024) {
    load8<false, TAIL>(xr, at, H, xh);
    load8<false, TAIL>(dr, at, H, a);
    load8<false, TAIL>(gamma, at, H, g);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      s1 = fmaf(a[j], g[j], s1);
      s2 = fmaf(a[j] * g[j], (xh[j] - mu) * r, s2);
    }
  }
  s1 = row_sum(s1, kMaxWaves, part[0]) / H;
  s2 = row_sum(s2, kMaxWaves, part[1]) / H;
  T* out = dx + static_cast<int64_t>(row) * H;
  for (int64_t at = threadIdx.x; at < n_vec; at += 1024) {
    load8<false, TAIL>(xr, at, H, xh);
    load8<false, TAIL>(dr, at, H, a);
    load8<false, TAIL>(gamma, at, H, g);
#pragma unroll
    for (int j = 0; j < kVec; ++j) a[j] = r * (a[j] * g[j] - s1 - (xh[j] - mu) * r * s2);
    store8<true, TAIL>(out, at, H, a);
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
#pragma unroll 16
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

constexpr int kMaxH = kMaxWaves * kWave * 4 * kVec;          // 32768: the longest row norm_kernel holds
constexpr int kMaxBackwardH = kMaxWaves * kWave * 2 * kVec;  // 16384: the longest of the backward kernel
constexpr int kPartials = kCus;                              // most blocks of the backward pass
constexpr int kJoinBytes = kMaxWaves * kWave * kVec * 2 * sizeof(float);  // 64 KB: 16 waves' sums

// Waves per row and rows at once per block of the backward pass: as many waves as the row has 512
// columns, as many rows as 16 waves hold, and a block a CU: twice the blocks at 10 waves each mean
// twice the partial rows, which cost more than they gain (4099 x 1001 f32: 24.6 against 19.6 us).
struct BackwardShape {
  int nv, waves, groups, blocks;
};

BackwardShape backward_shape(int T, int H) {
  BackwardShape b;
  b.nv = H <= kMaxBackwardH / 2 ? 1 : 2;
  b.waves = ceil_div(H, b.nv * kWave * kVec);
  b.groups = std::max(1, kMaxWaves / b.waves);
  b.blocks = static_cast<int>(std::min<int64_t>(kPartials, ceil_div64(T, b.groups)));
  return b;
}

int norm_partials(int T, int H) {
  return H <= kMaxBackwardH ? backward_shape(T, H).blocks : std::min(T, kPartials);
}

template <typename E, int NV>
int launch_norm(const void* x, const float* gamma, const float* beta, int T, int H, float eps, void* y,
                float* mean, float* rstd, hipStream_t s) {
  const int waves = ceil_div(H, NV * kWave * kVec), rows = waves == 1 ? 4 : 1;
  // as many blocks as the CUs hold at once (16 waves a CU at the registers of KEEP); when that is
  // every row, KEEP has nothing to keep for, and its registers only take waves from the CU
  const int64_t all = ceil_div64(T, rows), most = kCus * std::max(1, 16 / (waves * rows));
  const bool keep = NV <= 2 && all > 2 * most;
  const int64_t blocks = keep ? most : all;
  if (too_many(blocks, waves * rows * kWave))
    return fail(MOE_ERR_UNSUPPORTED, "moe_layer_norm: T=%d too large at H=%d", T, H);
  auto kernel = H % kVec == 0
                    ? (keep ? norm_kernel<E, NV, NV <= 2, false> : norm_kernel<E, NV, false, false>)
                    : (keep ? norm_kernel<E, NV, NV <= 2, true> : norm_kernel<E, NV, false, true>);
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(blocks)), dim3(waves * rows * kWave), 0, s,
                     static_cast<const E*>(x), gamma, beta, T, H, waves, eps, static_cast<E*>(y), mean,
                     rstd);
  MOE_LAUNCH_CHECK("moe_layer_norm: launch");
  return MOE_OK;
}

template <typename E>
int norm(const void* x, const float* gamma, const float* beta, int T, int H, float eps, void* y,
         float* mean, float* rstd, hipStream_t s) {
#define NORM(NV) return launch_norm<E, NV>(x, gamma, beta, T, H, eps, y, mean, rstd, s)
  // Few rows, which leave CUs idle: a vector a lane, so that a row's loads spread over more waves.
  // Many rows: two, so that fewer waves wait for one another.
  const int per = kWave * kVec;
  if (H <= per || (T <= kCus && H <= kMaxWaves * per)) NORM(1);
  if (H <= kMaxWaves * 2 * per) NORM(2);
  if (H <= kMaxH) NORM(4);
#undef NORM
  hipLaunchKernelGGL(norm_long_kernel<E>, dim3(T), dim3(1024), 0, s, static_cast<const E*>(x), gamma,
                     beta, H, eps, static_cast<E*>(y), mean, rstd);
  MOE_LAUNCH_CHECK("moe_layer_norm: launch");
  return MOE_OK;
}

template <typename E>
int norm_backward(const void* dy, const void* x, const float* gamma, const float* mean, const float* rstd,
                  int T, int H, void* dx, float* partial, hipStream_t s) {
  if (H <= kMaxBackwardH) {
    const BackwardShape b = backward_shape(T, H);
    auto kernel = H % kVec == 0
                      ? (b.nv == 1 ? norm_backward_kernel<E, 1, true, false> : norm_backward_kernel<E, 2, false, false>)
                      : (b.nv == 1 ? norm_backward_kernel<E, 1, true, true> : norm_backward_kernel<E, 2, false, true>);
    const size_t lds = b.groups > 1 && partial ? b.groups * 2 * static_cast<size_t>(H) * sizeof(float) : 0;
    MOE_HIP_CHECK(hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                      hipFuncAttributeMaxDynamicSharedMemorySize, kJoinBytes));
    hipLaunchKernelGGL(kernel, dim3(b.blocks), dim3(b.groups * b.waves * kWave), lds, s,
                       static_cast<const E*>(dy), static_cast<const E*>(x), gamma, mean, rstd, T, H,
                       b.waves, b.groups, static_cast<E*>(dx), partial);
    MOE_LAUNCH_CHECK("moe_layer_norm_backward: launch");
    return MOE_OK;
  }
  hipLaunchKernelGGL(norm_backward_long_kernel<E>, dim3(T), dim3(1024), 0, s, static_cast<const E*>(dy),
                     static_cast<const E*>(x), gamma, mean, rstd, H, static_cast<E*>(dx));
  MOE_LAUNCH_CHECK("moe_layer_norm_backward: launch");
  if (partial) {
    hipLaunchKernelGGL(norm_columns_kernel<E>, dim3(ceil_div(H, 256), norm_partials(T, H)), dim3(256), 0, s,
                       static_cast<const E*>(dy), static_cast<const E*>(x), mean, rstd, T, H, partial);
    MOE_LAUNCH_CHECK("moe_layer_norm_backward: columns launch");
  }
  return MOE_OK;
}

size_t norm_backward_ws(int T, int H) {
  return align_up(static_cast<size_t>(norm_partials(T, H)) * 2 * H * sizeof(float), 256);
}

}  // namespace
}  // namespace moe

extern "C" int moe_layer_norm(const void* x, const float* gamma, const float* beta, int T, int H,
                              float eps, moe_dtype dtype, void* y, float* mean, float* rstd,
                              moe_stream_t stream) {
  using namespace moe;
  if (T < 0 || H < 1 || !(eps >= 0.f) || (dtype != MOE_F32 && dtype != MOE_BF16))
    return fail(MOE_ERR_ARG, "moe_layer_norm: bad sizes T=%d H=%d, eps or dtype", T, H);
  if (H > kMaxRow || (H > kMaxH && too_many(T, 1024)))
    return fail(MOE_ERR_UNSUPPORTED, "moe_layer_norm: H=%d above %d, or T=%d too large for it", H, kMaxRow, T);
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
  if (H > kMaxRow || (H > kMaxBackwardH && too_many(T, 1024)))
    return fail(MOE_ERR_UNSUPPORTED, "moe_layer_norm_backward: H=%d above %d, or T=%d too large for it", H,
                kMaxRow, T);
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
                       dim3(kSumWaves * kWave), 0, s, partial, norm_partials(T, H), H, dgamma, dbeta);
    MOE_LAUNCH_CHECK("moe_layer_norm_backward: sum launch");
  }
  return debug_check(MOE_OK, "moe_layer_norm_backward", s, nullptr);
}
