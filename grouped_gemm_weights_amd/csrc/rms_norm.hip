// moe_rms_norm and moe_rms_norm_backward: the root-mean-square norm with the residual's addition, and
// an output in 8 bits with block scales (mx.h).
//
//   forward   s = x + residual (stored in the stream's type),  r = 1 / sqrt(mean s^2 + eps),
//             y = s r gamma,  q = mx(y)
//   backward  xh = s r,  a = dy gamma,  dx = dsum + r (a - xh mean(a xh)),  dgamma = sum_t dy xh
//
// Both are bound by HBM: a row is read once and held in registers as fp32; its one statistic is an
// fp32 sum over it.  y is quantised from fp32, not from its rounding to bf16.  Measured: bf16, 16384 x 7168
// with the residual, sum, y and 8-bit rows 191 us (5.6 TB/s); 64 x 7168 4.6 us on the GPU, 2-3 of them the
// launch; f32, 4099 x 1001 forward 15, backward 17 + 4 us.
#include <algorithm>

#include "mx.h"
#include "rows.h"

namespace moe {
namespace {

constexpr bool kTail = true;  // rows of any length

__device__ __forceinline__ float stored(float v, const uint16_t*) { return bf16_to_f32(f32_to_bf16(v)); }
__device__ __forceinline__ float stored(float v, const float*) { return v; }

template <typename T>
struct Outputs {
  T* sum;
  T* y;
  uint8_t* q;
  uint8_t* scales;
  float* rstd;
};

// How arrays of this size pass the caches.  Small ones take plain loads and stores: what one kernel writes
// the next finds in the 256 MB that all XCDs share.  Larger ones leave by non-temporal stores, and from
// 96 MB on come by such loads too, as in the backward pass, which reads three.  Measured (loads / stores,
// n: non-temporal): bf16, 16384 rows of 7168 n/n 192 us, -/n 201; of 2048 n/n 46.5, -/n 42.4, -/- 49.7; f32,
// 4099 rows of 1001 n/n 17.2, -/n 15.7, -/- 13.1; backward passes of these two n/n 51.8 and 24.8, -/- after
// a forward pass that leaves the sum behind 48 and 19.3, after one that does not 61 and 19.  Where other
// work has passed the cache in between (f32, both passes in turn on 345 MB) -/-, n/- and n/n take 39.5,
// 40.2 and 42.2 us.
enum Cache { kNear, kPast, kFar };
Cache cache(int64_t T, int H, int size) {
  const int64_t bytes = T * H * size;
  return bytes <= (int64_t{32} << 20) ? kNear : bytes < (int64_t{96} << 20) ? kPast : kFar;
}

// `waves` waves per row, each lane NV vectors of 8 elements: H <= waves * 64 * NV * 8.  Rows of one
// wave go four to a block, each wave on its own.  A block (wave) takes every `step`-th row.  KEEP:
// gamma stays in registers from row to row and the next row's loads are issued before this row's sum.
// TAIL: H is not a multiple of 8.  RES: with a residual.  CACHE: as cache() says.
template <typename T, int NV, bool KEEP, bool TAIL, bool RES, int CACHE>
__global__ __launch_bounds__(1024) void rms_kernel(const T* x, const T* res, const float* __restrict__ gamma,
                                                   int rows, int H, int waves, float eps, Outputs<T> out) {
  __shared__ __attribute__((aligned(16))) float part[2][kMaxWaves];
  // entries without a wave: nobody else writes them, and a barrier comes before the first read
  if (waves > 1 && threadIdx.x < 2 * kMaxWaves && threadIdx.x % kMaxWaves >= waves)
    (&part[0][0])[threadIdx.x] = 0.f;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int tid = waves == 1 ? threadIdx.x & (kWave - 1) : threadIdx.x, lanes = waves * kWave;
  const int64_t step = waves == 1 ? static_cast<int64_t>(gridDim.x) * 4 : gridDim.x;
  int64_t row = waves == 1 ? static_cast<int64_t>(blockIdx.x) * 4 + wave : blockIdx.x;
  Raw8<T> raw[NV], raw_res[RES ? NV : 1];
  float g[NV][kVec];
  auto fetch = [&]() {
    const int n = row < rows ? H : 0;
    const int64_t at = n ? row * H : 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      load_raw<CACHE == kFar, TAIL>(x + at, tid + i * lanes, n, raw[i]);
      if constexpr (RES) load_raw<CACHE == kFar, TAIL>(res + at, tid + i * lanes, n, raw_res[i]);
    }
  };
  fetch();
  if (KEEP)
#pragma unroll
    for (int i = 0; i < NV; ++i) load8<false, TAIL>(gamma, tid + i * lanes, H, g[i]);
  for (int turn = 0; row < rows; turn ^= 1) {
    const int64_t at_row = row;
    float v[NV][kVec];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unpack<TAIL>(raw[i], tid + i * lanes, H, v[i]);
      if constexpr (RES) {
        float b[kVec];
        unpack<TAIL>(raw_res[i], tid + i * lanes, H, b);
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[i][j] = stored(v[i][j] + b[j], x);
        if (out.sum) store8<CACHE != kNear, TAIL>(out.sum + at_row * H, tid + i * lanes, H, v[i]);
      }
#pragma unroll
      for (int j = 0; j < kVec; ++j) s = fmaf(v[i][j], v[i][j], s);
    }
    row += step;
    if (KEEP) fetch();
    // the sum's buffers alternate from row to row
    const float r = 1.f / sqrtf(row_sum(s, waves, part[turn]) / H + eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = tid + i * lanes;
      if (!KEEP) load8<false, TAIL>(gamma, at, H, g[i]);
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[i][j] = v[i][j] * r * g[i][j];
      if (out.y) store8<CACHE != kNear, TAIL>(out.y + at_row * H, at, H, v[i]);
      if (!TAIL && out.q)
        mx_store(v[i], static_cast<int64_t>(at) * kVec, H, out.q + at_row * H, out.scales + at_row * mx_pitch(H));
    }
    if (tid == 0 && out.rstd) out.rstd[at_row] = r;
    if (!KEEP) fetch();
  }
}

// Rows too long for registers (H > 32768): the row is read twice, the second time from L2.  sum may be
// x or the residual itself, so the second reading takes it and not the two that made it.
template <typename T>
__global__ __launch_bounds__(1024) void rms_long_kernel(const T* x, const T* res,
                                                        const float* __restrict__ gamma, int H, float eps,
                                                        Outputs<T> out) {
  __shared__ __attribute__((aligned(16))) float part[kMaxWaves];
  const int64_t first = static_cast<int64_t>(blockIdx.x) * H;
  const int64_t n_vec = (static_cast<int64_t>(H) + kVec - 1) / kVec;
  const int lane = threadIdx.x & (kWave - 1);
  auto load = [&](int64_t at, float (&v)[kVec], bool again) {
    if (again && res && out.sum) {
      load8<false, kTail>(out.sum + first, at, H, v);
      return;
    }
    load8<false, kTail>(x + first, at, H, v);
    if (!res) return;
    float b[kVec];
    load8<false, kTail>(res + first, at, H, b);
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = stored(v[j] + b[j], x);
  };
  float v[kVec], s = 0.f;
  // whole waves take part to the end: they exchange what they hold
  for (int64_t at = threadIdx.x; at - lane < n_vec; at += 1024) {
    load(at, v, false);
#pragma unroll
    for (int j = 0; j < kVec; ++j) s = fmaf(v[j], v[j], s);
    if (res && out.sum) store8<false, kTail>(out.sum + first, at, H, v);
  }
  const float r = 1.f / sqrtf(row_sum(s, kMaxWaves, part) / H + eps);
  for (int64_t at = threadIdx.x; at - lane < n_vec; at += 1024) {
    float g[kVec];
    load(at, v, true);
    load8<false, kTail>(gamma, at, H, g);
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = v[j] * r * g[j];
    if (out.y) store8<true, kTail>(out.y + first, at, H, v);
    if (out.q) mx_store(v, at * kVec, H, out.q + first, out.scales + blockIdx.x * mx_pitch(H));
  }
  if (threadIdx.x == 0 && out.rstd) out.rstd[blockIdx.x] = r;
}

// Backward.  `waves` waves share a row and the block has groups = blockDim / (64 waves) such teams;
// team g takes rows blockIdx * groups + g, then gridDim * groups further on.  Its lanes own fixed
// columns, so the sums over its rows for dgamma stay in registers; the block's teams are joined in LDS
// in team order and leave as one partial row of H floats (partial != nullptr).  Every team makes the
// same number of turns, so all waves meet at the barriers.  AHEAD: the next row's loads are issued
// before this row's sum and gamma stays in registers.  FAR: non-temporal loads and stores.
template <typename T, int NV, bool AHEAD, bool TAIL, bool FAR>
__global__ __launch_bounds__(1024) void rms_backward_kernel(
    const T* __restrict__ dy, const T* dsum, const T* __restrict__ x, const float* __restrict__ gamma,
    const float* __restrict__ rstd, int rows, int H, int waves, int groups, T* dx,
    float* __restrict__ partial) {
  extern __shared__ __attribute__((aligned(16))) float joined[];  // [groups][H]
  __shared__ __attribute__((aligned(16))) float part[2][kMaxWaves][kMaxWaves];  // [team][wave]
  const int lanes = waves * kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int group = wave / waves, tid = threadIdx.x - group * lanes;
  const int step = gridDim.x * groups;
  const int in_team = wave - group * waves;
  // entries past a team's waves: nobody else writes them, and a barrier comes before the first read
  if (waves > 1)
    for (int i = threadIdx.x; i < 2 * kMaxWaves * kMaxWaves; i += blockDim.x)
      if (i % kMaxWaves >= waves) (&part[0][0][0])[i] = 0.f;
  float sg[NV][kVec], g[NV][kVec];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (AHEAD) load8<false, TAIL>(gamma, tid + i * lanes, H, g[i]);
#pragma unroll
    for (int j = 0; j < kVec; ++j) sg[i][j] = 0.f;
  }
  Raw8<T> xn[NV], dn[NV], sn[NV];
  float r_n = 0.f;
  auto fetch = [&](int64_t r) {
    const int n = r < rows ? H : 0;  // a turn without a row: zeros
    const int64_t at = n ? r * H : 0;
    r_n = n ? rstd[r] : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      load_raw<FAR, TAIL>(x + at, tid + i * lanes, n, xn[i]);
      load_raw<FAR, TAIL>(dy + at, tid + i * lanes, n, dn[i]);
      load_raw<FAR, TAIL>(dsum + at, tid + i * lanes, dsum ? n : 0, sn[i]);
    }
  };
  int64_t first = static_cast<int64_t>(blockIdx.x) * groups, row = first + group;
  if (AHEAD) fetch(row);
  for (int turn = 0; first < rows; first += step, row += step, turn ^= 1) {
    if (!AHEAD) fetch(row);
    const float r = r_n;
    float a[NV][kVec], xh[NV][kVec], d[NV][kVec];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unpack<TAIL>(xn[i], tid + i * lanes, H, xh[i]);
      unpack<TAIL>(dn[i], tid + i * lanes, H, a[i]);
      unpack<TAIL>(sn[i], tid + i * lanes, dsum ? H : 0, d[i]);
    }
    if (AHEAD) fetch(row + step);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!AHEAD) load8<false, TAIL>(gamma, tid + i * lanes, H, g[i]);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        xh[i][j] *= r;
        sg[i][j] = fmaf(a[i][j], xh[i][j], sg[i][j]);
        a[i][j] *= g[i][j];
        s = fmaf(a[i][j], xh[i][j], s);
      }
    }
    s = wave_sum(s);
    if (waves > 1) {
      // the buffers alternate from row to row, so one barrier a row is enough
      if ((threadIdx.x & (kWave - 1)) == 0) part[turn][group][in_team] = s;
      __syncthreads();
      s = sum16(part[turn][group]);
    }
    s /= H;
    if (row >= rows) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) a[i][j] = fmaf(r, a[i][j] - xh[i][j] * s, d[i][j]);
      store8<FAR, TAIL>(dx + row * H, tid + i * lanes, H, a[i]);
    }
  }
  if (!partial) return;
  float* p = partial + static_cast<int64_t>(blockIdx.x) * H;
  if (groups == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) store8<false, TAIL>(p, tid + i * lanes, H, sg[i]);
    return;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) store8<false, TAIL>(joined + group * H, tid + i * lanes, H, sg[i]);
  __syncthreads();
  for (int c = threadIdx.x; c < H; c += blockDim.x) {
    float s = 0.f;
    for (int k = 0; k < groups; ++k) s += joined[k * H + c];
    p[c] = s;
  }
}

// Rows too long for registers: dx alone, the row read twice.
template <typename T>
__global__ __launch_bounds__(1024) void rms_backward_long_kernel(
    const T* __restrict__ dy, const T* dsum, const T* __restrict__ x, const float* __restrict__ gamma,
    const float* __restrict__ rstd, int H, T* dx) {
  __shared__ __attribute__((aligned(16))) float part[kMaxWaves];
  const int64_t first = static_cast<int64_t>(blockIdx.x) * H;
  const float r = rstd[blockIdx.x];
  const int64_t n_vec = (static_cast<int64_t>(H) + kVec - 1) / kVec;
  float a[kVec], xh[kVec], g[kVec];
  float s = 0.f;
  for (int64_t at = threadIdx.x; at < n_vec; at += 1024) {
    load8<false, kTail>(x + first, at, H, xh);
    load8<false, kTail>(dy + first, at, H, a);
    load8<false, kTail>(gamma, at, H, g);
#pragma unroll
    for (int j = 0; j < kVec; ++j) s = fmaf(a[j] * g[j], xh[j] * r, s);
  }
  s = row_sum(s, kMaxWaves, part) / H;
  for (int64_t at = threadIdx.x; at < n_vec; at += 1024) {
    float d[kVec];
    load8<false, kTail>(x + first, at, H, xh);
    load8<false, kTail>(dy + first, at, H, a);
    load8<false, kTail>(gamma, at, H, g);
    load8<false, kTail>(dsum + first, at, dsum ? H : 0, d);
#pragma unroll
    for (int j = 0; j < kVec; ++j) a[j] = fmaf(r, a[j] * g[j] - xh[j] * r * s, d[j]);
    store8<true, kTail>(dx + first, at, H, a);
  }
}

// Its column sums: one thread per column and block of rows, straight from x and dy.
template <typename T>
__global__ __launch_bounds__(256) void rms_columns_kernel(const T* __restrict__ dy, const T* __restrict__ x,
                                                          const float* __restrict__ rstd, int rows, int H,
                                                          float* __restrict__ partial) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= H) return;
  float s = 0.f;
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
    s = fmaf(d, v * rstd[row], s);
  }
  partial[static_cast<int64_t>(blockIdx.y) * H + c] = s;
}

// dgamma from n partial rows of H floats: 64 columns per block, 16 waves that each take every 16th
// row, joined in LDS in wave order.
__global__ __launch_bounds__(kMaxWaves* kWave) void rms_sum_kernel(const float* __restrict__ partial, int n,
                                                                   int H, float* __restrict__ dgamma) {
  __shared__ float s[kMaxWaves][kWave];
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kWave + lane;
  float v = 0.f;
  if (c < H) {
#pragma unroll 16
    for (int i = w; i < n; i += kMaxWaves) v += partial[static_cast<int64_t>(i) * H + c];
  }
  s[w][lane] = v;
  __syncthreads();
  if (w == 0 && c < H) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxWaves; ++i) v += s[i][lane];
    dgamma[c] = v;
  }
}

constexpr int kMaxH = kMaxWaves * kWave * 4 * kVec;          // 32768: the longest row rms_kernel holds
constexpr int kMaxBackwardH = kMaxWaves * kWave * 2 * kVec;  // 16384: the longest of the backward kernel

// Waves per row, rows at once per block and blocks of the backward pass: as many waves as the row has
// 512 columns, as many rows as 16 waves hold, and a block a CU (more would mean more partial rows).  Two
// turns of one block are shorter than the launch that would add two blocks' sums.
struct BackwardShape {
  int nv, waves, groups, blocks;
};

BackwardShape backward_shape(int T, int H) {
  BackwardShape b;
  b.nv = H <= kMaxBackwardH / 2 ? 1 : 2;
  b.waves = ceil_div(H, b.nv * kWave * kVec);
  b.groups = std::max(1, kMaxWaves / b.waves);
  b.blocks = T <= 2 * b.groups ? std::min(T, 1) : static_cast<int>(std::min<int64_t>(kCus, ceil_div64(T, b.groups)));
  return b;
}

int partials(int T, int H) {
  return H <= kMaxBackwardH ? backward_shape(T, H).blocks : std::min(T, kCus);
}

template <typename E, int NV, bool RES, int CACHE>
int launch_rms(const E* x, const E* res, const float* gamma, int T, int H, float eps, const Outputs<E>& out,
               hipStream_t s) {
  const int waves = ceil_div(H, NV * kWave * kVec), rows = waves == 1 ? 4 : 1;
  // as many blocks as the CUs hold at once (16 waves a CU at the registers of KEEP); when that is
  // every row, KEEP has nothing to keep for, and its registers only take waves from the CU
  const int64_t all = ceil_div64(T, rows), most = kCus * std::max(1, 16 / (waves * rows));
  const bool keep = NV <= 2 && all > 2 * most;
  const int64_t blocks = keep ? most : all;
  if (too_many(blocks, waves * rows * kWave))
    return fail(MOE_ERR_UNSUPPORTED, "moe_rms_norm: T=%d too large at H=%d", T, H);
  // Up to 2 * most blocks hold at most 512 * 16 waves of 512 NV elements: with NV <= 2 that is 32 MB, so
  // larger arrays are all KEEP
  constexpr bool always = NV <= 2 && CACHE != kNear, never = NV > 2;
  auto kernel = H % kVec == 0
                    ? (keep ? rms_kernel<E, NV, !never, false, RES, CACHE> : rms_kernel<E, NV, always, false, RES, CACHE>)
                    : (keep ? rms_kernel<E, NV, !never, true, RES, CACHE> : rms_kernel<E, NV, always, true, RES, CACHE>);
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(blocks)), dim3(waves * rows * kWave), 0, s, x, res,
                     gamma, T, H, waves, eps, out);
  MOE_LAUNCH_CHECK("moe_rms_norm: launch");
  return MOE_OK;
}

template <typename E>
int rms(const void* xv, const void* rv, const float* gamma, int T, int H, float eps, const Outputs<E>& out,
        hipStream_t s) {
  const E* x = static_cast<const E*>(xv);
  const E* res = static_cast<const E*>(rv);
  const Cache how = cache(T, H, sizeof(E));
#define RMS_OF(NV, RES) \
  (how == kNear ? launch_rms<E, NV, RES, kNear> : how == kPast ? launch_rms<E, NV, RES, kPast> : launch_rms<E, NV, RES, kFar>)
#define RMS(NV) return (res ? RMS_OF(NV, true) : RMS_OF(NV, false))(x, res, gamma, T, H, eps, out, s)
  // Few rows, which leave CUs idle: a vector a lane, so that a row's loads spread over more waves.
  // Many rows: two, so that fewer waves wait for one another.
  const int per = kWave * kVec;
  if (H <= per || (T <= kCus && H <= kMaxWaves * per)) RMS(1);
  if (H <= kMaxWaves * 2 * per) RMS(2);
  if (H <= kMaxH) RMS(4);
#undef RMS
#undef RMS_OF
  hipLaunchKernelGGL(rms_long_kernel<E>, dim3(T), dim3(1024), 0, s, x, res, gamma, H, eps, out);
  MOE_LAUNCH_CHECK("moe_rms_norm: launch");
  return MOE_OK;
}

template <typename E>
int rms_backward(const void* dyv, const void* dsv, const void* xv, const float* gamma, const float* rstd, int T,
                 int H, void* dxv, float* partial, hipStream_t s) {
  const E* dy = static_cast<const E*>(dyv);
  const E* dsum = static_cast<const E*>(dsv);
  const E* x = static_cast<const E*>(xv);
  E* dx = static_cast<E*>(dxv);
  if (H <= kMaxBackwardH) {
    const BackwardShape b = backward_shape(T, H);
    const bool far = cache(T, H, sizeof(E)) != kNear;
#define BACKWARD(NV, AHEAD, TAIL) \
  (far ? rms_backward_kernel<E, NV, AHEAD, TAIL, true> : rms_backward_kernel<E, NV, AHEAD, TAIL, false>)
    auto kernel = H % kVec == 0 ? (b.nv == 1 ? BACKWARD(1, true, false) : BACKWARD(2, false, false))
                                : (b.nv == 1 ? BACKWARD(1, true, true) : BACKWARD(2, false, true));
#undef BACKWARD
    const size_t lds = b.groups > 1 && partial ? b.groups * static_cast<size_t>(H) * sizeof(float) : 0;
    hipLaunchKernelGGL(kernel, dim3(b.blocks), dim3(b.groups * b.waves * kWave), lds, s, dy, dsum, x, gamma,
                       rstd, T, H, b.waves, b.groups, dx, partial);
    MOE_LAUNCH_CHECK("moe_rms_norm_backward: launch");
    return MOE_OK;
  }
  hipLaunchKernelGGL(rms_backward_long_kernel<E>, dim3(T), dim3(1024), 0, s, dy, dsum, x, gamma, rstd, H, dx);
  MOE_LAUNCH_CHECK("moe_rms_norm_backward: launch");
  if (partial) {
    hipLaunchKernelGGL(rms_columns_kernel<E>, dim3(ceil_div(H, 256), partials(T, H)), dim3(256), 0, s, dy, x,
                       rstd, T, H, partial);
    MOE_LAUNCH_CHECK("moe_rms_norm_backward: columns launch");
  }
  return MOE_OK;
}

size_t backward_ws(int T, int H) {
  return align_up(static_cast<size_t>(partials(T, H)) * H * sizeof(float), 256);
}

}  // namespace
}  // namespace moe

extern "C" int moe_rms_norm(const void* x, const void* residual, const float* gamma, int T, int H, float eps,
                            moe_dtype dtype, void* sum, void* y, uint8_t* q, uint8_t* scales, float* rstd,
                            moe_stream_t stream) {
  using namespace moe;
  const char* who = "moe_rms_norm";
  if (T < 0 || H < 1 || !(eps >= 0.f) || !is_dtype(dtype))
    return fail(MOE_ERR_ARG, "%s: bad sizes T=%d H=%d, eps or dtype", who, T, H);
  if (!q != !scales) return fail(MOE_ERR_ARG, "%s: q and scales come together", who);
  if (sum && !residual) return fail(MOE_ERR_ARG, "%s: a sum without a residual", who);
  if (H > kMaxRow || (H > kMaxH && too_many(T, 1024)))
    return fail(MOE_ERR_UNSUPPORTED, "%s: H=%d above %d, or T=%d too large for it", who, H, kMaxRow, T);
  if (q && H % kMxBlock != 0)
    return fail(MOE_ERR_UNSUPPORTED, "%s: H=%d is not a multiple of %d, as 8-bit rows need", who, H, kMxBlock);
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(scales)) % 16 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "%s: q or scales is not aligned to 16 bytes", who);
  if (T == 0) return MOE_OK;
  if (!x || !gamma || (!y && !q)) return fail(MOE_ERR_ARG, "%s: null pointer", who);
  hipStream_t s = as_stream(stream);
  const int rc =
      dtype == MOE_F32
          ? rms<float>(x, residual, gamma, T, H, eps,
                       Outputs<float>{static_cast<float*>(sum), static_cast<float*>(y), q, scales, rstd}, s)
          : rms<uint16_t>(x, residual, gamma, T, H, eps,
                          Outputs<uint16_t>{static_cast<uint16_t*>(sum), static_cast<uint16_t*>(y), q, scales, rstd},
                          s);
  return debug_check(rc, who, s, nullptr);
}

extern "C" int moe_rms_norm_backward_workspace_size(int T, int H, size_t* bytes) {
  using namespace moe;
  if (!bytes || T < 0 || H < 1) return fail(MOE_ERR_ARG, "moe_rms_norm_backward_workspace_size: bad arguments");
  *bytes = backward_ws(T, H);
  return MOE_OK;
}

extern "C" int moe_rms_norm_backward(const void* dy, const void* dsum, const void* x, const float* gamma,
                                     const float* rstd, int T, int H, moe_dtype dtype, void* dx, float* dgamma,
                                     void* ws, size_t ws_bytes, moe_stream_t stream) {
  using namespace moe;
  const char* who = "moe_rms_norm_backward";
  if (T < 0 || H < 1 || !is_dtype(dtype)) return fail(MOE_ERR_ARG, "%s: bad sizes T=%d H=%d or dtype", who, T, H);
  if (H > kMaxRow || (H > kMaxBackwardH && too_many(T, 1024)))
    return fail(MOE_ERR_UNSUPPORTED, "%s: H=%d above %d, or T=%d too large for it", who, H, kMaxRow, T);
  if (T > 0 && (!dy || !x || !gamma || !rstd || !dx)) return fail(MOE_ERR_ARG, "%s: null pointer", who);
  const size_t need = backward_ws(T, H);
  if (dgamma && need > 0 && (!ws || ws_bytes < need))
    return fail(MOE_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", who, ws_bytes, need);
  if (T == 0 && !dgamma) return MOE_OK;
  hipStream_t s = as_stream(stream);
  const int n = partials(T, H);
  float* partial = n == 1 ? dgamma : dgamma ? static_cast<float*>(ws) : nullptr;  // one row of sums is dgamma
  if (T > 0) {
    const int rc = dtype == MOE_F32 ? rms_backward<float>(dy, dsum, x, gamma, rstd, T, H, dx, partial, s)
                                    : rms_backward<uint16_t>(dy, dsum, x, gamma, rstd, T, H, dx, partial, s);
    if (rc) return rc;
  }
  if (dgamma && n != 1) {
    // no rows: zero sums
    hipLaunchKernelGGL(rms_sum_kernel, dim3(ceil_div(H, kWave)), dim3(kMaxWaves * kWave), 0, s, partial, n, H,
                       dgamma);
    MOE_LAUNCH_CHECK("moe_rms_norm_backward: sum launch");
  }
  return debug_check(MOE_OK, who, s, nullptr);
}
