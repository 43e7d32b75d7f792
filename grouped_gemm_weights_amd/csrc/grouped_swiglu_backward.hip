// moe_grouped_swiglu_backward: the gradient of the grouped SwiGLU experts.
//
// For the rows r of expert e (X = x_perm rows, dY = dy_perm rows, sg = sigmoid(g)):
//   g = X Wg^T,  u = X Wu^T                    (recomputed: the forward pass keeps only h)
//   dH = dY Wd
//   h = g sg u,  dU = dH g sg,  dG = dH u sg (1 + g (1 - sg))
//   dX = dG Wg + dU Wu
//   dWg = dG^T X,  dWu = dU^T X,  dWd = dY^T h
// 16 R H I operations, in four launches after the tile plan:
//   1. dH            (kept in fp32: dG and dU are its only roundings on the way to dX and dW)
//   2. g, u, then in the epilogue dG | dU as one [R][2I] matrix and h
//   3. dX = [dG dU] [Wg; Wu]: one product of depth 2I, as Wg and Wu lie one after the other
//   4. dW: [dWg; dWu] = [dG dU]^T X and dWd = dY^T h, one block per expert and output tile
//
// fp32 MFMA tiles (32x32x2), bf16 operands widened as they are staged.
#include <algorithm>

#include "common.h"

namespace moe {
namespace {

typedef float floatx16 __attribute__((ext_vector_type(16)));

struct Tile {
  int32_t expert;
  int32_t row0;
  int32_t rows;
  int32_t slot;
};

constexpr int kMaxSide = 1 << 20;  // largest H and I: bounds the grids
constexpr int kBM = 128, kBN = 128, kBK = 16;
constexpr int kLd = kBM + 4;  // LDS row (one k) of an operand tile

int64_t max_tiles(int64_t R, int E) { return ceil_div64(R, kBM) + std::min<int64_t>(E, R); }

struct BackwardWs {
  size_t dh_off, dgu_off, h_off, tiles_off, count_off, total;
};

BackwardWs backward_ws(int64_t R, int E, int I, moe_dtype dt) {
  const size_t n = static_cast<size_t>(R) * I;
  BackwardWs w;
  w.dh_off = 0;
  w.dgu_off = align_up(n * sizeof(float), 256);
  w.h_off = w.dgu_off + align_up(2 * n * elem_size(dt), 256);
  w.tiles_off = w.h_off + align_up(n * elem_size(dt), 256);
  w.count_off = w.tiles_off + align_up(static_cast<size_t>(max_tiles(R, E)) * sizeof(Tile), 256);
  w.total = w.count_off + 256;
  return w;
}

// Rows [lo, lo + count) of expert e, held to [0, R) whatever offsets says.
__device__ __forceinline__ int expert_rows(const int32_t* offsets, int e, int R, int* lo) {
  const int a = min(max(offsets[e], 0), R), b = min(max(offsets[e + 1], 0), R);
  *lo = a;
  return max(b - a, 0);
}

// Row tiles of BM rows per expert, expert-major.
__global__ __launch_bounds__(MOE_MAX_E) void backward_plan_kernel(
    const int32_t* __restrict__ offsets, int R, int E, int BM, const int32_t* __restrict__ slot_of,
    int n_slots, int tile_cap, Tile* __restrict__ tiles, int32_t* __restrict__ n_tiles,
    int32_t* status) {
  __shared__ int32_t s[MOE_MAX_E];
  const int e = threadIdx.x;
  int n = 0, lo = 0, cnt = 0, slot = -1;
  if (e < E) {
    cnt = expert_rows(offsets, e, R, &lo);
    if (cnt > 0) {
      slot = slot_of[e];
      // a slot outside the merged buffer is treated as absent, never read
      if (slot < 0 || slot >= n_slots) status_or(status, MOE_STATUS_EXPERT_ABSENT);
      else n = (cnt + BM - 1) / BM;
    }
  }
  s[e] = n;
  __syncthreads();
  for (int off = 1; off < MOE_MAX_E; off <<= 1) {
    const int32_t add = e >= off ? s[e - off] : 0;
    __syncthreads();
    s[e] += add;
    __syncthreads();
  }
  const int first = s[e] - n;
  for (int i = 0; i < n && first + i < tile_cap; ++i)
    tiles[first + i] = Tile{e, lo + i * BM, min(BM, cnt - i * BM), slot};
  if (e == 0) *n_tiles = min(s[MOE_MAX_E - 1], tile_cap);
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = f32_to_bf16(v); }

// One stage of an operand: 128 "outer" indices by 16 depth steps into LDS as [depth][outer], zero
// outside [0, n_outer) and [0, K).  KMAJOR: element (o, k) is at p[k * ld + o], else at
// p[o * ld + k].  `at(o)` maps a tile's outer index to the operand's (or -1).
template <bool KMAJOR, typename T, typename At>
__device__ __forceinline__ void stage(const T* __restrict__ p, int64_t ld, int k0, int K, At at,
                                      float* __restrict__ lds) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int i = 0; i < kBM * kBK / 256; ++i) {
    const int o = KMAJOR ? tid % kBM : tid / kBK + i * (256 / kBK);
    const int k = KMAJOR ? tid / kBM + i * (256 / kBM) : tid % kBK;
    const int src = at(o);
    float v = 0.f;
    if (src >= 0 && k0 + k < K)
      v = to_f32(KMAJOR ? p[static_cast<int64_t>(k0 + k) * ld + src]
                        : p[static_cast<int64_t>(src) * ld + k0 + k]);
    lds[k * kLd + o] = v;
  }
}

// acc[i][j] += A B over depth [0, K): 4 waves as 2 x 2, each 64 rows (i) by two 32-column blocks
// whose tile columns start at wcol[j].
template <bool A_KMAJOR, bool B_KMAJOR, typename TA, typename TB, typename AtA, typename AtB>
__device__ __forceinline__ void tile_product(const TA* __restrict__ A, int64_t lda, AtA at_a,
                                             const TB* __restrict__ B, int64_t ldb, AtB at_b, int K,
                                             const int (&wcol)[2], float* As, float* Bs,
                                             floatx16 (&acc)[2][2]) {
  const int lane = threadIdx.x & (kWave - 1);
  const int wm = (threadIdx.x / kWave) >> 1;
  for (int k0 = 0; k0 < K; k0 += kBK) {
    stage<A_KMAJOR>(A, lda, k0, K, at_a, As);
    stage<B_KMAJOR>(B, ldb, k0, K, at_b, Bs);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kBK; k += 2) {
      const int row = (k + (lane >> 5)) * kLd + (lane & 31);
      float a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) a[i] = As[row + wm * 64 + i * 32];
#pragma unroll
      for (int j = 0; j < 2; ++j) b[j] = Bs[row + wcol[j]];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[j], acc[i][j], 0, 0, 0);
    }
    __syncthreads();
  }
}

__device__ __forceinline__ void clear(floatx16 (&acc)[2][2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;
}

// Element q of 32x32 block i of this lane: row within the tile.
__device__ __forceinline__ int acc_row(int i, int q) {
  const int lane = threadIdx.x & (kWave - 1);
  return ((threadIdx.x / kWave) >> 1) * 64 + i * 32 + (q >> 2) * 8 + (lane >> 5) * 4 + (q & 3);
}

// C[r][n] = sum_k A[r][k] B[k][n] for the rows of each tile; B of the tile's expert starts at
// b_off of its block.
template <typename T, typename O>
__global__ __launch_bounds__(256) void rows_product_kernel(
    const T* __restrict__ A, int64_t lda, const char* __restrict__ wbase, int64_t expert_bytes,
    int64_t b_off, int N, int K, const Tile* __restrict__ tiles, const int32_t* __restrict__ n_tiles,
    O* __restrict__ C) {
  __shared__ float As[kBK * kLd], Bs[kBK * kLd];
  if (static_cast<int>(blockIdx.x) >= *n_tiles) return;
  const Tile t = tiles[blockIdx.x];
  const int n0 = blockIdx.y * kBN;
  const int wn = (threadIdx.x / kWave) & 1;
  const T* B = reinterpret_cast<const T*>(wbase + t.slot * expert_bytes + b_off);
  const int wcol[2] = {wn * 64, wn * 64 + 32};
  floatx16 acc[2][2];
  clear(acc);
  tile_product<false, true>(
      A + t.row0 * lda, lda, [&](int o) { return o < t.rows ? o : -1; }, B, N,
      [&](int o) { return n0 + o < N ? n0 + o : -1; }, K, wcol, As, Bs, acc);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int r = acc_row(i, q);
      if (r >= t.rows) continue;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = n0 + wcol[j] + (threadIdx.x & 31);
        if (c < N) put(C + static_cast<int64_t>(t.row0 + r) * N + c, acc[i][j][q]);
      }
    }
}

// g and u for 64 columns, then dG, dU and h from dH.
template <typename T>
__global__ __launch_bounds__(256) void gate_up_backward_kernel(
    const T* __restrict__ x, const char* __restrict__ wbase, int64_t expert_bytes, int H, int I,
    const Tile* __restrict__ tiles, const int32_t* __restrict__ n_tiles, const float* __restrict__ dh,
    T* __restrict__ dgu, T* __restrict__ h) {
  __shared__ float As[kBK * kLd], Bs[kBK * kLd];
  if (static_cast<int>(blockIdx.x) >= *n_tiles) return;
  const Tile t = tiles[blockIdx.x];
  const int n0 = blockIdx.y * (kBN / 2);
  const int wn = (threadIdx.x / kWave) & 1;
  const T* W = reinterpret_cast<const T*>(wbase + t.slot * expert_bytes);
  // B tile: 64 rows of Wg, then the same 64 rows of Wu, so a wave holds matching columns of both
  const int wcol[2] = {wn * 32, 64 + wn * 32};
  floatx16 acc[2][2];
  clear(acc);
  tile_product<false, false>(
      x + static_cast<int64_t>(t.row0) * H, H, [&](int o) { return o < t.rows ? o : -1; }, W, H,
      [&](int o) {
        const int c = n0 + (o & 63);
        return c < I ? c + (o >> 6) * I : -1;
      },
      H, wcol, As, Bs, acc);
  const int c = n0 + wn * 32 + (threadIdx.x & 31);
  if (c >= I) return;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int r = acc_row(i, q);
      if (r >= t.rows) continue;
      const int64_t row = t.row0 + r;
      const float g = acc[i][0][q], u = acc[i][1][q], d = dh[row * I + c];
      const float sg = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.4426950408889634f));
      const float silu = g * sg;
      put(dgu + row * 2 * I + c, d * u * (sg * (1.0f + g * (1.0f - sg))));
      put(dgu + row * 2 * I + I + c, d * silu);
      put(h + row * I + c, silu * u);
    }
}

// C[m][n] = sum over the expert's rows r of A[r][m] B[r][n], written at c_off of the expert's
// block of dw.  An expert without rows gets zeros, one outside the buffer nothing.
template <typename T>
__global__ __launch_bounds__(256) void weight_grad_kernel(
    const T* __restrict__ A, int M, const T* __restrict__ B, int N, const int32_t* __restrict__ offsets,
    int R, const int32_t* __restrict__ slot_of, int n_slots, int64_t expert_bytes, int64_t c_off,
    char* __restrict__ dw) {
  __shared__ float As[kBK * kLd], Bs[kBK * kLd];
  const int e = blockIdx.z;
  const int slot = slot_of[e];
  if (slot < 0 || slot >= n_slots) return;
  int lo;
  const int K = expert_rows(offsets, e, R, &lo);
  const int m0 = blockIdx.x * kBM, n0 = blockIdx.y * kBN;
  const int wn = (threadIdx.x / kWave) & 1;
  const int wcol[2] = {wn * 64, wn * 64 + 32};
  floatx16 acc[2][2];
  clear(acc);
  tile_product<true, true>(
      A + static_cast<int64_t>(lo) * M, M, [&](int o) { return m0 + o < M ? m0 + o : -1; },
      B + static_cast<int64_t>(lo) * N, N, [&](int o) { return n0 + o < N ? n0 + o : -1; }, K, wcol, As,
      Bs, acc);
  T* C = reinterpret_cast<T*>(dw + slot * expert_bytes + c_off);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int m = m0 + acc_row(i, q);
      if (m >= M) continue;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = n0 + wcol[j] + (threadIdx.x & 31);
        if (c < N) put(C + static_cast<int64_t>(m) * N + c, acc[i][j][q]);
      }
    }
}

template <typename T>
int run(const void* x_perm, const void* dy_perm, const int32_t* offsets, int R, int E, int H, int I,
        moe_dtype dt, const moe_wbuf* w, char* ws, void* dx_perm, void* dw, int32_t* status,
        hipStream_t s) {
  const BackwardWs L = backward_ws(R, E, I, dt);
  float* dh = reinterpret_cast<float*>(ws + L.dh_off);
  T* dgu = reinterpret_cast<T*>(ws + L.dgu_off);
  T* h = reinterpret_cast<T*>(ws + L.h_off);
  Tile* tiles = reinterpret_cast<Tile*>(ws + L.tiles_off);
  int32_t* n_tiles = reinterpret_cast<int32_t*>(ws + L.count_off);
  const T* x = static_cast<const T*>(x_perm);
  const T* dy = static_cast<const T*>(dy_perm);
  const char* wbase = static_cast<const char*>(w->base);
  const int64_t eb = w->expert_bytes;
  const int64_t HI = static_cast<int64_t>(H) * I * sizeof(T);
  if (R > 0) {
    const unsigned cap = static_cast<unsigned>(max_tiles(R, E));
    hipLaunchKernelGGL(backward_plan_kernel, dim3(1), dim3(MOE_MAX_E), 0, s, offsets, R, E, kBM,
                       w->slot_of, w->n_slots, static_cast<int>(cap), tiles, n_tiles, status);
    MOE_LAUNCH_CHECK("moe_grouped_swiglu_backward: plan");
    hipLaunchKernelGGL((rows_product_kernel<T, float>), dim3(cap, ceil_div(I, kBN)), dim3(256), 0, s, dy,
                       static_cast<int64_t>(H), wbase, eb, 2 * HI, I, H, tiles, n_tiles, dh);
    MOE_LAUNCH_CHECK("moe_grouped_swiglu_backward: dh");
    hipLaunchKernelGGL(gate_up_backward_kernel<T>, dim3(cap, ceil_div(I, kBN / 2)), dim3(256), 0, s, x,
                       wbase, eb, H, I, tiles, n_tiles, dh, dgu, h);
    MOE_LAUNCH_CHECK("moe_grouped_swiglu_backward: gate/up");
    if (dx_perm) {
      hipLaunchKernelGGL((rows_product_kernel<T, T>), dim3(cap, ceil_div(H, kBN)), dim3(256), 0, s, dgu,
                         2 * static_cast<int64_t>(I), wbase, eb, int64_t{0}, H, 2 * I, tiles, n_tiles,
                         static_cast<T*>(dx_perm));
      MOE_LAUNCH_CHECK("moe_grouped_swiglu_backward: dx");
    }
  }
  if (dw) {
    char* out = static_cast<char*>(dw);
    hipLaunchKernelGGL(weight_grad_kernel<T>, dim3(ceil_div(2 * I, kBM), ceil_div(H, kBN), E), dim3(256),
                       0, s, dgu, 2 * I, x, H, offsets, R, w->slot_of, w->n_slots, eb, int64_t{0}, out);
    MOE_LAUNCH_CHECK("moe_grouped_swiglu_backward: gate/up weights");
    hipLaunchKernelGGL(weight_grad_kernel<T>, dim3(ceil_div(H, kBM), ceil_div(I, kBN), E), dim3(256), 0,
                       s, dy, H, h, I, offsets, R, w->slot_of, w->n_slots, eb, 2 * HI, out);
    MOE_LAUNCH_CHECK("moe_grouped_swiglu_backward: down weights");
  }
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" int moe_grouped_swiglu_backward_workspace_size(int R, int E, int H, int I, moe_dtype dtype,
                                                          size_t* bytes) {
  using namespace moe;
  if (!bytes || R < 0 || E < 1 || H < 1 || I < 1 || (dtype != MOE_F32 && dtype != MOE_BF16))
    return fail(MOE_ERR_ARG, "moe_grouped_swiglu_backward_workspace_size: bad arguments");
  *bytes = backward_ws(R, E, I, dtype).total;
  return MOE_OK;
}

extern "C" int moe_grouped_swiglu_backward(const void* x_perm, const void* dy_perm,
                                           const int32_t* offsets, int R, int E, int H, int I,
                                           moe_dtype dtype, const moe_wbuf* w, void* ws,
                                           size_t ws_bytes, void* dx_perm, void* dw, int32_t* status,
                                           moe_stream_t stream) {
  using namespace moe;
  const char* who = "moe_grouped_swiglu_backward";
  if (R < 0 || E < 1 || H < 1 || I < 1 || (dtype != MOE_F32 && dtype != MOE_BF16))
    return fail(MOE_ERR_ARG, "%s: bad sizes R=%d E=%d H=%d I=%d or dtype", who, R, E, H, I);
  if (E > MOE_MAX_E) return fail(MOE_ERR_UNSUPPORTED, "%s: E=%d above %d", who, E, MOE_MAX_E);
  if (!w || !w->base || !w->slot_of || !offsets || (!dx_perm && !dw))
    return fail(MOE_ERR_ARG, "%s: null pointer", who);
  const int64_t eb = 3 * static_cast<int64_t>(H) * I * elem_size(dtype);
  if (w->expert_bytes != eb || w->n_experts != E)
    return fail(MOE_ERR_ARG, "%s: merged buffer holds %lld-byte blocks for E=%d, expected %lld for E=%d",
                who, static_cast<long long>(w->expert_bytes), w->n_experts, static_cast<long long>(eb), E);
  if (static_cast<int64_t>(H) * I >= (int64_t{1} << 30) || H > kMaxSide || I > kMaxSide)
    return fail(MOE_ERR_UNSUPPORTED, "%s: H=%d or I=%d above %d, or H*I 2^30 or more", who, H, I, kMaxSide);
  if (dtype == MOE_BF16 && (H % 8 != 0 || I % 8 != 0))
    return fail(MOE_ERR_UNSUPPORTED, "%s: H=%d and I=%d must be multiples of 8", who, H, I);
  const uintptr_t all = reinterpret_cast<uintptr_t>(x_perm) | reinterpret_cast<uintptr_t>(dy_perm) |
                        reinterpret_cast<uintptr_t>(w->base) | reinterpret_cast<uintptr_t>(dx_perm) |
                        reinterpret_cast<uintptr_t>(dw) | reinterpret_cast<uintptr_t>(ws);
  if (all % (dtype == MOE_BF16 ? 16 : 4) != 0)
    return fail(MOE_ERR_UNSUPPORTED, "%s: a pointer is not aligned to %d bytes", who,
                dtype == MOE_BF16 ? 16 : 4);
  const BackwardWs L = backward_ws(R, E, I, dtype);
  if (!ws || ws_bytes < L.total)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", who, ws_bytes, L.total);
  if (R > 0 && (!x_perm || !dy_perm)) return fail(MOE_ERR_ARG, "%s: null pointer", who);
  hipStream_t s = as_stream(stream);
  char* wsb = static_cast<char*>(ws);
  const int rc = dtype == MOE_F32 ? run<float>(x_perm, dy_perm, offsets, R, E, H, I, dtype, w, wsb,
                                               dx_perm, dw, status, s)
                                  : run<uint16_t>(x_perm, dy_perm, offsets, R, E, H, I, dtype, w, wsb,
                                                  dx_perm, dw, status, s);
  return debug_check(rc, who, s, status);
}
