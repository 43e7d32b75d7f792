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
// bf16: the tile product of mfma_tile.h; dH and dX read the weights transposed, dW both operands.
// f32: 64 x 64 tiles of the fp32 MFMA (32x32x2), staged through registers.
#include <algorithm>
#include <type_traits>

#include "mfma_tile.h"

namespace moe {
namespace {

struct Tile {
  int32_t expert;
  int32_t row0;
  int32_t rows;
  int32_t slot;
};

constexpr int kMaxSide = 1 << 20;  // largest H and I: bounds the grids
constexpr int kBM = 64, kBN = 64, kBK = 32;  // f32 tile
constexpr int kLd = kBM + 33;                // LDS row (one k) of an f32 operand tile
constexpr int kRowTile = 256;                // bf16: rows of a tile

int tile_rows(moe_dtype dt) { return dt == MOE_BF16 ? kRowTile : kBM; }

int64_t max_tiles(int64_t R, int E, moe_dtype dt) {
  return ceil_div64(R, tile_rows(dt)) + std::min<int64_t>(E, R);
}

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
  w.count_off = w.tiles_off + align_up(static_cast<size_t>(max_tiles(R, E, dt)) * sizeof(Tile), 256);
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

// dG, dU and h of one element, from g, u and dH.  exp2 and reciprocal are the hardware's (about 1
// ulp each); a sigmoid that saturates gives exact zeros, not NaN.
__device__ __forceinline__ void swiglu_grad(float g, float u, float d, float* dg, float* du, float* h) {
  const float sg = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.4426950408889634f));
  const float silu = g * sg;
  *dg = d * u * (sg * (1.0f + g * (1.0f - sg)));
  *du = d * silu;
  *h = silu * u;
}

// ---------------------------------------------------------------------------
// f32
// ---------------------------------------------------------------------------

// Tiles of 64 x 64, four waves of one 32 x 32 block each: small enough that the few rows of an
// expert still make blocks for every CU, several of which share a CU and hide one another's
// latency.  A stage is 32 of depth; the next two stages' loads are in flight while this one's
// MFMAs run, LDS is double-buffered and an even and an odd accumulator keep two MFMAs independent.

typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// This thread's 8 elements of a stage of an operand: 64 "outer" indices by 32 of depth, zero outside
// the operand.  KMAJOR: element (o, k) is at p[k * ld + o], else at p[o * ld + k]; either way four
// elements that lie together in memory are one load where all four exist.  Two pieces alternate,
// each a stage ahead of the other.  at(o) maps a tile's outer index to the operand's, or to -1;
// four from a multiple of 4 stay together (KMAJOR).
template <bool KMAJOR>
struct Piece {
  const float* p[2];  // this thread's elements of the stage to load next
  int n[2];           // how many of the four exist (KMAJOR: columns; else 4 or 0)
  int64_t step;       // two stages on
  int k;              // depth of the first of them within the operand
  float v[2][4];

  template <typename At>
  __device__ __forceinline__ void init(const float* base, int64_t ld, int k0, At at) {
    const int tid = threadIdx.x;
    k = k0 + (KMAJOR ? tid >> 4 : (tid & 7) * 4);
    step = 2 * kBK * (KMAJOR ? ld : 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int o = KMAJOR ? (tid & 15) * 4 : (tid >> 3) + i * 32;
      n[i] = 0;
      if (KMAJOR) {
        while (n[i] < 4 && at(o + n[i]) >= 0) ++n[i];
      } else if (at(o) >= 0) {
        n[i] = 4;
      }
      const int src = n[i] ? at(o) : 0;
      p[i] = base + (KMAJOR ? static_cast<int64_t>(k + 16 * i) * ld + src : static_cast<int64_t>(src) * ld + k);
    }
  }

  __device__ __forceinline__ void load(int K) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // of the four, those inside the depth too
      const int left = K - k;
      const int m = KMAJOR ? (left > 16 * i ? n[i] : 0) : min(n[i], left);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = 0.f;
      if (m == 4) {
        const f32x4_a4 q = *reinterpret_cast<const f32x4_a4*>(p[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = q[j];
      } else if (m > 0) {
#pragma unroll
        for (int j = 0; j < 3; ++j)
          if (j < m) v[i][j] = p[i][j];
      }
      p[i] += step;
    }
    k += 2 * kBK;
  }

  // To LDS as [depth][outer], rows of 97 floats: the transposing writes of a row operand and the
  // fragment reads (two depths of 32) spread over the banks.
  __device__ __forceinline__ void store(float* __restrict__ lds) const {
    const int tid = threadIdx.x;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int o = KMAJOR ? (tid & 15) * 4 + j : (tid >> 3) + i * 32;
        const int k = KMAJOR ? (tid >> 4) + i * 16 : (tid & 7) * 4 + j;
        lds[k * kLd + o] = v[i][j];
      }
  }
};

constexpr int kF32Lds = kBK * kLd;  // floats of one operand's stage

// The wave's 32 x 32 block (rows 32 (wave / 2), tile columns 32 (wave % 2)) of A B over depth
// [0, K).  lds: two stages of two operands.
template <bool A_KMAJOR, bool B_KMAJOR, typename AtA, typename AtB>
__device__ __forceinline__ floatx16 tile_product_f32(const float* __restrict__ A, int64_t lda, AtA at_a,
                                                     const float* __restrict__ B, int64_t ldb, AtB at_b,
                                                     int K, float* lds) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int ra = (lane >> 5) * kLd + (wave >> 1) * 32 + (lane & 31);
  const int rb = (lane >> 5) * kLd + (wave & 1) * 32 + (lane & 31) + kF32Lds;
  floatx16 even, odd;
#pragma unroll
  for (int q = 0; q < 16; ++q) even[q] = odd[q] = 0.f;
  Piece<A_KMAJOR> pa[2];
  Piece<B_KMAJOR> pb[2];
  auto load = [&](int i) {
    pa[i].load(K);
    pb[i].load(K);
  };
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    pa[i].init(A, lda, i * kBK, at_a);
    pb[i].init(B, ldb, i * kBK, at_b);
    load(i);
  }
  // stage i & 1, from its registers and into its LDS.  The barrier of the next stage orders these
  // reads before the same buffer is written again.
  auto stage = [&](int i) {
    float* cur = lds + i * 2 * kF32Lds;
    pa[i].store(cur);
    pb[i].store(cur + kF32Lds);
    __syncthreads();
    load(i);
#pragma unroll
    for (int k = 0; k < kBK; k += 4) {
      even = __builtin_amdgcn_mfma_f32_32x32x2f32(cur[k * kLd + ra], cur[k * kLd + rb], even, 0, 0, 0);
      odd = __builtin_amdgcn_mfma_f32_32x32x2f32(cur[(k + 2) * kLd + ra], cur[(k + 2) * kLd + rb], odd, 0, 0, 0);
    }
  };
  for (int k0 = 0; k0 < K; k0 += 2 * kBK) {
    stage(0);
    if (k0 + kBK < K) stage(1);
  }
  return even + odd;
}

// Row within the tile of element q of this lane's block; its tile column is 32 (wave % 2) + lane % 32.
__device__ __forceinline__ int acc_row(int q) {
  const int lane = threadIdx.x & (kWave - 1);
  return (threadIdx.x / kWave >> 1) * 32 + (q >> 2) * 8 + (lane >> 5) * 4 + (q & 3);
}
__device__ __forceinline__ int acc_col() { return (threadIdx.x / kWave & 1) * 32 + (threadIdx.x & 31); }

// C[r][n] = sum_k A[r][k] B[k][n] for the rows of each tile; B of the tile's expert starts at
// b_off of its block.
__global__ __launch_bounds__(256) void rows_product_f32_kernel(
    const float* __restrict__ A, int64_t lda, const char* __restrict__ wbase, int64_t expert_bytes,
    int64_t b_off, int N, int K, const Tile* __restrict__ tiles, const int32_t* __restrict__ n_tiles,
    float* __restrict__ C) {
  __shared__ float lds[4 * kF32Lds];
  if (static_cast<int>(blockIdx.x) >= *n_tiles) return;
  const Tile t = tiles[blockIdx.x];
  const int n0 = blockIdx.y * kBN;
  const float* B = reinterpret_cast<const float*>(wbase + t.slot * expert_bytes + b_off);
  const floatx16 acc = tile_product_f32<false, true>(
      A + t.row0 * lda, lda, [&](int o) { return o < t.rows ? o : -1; }, B, N,
      [&](int o) { return n0 + o < N ? n0 + o : -1; }, K, lds);
  const int c = n0 + acc_col();
  if (c >= N) return;
#pragma unroll
  for (int q = 0; q < 16; ++q)
    if (acc_row(q) < t.rows) C[static_cast<int64_t>(t.row0 + acc_row(q)) * N + c] = acc[q];
}

// g and u for 32 columns, then dG, dU and h from dH.  Each wave's 32 tile columns are 16 of Wg and
// the same 16 of Wu: lanes l and l ^ 16 hold g and u of one element.
__global__ __launch_bounds__(256) void gate_up_backward_f32_kernel(
    const float* __restrict__ x, const char* __restrict__ wbase, int64_t expert_bytes, int H, int I,
    const Tile* __restrict__ tiles, const int32_t* __restrict__ n_tiles, const float* __restrict__ dh,
    float* __restrict__ dgu, float* __restrict__ h) {
  __shared__ float lds[4 * kF32Lds];
  if (static_cast<int>(blockIdx.x) >= *n_tiles) return;
  const Tile t = tiles[blockIdx.x];
  const int n0 = blockIdx.y * (kBN / 2);
  const float* W = reinterpret_cast<const float*>(wbase + t.slot * expert_bytes);
  const int c = n0 + (threadIdx.x / kWave & 1) * 16 + (threadIdx.x & 15);
  const bool up = threadIdx.x & 16;
  // dH arrives while the products run; a lane past the tile or past I reads a place inside
  float d[16];
#pragma unroll
  for (int q = 0; q < 16; ++q)
    d[q] = dh[static_cast<int64_t>(t.row0 + min(acc_row(q), t.rows - 1)) * I + min(c, I - 1)];
  const floatx16 acc = tile_product_f32<false, false>(
      x + static_cast<int64_t>(t.row0) * H, H, [&](int o) { return o < t.rows ? o : -1; }, W, H,
      [&](int o) {
        const int c = n0 + (o >> 5) * 16 + (o & 15);
        return c < I ? c + (o >> 4 & 1) * I : -1;
      },
      H, lds);
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const float mate = __shfl_xor(acc[q], 16);
    if (acc_row(q) >= t.rows || c >= I) continue;
    const int64_t row = t.row0 + acc_row(q);
    float dg, du, hv;
    swiglu_grad(up ? mate : acc[q], up ? acc[q] : mate, d[q], &dg, &du, &hv);
    if (up) {
      dgu[row * 2 * I + I + c] = du;
    } else {
      dgu[row * 2 * I + c] = dg;
      h[row * I + c] = hv;
    }
  }
}

// C[m][n] = sum over the expert's rows r of A[r][m] B[r][n], written at c_off of the expert's
// block of dw.  An expert without rows gets zeros, one outside the buffer nothing.
__global__ __launch_bounds__(256) void weight_grad_f32_kernel(
    const float* __restrict__ A, int M, const float* __restrict__ B, int N,
    const int32_t* __restrict__ offsets, int R, const int32_t* __restrict__ slot_of, int n_slots,
    int64_t expert_bytes, int64_t c_off, char* __restrict__ dw) {
  __shared__ float lds[4 * kF32Lds];
  const int e = blockIdx.z;
  const int slot = slot_of[e];
  if (slot < 0 || slot >= n_slots) return;
  int lo;
  const int K = expert_rows(offsets, e, R, &lo);
  const int m0 = blockIdx.x * kBM, n0 = blockIdx.y * kBN;
  const floatx16 acc = tile_product_f32<true, true>(
      A + static_cast<int64_t>(lo) * M, M, [&](int o) { return m0 + o < M ? m0 + o : -1; },
      B + static_cast<int64_t>(lo) * N, N, [&](int o) { return n0 + o < N ? n0 + o : -1; }, K, lds);
  float* C = reinterpret_cast<float*>(dw + slot * expert_bytes + c_off);
  const int c = n0 + acc_col();
  if (c >= N) return;
#pragma unroll
  for (int q = 0; q < 16; ++q)
    if (m0 + acc_row(q) < M) C[static_cast<int64_t>(m0 + acc_row(q)) * N + c] = acc[q];
}

// ---------------------------------------------------------------------------
// bf16
// ---------------------------------------------------------------------------

// Work order: units of gm x gn output tiles, unit u on XCD u % 8 (workgroup i runs on XCD i % 8),
// so the workgroups that run together on an XCD share gm row panels and gn column panels in its L2.
struct Order {
  int gm, gn, n_gn;  // tiles of a unit; units across
};

__device__ __forceinline__ void place(const Order& o, int* m, int* n) {
  const int xcd = blockIdx.x % 8, local = blockIdx.x / 8;
  const int per = o.gm * o.gn;
  const int unit = local / per * 8 + xcd, at = local % per;
  *m = unit / o.n_gn * o.gm + at % o.gm;
  *n = unit % o.n_gn * o.gn + at / o.gm;
}

Order make_order(int64_t mt, int64_t nt, int64_t* grid) {
  // up to 4 x 8 tiles (32 CUs an XCD), the columns cut evenly, where that leaves every XCD a few
  // units, else single tiles
  Order o{4, static_cast<int>(ceil_div64(nt, ceil_div64(nt, 8))), 0};
  if (ceil_div64(mt, o.gm) * ceil_div64(nt, o.gn) < 32) o.gm = o.gn = 1;
  o.n_gn = static_cast<int>(ceil_div64(nt, o.gn));
  const int64_t units = ceil_div64(mt, o.gm) * o.n_gn;
  *grid = ceil_div64(units, 8) * 8 * o.gm * o.gn;
  return o;
}

__device__ __forceinline__ Tile load_tile(const Tile* tiles, int m) {
  const Tile t = tiles[m];
  return Tile{__builtin_amdgcn_readfirstlane(t.expert), __builtin_amdgcn_readfirstlane(t.row0),
              __builtin_amdgcn_readfirstlane(t.rows), __builtin_amdgcn_readfirstlane(t.slot)};
}

// Calls f with the smallest tile mode that holds `rows` rows.
template <typename F>
__device__ __forceinline__ void by_rows(int rows, F f) {
  if (rows > 192) f(std::integral_constant<int, 0>{});
  else if (rows > 128) f(std::integral_constant<int, 6>{});
  else if (rows > 64) f(std::integral_constant<int, 4>{});
  else if (rows > 32) f(std::integral_constant<int, 2>{});
  else f(std::integral_constant<int, 1>{});
}

// A tile's accumulators to C (its first row and column), of which rows x cols exist.
template <int MI>
__device__ __forceinline__ void store_tile(
    const floatx16 (&acc)[TileShape<MI, false>::MW][TileShape<MI, false>::NJ], lds_char* smem,
    uint16_t* C, int64_t ld, int rows, int cols) {
  using S = TileShape<MI, false>;
#pragma unroll
  for (int i = 0; i < S::MW; ++i) {
    const int r0 = S::first_row() + i * 32, c0 = S::first_col();
    store_block<S::NJ * 32>(smem, C + r0 * ld + c0, ld, rows - r0, cols - c0, [&](int j, int v) {
      return pack4(acc[i][j][v * 4], acc[i][j][v * 4 + 1], acc[i][j][v * 4 + 2], acc[i][j][v * 4 + 3]);
    });
  }
}

template <int MI>
__device__ __forceinline__ void store_tile(
    const floatx16 (&acc)[TileShape<MI, false>::MW][TileShape<MI, false>::NJ], lds_char*, float* C,
    int64_t ld, int rows, int cols) {
  using S = TileShape<MI, false>;
#pragma unroll
  for (int i = 0; i < S::MW; ++i) {
    const int r = lane_row<MI, false>(i);
    if (r >= rows) continue;
#pragma unroll
    for (int j = 0; j < S::NJ; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int c = S::first_col() + S::col(j) + lane_col(v);
        if (c < cols)
          *reinterpret_cast<floatx4*>(C + r * ld + c) =
              floatx4{acc[i][j][v * 4], acc[i][j][v * 4 + 1], acc[i][j][v * 4 + 2], acc[i][j][v * 4 + 3]};
      }
  }
}

// C[r][n] = sum_k A[r][k] B[k][n] for the rows of each tile; B of the tile's expert starts at
// b_off of its block.
template <int MI, typename O>
__device__ __forceinline__ void rows_product(const Tile& t, int n0, const uint16_t* A, int lda,
                                             const uint16_t* B, int N, int K, O* C, lds_char* smem) {
  using S = TileShape<MI, false>;
  Operand<false, S::ROWS> oa;
  Operand<true, 256> ob;
  oa.init(A + static_cast<int64_t>(t.row0) * lda, lda, K, [&](int r) { return r < t.rows ? r : -1; });
  ob.init(B + n0, N, K, [&](int c) { return n0 + c < N ? c : -1; });
  floatx16 acc[S::MW][S::NJ];
  tile_product<MI, false, false, true>(oa, ob, K, smem, acc);
  store_tile<MI>(acc, smem, C + static_cast<int64_t>(t.row0) * N + n0, N, t.rows, N - n0);
}

template <typename O>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void rows_product_kernel(
    const uint16_t* __restrict__ A, int lda, const char* __restrict__ wbase, int64_t expert_bytes,
    int64_t b_off, int N, int K, const Tile* __restrict__ tiles, const int32_t* __restrict__ n_tiles,
    Order order, O* __restrict__ C) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  int m, n;
  place(order, &m, &n);
  if (m >= *n_tiles || n * kTileN >= N) return;
  const Tile t = load_tile(tiles, m);
  const uint16_t* B = reinterpret_cast<const uint16_t*>(wbase + t.slot * expert_bytes + b_off);
  by_rows(t.rows, [&](auto mi) {
    rows_product<decltype(mi)::value>(t, n * kTileN, A, lda, B, N, K, C, (lds_char*)smem);
  });
}

// g and u for 128 columns, then dG, dU and h from dH.
template <int MI>
__device__ __forceinline__ void gate_up_backward(const Tile& t, int n0, const uint16_t* x,
                                                 const uint16_t* W, int H, int I, const float* dh,
                                                 uint16_t* dgu, uint16_t* h, lds_char* smem) {
  using S = TileShape<MI, true>;
  Operand<false, S::ROWS> oa;
  Operand<false, 256> ob;
  oa.init(x + static_cast<int64_t>(t.row0) * H, H, H, [&](int r) { return r < t.rows ? r : -1; });
  ob.init(W + static_cast<int64_t>(n0) * H, H, H,
          [&](int r) { return n0 + (r & 127) < I ? (r & 127) + (r >> 7) * I : -1; });
  floatx16 acc[S::MW][S::NJ];
  tile_product<MI, true, false, false>(oa, ob, H, smem, acc);
  constexpr int HALF = S::NJ / 2, COLS = HALF * 32;
  const int c0 = n0 + S::first_col(), cols = I - c0;
  if (cols <= 0) return;
#pragma unroll
  for (int i = 0; i < S::MW; ++i) {
    const int r0 = S::first_row() + i * 32, rows = t.rows - r0;
    if (rows <= 0) return;
    // dH of the lane's row, all of it in flight at once; a lane past the tile or past I reads a
    // place inside and its values are not stored
    const float* drow = dh + static_cast<int64_t>(t.row0 + min(lane_row<MI, true>(i), t.rows - 1)) * I;
    floatx4 d[HALF][4];
#pragma unroll
    for (int j = 0; j < HALF; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        d[j][v] = *reinterpret_cast<const floatx4*>(drow + min(c0 + j * 32 + lane_col(v), I - 4));
    u32x2 du[HALF][4], hv[HALF][4];
    const int64_t row = t.row0 + r0;
    store_block<COLS>(smem, dgu + row * 2 * I + c0, 2 * I, rows, cols, [&](int j, int v) {
      float a[4], b[4], c[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        swiglu_grad(acc[i][j][v * 4 + q], acc[i][j + HALF][v * 4 + q], d[j][v][q], &a[q], &b[q], &c[q]);
      du[j][v] = pack4(b[0], b[1], b[2], b[3]);
      hv[j][v] = pack4(c[0], c[1], c[2], c[3]);
      return pack4(a[0], a[1], a[2], a[3]);
    });
    store_block<COLS>(smem, dgu + row * 2 * I + I + c0, 2 * I, rows, cols,
                      [&](int j, int v) { return du[j][v]; });
    store_block<COLS>(smem, h + row * I + c0, I, rows, cols, [&](int j, int v) { return hv[j][v]; });
  }
}

__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void
gate_up_backward_kernel(const uint16_t* __restrict__ x, const char* __restrict__ wbase,
                        int64_t expert_bytes, int H, int I, const Tile* __restrict__ tiles,
                        const int32_t* __restrict__ n_tiles, Order order, const float* __restrict__ dh,
                        uint16_t* __restrict__ dgu, uint16_t* __restrict__ h) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  int m, n;
  place(order, &m, &n);
  if (m >= *n_tiles || n * (kTileN / 2) >= I) return;
  const Tile t = load_tile(tiles, m);
  const uint16_t* W = reinterpret_cast<const uint16_t*>(wbase + t.slot * expert_bytes);
  by_rows(t.rows, [&](auto mi) {
    gate_up_backward<decltype(mi)::value>(t, n * (kTileN / 2), x, W, H, I, dh, dgu, h, (lds_char*)smem);
  });
}

// C[m][n] = sum over the expert's rows r of A[r][m] B[r][n], written at c_off of the expert's
// block of dw.  An expert without rows gets zeros, one outside the buffer nothing.
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void weight_grad_kernel(
    const uint16_t* __restrict__ A, int M, const uint16_t* __restrict__ B, int N,
    const int32_t* __restrict__ offsets, int R, const int32_t* __restrict__ slot_of, int n_slots,
    int64_t expert_bytes, int64_t c_off, Order order, char* __restrict__ dw) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  using S = TileShape<0, false>;
  int m, n;
  place(order, &m, &n);
  const int e = blockIdx.y;
  const int m0 = m * kRowTile, n0 = n * kTileN;
  if (m0 >= M || n0 >= N) return;
  const int slot = __builtin_amdgcn_readfirstlane(slot_of[e]);
  if (slot < 0 || slot >= n_slots) return;
  int lo;
  const int K = __builtin_amdgcn_readfirstlane(expert_rows(offsets, e, R, &lo));
  lo = __builtin_amdgcn_readfirstlane(lo);
  Operand<true, 256> oa, ob;
  oa.init(A + static_cast<int64_t>(lo) * M + m0, M, K, [&](int c) { return m0 + c < M ? c : -1; });
  ob.init(B + static_cast<int64_t>(lo) * N + n0, N, K, [&](int c) { return n0 + c < N ? c : -1; });
  floatx16 acc[S::MW][S::NJ];
  tile_product<0, false, true, true>(oa, ob, K, (lds_char*)smem, acc);
  uint16_t* C = reinterpret_cast<uint16_t*>(dw + slot * expert_bytes + c_off);
  store_tile<0>(acc, (lds_char*)smem, C + static_cast<int64_t>(m0) * N + n0, N, M - m0, N - n0);
}

struct Call {
  const int32_t* offsets;
  int R, E, H, I;
  const moe_wbuf* w;
  char* ws;
  BackwardWs L;
  void* dx_perm;
  char* dw;
  int32_t* status;
  hipStream_t s;
};

int launch_plan(const Call& c, moe_dtype dt, Tile** tiles, int32_t** n_tiles, int64_t* cap) {
  *tiles = reinterpret_cast<Tile*>(c.ws + c.L.tiles_off);
  *n_tiles = reinterpret_cast<int32_t*>(c.ws + c.L.count_off);
  *cap = max_tiles(c.R, c.E, dt);
  hipLaunchKernelGGL(backward_plan_kernel, dim3(1), dim3(MOE_MAX_E), 0, c.s, c.offsets, c.R, c.E,
                     tile_rows(dt), c.w->slot_of, c.w->n_slots, static_cast<int>(*cap), *tiles, *n_tiles,
                     c.status);
  MOE_LAUNCH_CHECK("moe_grouped_swiglu_backward: plan");
  return MOE_OK;
}

int run_f32(const Call& c, const float* x, const float* dy) {
  const int E = c.E, H = c.H, I = c.I;
  float* dh = reinterpret_cast<float*>(c.ws + c.L.dh_off);
  float* dgu = reinterpret_cast<float*>(c.ws + c.L.dgu_off);
  float* h = reinterpret_cast<float*>(c.ws + c.L.h_off);
  const char* wbase = static_cast<const char*>(c.w->base);
  const int64_t eb = c.w->expert_bytes, HI = static_cast<int64_t>(H) * I * sizeof(float);
  if (c.R > 0) {
    Tile* tiles;
    int32_t* n_tiles;
    int64_t cap64;
    const int rc = launch_plan(c, MOE_F32, &tiles, &n_tiles, &cap64);
    if (rc) return rc;
    const unsigned cap = static_cast<unsigned>(cap64);
    hipLaunchKernelGGL(rows_product_f32_kernel, dim3(cap, ceil_div(I, kBN)), dim3(256), 0, c.s, dy,
                       static_cast<int64_t>(H), wbase, eb, 2 * HI, I, H, tiles, n_tiles, dh);
    MOE_LAUNCH_CHECK("moe_grouped_swiglu_backward: dh");
    hipLaunchKernelGGL(gate_up_backward_f32_kernel, dim3(cap, ceil_div(I, kBN / 2)), dim3(256), 0, c.s, x,
                       wbase, eb, H, I, tiles, n_tiles, dh, dgu, h);
    MOE_LAUNCH_CHECK("moe_grouped_swiglu_backward: gate/up");
    if (c.dx_perm) {
      hipLaunchKernelGGL(rows_product_f32_kernel, dim3(cap, ceil_div(H, kBN)), dim3(256), 0, c.s, dgu,
                         2 * static_cast<int64_t>(I), wbase, eb, int64_t{0}, H, 2 * I, tiles, n_tiles,
                         static_cast<float*>(c.dx_perm));
      MOE_LAUNCH_CHECK("moe_grouped_swiglu_backward: dx");
    }
  }
  if (c.dw) {
    hipLaunchKernelGGL(weight_grad_f32_kernel, dim3(ceil_div(2 * I, kBM), ceil_div(H, kBN), E), dim3(256),
                       0, c.s, dgu, 2 * I, x, H, c.offsets, c.R, c.w->slot_of, c.w->n_slots, eb,
                       int64_t{0}, c.dw);
    MOE_LAUNCH_CHECK("moe_grouped_swiglu_backward: gate/up weights");
    hipLaunchKernelGGL(weight_grad_f32_kernel, dim3(ceil_div(H, kBM), ceil_div(I, kBN), E), dim3(256), 0,
                       c.s, dy, H, h, I, c.offsets, c.R, c.w->slot_of, c.w->n_slots, eb, 2 * HI, c.dw);
    MOE_LAUNCH_CHECK("moe_grouped_swiglu_backward: down weights");
  }
  return MOE_OK;
}

// Enqueue a tile kernel: its 128 KB of LDS are above the default limit of a launch.
template <typename K, typename... A>
int launch_tiles(const char* what, K kernel, dim3 grid, hipStream_t s, A... args) {
  MOE_HIP_CHECK(hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                    hipFuncAttributeMaxDynamicSharedMemorySize, kTileLds));
  hipLaunchKernelGGL(kernel, grid, dim3(256), kTileLds, s, args...);
  MOE_LAUNCH_CHECK(what);
  return MOE_OK;
}

int run_bf16(const Call& c, const uint16_t* x, const uint16_t* dy) {
  const int H = c.H, I = c.I;
  float* dh = reinterpret_cast<float*>(c.ws + c.L.dh_off);
  uint16_t* dgu = reinterpret_cast<uint16_t*>(c.ws + c.L.dgu_off);
  uint16_t* h = reinterpret_cast<uint16_t*>(c.ws + c.L.h_off);
  const char* wbase = static_cast<const char*>(c.w->base);
  const int64_t eb = c.w->expert_bytes, HI = static_cast<int64_t>(H) * I * 2;
  int64_t grid;
  int rc;
  if (c.R > 0) {
    Tile* tiles;
    int32_t* n_tiles;
    int64_t cap;
    rc = launch_plan(c, MOE_BF16, &tiles, &n_tiles, &cap);
    if (rc) return rc;
    Order o = make_order(cap, ceil_div(I, kTileN), &grid);
    rc = launch_tiles("moe_grouped_swiglu_backward: dh", rows_product_kernel<float>,
                      dim3(static_cast<unsigned>(grid)), c.s, dy, H, wbase, eb, 2 * HI, I, H, tiles,
                      n_tiles, o, dh);
    if (rc) return rc;
    o = make_order(cap, ceil_div(I, kTileN / 2), &grid);
    rc = launch_tiles("moe_grouped_swiglu_backward: gate/up", gate_up_backward_kernel,
                      dim3(static_cast<unsigned>(grid)), c.s, x, wbase, eb, H, I, tiles, n_tiles, o, dh,
                      dgu, h);
    if (rc) return rc;
    if (c.dx_perm) {
      o = make_order(cap, ceil_div(H, kTileN), &grid);
      rc = launch_tiles("moe_grouped_swiglu_backward: dx", rows_product_kernel<uint16_t>,
                        dim3(static_cast<unsigned>(grid)), c.s, dgu, 2 * I, wbase, eb, int64_t{0}, H,
                        2 * I, tiles, n_tiles, o, static_cast<uint16_t*>(c.dx_perm));
      if (rc) return rc;
    }
  }
  if (c.dw) {
    Order o = make_order(ceil_div(2 * I, kRowTile), ceil_div(H, kTileN), &grid);
    rc = launch_tiles("moe_grouped_swiglu_backward: gate/up weights", weight_grad_kernel,
                      dim3(static_cast<unsigned>(grid), c.E), c.s, dgu, 2 * I, x, H, c.offsets, c.R,
                      c.w->slot_of, c.w->n_slots, eb, int64_t{0}, o, c.dw);
    if (rc) return rc;
    o = make_order(ceil_div(H, kRowTile), ceil_div(I, kTileN), &grid);
    rc = launch_tiles("moe_grouped_swiglu_backward: down weights", weight_grad_kernel,
                      dim3(static_cast<unsigned>(grid), c.E), c.s, dy, H, h, I, c.offsets, c.R,
                      c.w->slot_of, c.w->n_slots, eb, 2 * HI, o, c.dw);
    if (rc) return rc;
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
  if (static_cast<int64_t>(H) * I >= (int64_t{1} << 29) || H > kMaxSide || I > kMaxSide)
    return fail(MOE_ERR_UNSUPPORTED, "%s: H=%d or I=%d above %d, or H*I 2^29 or more", who, H, I, kMaxSide);
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
  const Call c{offsets, R, E, H, I, w, static_cast<char*>(ws), L, dx_perm, static_cast<char*>(dw), status, s};
  const int rc = dtype == MOE_F32
                     ? run_f32(c, static_cast<const float*>(x_perm), static_cast<const float*>(dy_perm))
                     : run_bf16(c, static_cast<const uint16_t*>(x_perm), static_cast<const uint16_t*>(dy_perm));
  return debug_check(rc, who, s, status);
}
