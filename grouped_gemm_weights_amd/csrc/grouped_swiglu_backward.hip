// moe_grouped_swiglu_backward: the gradient of the grouped SwiGLU experts.
//
// For the rows r of expert e (X = x_perm rows, dY = dy_perm rows, sg = sigmoid(g)):
//   g = X Wg^T,  u = X Wu^T                    (recomputed: the forward pass keeps only h)
//   dH = dY Wd
//   h = g sg u,  dU = dH g sg,  dG = dH u sg (1 + g (1 - sg))
//   dX = dG Wg + dU Wu
//   dWg = dG^T X,  dWu = dU^T X,  dWd = dY^T h
// 16 R H I operations, in three launches:
//   1. dH            (kept in fp32: dG and dU are its only roundings on the way to dX and dW)
//   2. g, u, then in the epilogue dG | dU as one [R][2I] matrix and h
//   3. dX = [dG dU] [Wg; Wu], one product of depth 2I, as Wg and Wu lie one after the other, and
//      dW: [dWg; dWu] = [dG dU]^T X and dWd = dY^T h, one block per expert and output tile.  The
//      three are independent, so the blocks of one fill the CUs that the last of another leave.
// A block finds its tile of rows from offsets by itself (find_tile: a scan over the experts in
// each wave, under 1 us of a block's time, against 4-5 us for a launch that lists the tiles).
// Measured, bf16, 65536 rows of 32 experts of 7168 x 2048: 1.69 + 3.6 + 8.15 ms (1140, 1070 and 1180
// TFLOP/s; the chip holds 1.7-1.9 GHz), so 1150 in all against 1400-1500 of one large library
// product.  256 experts of that size: 131072 rows 33.8 ms (910 TFLOP/s), 32768 rows 16.3 ms, 512 rows
// 10.0 ms, where 60 GB of weights (Wg and Wu twice) and gradients move at 6.0 TB/s.  24576 rows of 64
// experts of 2048 x 1408, skewed: 0.20 + 0.39 + 0.95 ms, where a weight gradient's depth is an expert's
// few hundred rows and its tile's start and stores are half its time.
//
// bf16: the tile product of mfma_tile.h; dH and dX read the weights transposed, dW both operands.
// dG, dU and h are rounded to bf16 between the second and third launch, as operands of bf16 MFMAs (the
// fp32 MFMA has a sixteenth of their rate) and as the forward pass rounds h; dH, which is no operand,
// is not.  Error against 64 bits 0.0023 relative, where rounding the outputs alone makes 0.0017.
// f32: 64 x 64 tiles of the fp32 MFMA (32x32x2), staged through registers.
//
// moe_clear_unmapped: zeros for the blocks of dw that belong to no expert.
#include "expert_tiles.h"

namespace moe {
namespace {

struct BackwardWs {
  size_t dh_off, dgu_off, h_off, total;
};

BackwardWs backward_ws(int64_t R, int I, moe_dtype dt) {
  const size_t n = static_cast<size_t>(R) * I;
  BackwardWs w;
  w.dh_off = 0;
  w.dgu_off = align_up(n * sizeof(float), 256);
  w.h_off = w.dgu_off + align_up(2 * n * elem_size(dt), 256);
  w.total = w.h_off + align_up(n * elem_size(dt), 256) + 256;
  return w;
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

template <int TR>
__global__ __launch_bounds__(256) void dh_f32_kernel(Experts x, const float* __restrict__ dy,
                                                     const char* __restrict__ wbase, int64_t expert_bytes,
                                                     int H, int I, float* __restrict__ dh) {
  __shared__ float lds[TileF32<TR>::LDS];
  rows_product_f32<TR>(x, blockIdx.x, blockIdx.y * TR, blockIdx.x == 0 && blockIdx.y == 0, dy, H, wbase,
                       expert_bytes, 2 * static_cast<int64_t>(H) * I * 4, I, H, dh, lds);
}

// g and u for TR / 2 columns, then dG, dU and h from dH.  Each 32 tile columns are 16 of Wg and the
// same 16 of Wu: lanes l and l ^ 16 hold g and u of one element.
template <int TR>
__global__ __launch_bounds__(256) void gate_up_backward_f32_kernel(
    Experts ex, const float* __restrict__ x, const char* __restrict__ wbase, int64_t expert_bytes, int H,
    int I, const float* __restrict__ dh, float* __restrict__ dgu, float* __restrict__ h) {
  using S = TileF32<TR>;
  __shared__ float lds[S::LDS];
  Tile t;
  if (!find_tile<TR>(ex, blockIdx.x, false, &t)) return;
  const int n0 = blockIdx.y * (TR / 2);
  const float* W = reinterpret_cast<const float*>(wbase + t.slot * expert_bytes);
  const int c = n0 + S::block_col() * 16 + (threadIdx.x & 15);
  const bool up = threadIdx.x & 16;
  // dH arrives while the products run; a lane past the tile or past I reads a place inside
  float d[S::NQ], acc[S::NQ];
#pragma unroll
  for (int q = 0; q < S::NQ; ++q)
    d[q] = dh[static_cast<int64_t>(t.row0 + min(S::row(q), t.rows - 1)) * I + min(c, I - 1)];
  tile_product_f32<TR, false, false>(
      x + static_cast<int64_t>(t.row0) * H, H, [&](int o) { return o < t.rows ? o : -1; }, W, H,
      [&](int o) {
        const int c = n0 + (o >> 5) * 16 + (o & 15);
        return c < I ? c + (o >> 4 & 1) * I : -1;
      },
      H, lds, acc);
#pragma unroll
  for (int q = 0; q < S::NQ; ++q) {
    const float mate = __shfl_xor(acc[q], 16);
    if (S::row(q) >= t.rows || c >= I) continue;
    const int64_t row = t.row0 + S::row(q);
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

// The third launch: dX, [dWg; dWu] and dWd.  Block ranges in this order, each possibly empty.
struct Ranges {
  int64_t dx, dwgu;  // blocks of dX, and of [dWg; dWu]
  int per_gu, per_d;  // blocks of an expert in the second and third range
};

// DX and DW: the tiles of dX and of the weight gradients.
template <int DX, int DW>
__global__ __launch_bounds__(256) void grads_f32_kernel(
    Experts ex, const float* __restrict__ x, const float* __restrict__ dy, const float* __restrict__ dgu,
    const float* __restrict__ h, const char* __restrict__ wbase, int64_t expert_bytes, int H, int I,
    Ranges ranges, float* __restrict__ dx, char* __restrict__ dw) {
  __shared__ float lds[std::max(TileF32<DX>::LDS, TileF32<DW>::LDS)];
  int64_t b = blockIdx.x;
  if (b < ranges.dx) {
    const int nh = (H + DX - 1) / DX;
    rows_product_f32<DX>(ex, static_cast<int>(b / nh), static_cast<int>(b % nh) * DX, false, dgu,
                     2 * static_cast<int64_t>(I), wbase, expert_bytes, 0, H, 2 * I, dx, lds);
    return;
  }
  b -= ranges.dx;
  const int nh = (H + DW - 1) / DW, ni = (I + DW - 1) / DW;
  if (b < ranges.dwgu) {
    const int e = static_cast<int>(b / ranges.per_gu), at = static_cast<int>(b % ranges.per_gu);
    weight_grad_f32<DW>(ex, e, at / nh * DW, at % nh * DW, dgu, 2 * I, x, H, expert_bytes, 0, dw, lds);
    return;
  }
  b -= ranges.dwgu;
  const int e = static_cast<int>(b / ranges.per_d), at = static_cast<int>(b % ranges.per_d);
  weight_grad_f32<DW>(ex, e, at / ni * DW, at % ni * DW, dy, H, h, I, expert_bytes,
                  2 * static_cast<int64_t>(H) * I * 4, dw, lds);
}

// ---------------------------------------------------------------------------
// bf16
// ---------------------------------------------------------------------------

template <int TR>
TILE_KERNEL dh_kernel(Experts ex, const uint16_t* __restrict__ dy, const char* __restrict__ wbase,
                      int64_t expert_bytes, int H, int I, Order order, float* __restrict__ dh) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  int m, n;
  place(order, blockIdx.x, &m, &n);
  rows_product<TR>(ex, m, n, m == 0 && n == 0, dy, H, wbase, expert_bytes,
                   2 * static_cast<int64_t>(H) * I * 2, I, H, dh, (lds_char*)smem);
}

// g and u for half a tile's columns, then dG, dU and h from dH.
template <int TR, int MI>
__device__ __forceinline__ void gate_up_tile(const Tile& t, int n0, const uint16_t* x,
                                             const uint16_t* W, int H, int I, const float* dh,
                                             uint16_t* dgu, uint16_t* h, lds_char* smem) {
  using S = TileShape<TR, MI, true>;
  constexpr int HALF = S::NJ / 2, COLS = HALF * 32, OUT = S::TN / 2;
  Operand<false, S::ROWS> oa;
  Operand<false, S::TN> ob;
  oa.init(x + static_cast<int64_t>(t.row0) * H, H, H, [&](int r) { return r < t.rows ? r : -1; });
  ob.init(W + static_cast<int64_t>(n0) * H, H, H,
          [&](int r) { return n0 + r % OUT < I ? r % OUT + r / OUT * I : -1; });
  floatx16 acc[S::MW][S::NJ];
  tile_product<TR, MI, true, false, false>(oa, ob, H, smem, acc);
  const int c0 = n0 + S::first_col(), cols = I - c0;
  if (cols <= 0) return;
#pragma unroll
  for (int i = 0; i < S::MW; ++i) {
    const int r0 = S::first_row() + i * 32, rows = t.rows - r0;
    if (rows <= 0) return;
    // dH of the lane's row, all of it in flight at once; a lane past the tile or past I reads a
    // place inside and its values are not stored
    const float* drow = dh + static_cast<int64_t>(t.row0 + min(lane_row<TR, MI, true>(i), t.rows - 1)) * I;
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

template <int TR>
TILE_KERNEL gate_up_kernel(Experts ex, const uint16_t* __restrict__ x, const char* __restrict__ wbase,
                           int64_t expert_bytes, int H, int I, Order order, const float* __restrict__ dh,
                           uint16_t* __restrict__ dgu, uint16_t* __restrict__ h) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  int m, n;
  place(order, blockIdx.x, &m, &n);
  const int n0 = n * (tile_columns(TR, true) / 2);
  Tile t;
  if (n0 >= I || !find_tile<TR>(ex, m, false, &t)) return;
  const uint16_t* W = reinterpret_cast<const uint16_t*>(wbase + t.slot * expert_bytes);
  by_rows<TR>(t.rows, [&](auto mi) {
    gate_up_tile<TR, decltype(mi)::value>(t, n0, x, W, H, I, dh, dgu, h, (lds_char*)smem);
  });
}

struct GradsOrder {
  Order dx, gu, d;  // of dX; of an expert's [dWg; dWu] and dWd
};

template <int TR>
TILE_KERNEL grads_kernel(Experts ex, const uint16_t* __restrict__ x, const uint16_t* __restrict__ dy,
                         const uint16_t* __restrict__ dgu, const uint16_t* __restrict__ h,
                         const char* __restrict__ wbase, int64_t expert_bytes, int H, int I,
                         Ranges ranges, GradsOrder order, uint16_t* __restrict__ dx,
                         char* __restrict__ dw) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  lds_char* lds = (lds_char*)smem;
  int m, n;
  int64_t b = blockIdx.x;
  if (b < ranges.dx) {
    place(order.dx, static_cast<int>(b), &m, &n);
    rows_product<TR>(ex, m, n, false, dgu, 2 * I, wbase, expert_bytes, 0, H, 2 * I, dx, lds);
    return;
  }
  b -= ranges.dx;
  const bool gu = b < ranges.dwgu;
  if (!gu) b -= ranges.dwgu;
  const int per = gu ? ranges.per_gu : ranges.per_d;
  const int e = static_cast<int>(b / per);
  place(gu ? order.gu : order.d, static_cast<int>(b % per), &m, &n);
  weight_grad<TR>(ex, e, m, n, gu ? dgu : dy, gu ? 2 * I : H, gu ? x : h, gu ? H : I, expert_bytes,
                  gu ? 0 : 2 * static_cast<int64_t>(H) * I * 2, dw, lds);
}

struct Call {
  Experts ex;
  int H, I;
  const char* wbase;
  int64_t expert_bytes;
  char* ws;
  BackwardWs L;
  void* dx_perm;
  char* dw;
  hipStream_t s;
};

template <int DX, int DW>
int launch_grads_f32(const Call& c, const float* x, const float* dy, const float* dgu, const float* h) {
  const int E = c.ex.E, H = c.H, I = c.I;
  Ranges r;
  r.dx = c.dx_perm ? max_tiles(c.ex.R, E, DX) * ceil_div(H, DX) : 0;
  r.per_gu = ceil_div(2 * I, DW) * ceil_div(H, DW);
  r.per_d = ceil_div(H, DW) * ceil_div(I, DW);
  r.dwgu = c.dw ? static_cast<int64_t>(E) * r.per_gu : 0;
  const int64_t blocks = r.dx + r.dwgu + (c.dw ? static_cast<int64_t>(E) * r.per_d : 0);
  if (blocks == 0) return MOE_OK;
  hipLaunchKernelGGL((grads_f32_kernel<DX, DW>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0, c.s, c.ex,
                     x, dy, dgu, h, c.wbase, c.expert_bytes, H, I, r, static_cast<float*>(c.dx_perm), c.dw);
  MOE_LAUNCH_CHECK("moe_grouped_swiglu_backward: gradients");
  return MOE_OK;
}

int run_f32(const Call& c, const float* x, const float* dy) {
  const int E = c.ex.E, H = c.H, I = c.I;
  float* dh = reinterpret_cast<float*>(c.ws + c.L.dh_off);
  float* dgu = reinterpret_cast<float*>(c.ws + c.L.dgu_off);
  float* h = reinterpret_cast<float*>(c.ws + c.L.h_off);
  const int64_t large = max_tiles(c.ex.R, E, 64);
  if (c.ex.R > 0) {
    bool small = small_tiles_f32(large * ceil_div(I, 64));
    int tr = small ? 32 : 64;
    hipLaunchKernelGGL(small ? dh_f32_kernel<32> : dh_f32_kernel<64>,
                       dim3(static_cast<unsigned>(max_tiles(c.ex.R, E, tr)), ceil_div(I, tr)), dim3(256), 0,
                       c.s, c.ex, dy, c.wbase, c.expert_bytes, H, I, dh);
    MOE_LAUNCH_CHECK("moe_grouped_swiglu_backward: dh");
    small = small_tiles_f32(large * ceil_div(I, 32));
    tr = small ? 32 : 64;
    hipLaunchKernelGGL(small ? gate_up_backward_f32_kernel<32> : gate_up_backward_f32_kernel<64>,
                       dim3(static_cast<unsigned>(max_tiles(c.ex.R, E, tr)), ceil_div(I, tr / 2)), dim3(256), 0,
                       c.s, c.ex, x, c.wbase, c.expert_bytes, H, I, dh, dgu, h);
    MOE_LAUNCH_CHECK("moe_grouped_swiglu_backward: gate/up");
  }
  const int64_t nh = ceil_div(H, 64), ni = ceil_div(I, 64);
  const bool small_dx = small_tiles_f32(large * nh);
  const bool small_dw = small_tiles_f32(E * nh * (ceil_div(2 * I, 64) + ni));
  auto launch = small_dx ? (small_dw ? launch_grads_f32<32, 32> : launch_grads_f32<32, 64>)
                         : (small_dw ? launch_grads_f32<64, 32> : launch_grads_f32<64, 64>);
  return launch(c, x, dy, dgu, h);
}

// Large tiles when dH and dX together have one for every CU, else small ones, of which there are 16
// times as many.  Measured, large against small: 954 tokens x 3 of 3 experts, 840 x 120 (75 large
// tiles) 91 / 46 us; 239 x 3 of 42, 88 x 120 (90) 34 / 17 us; 136 x 3 of 20, 3984 x 72 (357) 95 / 96 us;
// 1623 x 7 of 16, 984 x 616 (427) 234 / 390 us; 18 x 8 of 42, 1848 x 1296 (602) 416 / 573 us.
bool large_tiles(int R, int E, int H, int I) {
  return max_tiles(R, E, 256) * (ceil_div(H, 256) + ceil_div(I, 256)) >= 256;
}

template <int TR>
int run_bf16(const Call& c, const uint16_t* x, const uint16_t* dy) {
  const int E = c.ex.E, H = c.H, I = c.I;
  constexpr int TN = tile_columns(TR, false);
  float* dh = reinterpret_cast<float*>(c.ws + c.L.dh_off);
  uint16_t* dgu = reinterpret_cast<uint16_t*>(c.ws + c.L.dgu_off);
  uint16_t* h = reinterpret_cast<uint16_t*>(c.ws + c.L.h_off);
  const int64_t cap = max_tiles(c.ex.R, E, TR);
  int64_t n;
  if (c.ex.R > 0) {
    Order o = make_order(TR, cap, ceil_div(I, TN), &n);
    int rc = launch_tiles("moe_grouped_swiglu_backward: dh", dh_kernel<TR>, n, tile_lds(TR, false), c.s,
                          c.ex, dy, c.wbase, c.expert_bytes, H, I, o, dh);
    if (rc) return rc;
    o = make_order(TR, cap, ceil_div(I, tile_columns(TR, true) / 2), &n);
    rc = launch_tiles("moe_grouped_swiglu_backward: gate/up", gate_up_kernel<TR>, n, tile_lds(TR, true),
                      c.s, c.ex, x, c.wbase, c.expert_bytes, H, I, o, dh, dgu, h);
    if (rc) return rc;
  }
  GradsOrder o{};
  Ranges r{0, 0, 1, 1};
  int64_t blocks = 0;
  if (c.dx_perm && c.ex.R > 0) {
    o.dx = make_order(TR, cap, ceil_div(H, TN), &n);
    blocks = r.dx = n;
  }
  if (c.dw) {
    o.gu = make_order(TR, ceil_div(2 * I, TR), ceil_div(H, TN), &n);
    r.per_gu = static_cast<int>(n);
    o.d = make_order(TR, ceil_div(H, TR), ceil_div(I, TN), &n);
    r.per_d = static_cast<int>(n);
    r.dwgu = static_cast<int64_t>(E) * r.per_gu;
    blocks += r.dwgu + static_cast<int64_t>(E) * r.per_d;
  }
  if (blocks == 0) return MOE_OK;
  return launch_tiles("moe_grouped_swiglu_backward: gradients", grads_kernel<TR>, blocks,
                      tile_lds(TR, false), c.s, c.ex, x, dy, dgu, h, c.wbase, c.expert_bytes, H, I, r, o,
                      static_cast<uint16_t*>(c.dx_perm), c.dw);
}

// Zeros for the blocks of dw whose slot no expert maps to.  `parts` workgroups a slot, each of which
// looks the slot up in slot_of (4 KB at most, from L2) and leaves if an expert has it, so the cost is
// a launch and the bytes that have to be zero.  Measured, 256 slots of 88 MB: every slot taken 10.7 us,
// 37 of them free 0.6 ms (5.0 TB/s).
constexpr int64_t kClearBytes = 1 << 20;  // of a workgroup

__global__ __launch_bounds__(256) void clear_unmapped_kernel(const int32_t* __restrict__ slot_of, int E,
                                                             int parts, int64_t words,
                                                             uint32_t* __restrict__ dw) {
  typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
  const int slot = blockIdx.x / parts, part = blockIdx.x % parts;
  int mapped = 0;
  for (int e = threadIdx.x; e < E; e += 256) mapped |= slot_of[e] == slot;
  if (__syncthreads_or(mapped)) return;
  uint32_t* p = dw + slot * words;
  const int64_t begin = part * (kClearBytes / 4), end = min(begin + kClearBytes / 4, words);
  for (int64_t i = begin + threadIdx.x * 4; i < end; i += 1024) {
    if (i + 4 <= end) {
      __builtin_nontemporal_store(u32x4_a4{0, 0, 0, 0}, reinterpret_cast<u32x4_a4*>(p + i));
    } else {
      for (int64_t j = i; j < end; ++j) p[j] = 0;
    }
  }
}

}  // namespace
}  // namespace moe

extern "C" int moe_clear_unmapped(const moe_wbuf* w, void* dw, moe_stream_t stream) {
  using namespace moe;
  const char* who = "moe_clear_unmapped";
  if (!w || !w->slot_of || w->n_experts < 1 || w->n_slots < 0 || w->expert_bytes < 4 || w->expert_bytes % 4 != 0)
    return fail(MOE_ERR_ARG, "%s: bad merged buffer", who);
  if (w->n_experts > MOE_MAX_E) return fail(MOE_ERR_UNSUPPORTED, "%s: E=%d above %d", who, w->n_experts, MOE_MAX_E);
  const int64_t parts = (w->expert_bytes - 1) / kClearBytes + 1;  // no sum or product here can pass 64 bits
  if (parts > UINT32_MAX / 256 || too_many(parts * w->n_slots, 256))
    return fail(MOE_ERR_UNSUPPORTED, "%s: %d slots of %lld bytes are more than a launch takes", who, w->n_slots,
                static_cast<long long>(w->expert_bytes));
  if (w->n_slots == 0) return MOE_OK;
  if (!dw) return fail(MOE_ERR_ARG, "%s: null pointer", who);
  if (reinterpret_cast<uintptr_t>(dw) % 4 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "%s: a pointer is not aligned to 4 bytes", who);
  hipStream_t s = as_stream(stream);
  hipLaunchKernelGGL(clear_unmapped_kernel, dim3(static_cast<unsigned>(parts * w->n_slots)), dim3(256), 0, s,
                     w->slot_of, w->n_experts, static_cast<int>(parts), w->expert_bytes / 4,
                     static_cast<uint32_t*>(dw));
  MOE_LAUNCH_CHECK("moe_clear_unmapped: launch");
  return debug_check(MOE_OK, who, s, nullptr);
}

extern "C" int moe_grouped_swiglu_backward_workspace_size(int R, int E, int H, int I, moe_dtype dtype,
                                                          size_t* bytes) {
  using namespace moe;
  if (!bytes || R < 0 || E < 1 || H < 1 || I < 1 || (dtype != MOE_F32 && dtype != MOE_BF16))
    return fail(MOE_ERR_ARG, "moe_grouped_swiglu_backward_workspace_size: bad arguments");
  *bytes = backward_ws(R, I, dtype).total;
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
  if (eb / 3 >= (int64_t{1} << 30) || H > kMaxSide || I > kMaxSide)
    return fail(MOE_ERR_UNSUPPORTED, "%s: H=%d or I=%d above %d, or a matrix of 2^30 bytes or more", who, H,
                I, kMaxSide);
  if (dtype == MOE_BF16 && (H % 8 != 0 || I % 8 != 0))
    return fail(MOE_ERR_UNSUPPORTED, "%s: H=%d and I=%d must be multiples of 8", who, H, I);
  // the largest launch: small tiles of dX and of every expert's weight gradients
  const int64_t nh = ceil_div(H, 64), ni = ceil_div(I, 64);
  if (too_many((max_tiles(R, E, 64) + 8) * std::max(nh, 2 * ni) + E * (3 * nh * ni + 24), 256))
    return fail(MOE_ERR_UNSUPPORTED, "%s: R=%d rows of H=%d, I=%d are more than a launch takes", who, R, H, I);
  const uintptr_t all = reinterpret_cast<uintptr_t>(x_perm) | reinterpret_cast<uintptr_t>(dy_perm) |
                        reinterpret_cast<uintptr_t>(w->base) | reinterpret_cast<uintptr_t>(dx_perm) |
                        reinterpret_cast<uintptr_t>(dw) | reinterpret_cast<uintptr_t>(ws);
  if (all % (dtype == MOE_BF16 ? 16 : 4) != 0)
    return fail(MOE_ERR_UNSUPPORTED, "%s: a pointer is not aligned to %d bytes", who,
                dtype == MOE_BF16 ? 16 : 4);
  const BackwardWs L = backward_ws(R, I, dtype);
  if (!ws || ws_bytes < L.total)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", who, ws_bytes, L.total);
  if (R > 0 && (!x_perm || !dy_perm)) return fail(MOE_ERR_ARG, "%s: null pointer", who);
  hipStream_t s = as_stream(stream);
  const Call c{Experts{offsets, w->slot_of, R, E, w->n_slots, status}, H, I,
               static_cast<const char*>(w->base), eb, static_cast<char*>(ws), L, dx_perm,
               static_cast<char*>(dw), s};
  int rc;
  if (dtype == MOE_F32) {
    const float* x = static_cast<const float*>(x_perm);
    const float* dy = static_cast<const float*>(dy_perm);
    rc = run_f32(c, x, dy);
  } else {
    const uint16_t* x = static_cast<const uint16_t*>(x_perm);
    const uint16_t* dy = static_cast<const uint16_t*>(dy_perm);
    rc = large_tiles(R, E, H, I) ? run_bf16<256>(c, x, dy) : run_bf16<64>(c, x, dy);
  }
  return debug_check(rc, who, s, status);
}
