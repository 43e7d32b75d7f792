// moe_grouped_gemm, its gradient, and moe_grouped_gemm_mx: one product per expert over ragged rows.
//
//   y[r] = x[r] W_e^T for the rows r of expert e,     dx[r] = dy[r] W_e,     dW_e = sum_r dy[r]^T x[r]
//
// The 8-bit form takes e4m3 rows and weights with a scale for each 32 values (mx.h).
//
// The forward products of both types run on the tile loop of row_tile.h (256 x 256, 64 x 256 for few tiles,
// 64 x 64 with the depth split over the waves for fewer), the gradients on that of mfma_tile.h, whose
// operands run across the depth, and f32 on tiles of the fp32 MFMA (expert_tiles.h).  Blocks find their
// tile from offsets by themselves.  Many rows are bound by the MFMA pipes, few by the weights' bytes.
// Measured: 64 tokens x 8 on 64 experts of 7168 x 4096 in 8 bits 327 us (5.9 TB/s); 65536 rows of 32 such
// experts 1.56 ms (2470 TFLOP/s).
#include "expert_tiles.h"
#include "row_tile.h"

namespace moe {
namespace {

// What a product reads its second operand from: the matrices [N][K] at `off` of each expert's block, their
// scales (8 bits) at `scales_off`.
struct Weights {
  const char* base;
  int64_t expert_bytes, off, scales_off;
};

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------

template <int TR>
__global__ __launch_bounds__(256) void product_f32_kernel(Experts ex, Source src, const float* __restrict__ x,
                                                          Weights w, int K, int N, int col_blocks,
                                                          float* __restrict__ y) {
  __shared__ float lds[TileF32<TR>::LDS];
  rows_product_f32<TR, true>(ex, blockIdx.x / col_blocks, blockIdx.x % col_blocks * TR, blockIdx.x == 0, x, K, w.base,
                             w.expert_bytes, w.off, N, K, y, lds, src);
}

// A tile's f32 outputs, 32 rows by 64 columns at a time.  From the accumulators a lane would store 16 bytes of
// a row of its own; through LDS, whose rows are padded by 16 bytes, a row leaves as two whole lines.
// Measured, from the accumulators, through LDS with plain and with non-temporal stores: 16384 rows of 512 x
// 4096, bf16 126 / 118 / 107 us; 32768 rows of 64 experts of 2048 x 7168, 8 bits 1072 / 1029 / 1018 us.
template <int MI>
__device__ __forceinline__ void store_rows(
    const floatx16 (&acc)[TileShape<256, MI, false>::MW][TileShape<256, MI, false>::NJ], lds_char* smem, float* C,
    int64_t ld, int rows, int cols) {
  using S = TileShape<256, MI, false>;
  static_assert(S::NJ % 2 == 0, "two column blocks at a time");
  constexpr int PITCH = 64 * 4 + 16;
  typedef __attribute__((address_space(3))) floatx4 lds_floatx4;
  const int lane = threadIdx.x & (kWave - 1), c = lane % 16 * 4;
  lds_char* mine = smem + (threadIdx.x / kWave) * 16384;
#pragma unroll
  for (int i = 0; i < S::MW; ++i)
#pragma unroll
    for (int j = 0; j < S::NJ; j += 2) {
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        const floatx16& a = acc[i][j + v / 4];
        const int e = v % 4 * 4;
        *reinterpret_cast<lds_floatx4*>(mine + (lane & 31) * PITCH + (v / 4 * 32 + lane_col(v % 4)) * 4) =
            floatx4{a[e], a[e + 1], a[e + 2], a[e + 3]};
      }
      wave_lds_sync();
      const int r0 = S::first_row() + i * 32, c0 = S::first_col() + S::col(j);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int r = k * 4 + lane / 16;
        const floatx4 d = *reinterpret_cast<lds_floatx4*>(mine + r * PITCH + c * 4);
        floatx4* to = reinterpret_cast<floatx4*>(C + (r0 + r) * ld + c0 + c);
        if (r0 + r < rows && c0 + c < cols) __builtin_nontemporal_store(d, to);
      }
      wave_lds_sync();
    }
}
template <int MI>
__device__ __forceinline__ void store_rows(
    const floatx16 (&acc)[TileShape<256, MI, false>::MW][TileShape<256, MI, false>::NJ], lds_char* smem, uint16_t* C,
    int64_t ld, int rows, int cols) {
  store_tile<256, MI>(acc, smem, C, ld, rows, cols);
}

template <Kind KIND, int MI, typename O>
__device__ __forceinline__ void row_tile(const Tile& t, int n0, const Source& src, const char* x, const uint8_t* xs,
                                         const char* B, const uint8_t* bs, int K, int N, int start, O* y,
                                         lds_char* smem) {
  using S = TileShape<256, MI, false>;
  const int bytes = K * value_bytes(KIND);
  const bool gather = src.src_of;
  const auto row = [&](int r) { return r >= t.rows ? -1 : gather ? src.at(t.row0 + r) : r; };
  const auto col = [&](int c) { return n0 + c < N ? c : -1; };
  RowOperand<S::ROWS> oa;
  RowOperand<S::TN> ob;
  oa.init(gather ? x : x + static_cast<int64_t>(t.row0) * bytes, bytes, start, row);
  ob.init(B + static_cast<int64_t>(n0) * bytes, bytes, start, col);
  ScaleRows sa, sb;
  if constexpr (KIND != Kind::kBf16) {
    const int64_t pitch = mx_pitch(K);
    sa.init(gather ? xs : xs + t.row0 * pitch, pitch, start / kMxBlock, row);
    sb.init(bs + n0 * pitch, pitch, start / kMxBlock, col);
  }
  floatx16 acc[S::MW][S::NJ];
  RowProduct<KIND, MI> p{oa, ob, sa, sb, acc};
  p.run(bytes, smem);
  store_rows<MI>(acc, smem, y + static_cast<int64_t>(t.row0) * N + n0, N, t.rows, N - n0);
}

// Tiles of TR rows (256 or 64) by 256 columns.  phases: how many 512-byte parts of a row the units of tiles
// take turns to start at (1: all at the row's start).  Where a row is a multiple of 2 KB, all tiles at one
// depth would ask few of the memory channels; the tiles of a unit go together, since they read the same
// rows.  Measured at 32 experts of 2048 columns, the same start against these: 8 rows each, bf16, depth
// 2048 65.8 / 48.3 us, 4096 129 / 101 us; 128 rows each, bf16, 2048 70 / 56 us, 4096 131 / 102 us, 8 bits,
// 4096 74 / 60 us; 2048 rows each of 8 experts of 4096 x 4096 428 / 427 us.  (A start of its own for every
// tile took 57 and 93 us at 8 rows, and 470 at 2048.)
template <Kind KIND, int TR, typename O>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void row_kernel(
    Experts ex, Source src, const char* __restrict__ x, const uint8_t* __restrict__ xs, Weights w, int K, int N,
    Order order, int phases, O* __restrict__ y) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  int m, n;
  place(order, blockIdx.x, &m, &n);
  const int n0 = n * 256;
  Tile t;
  if (n0 >= N || !find_tile<TR, true>(ex, m, m == 0 && n == 0, &t)) return;
  const char* block = w.base + t.slot * w.expert_bytes;
  const int start = static_cast<int>((blockIdx.x / 8 / (order.gm * order.gn) * 8 + blockIdx.x % 8) % phases) * 512;
  const auto run = [&](auto mi) {
    row_tile<KIND, decltype(mi)::value>(t, n0, src, x, xs, block + w.off,
                                        reinterpret_cast<const uint8_t*>(block) + w.scales_off, K, N, start, y,
                                        (lds_char*)smem);
  };
  if constexpr (TR == 256) by_rows<256>(t.rows, run);
  else if (t.rows > 32) run(std::integral_constant<int, 2>{});
  else run(std::integral_constant<int, 1>{});
}

// Tiles of 64 rows by 64 columns, the depth split over the waves.
template <Kind KIND, typename O>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 2))) void split_kernel(
    Experts ex, Source src, const char* __restrict__ x, const uint8_t* __restrict__ xs, Weights w, int K, int N,
    int col_blocks, O* __restrict__ y) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const int m = blockIdx.x / col_blocks, n0 = blockIdx.x % col_blocks * 64;
  Tile t;
  if (!find_tile<64>(ex, m, blockIdx.x == 0, &t)) return;
  const int bytes = K * value_bytes(KIND);
  const int64_t pitch = KIND == Kind::kBf16 ? 0 : mx_pitch(K);
  const char* block = w.base + t.slot * w.expert_bytes;
  const bool gather = src.src_of;
  const auto run = [&](auto mw) {
    SplitProduct<KIND, decltype(mw)::value> p;
    p.init(gather ? x : x + static_cast<int64_t>(t.row0) * bytes, block + w.off + static_cast<int64_t>(n0) * bytes,
           gather ? xs : xs + t.row0 * pitch, reinterpret_cast<const uint8_t*>(block) + w.scales_off + n0 * pitch, bytes,
           pitch, [&](int r) { return r >= t.rows ? -1 : gather ? src.at(t.row0 + r) : r; },
           [&](int c) { return n0 + c < N ? c : -1; });
    p.run(bytes, (lds_char*)smem, [&](int r, int c, floatx4 s) {
      if (r >= t.rows || n0 + c >= N) return;
      O* out = y + static_cast<int64_t>(t.row0 + r) * N + n0 + c;
      if constexpr (sizeof(O) == 4) *reinterpret_cast<floatx4*>(out) = s;
      else *reinterpret_cast<u32x2*>(out) = pack4(s[0], s[1], s[2], s[3]);
    });
  };
  if (t.rows > 32) run(std::integral_constant<int, 2>{});
  else run(std::integral_constant<int, 1>{});
}

// dX and dW in one launch where their tiles are alike: the blocks of one fill the CUs that the last of the other leave.
struct GradRanges {
  int64_t dx;  // blocks of dX
  int per;     // blocks of an expert's dW
};

// Without dX nobody else looks for experts that have rows and no slot.
template <int TR>
__device__ __forceinline__ void report_absent(const Experts& ex, bool first) {
  Tile t;
  if (first) find_tile<TR>(ex, -1, true, &t);
}

template <int TR>
TILE_KERNEL grads_kernel(Experts ex, const uint16_t* __restrict__ x, const uint16_t* __restrict__ dy, Weights w, int K,
                         int N, GradRanges ranges, Order odx, Order odw, uint16_t* __restrict__ dx,
                         char* __restrict__ dw) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  int m, n;
  int64_t b = blockIdx.x;
  if (b < ranges.dx) {
    place(odx, static_cast<int>(b), &m, &n);
    rows_product<TR, true>(ex, m, n, m == 0 && n == 0, dy, N, w.base, w.expert_bytes, w.off, K, N, dx, (lds_char*)smem);
    return;
  }
  report_absent<TR>(ex, blockIdx.x == 0);
  b -= ranges.dx;
  place(odw, static_cast<int>(b % ranges.per), &m, &n);
  weight_grad<TR>(ex, static_cast<int>(b / ranges.per), m, n, dy, N, x, K, w.expert_bytes, w.off, dw, (lds_char*)smem);
}

template <int DX, int DW>
__global__ __launch_bounds__(256) void grads_f32_kernel(Experts ex, const float* __restrict__ x,
                                                        const float* __restrict__ dy, Weights w, int K, int N,
                                                        GradRanges ranges, float* __restrict__ dx,
                                                        char* __restrict__ dw) {
  __shared__ float lds[std::max(TileF32<DX>::LDS, TileF32<DW>::LDS)];
  int64_t b = blockIdx.x;
  if (b < ranges.dx) {
    const int nk = (K + DX - 1) / DX;
    rows_product_f32<DX>(ex, static_cast<int>(b / nk), static_cast<int>(b % nk) * DX, b == 0, dy, N, w.base,
                         w.expert_bytes, w.off, K, N, dx, lds);
    return;
  }
  report_absent<DX>(ex, blockIdx.x == 0);
  b -= ranges.dx;
  const int nk = (K + DW - 1) / DW, at = static_cast<int>(b % ranges.per);
  weight_grad_f32<DW>(ex, static_cast<int>(b / ranges.per), at / nk * DW, at % nk * DW, dy, N, x, K, w.expert_bytes,
                      w.off, dw, lds);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

struct Call {
  const char* who;
  Experts ex;
  Source src;
  Weights w;
  int K, N;
  hipStream_t s;
};

// The tallest unit of 4, 2 or 1 by up to 8 tiles (columns cut evenly) that leaves every XCD four, else single
// tiles: tiles of one row panel that run together on an XCD read it once into its L2.  Measured, 256 rows
// each of 32 experts of 2112 x 2048, 1 x 8 against single tiles, which read x again for each column tile:
// bf16 73 / 88 us, 8 bits 45 / 60 us; 8 bits of 4224 x 2048 76 / 108 us.
Order row_order(int64_t mt, int64_t nt, int64_t* blocks) {
  Order o{4, static_cast<int>(ceil_div64(nt, ceil_div64(nt, 8))), 0};
  while (o.gm > 1 && ceil_div64(mt, o.gm) * ceil_div64(nt, o.gn) < 32) o.gm /= 2;
  if (ceil_div64(mt, o.gm) * ceil_div64(nt, o.gn) < 32) o.gm = o.gn = 1;
  o.n_gn = static_cast<int>(ceil_div64(nt, o.gn));
  *blocks = ceil_div64(ceil_div64(mt, o.gm) * o.n_gn, 8) * 8 * o.gm * o.gn;
  return o;
}

// What a forward product launches, by how many tiles each kind would have (with one for every expert more
// than there can be):
//   split  up to two a CU.  Measured, 4 experts, split against 64 x 256: bf16, 8 rows each of 4096 x 512
//          9.9 / 34.8 us, 128 rows of 2048 x 2048 13.2 / 21.7 us, 256 rows (640 tiles) 21.4 / 22.0 us; 64 rows
//          of 32 experts of 2112 x 2048 (2048 tiles) 72 / 54 us.
//   64     up to one a CU.  Against 256 x 256: bf16, 1024 rows each of 4096 x 512 40 / 72 us, of 1024 x 768
//          15 / 25 us; of 2048 x 2048 (544 tiles) 47 / 43 us.
struct RowPlan {
  enum Tiles { kSplit, k64, k256 } tiles;
  Order order;  // of all but split tiles
  int64_t blocks;
};

RowPlan plan_rows(int R, int E, int N) {
  const int64_t small = max_tiles(R, E, 64);
  RowPlan p{RowPlan::kSplit, Order{}, small * ceil_div(N, 64)};
  if (p.blocks <= 2 * kCus) return p;
  p.tiles = small * ceil_div(N, 256) <= kCus ? RowPlan::k64 : RowPlan::k256;
  p.order = row_order(p.tiles == RowPlan::k64 ? small : max_tiles(R, E, 256), ceil_div(N, 256), &p.blocks);
  return p;
}

template <Kind KIND, int TR, typename O>
int launch_rows(const Call& c, const RowPlan& p, const void* x, const uint8_t* xs, void* y) {
  const int bytes = c.K * value_bytes(KIND);
  const int phases = bytes % 2048 == 0 ? bytes / 512 : 1;
  return launch_tiles(c.who, row_kernel<KIND, TR, O>, p.blocks, row_tile_lds(KIND), c.s, c.ex, c.src,
                      static_cast<const char*>(x), xs, c.w, c.K, c.N, p.order, phases, static_cast<O*>(y));
}

template <Kind KIND, typename O>
int run_rows(const Call& c, const RowPlan& p, const void* x, const uint8_t* xs, void* y) {
  if (p.tiles == RowPlan::k256) return launch_rows<KIND, 256, O>(c, p, x, xs, y);
  if (p.tiles == RowPlan::k64) return launch_rows<KIND, 64, O>(c, p, x, xs, y);
  return launch_tiles(c.who, split_kernel<KIND, O>, p.blocks, SplitProduct<KIND, 2>::LDS, c.s, c.ex, c.src,
                      static_cast<const char*>(x), xs, c.w, c.K, c.N, ceil_div(c.N, 64), static_cast<O*>(y));
}

// The same in f32: tiles of 64 x 64 or 32 x 32.
struct F32Plan {
  int tr;
  int64_t blocks;
};

F32Plan plan_f32(int R, int E, int N) {
  const int64_t large = max_tiles(R, E, 64) * ceil_div(N, 64);
  if (small_tiles_f32(large)) return {32, max_tiles(R, E, 32) * ceil_div(N, 32)};
  return {64, large};
}

int run_f32(const Call& c, const F32Plan& p, const void* x, void* y) {
  hipLaunchKernelGGL(p.tr == 32 ? product_f32_kernel<32> : product_f32_kernel<64>, dim3(static_cast<unsigned>(p.blocks)),
                     dim3(256), 0, c.s, c.ex, c.src, static_cast<const float*>(x), c.w, c.K, c.N, ceil_div(c.N, p.tr),
                     static_cast<float*>(y));
  MOE_LAUNCH_CHECK(c.who);
  return MOE_OK;
}

// A launch of the gradients: dX, dW or both.
struct GradPlan {
  int dx, dw;  // tile sizes, 0 for what it leaves out (bf16: the same one where it has both)
  GradRanges r;
  Order odx, odw;  // bf16
  int64_t blocks;
};

GradPlan plan_grads(int R, int E, int K, int N, int dx, int dw) {
  GradPlan p{dx, dw, GradRanges{0, 1}, Order{}, Order{}, 0};
  int64_t n;
  if (dx) {
    p.odx = make_order(dx, max_tiles(R, E, dx), ceil_div(K, dx), &n);
    p.blocks = p.r.dx = n;
  }
  if (dw) {
    p.odw = make_order(dw, ceil_div(N, dw), ceil_div(K, dw), &n);
    p.r.per = static_cast<int>(n);
    p.blocks += E * n;
  }
  return p;
}

GradPlan plan_grads_f32(int R, int E, int K, int N, bool dx, bool dw) {
  const int64_t nk = ceil_div(K, 64);
  const int tx = small_tiles_f32(max_tiles(R, E, 64) * nk) ? 32 : 64, tw = small_tiles_f32(E * nk * ceil_div(N, 64)) ? 32 : 64;
  GradPlan p{tx, tw, GradRanges{0, 1}, Order{}, Order{}, 0};
  p.r.dx = dx ? max_tiles(R, E, tx) * ceil_div(K, tx) : 0;
  p.r.per = ceil_div(N, tw) * ceil_div(K, tw);
  p.blocks = p.r.dx + (dw ? static_cast<int64_t>(E) * p.r.per : 0);
  return p;
}

template <int TR>
int launch_grads(const Call& c, const GradPlan& p, const void* x, const void* dy, void* dx, void* dw) {
  return launch_tiles(c.who, grads_kernel<TR>, p.blocks, tile_lds(TR, false), c.s, c.ex, static_cast<const uint16_t*>(x),
                      static_cast<const uint16_t*>(dy), c.w, c.K, c.N, p.r, p.odx, p.odw, static_cast<uint16_t*>(dx),
                      static_cast<char*>(dw));
}

int run_grads(const Call& c, const GradPlan& p, const void* x, const void* dy, void* dx, void* dw) {
  if (p.blocks == 0) return MOE_OK;
  return std::max(p.dx, p.dw) == 256 ? launch_grads<256>(c, p, x, dy, dx, dw) : launch_grads<64>(c, p, x, dy, dx, dw);
}

int run_grads_f32(const Call& c, const GradPlan& p, const void* x, const void* dy, void* dx, void* dw) {
  if (p.blocks == 0) return MOE_OK;
  auto kernel = p.dx == 32 ? (p.dw == 32 ? grads_f32_kernel<32, 32> : grads_f32_kernel<32, 64>)
                           : (p.dw == 32 ? grads_f32_kernel<64, 32> : grads_f32_kernel<64, 64>);
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(p.blocks)), dim3(256), 0, c.s, c.ex, static_cast<const float*>(x),
                     static_cast<const float*>(dy), c.w, c.K, c.N, p.r, static_cast<float*>(dx), static_cast<char*>(dw));
  MOE_LAUNCH_CHECK(c.who);
  return MOE_OK;
}

// The checks that all three calls share.  `unit`: what K and N (8 bits: N) are multiples of; x_rows: rows
// of a gathered x, 0 without.
int check(const char* who, int R, int E, int K, int N, int unit, int bytes, const moe_wbuf* w, int64_t w_off,
          const int32_t* offsets, int64_t x_rows) {
  if (R < 0 || E < 1 || K < 1 || N < 1) return fail(MOE_ERR_ARG, "%s: bad sizes R=%d E=%d K=%d N=%d", who, R, E, K, N);
  if (E > MOE_MAX_E) return fail(MOE_ERR_UNSUPPORTED, "%s: E=%d above %d", who, E, MOE_MAX_E);
  if (!w || !w->base || !w->slot_of || !offsets) return fail(MOE_ERR_ARG, "%s: null pointer", who);
  if (K > kMaxSide || N > kMaxSide || static_cast<int64_t>(N) * K * bytes >= (int64_t{1} << 30))
    return fail(MOE_ERR_UNSUPPORTED, "%s: K=%d or N=%d above %d, or a matrix of 2^30 bytes or more", who, K, N,
                kMaxSide);
  if (K % unit != 0 || N % (unit > 8 ? 8 : unit) != 0)
    return fail(MOE_ERR_UNSUPPORTED, "%s: K=%d must be a multiple of %d and N=%d of %d", who, K, unit, N,
                unit > 8 ? 8 : unit);
  const int64_t matrix = static_cast<int64_t>(N) * K * bytes;
  if (w->n_experts != E || w_off < 0 || w->expert_bytes < matrix || w_off > w->expert_bytes - matrix)
    return fail(MOE_ERR_ARG, "%s: a %lld-byte matrix at %lld does not lie in the merged buffer's %lld-byte blocks for E=%d",
                who, static_cast<long long>(matrix), static_cast<long long>(w_off),
                static_cast<long long>(w->expert_bytes), w->n_experts);
  if (x_rows * K * bytes >= (int64_t{1} << 31))
    return fail(MOE_ERR_UNSUPPORTED, "%s: a gathered x of 2^31 bytes or more", who);
  return MOE_OK;
}

int check_blocks(const char* who, int64_t blocks) {
  if (too_many(blocks, 256))
    return fail(MOE_ERR_UNSUPPORTED, "%s: %lld workgroups are more than a launch takes", who,
                static_cast<long long>(blocks));
  return MOE_OK;
}

int check_aligned(const char* who, uintptr_t all, int to) {
  if (all % to != 0) return fail(MOE_ERR_UNSUPPORTED, "%s: a pointer or an offset is not aligned to %d bytes", who, to);
  return MOE_OK;
}

uintptr_t bits(const void* p) { return reinterpret_cast<uintptr_t>(p); }

}  // namespace
}  // namespace moe

extern "C" int moe_grouped_gemm(const void* x, const int32_t* src_of, int top_k, const int32_t* offsets, int R, int E,
                                int K, int N, moe_dtype dtype, const moe_wbuf* w, int64_t w_off, moe_dtype y_dtype,
                                void* y, int32_t* status, moe_stream_t stream) {
  using namespace moe;
  const char* who = "moe_grouped_gemm";
  if (!is_dtype(dtype) || !is_dtype(y_dtype) || (src_of && top_k < 1))
    return fail(MOE_ERR_ARG, "%s: bad dtype or top_k=%d", who, top_k);
  const int64_t x_rows = src_of ? (static_cast<int64_t>(R) + top_k - 1) / top_k : 0;
  int rc = check(who, R, E, K, N, dtype == MOE_F32 ? 1 : 8, elem_size(dtype), w, w_off, offsets, x_rows);
  if (rc) return rc;
  if (dtype == MOE_F32 && y_dtype != MOE_F32)
    return fail(MOE_ERR_UNSUPPORTED, "%s: f32 products have f32 outputs", who);
  const F32Plan f32 = plan_f32(R, E, N);
  const RowPlan rows = plan_rows(R, E, N);
  rc = check_blocks(who, dtype == MOE_F32 ? f32.blocks : rows.blocks);
  if (rc) return rc;
  rc = check_aligned(who, bits(x) | bits(w->base) | bits(y) | static_cast<uintptr_t>(w->expert_bytes | w_off),
                     dtype == MOE_F32 ? 4 : 16);
  if (rc) return rc;
  if (R == 0) return MOE_OK;
  if (!x || !y) return fail(MOE_ERR_ARG, "%s: null pointer", who);
  hipStream_t s = as_stream(stream);
  const Call c{who, Experts{offsets, w->slot_of, R, E, w->n_slots, status}, Source{src_of, top_k, static_cast<int>(x_rows)},
               Weights{static_cast<const char*>(w->base), w->expert_bytes, w_off, 0}, K, N, s};
  rc = dtype == MOE_F32 ? run_f32(c, f32, x, y)
                        : y_dtype == MOE_F32 ? run_rows<Kind::kBf16, float>(c, rows, x, nullptr, y)
                                           : run_rows<Kind::kBf16, uint16_t>(c, rows, x, nullptr, y);
  return debug_check(rc, who, s, status);
}

extern "C" int moe_grouped_gemm_mx(const uint8_t* x, const uint8_t* x_scales, const int32_t* src_of, int top_k,
                                   const int32_t* offsets, int R, int E, int K, int N, const moe_wbuf* w, int64_t w_off,
                                   int64_t s_off, moe_dtype y_dtype, void* y, int32_t* status, moe_stream_t stream) {
  using namespace moe;
  const char* who = "moe_grouped_gemm_mx";
  if (!is_dtype(y_dtype) || (src_of && top_k < 1)) return fail(MOE_ERR_ARG, "%s: bad dtype or top_k=%d", who, top_k);
  const int64_t x_rows = src_of ? (static_cast<int64_t>(R) + top_k - 1) / top_k : 0;
  int rc = check(who, R, E, K, N, kMxBlock, 1, w, w_off, offsets, x_rows);
  if (rc) return rc;
  const int64_t scales = N * mx_pitch(K);
  if (s_off < 0 || w->expert_bytes < scales || s_off > w->expert_bytes - scales)
    return fail(MOE_ERR_ARG, "%s: %lld bytes of scales at %lld do not lie in the merged buffer's %lld-byte blocks", who,
                static_cast<long long>(scales), static_cast<long long>(s_off), static_cast<long long>(w->expert_bytes));
  const RowPlan rows = plan_rows(R, E, N);
  rc = check_blocks(who, rows.blocks);
  if (rc) return rc;
  rc = check_aligned(who, bits(x) | bits(x_scales) | bits(w->base) | bits(y) |
                              static_cast<uintptr_t>(w->expert_bytes | w_off | s_off), 16);
  if (rc) return rc;
  if (R == 0) return MOE_OK;
  if (!x || !x_scales || !y) return fail(MOE_ERR_ARG, "%s: null pointer", who);
  hipStream_t s = as_stream(stream);
  const Call c{who, Experts{offsets, w->slot_of, R, E, w->n_slots, status}, Source{src_of, top_k, static_cast<int>(x_rows)},
               Weights{static_cast<const char*>(w->base), w->expert_bytes, w_off, s_off}, K, N, s};
  rc = y_dtype == MOE_F32 ? run_rows<Kind::kMxExact, float>(c, rows, x, x_scales, y)
                          : run_rows<Kind::kMx, uint16_t>(c, rows, x, x_scales, y);
  return debug_check(rc, who, s, status);
}

extern "C" int moe_grouped_gemm_backward(const void* x, const void* dy, const int32_t* offsets, int R, int E, int K,
                                         int N, moe_dtype dtype, const moe_wbuf* w, int64_t w_off, void* dx, void* dw,
                                         int32_t* status, moe_stream_t stream) {
  using namespace moe;
  const char* who = "moe_grouped_gemm_backward";
  if (!is_dtype(dtype)) return fail(MOE_ERR_ARG, "%s: bad dtype", who);
  int rc = check(who, R, E, K, N, dtype == MOE_F32 ? 1 : 8, elem_size(dtype), w, w_off, offsets, 0);
  if (rc) return rc;
  if (!dx && !dw) return fail(MOE_ERR_ARG, "%s: null pointer", who);
  const bool has_dx = dx && R > 0, has_dw = dw;
  GradPlan first, second{};
  if (dtype == MOE_F32) {
    first = plan_grads_f32(R, E, K, N, has_dx, has_dw);
  } else {
    // Large tiles for dX when it has one for every CU; for dW when it has one for every other CU, or every
    // fourth beside large tiles of dX.  Where the two differ they are launches of their own.  Measured
    // (both gradients and the forward product), dW in dX's size against its own: 32 rows each of 8 experts
    // of 2048 x 2048 (512 tiles) 61 / 51 us, 1373 rows each of 12 of 88 x 3024 (144) 138 / 130 us, 12 rows
    // each of 23 of 88 x 1168 (115) 13.8 / 20.6 us; beside large dX 4096 rows each of 8 of 512 x 1024 (64)
    // 167 / 200 us, 65536 rows of 512 x 512 (4) 1091 / 332 us.
    const bool large_dx = has_dx && max_tiles(R, E, 256) * ceil_div(K, 256) >= kCus;
    const bool large_dw = static_cast<int64_t>(E) * ceil_div(N, 256) * ceil_div(K, 256) >= (large_dx ? kCus / 4 : kCus / 2);
    const int tx = has_dx ? (large_dx ? 256 : 64) : 0, tw = has_dw ? (large_dw ? 256 : 64) : 0;
    const bool apart = tx && tw && tx != tw;
    first = plan_grads(R, E, K, N, tx, apart ? 0 : tw);
    if (apart) second = plan_grads(R, E, K, N, 0, tw);
  }
  rc = check_blocks(who, std::max(first.blocks, second.blocks));
  if (rc) return rc;
  rc = check_aligned(who, bits(x) | bits(dy) | bits(w->base) | bits(dx) | bits(dw) |
                              static_cast<uintptr_t>(w->expert_bytes | w_off), dtype == MOE_F32 ? 4 : 16);
  if (rc) return rc;
  if (R > 0 && (!x || !dy)) return fail(MOE_ERR_ARG, "%s: null pointer", who);
  hipStream_t s = as_stream(stream);
  const Call c{who, Experts{offsets, w->slot_of, R, E, w->n_slots, status}, Source{},
               Weights{static_cast<const char*>(w->base), w->expert_bytes, w_off, 0}, K, N, s};
  if (dtype == MOE_F32) {
    rc = run_grads_f32(c, first, x, dy, dx, dw);
  } else {
    rc = run_grads(c, first, x, dy, dx, dw);
    if (!rc) rc = run_grads(c, second, x, dy, dx, dw);
  }
  return debug_check(rc, who, s, status);
}
