// moe_grouped_gemm, its gradient, and moe_grouped_gemm_mx: one product per expert over ragged rows.
//
//   y[r] = x[r] W_e^T for the rows r of expert e,     dx[r] = dy[r] W_e,     dW_e = sum_r dy[r]^T x[r]
//
// The 8-bit form takes e4m3 rows and weights with a scale for each 32 values (mx.h).
//
// Two kinds of kernel:
//   stream  few rows an expert: tiles of up to 64 rows x 64 columns whose weights go from HBM straight
//           to MFMA operands (no LDS), the depth split over the block's waves; bound by weight bytes.
//   tile    256 x 256 (64 x 64) tiles through LDS (mfma_tile.h, mx_tile.h); bound by the MFMA pipes.
#include "expert_tiles.h"
#include "row_tile.h"

#ifndef NTW
#define NTW false
#endif
#ifndef D1
#define D1 4
#define D2 3
#define D4 2
#endif
#ifndef OCC
#define OCC
#endif
namespace moe {
namespace {

// What a product reads its second operand from: the matrices [N][K] at `off` of each expert's block,
// their scales (8 bits) at `scales_off`.
struct Weights {
  const char* base;
  int64_t expert_bytes, off, scales_off;
};

// ---------------------------------------------------------------------------
// stream
// ---------------------------------------------------------------------------

constexpr int kStreamCols = 64;
constexpr int kChunk = 128;  // bytes of a row that a wave takes at a time

// One operand: blocks of 16 rows, a lane row lane % 16 and, of each chunk, 16 bytes at 16 (lane / 16)
// and 16 bytes 64 further on (what the MFMAs take from a lane).  The block's four waves take every
// fourth chunk.  MX: and the chunk's word of four scales.
template <bool MX, int BLOCKS, bool NT>
struct Stream {
  uint64_t base, scales;  // wave-uniform: where the chunk to load next starts
  uint32_t voff[BLOCKS], soff[BLOCKS];

  template <typename Src>
  __device__ __forceinline__ void init(const char* p, int64_t row_bytes, const uint8_t* s, int64_t pitch, Src src) {
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    base = reinterpret_cast<uint64_t>(p) + wave * kChunk;
    scales = reinterpret_cast<uint64_t>(s) + wave * 4;
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b) {
      const int r = src(b * 16 + (lane & 15));
      voff[b] = r < 0 ? kOutside : static_cast<uint32_t>(r * row_bytes + (lane >> 4) * 16);
      soff[b] = r < 0 ? kOutside : static_cast<uint32_t>(r * pitch);
    }
  }
  // left: bytes of a row from the chunk on; what is past them reads as zeros
  __device__ __forceinline__ void load(int left, u32x4 (&v)[BLOCKS][2], uint32_t (&s)[BLOCKS]) {
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(base), 0, kOutside, 0x00020000);
    const int k = (threadIdx.x & 48);
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b) {
      v[b][0] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, k < left ? voff[b] : kOutside, 0, NT ? 2 : 0));
      v[b][1] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, k + 64 < left ? voff[b] + 64 : kOutside, 0, NT ? 2 : 0));
    }
    if constexpr (MX) {
      const __amdgpu_buffer_rsrc_t q =
          __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(scales), 0, kOutside, 0x00020000);
#pragma unroll
      for (int b = 0; b < BLOCKS; ++b) s[b] = __builtin_amdgcn_raw_buffer_load_b32(q, left > 0 ? soff[b] : kOutside, 0, 0);
    }
    base += 4 * kChunk;
    scales += 16;
  }
};

// Sixteen e4m3 values times 2^(byte - 127) as bf16, which holds them exactly.
__device__ __forceinline__ void expand(const u32x4& v, uint32_t byte, bf16x8 (&out)[2]) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const float scale = __uint_as_float(byte << 23);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    bf16x2 p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = i % 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * h + i / 2], scale, true)
                   : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * h + i / 2], scale, false);
    out[h] = bf16x8{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
  }
}

// A chunk of one block of 16 rows as MFMA operands, 8 bits expanded.  word: its four scales; a lane's
// first 16 bytes are half of block 0 or 1, the others of block 2 or 3.
template <bool MX>
struct Operands {
  static constexpr int N = MX ? 4 : 2;
  bf16x8 v[N];
  __device__ __forceinline__ void set(const u32x4 (&raw)[2], uint32_t word) {
    if constexpr (MX) {
      const uint32_t s = word >> (threadIdx.x >> 2 & 8);
      bf16x8 h[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        expand(raw[i], s >> 16 * i & 0xff, h);
        v[2 * i] = h[0];
        v[2 * i + 1] = h[1];
      }
    } else {
      v[0] = __builtin_bit_cast(bf16x8, raw[0]);
      v[1] = __builtin_bit_cast(bf16x8, raw[1]);
    }
  }
};

// Tiles of 16 MF rows by 64 columns.  D: chunks in flight per wave.
template <bool MX, int MF, int D, typename O>
__global__ __launch_bounds__(256 OCC) void stream_kernel(Experts ex, Source src, const char* __restrict__ x,
                                                     const uint8_t* __restrict__ xs, Weights w, int K, int N,
                                                     int col_blocks, O* __restrict__ y) {
  constexpr int NF = kStreamCols / 16;
  __shared__ __attribute__((aligned(16))) floatx4 sums[4][MF * NF][kWave];
  Tile t;
  const int m = blockIdx.x / col_blocks, n0 = blockIdx.x % col_blocks * kStreamCols;
  if (!find_tile<16 * MF>(ex, m, blockIdx.x == 0, &t)) return;
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t row_bytes = static_cast<int64_t>(K) * (MX ? 1 : 2), pitch = MX ? mx_pitch(K) : 0;
  const char* block = w.base + t.slot * w.expert_bytes;
  const bool gather = src.src_of;
  Stream<MX, MF, false> a;
  Stream<MX, NF, NTW> b;
  a.init(gather ? x : x + t.row0 * row_bytes, row_bytes, gather ? xs : xs + t.row0 * pitch, pitch,
         [&](int r) { return r >= t.rows ? -1 : gather ? src.at(t.row0 + r) : r; });
  b.init(block + w.off + n0 * row_bytes, row_bytes,
         reinterpret_cast<const uint8_t*>(block) + w.scales_off + n0 * pitch, pitch,
         [&](int c) { return n0 + c < N ? c : -1; });
  floatx4 acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  u32x4 va[D][MF][2], vb[D][NF][2];
  uint32_t sa[D][MF], sb[D][NF];
  int left = static_cast<int>(row_bytes) - wave * kChunk;
  auto load = [&](auto d) {
    constexpr int I = decltype(d)::value;
    b.load(left, vb[I], sb[I]);
    a.load(left, va[I], sa[I]);
    left -= 4 * kChunk;
  };
  each<0, D>(load);
  // every wave makes the same number of steps; those past its depth add zeros
  for (int at = 0; at < row_bytes; at += 4 * kChunk * D) {
    each<0, D>([&](auto d) {
      constexpr int I = decltype(d)::value;
      Operands<MX> oa[MF], ob;
#pragma unroll
      for (int i = 0; i < MF; ++i) oa[i].set(va[I][i], sa[I][i]);
      // the transposed block: a lane ends with four consecutive columns of one row
#pragma unroll
      for (int j = 0; j < NF; ++j) {
        ob.set(vb[I][j], sb[I][j]);
#pragma unroll
        for (int h = 0; h < Operands<MX>::N; ++h)
#pragma unroll
          for (int i = 0; i < MF; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ob.v[h], oa[i].v[h], acc[i][j], 0, 0, 0);
      }
      load(d);
    });
  }
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) sums[wave][i * NF + j][lane] = acc[i][j];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MF; ++i) {  // wave w joins column block w
    const int f = i * NF + wave;
    const floatx4 s = (sums[0][f][lane] + sums[1][f][lane]) + (sums[2][f][lane] + sums[3][f][lane]);
    const int r = i * 16 + (lane & 15), c = n0 + wave * 16 + (lane >> 4) * 4;
    if (r >= t.rows || c >= N) continue;
    O* out = y + static_cast<int64_t>(t.row0 + r) * N + c;
    if constexpr (sizeof(O) == 4) *reinterpret_cast<floatx4*>(out) = s;
    else *reinterpret_cast<u32x2*>(out) = pack4(s[0], s[1], s[2], s[3]);
  }
}

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

template <Kind KIND, int MI, typename O>
__device__ __forceinline__ void row_tile(const Tile& t, int n0, const Source& src, const char* x, const uint8_t* xs,
                                         const char* B, const uint8_t* bs, int K, int N, O* y, lds_char* smem) {
  using S = TileShape<256, MI, false>;
  const int bytes = K * value_bytes(KIND);
  const bool gather = src.src_of;
  const auto row = [&](int r) { return r >= t.rows ? -1 : gather ? src.at(t.row0 + r) : r; };
  const auto col = [&](int c) { return n0 + c < N ? c : -1; };
  RowOperand<S::ROWS> oa;
  RowOperand<S::TN> ob;
  oa.init(gather ? x : x + static_cast<int64_t>(t.row0) * bytes, bytes, row);
  ob.init(B + static_cast<int64_t>(n0) * bytes, bytes, col);
  ScaleRows sa, sb;
  if constexpr (KIND != Kind::kBf16) {
    const int64_t pitch = mx_pitch(K);
    sa.init(gather ? xs : xs + t.row0 * pitch, pitch, row);
    sb.init(bs + n0 * pitch, pitch, col);
  }
  floatx16 acc[S::MW][S::NJ];
  RowProduct<KIND, MI> p{oa, ob, sa, sb, acc};
  p.run(bytes, smem);
  store_tile<256, MI>(acc, smem, y + static_cast<int64_t>(t.row0) * N + n0, N, t.rows, N - n0);
}

template <Kind KIND, typename O>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void row_kernel(
    Experts ex, Source src, const char* __restrict__ x, const uint8_t* __restrict__ xs, Weights w, int K, int N,
    Order order, O* __restrict__ y) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  int m, n;
  place(order, blockIdx.x, &m, &n);
  const int n0 = n * 256;
  Tile t;
  if (n0 >= N || !find_tile<256, true>(ex, m, m == 0 && n == 0, &t)) return;
  const char* block = w.base + t.slot * w.expert_bytes;
  by_rows<256>(t.rows, [&](auto mi) {
    row_tile<KIND, decltype(mi)::value>(t, n0, src, x, xs, block + w.off,
                                        reinterpret_cast<const uint8_t*>(block) + w.scales_off, K, N, y,
                                        (lds_char*)smem);
  });
}

// dX and dW in one launch: the blocks of one fill the CUs that the last of the other leave.
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
    rows_product<TR, false, true>(ex, m, n, m == 0 && n == 0, dy, N, w.base, w.expert_bytes, w.off, K, N, dx, (lds_char*)smem);
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

template <bool MX, int MF, int D, typename O>
int launch_stream(const Call& c, const void* x, const uint8_t* xs, void* y) {
  const int nb = ceil_div(c.N, kStreamCols);
  const int64_t blocks = max_tiles(c.ex.R, c.ex.E, 16 * MF) * nb;
  hipLaunchKernelGGL((stream_kernel<MX, MF, D, O>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0, c.s, c.ex,
                     c.src, static_cast<const char*>(x), xs, c.w, c.K, c.N, nb, static_cast<O*>(y));
  MOE_LAUNCH_CHECK(c.who);
  return MOE_OK;
}

// Tile height of the stream kernel by the rows that an expert has on average.
template <bool MX, typename O>
int run_stream(const Call& c, const void* x, const uint8_t* xs, void* y) {
  const int64_t per = c.ex.R / c.ex.E;
  if (per <= 8) return launch_stream<MX, 1, D1, O>(c, x, xs, y);
  if (per <= 24) return launch_stream<MX, 2, D2, O>(c, x, xs, y);
  return launch_stream<MX, 4, D4, O>(c, x, xs, y);
}

// Whether the stream kernel takes a product.
#ifndef FEW
#define FEW 64
#endif
bool few_rows(int R, int E) { return R <= FEW * static_cast<int64_t>(E); }

template <Kind KIND, typename O>
int run_rows(const Call& c, const void* x, const uint8_t* xs, void* y) {
  int64_t n;
  const Order o = make_order(256, max_tiles(c.ex.R, c.ex.E, 256), ceil_div(c.N, 256), &n);
  return launch_tiles(c.who, row_kernel<KIND, O>, n, row_tile_lds(KIND), c.s, c.ex, c.src, static_cast<const char*>(x),
                      xs, c.w, c.K, c.N, o, static_cast<O*>(y));
}

template <typename O>
int run_bf16(const Call& c, const void* x, void* y) {
  if (few_rows(c.ex.R, c.ex.E)) return run_stream<false, O>(c, x, nullptr, y);
  return run_rows<Kind::kBf16, O>(c, x, nullptr, y);
}

int run_f32(const Call& c, const void* x, void* y) {
  const bool small = small_tiles_f32(max_tiles(c.ex.R, c.ex.E, 64) * ceil_div(c.N, 64));
  const int tr = small ? 32 : 64, nb = ceil_div(c.N, tr);
  hipLaunchKernelGGL(small ? product_f32_kernel<32> : product_f32_kernel<64>,
                     dim3(static_cast<unsigned>(max_tiles(c.ex.R, c.ex.E, tr) * nb)), dim3(256), 0, c.s, c.ex, c.src,
                     static_cast<const float*>(x), c.w, c.K, c.N, nb, static_cast<float*>(y));
  MOE_LAUNCH_CHECK(c.who);
  return MOE_OK;
}

template <int TR>
int launch_grads(const Call& c, const void* x, const void* dy, void* dx, void* dw) {
  GradRanges r{0, 1};
  Order odx{}, odw{};
  int64_t n, blocks = 0;
  if (dx && c.ex.R > 0) {
    odx = make_order(TR, max_tiles(c.ex.R, c.ex.E, TR), ceil_div(c.K, tile_columns(TR, false)), &n);
    blocks = r.dx = n;
  }
  if (dw) {
    odw = make_order(TR, ceil_div(c.N, TR), ceil_div(c.K, tile_columns(TR, false)), &n);
    r.per = static_cast<int>(n);
    blocks += c.ex.E * n;
  }
  if (blocks == 0) return MOE_OK;
  return launch_tiles(c.who, grads_kernel<TR>, blocks, tile_lds(TR, false), c.s, c.ex, static_cast<const uint16_t*>(x),
                      static_cast<const uint16_t*>(dy), c.w, c.K, c.N, r, odx, odw, static_cast<uint16_t*>(dx),
                      static_cast<char*>(dw));
}

template <int DX, int DW>
int launch_grads_f32(const Call& c, const void* x, const void* dy, void* dx, void* dw) {
  GradRanges r;
  r.dx = dx ? max_tiles(c.ex.R, c.ex.E, DX) * ceil_div(c.K, DX) : 0;
  r.per = ceil_div(c.N, DW) * ceil_div(c.K, DW);
  const int64_t blocks = r.dx + (dw ? static_cast<int64_t>(c.ex.E) * r.per : 0);
  if (blocks == 0) return MOE_OK;
  hipLaunchKernelGGL((grads_f32_kernel<DX, DW>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0, c.s, c.ex,
                     static_cast<const float*>(x), static_cast<const float*>(dy), c.w, c.K, c.N, r,
                     static_cast<float*>(dx), static_cast<char*>(dw));
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
  // the largest launch: small tiles of the rows and of every expert's weight gradient
  const int64_t side = std::max(ceil_div(K, 32), ceil_div(N, 32));
  if (too_many((max_tiles(R, E, 16) + 8) * side + static_cast<int64_t>(E) * ceil_div(K, 32) * ceil_div(N, 32) + 24, 256))
    return fail(MOE_ERR_UNSUPPORTED, "%s: R=%d rows of K=%d, N=%d are more than a launch takes", who, R, K, N);
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
  rc = check_aligned(who, bits(x) | bits(w->base) | bits(y) | static_cast<uintptr_t>(w->expert_bytes | w_off),
                     dtype == MOE_F32 ? 4 : 16);
  if (rc) return rc;
  if (R == 0) return MOE_OK;
  if (!x || !y) return fail(MOE_ERR_ARG, "%s: null pointer", who);
  hipStream_t s = as_stream(stream);
  const Call c{who, Experts{offsets, w->slot_of, R, E, w->n_slots, status}, Source{src_of, top_k, static_cast<int>(x_rows)},
               Weights{static_cast<const char*>(w->base), w->expert_bytes, w_off, 0}, K, N, s};
  rc = dtype == MOE_F32 ? run_f32(c, x, y)
                        : y_dtype == MOE_F32 ? run_bf16<float>(c, x, y) : run_bf16<uint16_t>(c, x, y);
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
  rc = check_aligned(who, bits(x) | bits(x_scales) | bits(w->base) | bits(y) |
                              static_cast<uintptr_t>(w->expert_bytes | w_off | s_off), 16);
  if (rc) return rc;
  if (R == 0) return MOE_OK;
  if (!x || !x_scales || !y) return fail(MOE_ERR_ARG, "%s: null pointer", who);
  hipStream_t s = as_stream(stream);
  const Call c{who, Experts{offsets, w->slot_of, R, E, w->n_slots, status}, Source{src_of, top_k, static_cast<int>(x_rows)},
               Weights{static_cast<const char*>(w->base), w->expert_bytes, w_off, s_off}, K, N, s};
  rc = y_dtype == MOE_F32 ? run_rows<Kind::kMxExact, float>(c, x, x_scales, y)
                          : run_rows<Kind::kMx, uint16_t>(c, x, x_scales, y);
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
  rc = check_aligned(who, bits(x) | bits(dy) | bits(w->base) | bits(dx) | bits(dw) |
                              static_cast<uintptr_t>(w->expert_bytes | w_off), dtype == MOE_F32 ? 4 : 16);
  if (rc) return rc;
  if (R > 0 && (!x || !dy)) return fail(MOE_ERR_ARG, "%s: null pointer", who);
  hipStream_t s = as_stream(stream);
  const Call c{who, Experts{offsets, w->slot_of, R, E, w->n_slots, status}, Source{},
               Weights{static_cast<const char*>(w->base), w->expert_bytes, w_off, 0}, K, N, s};
  if (dtype == MOE_F32) {
    const int64_t nk = ceil_div(K, 64);
    const bool small_dx = small_tiles_f32(max_tiles(R, E, 64) * nk);
    const bool small_dw = small_tiles_f32(E * nk * ceil_div(N, 64));
    auto launch = small_dx ? (small_dw ? launch_grads_f32<32, 32> : launch_grads_f32<32, 64>)
                           : (small_dw ? launch_grads_f32<64, 32> : launch_grads_f32<64, 64>);
    rc = launch(c, x, dy, R > 0 ? dx : nullptr, dw);
  } else {
    // large tiles when dX has one for every CU, else small ones, of which there are 16 times as many
    rc = max_tiles(R, E, 256) * ceil_div(K, 256) >= kCus ? launch_grads<256>(c, x, dy, dx, dw)
                                                         : launch_grads<64>(c, x, dy, dx, dw);
  }
  return debug_check(rc, who, s, status);
}
