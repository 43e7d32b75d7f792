// Products grouped by expert, shared by the kernels that run them: the list of row tiles, tiles of the
// fp32 MFMA, tiles of the bf16 one (mfma_tile.h) and the order in which workgroups take them.
#pragma once

#include <algorithm>
#include <type_traits>

#include "mfma_tile.h"
#include "rows.h"

namespace moe {

constexpr int kMaxSide = 1 << 20;  // largest H and I: bounds the grids

// Most tiles of `tr` rows that R rows of E experts can make.
inline int64_t max_tiles(int64_t R, int E, int tr) { return ceil_div64(R, tr) + std::min<int64_t>(E, R); }

// The experts' rows and slots.
struct Experts {
  const int32_t* offsets;
  const int32_t* slot_of;
  int R, E, n_slots;
  int32_t* status;
};

// Rows [lo, lo + count) of expert e, held to [0, R) whatever offsets says.
__device__ __forceinline__ int expert_rows(const Experts& x, int e, int* lo) {
  const int a = min(max(x.offsets[e], 0), x.R), b = min(max(x.offsets[e + 1], 0), x.R);
  *lo = a;
  return max(b - a, 0);
}

struct Tile {
  int row0, rows, slot;
};

// Tile m of the list that cuts each expert's rows into tiles of TR, expert by expert, leaving out
// experts without a slot in the merged buffer (a slot outside it is treated as absent, never
// read; `report`: their status bit is set).  False past the last tile.  Wave-uniform.
// LARGE_FIRST: tiles of more than TR / 2 rows come before the others, so that what the last CUs wait
// for is a small one.  Measured, expert by expert / large first: bf16, 4096 tokens x 6 on 64 skewed experts
// of 1408 x 2048 179 / 172 us, with the gradients 580 / 569; 2048 x 6 on 64 of 2048 x 1408 132 / 131; with less
// skew it costs up to 4 %: 1024 x 8 on 32 of 4096 x 2048 180 / 186, 8 bits, 8192 x 8 on 32 of 7168 x 4096
// 1543 / 1567.
template <int TR, bool LARGE_FIRST = false>
__device__ __forceinline__ bool find_tile(const Experts& x, int m, bool report, Tile* t) {
  const int lane = threadIdx.x & (kWave - 1);
  const int per = (x.E + kWave - 1) / kWave;  // experts of a lane
  const int e0 = min(lane * per, x.E), e1 = min(e0 + per, x.E);
  // of an expert's `cnt` rows: tiles of the first kind (up to 2^31 - 1 rows, so the sum is unsigned), and
  // whether its last tile is of the second
  const auto first_kind = [](int cnt) {
    return static_cast<int>((static_cast<uint32_t>(cnt) + (LARGE_FIRST ? TR / 2 : TR) - 1) / TR);
  };
  const auto second_kind = [](int cnt) { return LARGE_FIRST && cnt % TR > 0 && cnt % TR <= TR / 2 ? 1 : 0; };
  int n = 0, n2 = 0, cnt = 0, lo = 0, slot = 0;
  for (int e = e0; e < e1; ++e) {
    cnt = expert_rows(x, e, &lo);
    slot = x.slot_of[e];  // unconditional: it is on its way together with the offsets
    if (slot >= 0 && slot < x.n_slots) {
      n += first_kind(cnt);
      n2 += second_kind(cnt);
    } else if (report && cnt > 0) {
      status_or(x.status, MOE_STATUS_EXPERT_ABSENT);
    }
  }
  int end = wave_scan(n);  // tiles up to and with this lane's experts
  bool second = false;
  if constexpr (LARGE_FIRST) {
    const int all = __builtin_amdgcn_readlane(end, kWave - 1);
    second = m >= all;
    if (second) {
      m -= all;
      n = n2;
      end = wave_scan(n);
    }
  }
  const uint64_t mine = __ballot(m >= end - n && m < end);
  if (mine == 0) return false;
  int left = m - (end - n);  // of this lane's tiles
  int row0 = lo, rows = cnt;
  const auto cut = [&](int i) {
    row0 = lo + i * TR;
    rows = min(TR, cnt - i * TR);
  };
  if (per == 1) {
    cut(second ? cnt / TR : left);
  } else {
    for (int e = e0; e < e1; ++e) {
      cnt = expert_rows(x, e, &lo);
      const int s = x.slot_of[e];
      if (s < 0 || s >= x.n_slots) continue;
      const int tiles = second ? second_kind(cnt) : first_kind(cnt);
      if (left >= 0 && left < tiles) {
        cut(second ? cnt / TR : left);
        slot = s;
      }
      left -= tiles;
    }
  }
  const int owner = __builtin_ctzll(mine);
  t->row0 = __builtin_amdgcn_readlane(row0, owner);
  t->rows = __builtin_amdgcn_readlane(rows, owner);
  t->slot = __builtin_amdgcn_readlane(slot, owner);
  return true;
}

// ---------------------------------------------------------------------------
// f32
// ---------------------------------------------------------------------------

// Tiles of TR x TR, four waves:
//   64  a wave a 32 x 32 block, stages of 32 of depth
//   32  every wave the whole tile and a quarter of each stage's depth (64); the four sums are
//       added in LDS in wave order.  For products too small to fill the CUs with large tiles: four
//       times as many blocks, each with half as many stages of half as many MFMAs a wave.
// The loads of a stage are issued two stages ahead, LDS is double-buffered and an even and an odd
// accumulator keep two MFMAs independent.  Measured: 8192 rows of 8 experts of 1023 x 1001 1.29 ms
// (104 of the fp32 MFMA's 140 TFLOP/s that a large library product reaches), 1024 rows of 8
// experts of 256 x 512 51 us, one token x 3 of 280 x 273 19 us (launches and depth loops).
template <int TR>
struct TileF32 {
  static constexpr int K = TR == 64 ? 32 : 64;   // depth of a stage
  static constexpr int N = TR * K / 256;         // elements of an operand's stage per thread
  static constexpr int LD = TR + 1;              // LDS row (one k): writes along k spread over the banks
  static constexpr int STAGE = K * LD;           // floats of one operand's stage
  static constexpr int LDS = 4 * STAGE;          // two stages of two operands
  static constexpr int NQ = TR == 64 ? 16 : 4;   // elements of C per lane
  // row and column within the tile of this lane's element q
  static __device__ __forceinline__ int row(int q) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    return TR == 64 ? (wave >> 1) * 32 + (q >> 2) * 8 + (lane >> 5) * 4 + (q & 3)
                    : wave * 8 + (lane >> 5) * 4 + q;
  }
  static __device__ __forceinline__ int block_col() { return TR == 64 ? threadIdx.x / kWave & 1 : 0; }
  static __device__ __forceinline__ int col() { return block_col() * 32 + (threadIdx.x & 31); }
};

// How the stages of an operand are loaded: TR "outer" indices by K of depth, each load of a wave one
// or two runs that lie together in memory.  A lane outside the operand has an offset past the
// buffer's range, for which the hardware returns zero: no load is behind a branch, so none has to
// arrive before the branch ends.  KMAJOR: element (o, k) is at p[k * ld + o], else at p[o * ld + k].
template <int TR, bool KMAJOR>
struct OperandF32 {
  using T = TileF32<TR>;
  static constexpr int STEP = 256 / (KMAJOR ? TR : T::K);  // k's (outer indices) from element to element
  uint64_t base;        // wave-uniform: where the stage to load next starts
  uint32_t step;        // bytes from a stage to the next
  int left;             // steps of depth from there on
  int k;                // depth of this thread's element 0 within a stage
  uint32_t voff[T::N];  // kOutside for what does not exist

  // at(o) maps a tile's outer index to the operand's, or to -1
  template <typename At>
  __device__ __forceinline__ void init(const float* p, int64_t ld, int depth, At at) {
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    base = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u))) |
           static_cast<uint64_t>(static_cast<uint32_t>(
               __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u >> 32)))) << 32;
    step = static_cast<uint32_t>(T::K * (KMAJOR ? ld : 1) * 4);
    left = depth;
    k = KMAJOR ? threadIdx.x / TR : threadIdx.x % T::K;
#pragma unroll
    for (int i = 0; i < T::N; ++i) {
      const int src = at(outer(i));
      voff[i] = src < 0 ? kOutside
                        : static_cast<uint32_t>(KMAJOR ? (k + STEP * i) * ld + src : src * ld + k) * 4u;
    }
  }
  __device__ __forceinline__ int outer(int i) const {
    return KMAJOR ? threadIdx.x % TR : threadIdx.x / T::K + STEP * i;
  }
  // Element I of the next stage (the depth past the operand reads zeros: no branch, which would end
  // the compiler's block).
  template <int I>
  __device__ __forceinline__ void load(float (&v)[T::N]) const {
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(base), 0, kOutside, 0x00020000);
    const uint32_t at = k + (KMAJOR ? STEP * I : 0) < left ? voff[I] : kOutside;
    v[I] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0));
  }
  __device__ __forceinline__ void next_stage() {
    base += step;
    left -= T::K;
  }
  // Element I to LDS as [depth][outer].
  template <int I>
  __device__ __forceinline__ void store(const float (&v)[T::N], float* lds) const {
    lds[(k + (KMAJOR ? STEP * I : 0)) * T::LD + outer(I)] = v[I];
  }
};

// This lane's elements of the tile of A B over depth [0, K).  lds: TileF32<TR>::LDS floats.
template <int TR, bool A_KMAJOR, bool B_KMAJOR, typename AtA, typename AtB>
__device__ __forceinline__ void tile_product_f32(const float* __restrict__ A, int64_t lda, AtA at_a,
                                                 const float* __restrict__ B, int64_t ldb, AtB at_b, int K,
                                                 float* lds, float (&c)[TileF32<TR>::NQ]) {
  using T = TileF32<TR>;
  constexpr int KW = TR == 64 ? T::K : T::K / 4;  // a wave's depth of a stage
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int k_lane = (lane >> 5) + (TR == 64 ? 0 : wave * KW);
  const int ra = k_lane * T::LD + (TR == 64 ? (wave >> 1) * 32 : 0) + (lane & 31);
  const int rb = k_lane * T::LD + T::col() + T::STAGE;
  floatx16 even, odd;
#pragma unroll
  for (int q = 0; q < 16; ++q) even[q] = odd[q] = 0.f;
  OperandF32<TR, A_KMAJOR> oa;
  OperandF32<TR, B_KMAJOR> ob;
  oa.init(A, lda, K, at_a);
  ob.init(B, ldb, K, at_b);
  float va[2][T::N], vb[2][T::N];
  constexpr int NM = KW / 2, NP = NM / 4;  // MFMAs of a stage; fragments read a stage early
  float fa[2][NM], fb[2][NM];
  auto read = [&](auto i, auto t, const float* from) {
    constexpr int I = decltype(i)::value, P = decltype(t)::value;
    fa[I][P] = from[2 * P * T::LD + ra];
    fb[I][P] = from[2 * P * T::LD + rb];
  };
  // A stage of parity I whose first fragments are read.  A wave is often alone on its SIMD, so every
  // other instruction goes beside an MFMA: first this stage's other fragments and the loads of the
  // stage two ahead (into the registers the last stage emptied), then the next stage's elements to
  // LDS, and past the barrier, which the reads of this buffer precede, its first fragments.
  auto stage = [&](auto ic) {
    constexpr int I = decltype(ic)::value;
    const float* cur = lds + I * 2 * T::STAGE;
    float* next = lds + (1 - I) * 2 * T::STAGE;
    each<0, NM>([&](auto tc) {
      constexpr int t = decltype(tc)::value;
      if constexpr (t == NM - NP) __syncthreads();
      floatx16& acc = t % 2 ? odd : even;
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(fa[I][t], fb[I][t], acc, 0, 0, 0);
      each<0, NM>([&](auto f) {
        constexpr int F = decltype(f)::value;
        if constexpr (F >= NP && (F - NP) * (NM / 2) / (NM - NP) == t) read(ic, f, cur);
        if constexpr (F < NP && t == NM - NP + F) read(std::integral_constant<int, 1 - I>{}, f, next);
      });
      each<0, T::N>([&](auto e) {
        constexpr int X = decltype(e)::value;
        if constexpr (X * (NM / 2) / T::N == t) {
          oa.template load<X>(va[I]);
          ob.template load<X>(vb[I]);
        }
        if constexpr (NM / 4 + X * (NM / 2) / T::N == t) {
          oa.template store<X>(va[1 - I], next);
          ob.template store<X>(vb[1 - I], next + T::STAGE);
        }
      });
      __builtin_amdgcn_sched_barrier(0);
    });
    oa.next_stage();
    ob.next_stage();
  };
  each<0, 2>([&](auto i) {
    each<0, T::N>([&](auto e) {
      oa.template load<decltype(e)::value>(va[decltype(i)::value]);
      ob.template load<decltype(e)::value>(vb[decltype(i)::value]);
    });
    oa.next_stage();
    ob.next_stage();
  });
  each<0, T::N>([&](auto e) {
    oa.template store<decltype(e)::value>(va[0], lds);
    ob.template store<decltype(e)::value>(vb[0], lds + T::STAGE);
  });
  __syncthreads();
  each<0, NP>([&](auto t) { read(std::integral_constant<int, 0>{}, t, lds); });
  int stages = static_cast<int>((static_cast<uint32_t>(K) + T::K - 1) / T::K);
  for (; stages >= 2; stages -= 2) each<0, 2>(stage);
  if (stages > 0) stage(std::integral_constant<int, 0>{});
  const floatx16 sum = even + odd;
  if constexpr (TR == 64) {
#pragma unroll
    for (int q = 0; q < 16; ++q) c[q] = sum[q];
  } else {
    __syncthreads();  // the stages' reads are done
#pragma unroll
    for (int q = 0; q < 16; ++q) lds[(wave * 16 + q) * kWave + lane] = sum[q];
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float* p = lds + (wave * 4 + q) * kWave + lane;
      c[q] = p[0] + p[16 * kWave] + p[32 * kWave] + p[48 * kWave];
    }
  }
}

// Where the rows of a product's first operand are: row r itself, or, gathered, src_of[r] / k of `rows`
// rows (one outside them reads as zeros).
struct Source {
  const int32_t* src_of;  // nullptr: not gathered
  int k, rows;
  __device__ __forceinline__ int at(int r) const {
    const int a = src_of[r], row = a / k;
    return a >= 0 && row < rows ? row : -1;
  }
};

// C[r][n] = sum_k A[r][k] B[k][n], or with B_ROWS sum_k A[r][k] B[n][k], for tile m's rows and columns
// n0 .. n0 + TR - 1; B of the tile's expert starts at b_off of its block.
template <int TR, bool B_ROWS = false>
__device__ __forceinline__ void rows_product_f32(const Experts& x, int m, int n0, bool report,
                                                 const float* A, int64_t lda, const char* wbase,
                                                 int64_t expert_bytes, int64_t b_off, int N, int K,
                                                 float* C, float* lds, Source src = {}) {
  Tile t;
  if (!find_tile<TR>(x, m, report, &t)) return;
  using S = TileF32<TR>;
  const float* B = reinterpret_cast<const float*>(wbase + t.slot * expert_bytes + b_off);
  float acc[S::NQ];
  const bool gather = src.src_of;
  tile_product_f32<TR, false, !B_ROWS>(
      gather ? A : A + t.row0 * lda, lda,
      [&](int o) { return o >= t.rows ? -1 : gather ? src.at(t.row0 + o) : o; }, B, B_ROWS ? K : N,
      [&](int o) { return n0 + o < N ? n0 + o : -1; }, K, lds, acc);
  const int c = n0 + S::col();
  if (c >= N) return;
#pragma unroll
  for (int q = 0; q < S::NQ; ++q)
    if (S::row(q) < t.rows) C[static_cast<int64_t>(t.row0 + S::row(q)) * N + c] = acc[q];
}

// C[m][n] = sum over expert e's rows r of A[r][m] B[r][n], written at c_off of the expert's block of
// dw.  An expert without rows gets zeros, one outside the buffer nothing.
template <int TR>
__device__ __forceinline__ void weight_grad_f32(const Experts& x, int e, int m0, int n0, const float* A,
                                                int M, const float* B, int N, int64_t expert_bytes,
                                                int64_t c_off, char* dw, float* lds) {
  int lo;
  const int K = expert_rows(x, e, &lo), slot = x.slot_of[e];
  if (slot < 0 || slot >= x.n_slots) return;
  using S = TileF32<TR>;
  float acc[S::NQ];
  tile_product_f32<TR, true, true>(
      A + static_cast<int64_t>(lo) * M, M, [&](int o) { return m0 + o < M ? m0 + o : -1; },
      B + static_cast<int64_t>(lo) * N, N, [&](int o) { return n0 + o < N ? n0 + o : -1; }, K, lds, acc);
  float* C = reinterpret_cast<float*>(dw + slot * expert_bytes + c_off);
  const int c = n0 + S::col();
  if (c >= N) return;
#pragma unroll
  for (int q = 0; q < S::NQ; ++q)
    if (m0 + S::row(q) < M) C[static_cast<int64_t>(m0 + S::row(q)) * N + c] = acc[q];
}

// Small tiles for a product with fewer than two large ones a CU.  Measured, large against small: dH
// of 128 rows, depth 1024 (144 large tiles) 25 / 15 us; 1024 rows, depth 256 (192) 10.4 / 9.1; 2048
// rows, depth 512 (320) 24 / 21; 4096 rows, depth 512 (576) 33 / 34; 8192 rows, depth 1023 (2176)
// 175 / 227.
inline bool small_tiles_f32(int64_t large) { return large < 2 * kCus; }

// ---------------------------------------------------------------------------
// bf16
// ---------------------------------------------------------------------------

// Work order: units of gm x gn output tiles, unit u on XCD u % 8 (workgroup i runs on XCD i % 8),
// so the workgroups that run together on an XCD share gm row panels and gn column panels in its L2.
struct Order {
  int gm, gn, n_gn;  // tiles of a unit; units across
};

__device__ __forceinline__ void place(const Order& o, int block, int* m, int* n) {
  const int xcd = block % 8, local = block / 8;
  const int per = o.gm * o.gn;
  const int unit = local / per * 8 + xcd, at = local % per;
  *m = unit / o.n_gn * o.gm + at % o.gm;
  *n = unit % o.n_gn * o.gn + at / o.gm;
}

// Calls f with the smallest tile mode that holds `rows` rows.
template <int TR, typename F>
__device__ __forceinline__ void by_rows(int rows, F f) {
  if constexpr (TR == 256) {
    if (rows > 192) f(std::integral_constant<int, 0>{});
    else if (rows > 128) f(std::integral_constant<int, 6>{});
    else if (rows > 64) f(std::integral_constant<int, 4>{});
    else if (rows > 32) f(std::integral_constant<int, 2>{});
    else f(std::integral_constant<int, 1>{});
  } else {
    f(std::integral_constant<int, 0>{});
  }
}

// A tile's accumulators to C (its first row and column), of which rows x cols exist.
template <int TR, int MI>
__device__ __forceinline__ void store_tile(
    const floatx16 (&acc)[TileShape<TR, MI, false>::MW][TileShape<TR, MI, false>::NJ], lds_char* smem,
    uint16_t* C, int64_t ld, int rows, int cols) {
  using S = TileShape<TR, MI, false>;
#pragma unroll
  for (int i = 0; i < S::MW; ++i) {
    const int r0 = S::first_row() + i * 32, c0 = S::first_col();
    store_block<S::NJ * 32>(smem, C + r0 * ld + c0, ld, rows - r0, cols - c0, [&](int j, int v) {
      return pack4(acc[i][j][v * 4], acc[i][j][v * 4 + 1], acc[i][j][v * 4 + 2], acc[i][j][v * 4 + 3]);
    });
  }
}

template <int TR, int MI>
__device__ __forceinline__ void store_tile(
    const floatx16 (&acc)[TileShape<TR, MI, false>::MW][TileShape<TR, MI, false>::NJ], lds_char*, float* C,
    int64_t ld, int rows, int cols) {
  using S = TileShape<TR, MI, false>;
#pragma unroll
  for (int i = 0; i < S::MW; ++i) {
    const int r = lane_row<TR, MI, false>(i);
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

// C[r][n] = sum_k A[r][k] B[k][n] for the rows of a tile and columns n0 .. n0 + TN - 1.
template <int TR, int MI, typename O>
__device__ __forceinline__ void rows_tile(const Tile& t, int n0, const uint16_t* A, int lda,
                                          const uint16_t* B, int N, int K, O* C, lds_char* smem) {
  using S = TileShape<TR, MI, false>;
  Operand<false, S::ROWS> oa;
  Operand<true, S::TN> ob;
  oa.init(A + static_cast<int64_t>(t.row0) * lda, lda, K, [&](int r) { return r < t.rows ? r : -1; });
  ob.init(B + n0, N, K, [&](int c) { return n0 + c < N ? c : -1; });
  floatx16 acc[S::MW][S::NJ];
  tile_product<TR, MI, false, false, true>(oa, ob, K, smem, acc);
  store_tile<TR, MI>(acc, smem, C + static_cast<int64_t>(t.row0) * N + n0, N, t.rows, N - n0);
}

// The same for tile (m, n) of the list; B of the tile's expert starts at b_off of its block.
template <int TR, bool LARGE_FIRST = false, typename O>
__device__ __forceinline__ void rows_product(const Experts& x, int m, int n, bool report,
                                             const uint16_t* A, int lda, const char* wbase,
                                             int64_t expert_bytes, int64_t b_off, int N, int K, O* C,
                                             lds_char* smem) {
  const int n0 = n * tile_columns(TR, false);
  Tile t;
  if (n0 >= N || !find_tile<TR, LARGE_FIRST>(x, m, report, &t)) return;
  const uint16_t* B = reinterpret_cast<const uint16_t*>(wbase + t.slot * expert_bytes + b_off);
  by_rows<TR>(t.rows, [&](auto mi) {
    rows_tile<TR, decltype(mi)::value>(t, n0, A, lda, B, N, K, C, smem);
  });
}

#define TILE_KERNEL \
  __global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(TR == 256 ? 1 : 2, TR == 256 ? 1 : 2))) void

// C[m][n] = sum over expert e's rows r of A[r][m] B[r][n], written at c_off of the expert's block of
// dw.  An expert without rows gets zeros, one outside the buffer nothing.
template <int TR>
__device__ __forceinline__ void weight_grad(const Experts& x, int e, int m, int n, const uint16_t* A, int M,
                                            const uint16_t* B, int N, int64_t expert_bytes,
                                            int64_t c_off, char* dw, lds_char* smem) {
  using S = TileShape<TR, 0, false>;
  const int m0 = m * TR, n0 = n * S::TN;
  if (m0 >= M || n0 >= N) return;
  int lo;
  const int K = __builtin_amdgcn_readfirstlane(expert_rows(x, e, &lo));
  const int slot = __builtin_amdgcn_readfirstlane(x.slot_of[e]);
  lo = __builtin_amdgcn_readfirstlane(lo);
  if (slot < 0 || slot >= x.n_slots) return;
  Operand<true, TR> oa;
  Operand<true, S::TN> ob;
  oa.init(A + static_cast<int64_t>(lo) * M + m0, M, K, [&](int c) { return m0 + c < M ? c : -1; });
  ob.init(B + static_cast<int64_t>(lo) * N + n0, N, K, [&](int c) { return n0 + c < N ? c : -1; });
  floatx16 acc[S::MW][S::NJ];
  tile_product<TR, 0, false, true, true>(oa, ob, K, smem, acc);
  uint16_t* C = reinterpret_cast<uint16_t*>(dw + slot * expert_bytes + c_off);
  store_tile<TR, 0>(acc, smem, C + static_cast<int64_t>(m0) * N + n0, N, M - m0, N - n0);
}

// blocks: a multiple of 8.
inline Order make_order(int tr, int64_t mt, int64_t nt, int64_t* blocks) {
  // large tiles: up to 4 x 8 (32 CUs an XCD), the columns cut evenly, where that leaves every XCD a
  // few units, else single tiles
  Order o{4, static_cast<int>(ceil_div64(nt, ceil_div64(nt, 8))), 0};
  if (tr != 256 || ceil_div64(mt, o.gm) * ceil_div64(nt, o.gn) < 32) o.gm = o.gn = 1;
  o.n_gn = static_cast<int>(ceil_div64(nt, o.gn));
  const int64_t units = ceil_div64(mt, o.gm) * o.n_gn;
  *blocks = ceil_div64(units, 8) * 8 * o.gm * o.gn;
  return o;
}

// Enqueue a tile kernel: its LDS is above the default limit of a launch.
template <typename K, typename... A>
int launch_tiles(const char* what, K kernel, int64_t blocks, int lds, hipStream_t s, A... args) {
  MOE_HIP_CHECK(hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                    hipFuncAttributeMaxDynamicSharedMemorySize, lds));
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), lds, s, args...);
  MOE_LAUNCH_CHECK(what);
  return MOE_OK;
}

}  // namespace moe
