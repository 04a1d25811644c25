// kernels_f8block.hip -- fp8 GEMM with block scales, dense and per group:
//   Y[m][n] = sum_b xs[m][b] ws[n / 128][b] sum_{k in block b} X[m][k] W[n][k]
// over blocks b of 128 k.  The matrix instruction forms each block's inner
// sum in fp32 (v_mfma_scale_f32_16x16x128_f8f6f4 with unit scales spans
// exactly one block), and one fp32 multiply-add per result folds it into the
// accumulator with the product of the two scales.  The result is rounded once,
// to bf16.
#include <algorithm>

#include "gmi_device.hpp"
#include "gmi_internal.hpp"

namespace gmi {

// 16 x 16 x 128: operand lane l holds 32 bytes of row l % 16, k-group l / 16;
// result lane l, element j is D[4 (l / 16) + j][l % 16].  Which 32 of the 128
// k a group holds is free as long as both operands agree.
__device__ __forceinline__ f32x4 mfma16_f8(u32x8 a, u32x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_bit_cast(i32x8, a), __builtin_bit_cast(i32x8, b),
                                                          c, 0, 0, 0, 127, 0, 127);
}
__device__ __forceinline__ u32x8 join(u32x4 lo, u32x4 hi) {
  return u32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}
__device__ __forceinline__ float buf_loadf(rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0));
}

constexpr int SK_WAVES = 8, SK_N = 32;

// Up to 16 TM rows by SK_N columns: the waves take the k-blocks in turn,
// loading both operands from memory straight into registers (a weight is read
// once), and add their sums through LDS in wave order.
template <int TM>
__device__ __forceinline__ void skinny_tile(const F8BlockLaunch& a, int64_t row0, int rows, const uint8_t* W,
                                            const float* ws, int n0, f32x4 (*red)[4][SK_N / 16][64]) {
  constexpr int NB = SK_N / 16;
  const int lane = threadIdx.x & 63, wave = wave_id(), r = lane & 15, h = lane >> 4;
  const int kb_n = (a.K + 127) / 128;
  const int ncols = min(SK_N, a.N - n0);
  const rsrc_t rx = make_rsrc(a.X + row0 * a.ldx, (uint32_t)((int64_t)(rows - 1) * a.ldx + a.K));
  const rsrc_t rw = make_rsrc(W + (int64_t)n0 * a.ldw, (uint32_t)((int64_t)(ncols - 1) * a.ldw + a.K));
  const rsrc_t rs = make_rsrc(a.xs + row0 * a.ldxs, (uint32_t)((int64_t)(rows - 1) * a.ldxs + kb_n) * 4u);
  const float* wsr = ws + (int64_t)(n0 / 128) * a.ldws;
  f32x4 acc[TM][NB];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{};
  for (int kb = wave; kb < kb_n; kb += SK_WAVES) {
    // chunks h and h + 4 of the block's eight; those past K read as zeros
    const uint32_t k0 = kb * 128 + h * 16, k1 = k0 + 64;
    const bool in0 = (int)k0 < a.K, in1 = (int)k1 < a.K;
    u32x8 w[NB], x[TM];
    float s[TM];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const bool ok = 16 * j + r < ncols;
      const uint32_t o = (uint32_t)(16 * j + r) * (uint32_t)a.ldw;
      w[j] = join(buf_load16(rw, ok && in0 ? o + k0 : OOB), buf_load16(rw, ok && in1 ? o + k1 : OOB));
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const bool ok = 16 * i + r < rows;
      const uint32_t o = (uint32_t)(16 * i + r) * (uint32_t)a.ldx;
      x[i] = join(buf_load16(rx, ok && in0 ? o + k0 : OOB), buf_load16(rx, ok && in1 ? o + k1 : OOB));
      s[i] = buf_loadf(rs, ok ? ((uint32_t)(16 * i + r) * (uint32_t)a.ldxs + kb) * 4u : OOB) * wsr[kb];
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const f32x4 p = mfma16_f8(w[j], x[i], f32x4{});
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(s[i], p[e], acc[i][j][e]);
      }
  }
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) red[wave][i][j][lane] = acc[i][j];
  __syncthreads();
  // item: 4 consecutive columns of one row
  for (int it = threadIdx.x; it < TM * NB * 64; it += SK_WAVES * 64) {
    const int l = it & 63, j = it / 64 % NB, i = it / (64 * NB);
    f32x4 v{};
#pragma unroll
    for (int w = 0; w < SK_WAVES; ++w) v += red[w][i][j][l];
    const int m = 16 * i + (l & 15), n = n0 + 16 * j + 4 * (l >> 4);
    if (m >= rows || n >= a.N) continue;
    uint16_t* y = a.Y + (row0 + m) * a.ldy + n;
    if (n + 4 <= a.N) {
      *(u32x2*)y = u32x2{pack2<DT_BF16>(v[0], v[1]), pack2<DT_BF16>(v[2], v[3])};
    } else {
      for (int e = 0; e < a.N - n; ++e) y[e] = (uint16_t)to_bits<DT_BF16>(v[e]);
    }
  }
  __syncthreads();
}

// grid.x: column blocks; grid.y: groups (one without offsets); groups of more
// than max_rows rows are another kernel's
__global__ __launch_bounds__(SK_WAVES * 64) void k_f8_skinny(F8BlockLaunch a, int max_rows) {
  __shared__ f32x4 red[SK_WAVES][4][SK_N / 16][64];
  const int n0 = blockIdx.x * SK_N;
  int64_t lo, hi;
  const uint8_t* W = a.W;
  const float* ws = a.ws;
  if (a.offsets) {
    const int g = blockIdx.y;
    lo = min(max(a.offsets[g], 0), a.M);
    hi = min(max(a.offsets[g + 1], 0), a.M);
    W += (int64_t)g * a.w_stride;
    ws += (int64_t)g * a.ws_stride;
  } else {
    lo = 0;
    hi = a.M;
  }
  if (hi - lo > max_rows) return;
  for (int64_t m0 = lo; m0 < hi; m0 += 64) {
    const int rows = (int)min((int64_t)64, hi - m0);
    if (rows <= 16)
      skinny_tile<1>(a, m0, rows, W, ws, n0, red);
    else if (rows <= 32)
      skinny_tile<2>(a, m0, rows, W, ws, n0, red);
    else
      skinny_tile<4>(a, m0, rows, W, ws, n0, red);
  }
}

// ---------------------------------------------------------------------------
// Tiled kernel: BM x BN output tiles, WM x WN waves, k-tiles of 128 (one scale
// block).  Operand k-tiles stream from memory straight into LDS: three slots
// for X, two for W, so that while k-tile kt is multiplied, W of kt + 1 and X
// of kt + 2 are on their way.  A wave multiplies MI x NJ blocks of 16 x 16;
// each matrix instruction starts from zero and spans a whole scale block, and
// its four results per lane are folded with one multiply-add each, a few
// instructions later, while the next ones run.
//
// The instruction's first operand is W, so a lane's results are four
// consecutive columns of one row of Y, and one lane value per 16 rows holds
// the scale.  W rows are dealt to the blocks so that blocks 2p and 2p + 1 of
// lane group h hold columns 32 p + 8 h .. + 7: eight consecutive columns, one
// 16-byte store.
//
// LDS rows are 128 bytes, two to a 256-byte bank line; chunk c of row r sits
// in slot c ^ swizzle(r), so that the 16 rows of a fragment read hit all
// banks: rows r .. r + 15 of X vary bits 0-3, the dealt rows of W bits 0, 1, 3
// and 4.
// ---------------------------------------------------------------------------
template <int BM_, int BN_, int WM_, int WN_>
struct F8Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NW = WM * WN, THREADS = 64 * NW;
  static constexpr int WTM = BM / WM, WTN = BN / WN, MI = WTM / 16, NJ = WTN / 16;
  static constexpr int SA = 3, SB = 2;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, LDS = SA * A_BYTES + SB * B_BYTES;
  static constexpr int PA = BM / (8 * NW), PB = BN / (8 * NW);  // 1 KB copies (8 rows) per wave
  static constexpr int WGS_PER_CU = 160 * 1024 / LDS >= 2 ? 2 : 1;
  static_assert(WTM <= 64 && WTN <= 128 && NJ % 2 == 0 && NW % 4 == 0 && PA >= 1 && PB >= 1, "tile");
  static_assert(LDS <= 160 * 1024, "LDS budget");
};
__device__ __forceinline__ int swz_x(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int swz_w(int row) { return ((row >> 1) & 1) | ((row >> 2) & 6); }

// One operand's copies: rows row0 .. of a [rows][ld] byte matrix; copy i of
// wave w fills tile rows 8 (NW i + w) + lane / 8.  Rows past the end and
// chunks at or past K (every chunk, past the last k-tile) land as zeros.
template <int P, int NW, bool IS_W>
struct F8Loader {
  rsrc_t rs;
  uint32_t voff[P];
  int kc;  // first k of this lane's chunk in k-tile 0
  int K;
  __device__ __forceinline__ void init(const uint8_t* base, int64_t ld, int64_t row0, int rows, int K_) {
    const int left = rows < 8 * NW * P ? rows : 8 * NW * P;
    rs = make_rsrc(base + row0 * ld, (uint32_t)((int64_t)(left - 1) * ld + K_));
    const int lane = threadIdx.x & 63, row = 8 * wave_id() + (lane >> 3);
    const int chunk = (lane & 7) ^ (IS_W ? swz_w(row) : swz_x(row));
    kc = chunk * 16;
    K = K_;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int r = row + 8 * NW * i;
      voff[i] = r < left ? (uint32_t)r * (uint32_t)ld + (uint32_t)kc : OOB;
    }
  }
  __device__ __forceinline__ void issue(int i, int kt, char* tile) const {
    const uint32_t o = kt * 128 + kc < K ? voff[i] : OOB;
    dma16s(rs, o, (uint32_t)kt * 128u, tile + (NW * i + wave_id()) * 1024);
  }
};

// barrier that no LDS access moves across in the compiler
__device__ __forceinline__ void publish() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <class T>
__device__ __forceinline__ void f8_tile(char* lds, const F8BlockLaunch& a, int64_t row0, int rows, const uint8_t* W,
                                        const float* ws, int n0) {
  constexpr int MI = T::MI, NJ = T::NJ, NP = 4;
  char* const la = lds;
  char* const lb = lds + T::SA * T::A_BYTES;
  const int lane = threadIdx.x & 63, wave = wave_id(), r = lane & 15, h = lane >> 4;
  const int wm = wave / T::WN * T::WTM, wn = wave % T::WN * T::WTN;
  const int nk = (a.K + 127) / 128, cols = a.N - n0;
  F8Loader<T::PA, T::NW, false> al;
  F8Loader<T::PB, T::NW, true> bl;
  al.init(a.X, a.ldx, row0, rows, a.K);
  bl.init(W, a.ldw, n0, cols, a.K);
  const rsrc_t rxs = make_rsrc(a.xs + row0 * a.ldxs, (uint32_t)((int64_t)(rows < T::BM ? rows - 1 : T::BM - 1) * a.ldxs + nk) * 4u);
  // the wave's columns lie in one block of 128 weight rows (past N: no scale)
  const bool has_cols = n0 + wn < a.N;
  const rsrc_t rws = make_rsrc(ws + (has_cols ? (int64_t)((n0 + wn) / 128) * a.ldws : 0), has_cols ? (uint32_t)nk * 4u : 0u);
  const int srow = wm + lane % T::WTM;
  const uint32_t xo = srow < rows ? (uint32_t)srow * (uint32_t)a.ldxs * 4u : OOB;
  auto scale_x = [&](int kt) {
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rxs, (int)(kt < nk ? xo : OOB), kt * 4, 0));
  };
  auto scale_w = [&](int kt) {
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rws, (int)(kt < nk ? 0u : OOB), kt * 4, 0));
  };
  const bool busy = wm < rows;  // waves below the last row only copy

  // lane offsets of the fragments: chunks 2 h and 2 h + 1 of the row
  const int ra = wm + r, rb = wn + 8 * (r >> 2) + (r & 3);
  const uint32_t a0 = ra * 128 + (((2 * h) ^ swz_x(ra)) << 4), a1 = ra * 128 + (((2 * h + 1) ^ swz_x(ra)) << 4);
  const uint32_t b0 = rb * 128 + (((2 * h) ^ swz_w(rb)) << 4), b1 = rb * 128 + (((2 * h + 1) ^ swz_w(rb)) << 4);

  f32x4 acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{};

  float sx = scale_x(0), sw = scale_w(0);
#pragma unroll
  for (int i = 0; i < T::PA; ++i) al.issue(i, 0, la);
#pragma unroll
  for (int i = 0; i < T::PB; ++i) bl.issue(i, 0, lb);
#pragma unroll
  for (int i = 0; i < T::PA; ++i) al.issue(i, 1, la + T::A_BYTES);
  wait_vm_le<T::PA>();
  publish();
  int sa = 0, sb = 0;
  for (int kt = 0; kt < nk; ++kt) {
    const char* pa = la + sa * T::A_BYTES;
    const char* pb = lb + sb * T::B_BYTES;
    char* na = la + (sa == 0 ? 2 : sa - 1) * T::A_BYTES;  // slot of k-tile kt + 2
    char* nb = lb + (sb ^ 1) * T::B_BYTES;
    const float s = sx * sw;
    sx = scale_x(kt + 1);
    sw = scale_w(kt + 1);
    if (busy) {
      u32x8 fa[MI], fb[2];
      float sc[MI];
      fb[0] = join(*(const u32x4*)(pb + b0), *(const u32x4*)(pb + b1));
#pragma unroll
      for (int i = 0; i < MI; ++i)
        fa[i] = join(*(const u32x4*)(pa + a0 + i * 2048), *(const u32x4*)(pa + a1 + i * 2048));
#pragma unroll
      for (int i = 0; i < MI; ++i) sc[i] = __shfl(s, (16 * i + r) % T::WTM);
      f32x4 part[NP];
      constexpr int STEPS = MI * NJ, C = T::PA + T::PB;
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int t = 0; t < STEPS + NP - 1; ++t) {
        if (t < STEPS) {
          const int j = t / MI, i = t % MI;
          part[t % NP] = mfma16_f8(fb[j & 1], fa[i], f32x4{});
          if (i == 0 && j + 1 < NJ) {
            const int o = (32 * ((j + 1) / 2) + 4 * ((j + 1) & 1)) * 128;
            fb[(j + 1) & 1] = join(*(const u32x4*)(pb + b0 + o), *(const u32x4*)(pb + b1 + o));
          }
          // the copies, spread over the first half of the steps, W's first
#pragma unroll
          for (int c = t * C * 2 / STEPS; c < (t + 1) * C * 2 / STEPS; ++c) {
            if (c < T::PB) bl.issue(c, kt + 1, nb);
            else if (c < C) al.issue(c - T::PB, kt + 2, na);
          }
        }
        if (t >= NP - 1) {
          const int u = t - (NP - 1), j = u / MI, i = u % MI;
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(sc[i], part[u % NP][e], acc[i][j][e]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < T::PB; ++i) bl.issue(i, kt + 1, nb);
#pragma unroll
      for (int i = 0; i < T::PA; ++i) al.issue(i, kt + 2, na);
    }
    // W of kt + 1 (and X of kt + 1, issued before) has landed; X of kt + 2 may be in flight
    wait_vm_le<T::PA>();
    publish();
    sa = sa == 2 ? 0 : sa + 1;
    sb ^= 1;
  }
  wait_vm_le<0>();  // nothing lands in LDS after the tile

  if (!busy) return;
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int rr = tid & 15, hh = (tid & 63) >> 4;
  const int left = rows < T::BM ? rows : T::BM;
  const rsrc_t ry = make_rsrc(a.Y + row0 * a.ldy + n0, (uint32_t)((int64_t)(left - 1) * a.ldy + cols) * 2u);
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int m = wm + 16 * i + rr;
    const uint32_t ro = m < left ? (uint32_t)m * (uint32_t)a.ldy * 2u : OOB;
#pragma unroll
    for (int p = 0; p < NJ / 2; ++p) {
      const int n = wn + 32 * p + 8 * hh;
      const f32x4 v0 = acc[i][2 * p], v1 = acc[i][2 * p + 1];
      if (n + 8 <= cols) {
        buf_store16_wb(ry, ro + (uint32_t)n * 2u,
                       u32x4{pack2<DT_BF16>(v0[0], v0[1]), pack2<DT_BF16>(v0[2], v0[3]), pack2<DT_BF16>(v1[0], v1[1]),
                             pack2<DT_BF16>(v1[2], v1[3])});
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (n + e < cols)
            buf_store2(ry, ro + (uint32_t)(n + e) * 2u, to_bits<DT_BF16>(e < 4 ? v0[e & 3] : v1[e & 3]));
      }
    }
  }
}

// Workgroup -> tile: each XCD takes a run of consecutive tiles, which share
// operand panels in its L2; inside a problem bands of m-tiles (raster).
__device__ __forceinline__ int xcd_tile(int b, int total) {
  const int per = (total + XCDS - 1) / XCDS;
  const int t = (b % XCDS) * per + b / XCDS;
  return b / XCDS < per && t < total ? t : -1;
}

template <class T>
__global__ __launch_bounds__(T::THREADS, T::WGS_PER_CU) void k_f8_tiled(F8BlockLaunch a) {
  __shared__ __attribute__((aligned(16))) char lds[T::LDS];
  const int tm = (a.M + T::BM - 1) / T::BM, tn = (a.N + T::BN - 1) / T::BN;
  const int tile = xcd_tile(blockIdx.x, tm * tn);
  if (tile < 0) return;
  int mi, ni;
  raster(tile, tm, tn, mi, ni);
  f8_tile<T>(lds, a, (int64_t)mi * T::BM, a.M - mi * T::BM, a.W, a.ws, ni * T::BN);
}

// Group table: groups with more than SK_ROWS rows, in decreasing order of the
// rows a tile uses (long tiles first), with the prefix sums of their tiles.
struct F8Group {
  int32_t lo, m, g, tile_start;
};
constexpr int SK_ROWS = 64;      // rows up to which a group runs through the skinny kernel
constexpr int SK_ONLY_ROWS = 256;  // row capacity up to which the grouped call uses it alone

__global__ __launch_bounds__(kMaxOffsetGroupCount) void k_f8_group_table(F8BlockLaunch a, int bm, int tn, int32_t* total,
                                                                        F8Group* table) {
  __shared__ int32_t key[kMaxOffsetGroupCount];
  __shared__ int32_t scan[2][kMaxOffsetGroupCount];
  const int g = threadIdx.x;
  int lo = 0, m = 0;
  if (g < a.count) {
    lo = min(max(a.offsets[g], 0), a.M);
    m = max(min(max(a.offsets[g + 1], 0), a.M) - lo, 0);
  }
  const bool big = m > SK_ROWS;
  const int work = big ? min(m, bm) : 0, tiles = big ? (m + bm - 1) / bm * tn : 0;
  key[g] = work;
  scan[0][g] = 0;
  __syncthreads();
  int rank = g;
  if (g < a.count) {
    rank = 0;
    for (int q = 0; q < a.count; ++q) rank += (key[q] > work) || (key[q] == work && q < g);
    scan[0][rank] = tiles;
  }
  __syncthreads();
  int cur = 0;
  for (int d = 1; d < kMaxOffsetGroupCount; d <<= 1) {
    scan[cur ^ 1][g] = scan[cur][g] + (g >= d ? scan[cur][g - d] : 0);
    cur ^= 1;
    __syncthreads();
  }
  if (g < a.count) table[rank] = F8Group{lo, m, g, scan[cur][rank] - tiles};
  if (g == 0) *total = scan[cur][a.count - 1];
}

template <class T>
__global__ __launch_bounds__(T::THREADS, T::WGS_PER_CU) void k_f8_tiled_grouped(F8BlockLaunch a, const int32_t* total,
                                                                              const F8Group* table) {
  __shared__ __attribute__((aligned(16))) char lds[T::LDS];
  const int tile = xcd_tile(blockIdx.x, *total);
  if (tile < 0) return;
  // the last group whose first tile is not past this one: groups without
  // tiles come last and start at the total
  int n = 0;
  const int lane = threadIdx.x & 63;
  for (int q = lane; q < a.count; q += 64) n += table[q].tile_start <= tile;
  for (int d = 1; d < 64; d <<= 1) n += __shfl_xor(n, d);
  const F8Group d = table[__builtin_amdgcn_readfirstlane(n) - 1];
  const int local = tile - d.tile_start, tm = (d.m + T::BM - 1) / T::BM, tn = (a.N + T::BN - 1) / T::BN;
  if (local >= tm * tn) return;  // offsets out of order: the sums may not fit
  int mi, ni;
  raster(local, tm, tn, mi, ni);
  f8_tile<T>(lds, a, (int64_t)d.lo + (int64_t)mi * T::BM, d.m - mi * T::BM, a.W + (int64_t)d.g * a.w_stride,
             a.ws + (int64_t)d.g * a.ws_stride, ni * T::BN);
}

using F8T256 = F8Tile<256, 256, 4, 2>;
using F8T128 = F8Tile<128, 128, 2, 2>;

static hipError_t launch_skinny(const F8BlockLaunch& a, int max_rows, hipStream_t stream) {
  const int nb = (a.N + SK_N - 1) / SK_N;
  const int gy = a.offsets ? a.count : 1;
  hipLaunchKernelGGL(k_f8_skinny, dim3(nb, gy), dim3(SK_WAVES * 64), 0, stream, a, max_rows);
  return hipGetLastError();
}

size_t f8_block_workspace(int, int, int) { return 0; }
size_t f8_block_grouped_workspace(int count) { return 16 + sizeof(F8Group) * (size_t)count; }

static int64_t tiles_of(const F8BlockLaunch& a, int bm, int bn) {
  return ((int64_t)a.M + bm - 1) / bm * (((int64_t)a.N + bn - 1) / bn);
}

hipError_t launch_f8_block(const F8BlockLaunch& a, void*, size_t, hipStream_t stream) {
  if (a.M <= SK_ROWS) return launch_skinny(a, a.M, stream);
  if (tiles_of(a, 256, 256) >= device_cu_count()) {
    const unsigned grid = (unsigned)((tiles_of(a, 256, 256) + XCDS - 1) / XCDS * XCDS);
    hipLaunchKernelGGL((k_f8_tiled<F8T256>), dim3(grid), dim3(F8T256::THREADS), 0, stream, a);
  } else {
    const unsigned grid = (unsigned)((tiles_of(a, 128, 128) + XCDS - 1) / XCDS * XCDS);
    hipLaunchKernelGGL((k_f8_tiled<F8T128>), dim3(grid), dim3(F8T128::THREADS), 0, stream, a);
  }
  return hipGetLastError();
}

hipError_t launch_f8_block_grouped(const F8BlockLaunch& a, void* workspace, hipStream_t stream) {
  if (a.M <= SK_ONLY_ROWS) return launch_skinny(a, a.M, stream);
  int32_t* total = (int32_t*)workspace;
  F8Group* table = (F8Group*)((char*)workspace + 16);
  using T = F8T256;
  const int tn = (a.N + T::BN - 1) / T::BN;
  hipLaunchKernelGGL(k_f8_group_table, dim3(1), dim3(kMaxOffsetGroupCount), 0, stream, a, T::BM, tn, total, table);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // the tile total is known on the device only: every group with its own
  // partial tile bounds it
  const int64_t most = ((int64_t)a.M / T::BM + std::min<int64_t>(a.count, a.M / (SK_ROWS + 1))) * tn;
  const unsigned grid = (unsigned)((most + XCDS - 1) / XCDS * XCDS);
  if (grid > 0) {
    hipLaunchKernelGGL((k_f8_tiled_grouped<T>), dim3(grid), dim3(T::THREADS), 0, stream, a, total, table);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return launch_skinny(a, SK_ROWS, stream);
}

}  // namespace gmi
