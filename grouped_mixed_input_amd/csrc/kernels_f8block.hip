// kernels_f8block.hip -- fp8 GEMM with block scales, dense and per group:
//   Y[m][n] = sum_b xs[m][b] ws[n / 128][b] sum_{k in block b} X[m][k] W[n][k]
// over blocks b of 128 k.  The matrix instruction forms each block's inner
// sum in fp32 (v_mfma_scale_f32_16x16x128_f8f6f4 with unit scales spans
// exactly one block), and one fp32 multiply-add per result folds it into the
// accumulator with the product of the two scales.  The result is rounded once,
// to bf16.  The instruction's own sums are coarser than fp32: it takes eight
// consecutive k at a time and truncates their products toward zero at 2^-13 of
// the largest (probed, and modelled to the bit by the tests; the 16x16x32 fp8
// form keeps as many).  That is less than 8.6e-4 of the sum of magnitudes
// whatever the operands and 2e-5 over 128 random terms, where bf16 rounds at
// 2^-8 of the result.  There is no finer fp8 form; converting to bf16 first
// would halve the matrix rate.
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
__device__ __forceinline__ float buf_loadfs(rsrc_t r, uint32_t off, uint32_t soff) {
  return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, (int)soff, 0));
}

constexpr int SK_WAVES = 8, SK_N = 32;

// One of several splits of K, as a problem of its own: `splits` runs of whole
// k-blocks of even length, the sums in fp32 to a.part + split * M * ldp.
__device__ __forceinline__ F8BlockLaunch k_split(F8BlockLaunch a, int split) {
  if (a.splits <= 1) return a;
  const int kb_n = (a.K + 127) / 128, b0 = (int)((int64_t)kb_n * split / a.splits),
            b1 = (int)((int64_t)kb_n * (split + 1) / a.splits);
  a.X += b0 * 128;
  a.W += b0 * 128;
  a.xs += b0;
  a.ws += b0;
  a.K = min(a.K, b1 * 128) - b0 * 128;
  a.part += (int64_t)split * a.M * a.ldp;
  return a;
}

// Up to 16 TM rows by SK_N columns: the waves take the k-blocks in turn and add
// their sums through LDS in wave order.  Weights, read once, go from memory to
// a ring of D slots of LDS that a wave keeps to itself (no barrier): a copy then
// moves whole 128-byte lines of 8 rows, where loads into the instruction's
// registers take each line in two halves.  X, in the L2 after the first
// workgroup's reads, goes straight to registers.  Past the last k-block the
// loads return zeros without memory traffic.  Bound by memory: 128 experts, 128
// rows 59 us (6.4 TB/s); 16 rows, 8192 x 8192 16.8 us (4.0, launch included), 12.4
// where the memory-side cache holds the weights.
// Two k-blocks per wave in flight; with three or four the loads only queue
// (experts 81-85 us).
template <int TM, int D, bool NT>
__device__ __forceinline__ void skinny_tile(const F8BlockLaunch& a, int64_t row0, int rows, const uint8_t* W,
                                            const float* ws, int n0, char* lds) {
  constexpr int NB = SK_N / 16;
  const int lane = threadIdx.x & 63, wave = wave_id(), r = lane & 15, h = lane >> 4;
  const int kb_n = (a.K + 127) / 128;
  const int ncols = min(SK_N, a.N - n0);
  const rsrc_t rx = make_rsrc(a.X + row0 * a.ldx, (uint32_t)((int64_t)(rows - 1) * a.ldx + a.K));
  const rsrc_t rw = make_rsrc(W + (int64_t)n0 * a.ldw, (uint32_t)((int64_t)(ncols - 1) * a.ldw + a.K));
  const rsrc_t rs = make_rsrc(a.xs + row0 * a.ldxs, (uint32_t)((int64_t)(rows - 1) * a.ldxs + kb_n) * 4u);
  const rsrc_t rws = make_rsrc(ws + (int64_t)(n0 / 128) * a.ldws, (uint32_t)kb_n * 4u);
  f32x4 acc[TM][NB];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{};
  // copy q: rows 8 q + lane / 8 of the weights; chunk c of row n lies in slot c ^ (n / 2 % 8)
  constexpr int WC = SK_N / 8;
  char* const ring = lds + wave * (D * SK_N * 128);
  uint32_t wo[WC], wc[WC], xo[TM], so[TM];
#pragma unroll
  for (int q = 0; q < WC; ++q) {
    const int n = 8 * q + (lane >> 3);
    wc[q] = ((lane & 7) ^ ((n >> 1) & 7)) * 16;
    wo[q] = n < ncols ? (uint32_t)n * (uint32_t)a.ldw + wc[q] : OOB;
  }
  uint32_t f0[NB], f1[NB];  // this lane's chunks h and h + 4 of its rows
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int n = 16 * j + r;
    f0[j] = n * 128 + ((h ^ ((n >> 1) & 7)) << 4);
    f1[j] = n * 128 + (((h + 4) ^ ((n >> 1) & 7)) << 4);
  }
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const bool ok = 16 * i + r < rows;
    xo[i] = ok ? (uint32_t)(16 * i + r) * (uint32_t)a.ldx + h * 16 : OOB;
    so[i] = ok ? (uint32_t)(16 * i + r) * (uint32_t)a.ldxs * 4u : OOB;
  }
  u32x8 x[D][TM];
  float sx[D][TM], sw[D];
  // column blocks start at different k-blocks: rows a power of two apart would
  // otherwise send every workgroup to the same few memory channels at a time
  // (K = 8192, 16 rows: 20.5 us against 15.8)
  const int rot = kb_n > 0 ? (int)(blockIdx.x + blockIdx.y) % kb_n : 0;
  auto load = [&](int d, int kb) {
    if (kb < kb_n) kb = kb + rot < kb_n ? kb + rot : kb + rot - kb_n;
    // chunks h and h + 4 of the block's eight; those past K read as zeros
    const uint32_t k0 = (uint32_t)kb * 128u;
    const bool in0 = (int)k0 + h * 16 < a.K, in1 = (int)k0 + h * 16 + 64 < a.K;
#pragma unroll
    for (int q = 0; q < WC; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(ring + d * (SK_N * 128) + q * 1024), 16,
                                               (int)(k0 + wc[q] < (uint32_t)a.K ? wo[q] : OOB), (int)k0, 0,
                                               NT ? CPOL_NT : 0);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      x[d][i] = join(buf_load16s(rx, in0 ? xo[i] : OOB, k0), buf_load16s(rx, in1 ? xo[i] : OOB, k0 + 64));
      sx[d][i] = buf_loadfs(rs, kb < kb_n ? so[i] : OOB, (uint32_t)kb * 4u);
    }
    sw[d] = buf_loadfs(rws, kb < kb_n ? 0u : OOB, (uint32_t)kb * 4u);
  };
#pragma unroll
  for (int d = 0; d < D; ++d) {
    load(d, wave + d * SK_WAVES);
    __builtin_amdgcn_sched_barrier(0);  // in ring order, as the loop's waits count them
  }
  for (int kb0 = wave; kb0 < kb_n; kb0 += D * SK_WAVES) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      // this slot's copies and everything behind them up to the newest D - 1
      // k-blocks have arrived
      wait_vm_le<(D - 1) * (WC + 3 * TM + 1)>();
      asm volatile("" ::: "memory");
      u32x8 w[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j)
        w[j] = join(*(const u32x4*)(ring + d * (SK_N * 128) + f0[j]), *(const u32x4*)(ring + d * (SK_N * 128) + f1[j]));
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const float s = sx[d][i] * sw[d];  // both zero past the last k-block
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const f32x4 p = mfma16_f8(w[j], x[d][i], f32x4{});
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(s, p[e], acc[i][j][e]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      wait_lgkm();  // the slot has been read
      load(d, kb0 + (d + D) * SK_WAVES);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  wait_vm_le<0>();  // the sums take the place of the rings, where nothing lands any more
  __syncthreads();
  f32x4(*red)[TM][NB][64] = (f32x4(*)[TM][NB][64])lds;
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
    if (a.part) {  // its rows are padded to 8 columns
      *(f32x4*)(a.part + (row0 + m) * a.ldp + n) = v;
      continue;
    }
    uint16_t* y = a.Y + (row0 + m) * a.ldy + n;
    if (n + 4 <= a.N) {
      *(u32x2*)y = u32x2{pack2<DT_BF16>(v[0], v[1]), pack2<DT_BF16>(v[2], v[3])};
    } else {
      for (int e = 0; e < a.N - n; ++e) y[e] = (uint16_t)to_bits<DT_BF16>(v[e]);
    }
  }
  __syncthreads();
}

// grid.x: column blocks; grid.y: groups (one without offsets); grid.z: splits
// of K.  TMAX: row blocks of 16 a workgroup holds at a time.  Up to 32 rows two
// workgroups of 128 registers per lane share a CU; 64 rows take the registers
// of both (capped at 128 they spill: 77 us against 66 with 128 experts).
// NT: weights past the caches.
template <int TMAX, bool NT>
__global__ __launch_bounds__(SK_WAVES * 64, TMAX <= 2 ? 4 : 2) void k_f8_skinny(F8BlockLaunch rec) {
  constexpr int D = 2;
  static_assert(16 * TMAX * SK_N * 4 <= D * SK_N * 128, "a wave's sums fit its ring");
  __shared__ __attribute__((aligned(16))) char lds[SK_WAVES * D * SK_N * 128];
  const F8BlockLaunch a = k_split(rec, blockIdx.z);
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
  for (int64_t m0 = lo; m0 < hi; m0 += 16 * TMAX) {
    const int rows = (int)min((int64_t)(16 * TMAX), hi - m0);
    if (rows <= 16)
      skinny_tile<1, D, NT>(a, m0, rows, W, ws, n0, lds);
    else if (rows <= 32)
      skinny_tile<2, D, NT>(a, m0, rows, W, ws, n0, lds);
    else if constexpr (TMAX > 2)
      skinny_tile<4, D, NT>(a, m0, rows, W, ws, n0, lds);
  }
}

// ---------------------------------------------------------------------------
// Tiled kernel: BM x BN output tiles, WM x WN waves, k-tiles of 128 (one scale
// block).  4096 x 8192 x 8192: 231-248 us, 2.2-2.4 PFLOP/s, the matrix pipe busy
// 52% of the cycles at the card's power limit.  Operand k-tiles stream from
// memory straight into LDS rings of SA slots for X and SB for W.  A wave
// multiplies MI x NJ blocks of 16 x 16; each matrix instruction starts from zero
// and spans a whole scale block, and its four results per lane are folded with
// one multiply-add each, a few instructions later, while the next ones run.
//
// A k-tile's X fragments are all held in registers, so its X slot is free after
// the first column of blocks (EARLY_X: a barrier there, and the copies of X two
// k-tiles on start that much earlier, 258 to 252 us at 4096 x 8192 x 8192).
// The main barrier stands before the last column: by then every wave holds all
// it needs of this k-tile, so its slots are free, and k-tile kt + 1 has landed,
// so its fragments are read behind the last column's matrix instructions (each
// X fragment right after its last use).
//
// The instruction's first operand is W, so a lane's results are four
// consecutive columns of one row of Y, and one lane value per 16 rows holds
// the scale.  W rows are dealt to the blocks so that blocks 2p and 2p + 1 of
// lane group h hold columns 32 p + 8 h .. + 7: eight consecutive columns, one
// 16-byte store.
//
// LDS rows are 128 bytes, two to a 256-byte bank line; chunk c of row r sits
// in slot c ^ swizzle(r).  A 128-bit read serves lanes 0-3, 12-15 and 20-27
// together (then 4-11 with 16-19 and 28-31, and the upper half alike), so lane
// group h reads chunk h and then chunk h + 4: groups 0 and 1 then differ in
// bit 0 of the chunk, which keeps their banks apart (in bit 1, the two halves
// of the 16 rows would meet and every read take twice as long).
//
// Row scales are copied to LDS in strips of four k-tiles by one wave per 64
// rows.  (A load per wave and k-tile touches a line per row and asks the L1 for
// as many lines as the operands' copies do: 271 us against 239 without them.)
// ---------------------------------------------------------------------------
template <int BM_, int BN_, int WM_, int WN_, int SA_, int SB_, bool EARLY_X_, bool NT_ = false, int ROWS_ = BM_ / WM_>
struct F8Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NW = WM * WN, THREADS = 64 * NW;
  static constexpr int WTM = BM / WM, WTN = BN / WN, MI = ROWS_ / 16, NJ = WTN / 16;  // (the first ROWS_ of a wave's rows)
  static constexpr int SA = SA_, SB = SB_;
  static constexpr bool EARLY_X = EARLY_X_, NT = NT_;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  static constexpr int S_BYTES = BM * 16;
  static constexpr int LDS = SA * A_BYTES + SB * B_BYTES + 2 * S_BYTES;
  static constexpr int PA = BM / (8 * NW), PB = BN / (8 * NW);  // 1 KB copies (8 rows) per wave
  static constexpr int WGS_PER_CU = 160 * 1024 / LDS >= 2 ? 2 : 1;
  // copies that may be in flight when k-tile kt + 1 has to be there: those
  // behind the later of its W and its X (scale loads not counted: fewer)
  static constexpr int LATER = EARLY_X ? PA : (SA - 2) * (PA + PB);
  static_assert(WTM == 64 && WTN <= 128 && NJ % 2 == 0 && NW % 4 == 0 && PA >= 1 && PB >= 1, "tile");
  static_assert(EARLY_X ? SA == 2 && SB == 2 : SA >= 2 && SA == SB, "ring");
  static_assert(LDS <= 160 * 1024, "LDS budget");
};
__device__ __forceinline__ int swz_x(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int swz_w(int row) { return ((row >> 1) & 1) | ((row >> 2) & 6); }

// One operand's copies: rows row0 .. of a [rows][ld] byte matrix; copy i of
// wave w fills tile rows 8 (NW i + w) + lane / 8.  Rows past the end and
// chunks at or past K (every chunk, past the last k-tile) land as zeros.
template <int P, int NW, bool IS_W, bool NTW = false>
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
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(tile + (NW * i + wave_id()) * 1024), 16, (int)o,
                                             (int)(kt * 128), 0, NTW ? CPOL_NT : 0);
  }
};

// barrier that no LDS access moves across in the compiler
__device__ __forceinline__ void publish() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// wave-uniform fp32 through the scalar cache (read only)
typedef const __attribute__((address_space(4))) float uniform_float;

template <class T>
__device__ __forceinline__ void f8_tile(char* lds, const F8BlockLaunch& a, int64_t row0, int rows, const uint8_t* W,
                                        const float* ws, int n0, int turn) {
  constexpr int MI = T::MI, NJ = T::NJ, NP = 4;
  char* const la = lds;
  char* const lb = la + T::SA * T::A_BYTES;
  const int lane = threadIdx.x & 63, wave = wave_id(), r = lane & 15, h = lane >> 4;
  const int wm = wave / T::WN * T::WTM, wn = wave % T::WN * T::WTN;
  const int nk = (a.K + 127) / 128, cols = a.N - n0;
  F8Loader<T::PA, T::NW, false> al;
  F8Loader<T::PB, T::NW, true, T::NT> bl;
  al.init(a.X, a.ldx, row0, rows, a.K);
  bl.init(W, a.ldw, n0, cols, a.K);
  const rsrc_t rxs = make_rsrc(
      a.xs + row0 * a.ldxs, (uint32_t)((int64_t)(rows < T::BM ? rows - 1 : T::BM - 1) * a.ldxs + nk) * 4u);
  // the wave's columns lie in one block of 128 weight rows (past N any will
  // do: those results are dropped)
  uniform_float* wsr = (uniform_float*)(uint64_t)(ws + (n0 + wn < a.N ? (int64_t)((n0 + wn) / 128) * a.ldws : 0));
  const int srow = wave * 64 + lane;  // waves 0 .. WM - 1 copy the scales
  const uint32_t xo = srow < rows ? (uint32_t)srow * (uint32_t)a.ldxs * 4u : OOB;
  // The k-tiles are taken in rotation from a place that the caller chooses
  // (turn), in steps of four, the scales' unit.
  const int k0 = nk > 0 && nk % 4 == 0 ? 4 * turn % nk : 0;
  auto nth = [&](int kt) { return kt >= nk ? nk : kt + k0 < nk ? kt + k0 : kt + k0 - nk; };
  // Strips of row scales: 64 rows by four k-tiles from `from` on (the last
  // four, near the end; fewer than four in all lie k-tile by k-tile), two buffers.
  char* const ls = lb + T::SB * T::B_BYTES;
  const int s_row = nk >= 4 ? 16 : 4, s_kt = nk >= 4 ? 4 : 256;
  auto from = [&](int kk) { return nk >= 4 ? min(kk, nk - 4) : 0; };
  auto copy_scales = [&](int kk, int buf) {
    if (wave >= T::WM) return;
    char* const dst = ls + buf * T::S_BYTES + wave * 1024;
    if (nk >= 4) {
      dma16s(rxs, xo, (uint32_t)from(kk) * 4u, dst);
    } else {
      for (int e = 0; e < nk; ++e) dma4(rxs, xo + e * 4u, dst + e * 256);
    }
  };
  const bool busy = wm < rows;  // waves below the last row only copy

  // lane offsets of the fragments: chunks h and h + 4 of the row
  const int ra = wm + r, rb = wn + 8 * (r >> 2) + (r & 3);
  const uint32_t a0 = ra * 128 + ((h ^ swz_x(ra)) << 4), a1 = ra * 128 + (((h + 4) ^ swz_x(ra)) << 4);
  const uint32_t b0 = rb * 128 + ((h ^ swz_w(rb)) << 4), b1 = rb * 128 + (((h + 4) ^ swz_w(rb)) << 4);

  // the c-th of the copies that take the slots of k-tile kt
  constexpr int C = T::PA + T::PB;
  auto copy_x = [&](int c, int kt, char* slot) { al.issue(c, nth(kt + T::SA), slot); };
  auto copy_w = [&](int c, int kt, char* slot) { bl.issue(c, nth(kt + T::SB), slot); };

  f32x4 acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{};

  if (nk > 0) {
    copy_scales(k0, 0);
    copy_scales(nth(4), 1);
#pragma unroll
    for (int p = 0; p < T::SA; ++p) {
#pragma unroll
      for (int c = 0; c < T::PA; ++c) copy_x(c, p - T::SA, la + p * T::A_BYTES);
#pragma unroll
      for (int c = 0; c < T::PB; ++c) copy_w(c, p - T::SB, lb + p * T::B_BYTES);
    }
    // k-tile 0: what was issued behind its W and X may be in flight
    wait_vm_le<(T::SA - 1) * C>();
    publish();
    int sa = 0, sb = 0;  // slots of k-tile kt
    u32x8 fa[MI], fb[2];
    float sc[MI], sn[MI];
    float sw = wsr[k0];  // of k-tile kt + 1 inside the loop
    // row scales of the kt-th k-tile for the blocks of 16 rows
    auto read_scales = [&](int kt, float (&out)[MI]) {
      const int kk = min(nth(kt), nk - 1);
      const char* const p = ls + (kt / 4 & 1) * T::S_BYTES + wm * 16 + (kk - from(kk & ~3)) * s_kt;
#pragma unroll
      for (int i = 0; i < MI; ++i) out[i] = *(const float*)(p + (16 * i + r) * s_row);
    };
    if (busy) {
      fb[0] = join(*(const u32x4*)(lb + b0), *(const u32x4*)(lb + b1));
#pragma unroll
      for (int i = 0; i < MI; ++i)
        fa[i] = join(*(const u32x4*)(la + a0 + i * 2048), *(const u32x4*)(la + a1 + i * 2048));
      read_scales(0, sc);
#pragma unroll
      for (int i = 0; i < MI; ++i) sc[i] *= sw;
    }
    sw = wsr[nk > 1 ? nth(1) : 0];
    for (int kt = 0; kt < nk; ++kt) {
      // first of four k-tiles: everyone is past the other buffer, the next four go there
      if (kt > 0 && kt % 4 == 0) copy_scales(nth(kt + 4), (kt / 4 + 1) & 1);
      char* const ca = la + sa * T::A_BYTES;  // this k-tile's slots: free behind the barrier
      char* const cb = lb + sb * T::B_BYTES;
      sa = sa + 1 == T::SA ? 0 : sa + 1;
      sb = sb + 1 == T::SB ? 0 : sb + 1;
      const char* const na = la + sa * T::A_BYTES;
      const char* const nb = lb + sb * T::B_BYTES;
      constexpr int STEPS = MI * NJ, LAST = MI * (NJ - 1);
      if (busy) {
        f32x4 part[NP];
        float swn = 0.0f;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < STEPS + NP - 1; ++t) {
          const int j = t / MI, i = t % MI;
          if (T::EARLY_X && t == MI) {
            publish();  // every wave holds its X fragments
            __builtin_amdgcn_sched_barrier(0);
          }
          if (t == LAST) {
            wait_lgkm();  // the last fragments of this k-tile are in registers
            wait_vm_le<T::LATER>();
            publish();
            fb[0] = join(*(const u32x4*)(nb + b0), *(const u32x4*)(nb + b1));
            read_scales(kt + 1, sn);
            const float sw2 = wsr[kt + 2 < nk ? nth(kt + 2) : 0];
            swn = sw;
            sw = sw2;
            __builtin_amdgcn_sched_barrier(0);
          }
          if (t < STEPS) {
            part[t % NP] = mfma16_f8(fb[j & 1], fa[i], f32x4{});
            if (i == 0 && j + 1 < NJ) {
              const int o = (32 * ((j + 1) / 2) + 4 * ((j + 1) & 1)) * 128;
              fb[(j + 1) & 1] = join(*(const u32x4*)(cb + b0 + o), *(const u32x4*)(cb + b1 + o));
            }
            if (T::EARLY_X && j == 1) {
#pragma unroll
              for (int c = i * T::PA / MI; c < (i + 1) * T::PA / MI; ++c) copy_x(c, kt, ca);
            }
            if (t >= LAST) {
#pragma unroll
              for (int c = i * C / MI; c < (i + 1) * C / MI; ++c) {
                if (c >= T::PA) copy_w(c - T::PA, kt, cb);
                else if (!T::EARLY_X) copy_x(c, kt, ca);
              }
            }
          }
          if (t >= NP - 1) {
            const int u = t - (NP - 1), j2 = u / MI, i2 = u % MI;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i2][j2][e] = __builtin_fmaf(sc[i2], part[u % NP][e], acc[i2][j2][e]);
          }
          if (t >= LAST && t < STEPS)
            fa[i] = join(*(const u32x4*)(na + a0 + i * 2048), *(const u32x4*)(na + a1 + i * 2048));
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < MI; ++i) sc[i] = sn[i] * swn;
      } else {
        if constexpr (T::EARLY_X) {
          publish();
#pragma unroll
          for (int c = 0; c < T::PA; ++c) copy_x(c, kt, ca);
        }
        wait_vm_le<T::LATER>();
        publish();
#pragma unroll
        for (int c = 0; c < C; ++c) {
          if (c >= T::PA) copy_w(c - T::PA, kt, cb);
          else if (!T::EARLY_X) copy_x(c, kt, ca);
        }
      }
    }
  }
  wait_vm_le<0>();  // nothing lands in LDS after the tile

  if (!busy) return;
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int rr = tid & 15, hh = (tid & 63) >> 4;
  const int left = rows < T::BM ? rows : T::BM;
  if (a.part) {  // its rows are padded to 8 columns
    const int pad = (cols + 7) / 8 * 8;
    const rsrc_t rp = make_rsrc(a.part + row0 * a.ldp + n0, (uint32_t)((int64_t)(left - 1) * a.ldp + pad) * 4u);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int m = wm + 16 * i + rr;
#pragma unroll
      for (int p = 0; p < NJ / 2; ++p) {
        const int n = wn + 32 * p + 8 * hh;
        const uint32_t o = m < left && n < cols ? ((uint32_t)m * (uint32_t)a.ldp + (uint32_t)n) * 4u : OOB;
        buf_store16_wb(rp, o, __builtin_bit_cast(u32x4, acc[i][2 * p]));
        buf_store16_wb(rp, o + 16u, __builtin_bit_cast(u32x4, acc[i][2 * p + 1]));
      }
    }
    return;
  }
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
__global__ __launch_bounds__(T::THREADS, T::WGS_PER_CU) void k_f8_tiled(F8BlockLaunch rec) {
  __shared__ __attribute__((aligned(16))) char lds[T::LDS];
  const F8BlockLaunch a = k_split(rec, blockIdx.y);
  const int tm = (a.M + T::BM - 1) / T::BM, tn = (a.N + T::BN - 1) / T::BN;
  const int tile = xcd_tile(blockIdx.x, tm * tn);
  if (tile < 0) return;
  int mi, ni;
  raster(tile, tm, tn, mi, ni);
  f8_tile<T>(lds, a, (int64_t)mi * T::BM, a.M - mi * T::BM, a.W, a.ws, ni * T::BN, 0);
}

// Y = the splits' sums, added in order; 8 columns a thread
__global__ __launch_bounds__(256) void k_f8_join(F8BlockLaunch a) {
  const int64_t per = a.ldp / 8, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.M * per) return;
  const int64_t m = i / per, n = i % per * 8;
  f32x4 v0{}, v1{};
  for (int s = 0; s < a.splits; ++s) {
    const f32x4* p = (const f32x4*)(a.part + ((int64_t)s * a.M + m) * a.ldp + n);
    v0 += p[0];
    v1 += p[1];
  }
  uint16_t* y = a.Y + m * a.ldy + n;
  if (n + 8 <= a.N) {
    *(u32x4*)y = u32x4{pack2<DT_BF16>(v0[0], v0[1]), pack2<DT_BF16>(v0[2], v0[3]), pack2<DT_BF16>(v1[0], v1[1]),
                       pack2<DT_BF16>(v1[2], v1[3])};
  } else {
    for (int e = 0; e < a.N - n; ++e) y[e] = (uint16_t)to_bits<DT_BF16>(e < 4 ? v0[e & 3] : v1[e & 3]);
  }
}

using F8T256 = F8Tile<256, 256, 4, 2, 2, 2, true>;
using F8T128 = F8Tile<128, 128, 2, 2, 2, 2, true>;
// The grouped call's tile shapes.  UNIT rows and columns at most, a group's last
// rows in the smallest shape that holds them; weights of short tiles are read
// once and pass the L2 by (nt: 128 experts of 64 rows 205 to 194 us), three
// k-tiles deep (two: 309 us against 285 in the mix below).  TINY multiplies only
// 32 rows.  LONG: groups of more rows than this mostly wait for the matrix pipe.
struct F8Large {
  static constexpr int UNIT = 256, LONG = 128, THREADS = 512, WGS = 1;
  using Full = F8T256;
  using Half = F8Tile<128, 256, 2, 4, 3, 3, false, true>;
  using Short = F8Tile<64, 256, 1, 8, 3, 3, false, true>;
  using Tiny = F8Tile<64, 256, 1, 8, 3, 3, false, true, 32>;
};
// where those tiles would not fill the device (4 groups, 1000 rows, N 512, K
// 1024: 22.9 us; these take 14.5)
struct F8Small {
  static constexpr int UNIT = 128, LONG = 64, THREADS = 256, WGS = 2;
  using Full = F8T128;
  using Half = F8T128;
  using Short = F8Tile<64, 128, 1, 4, 3, 3, false, true>;
  using Tiny = F8Tile<64, 128, 1, 4, 3, 3, false, true, 32>;
};
constexpr int SK_ROWS = 64;  // rows up to which the skinny kernel runs
constexpr int SPLIT_MOST = 8;

// Tiles of the grouped call.  A group's rows are cut into units; long groups
// mostly wait for the matrix pipe, short ones for their weights to come from
// memory, so the two lists of tiles are dealt out in turn, in proportion, and
// the device computes and reads at the same time (275 us against 283 one list
// after the other: 128 experts, 16384 skewed rows, N 2048, K 4096; now 263);
// some short tiles are kept for the end, where they even out the finish.
// Workgroups that stay and fetch tiles from a counter measured 5% slower than
// letting the hardware place them.
struct F8Lists {
  int32_t total[2];  // tiles of the long and of the short groups
  int32_t start[2][kMaxOffsetGroupCount];  // exclusive sums over the groups
};
// rows lo .. m (of the next group) clipped to the operand: first row and count
__device__ __forceinline__ void clip_rows(const F8BlockLaunch& a, int& lo, int& m) {
  lo = min(max(lo, 0), a.M);
  m = max(min(max(m, 0), a.M) - lo, 0);
}
__device__ __forceinline__ void group_rows(const F8BlockLaunch& a, int g, int& lo, int& m) {
  lo = a.offsets[g];
  m = a.offsets[g + 1];
  clip_rows(a, lo, m);
}

__global__ __launch_bounds__(kMaxOffsetGroupCount) void k_f8_group_table(F8BlockLaunch a, int unit, int above, F8Lists* lists) {
  __shared__ int32_t sums[2][kMaxOffsetGroupCount / 64];
  const int g = threadIdx.x, lane = g & 63, wave = g >> 6;
  int lo, m = 0;
  if (g < a.count) group_rows(a, g, lo, m);
  const int tiles = (m + unit - 1) / unit * ((a.N + unit - 1) / unit);
  int v[2] = {m > above ? tiles : 0, m > above ? 0 : tiles}, s[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    s[c] = v[c];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(s[c], d);
      if (lane >= d) s[c] += o;
    }
    if (lane == 63) sums[c][wave] = s[c];
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    for (int w = 0; w < wave; ++w) s[c] += sums[c][w];
    if (g < a.count) lists->start[c][g] = s[c] - v[c];
    if (g == kMaxOffsetGroupCount - 1) lists->total[c] = s[c];
  }
}

// Tiles go to the XCDs in chunks of CHUNK neighbours of one list, the chunks in
// turn: a chunk of long tiles is a block of 4 by 2, a chunk of short ones mostly
// a group's rows with all its weights, so an XCD fetches few panels for it
// (chunks of 8 neighbours of the mixed order: 1553 MB past the L2 against 1270).
constexpr int CHUNK = 8, BAND = 4;

template <class G>
__global__ __launch_bounds__(G::THREADS, G::WGS) void k_f8_tiled_grouped(F8BlockLaunch a, const F8Lists* lists, int tail) {
  constexpr int FULL = G::Full::LDS, HALF = G::Half::LDS, SHORT = G::Short::LDS;
  __shared__ __attribute__((aligned(16))) char lds[FULL > HALF ? (FULL > SHORT ? FULL : SHORT) : (HALF > SHORT ? HALF : SHORT)];
  static_assert(G::Full::THREADS == G::THREADS && G::Half::THREADS == G::THREADS && G::Short::THREADS == G::THREADS &&
                    G::Tiny::THREADS == G::THREADS && G::Tiny::LDS == SHORT,
                "one workgroup size");
  const int lane = threadIdx.x & 63, turn_of_xcd = blockIdx.x / XCDS;
  const int p = turn_of_xcd / CHUNK * XCDS + blockIdx.x % XCDS;  // chunk
  // All that finding the tile needs of the first 128 groups is asked for at
  // once: one trip to memory before the first copy instead of four.
  const int nl = lists->total[0], ns = lists->total[1];
  int first[2][2], row[2], next[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int q = min(lane + 64 * i, a.count - 1);
    first[i][0] = lists->start[0][q];
    first[i][1] = lists->start[1][q];
    row[i] = a.offsets[q];
    next[i] = a.offsets[q + 1];
  }
  const int cl = (nl + CHUNK - 1) / CHUNK, cs = (ns + CHUNK - 1) / CHUNK;
  if (p >= cl + cs) return;
  // chunks of short tiles before chunk p: spread evenly over the long ones up
  // to the last `tail`
  const int spread = max(cs - tail, 0), mixed = cl + spread;
  int cls = 1, tile = p - cl;
  if (p < mixed) {
    const int before = (int)((int64_t)p * spread / mixed), after = (int)((int64_t)(p + 1) * spread / mixed);
    cls = after > before;
    tile = cls ? before : p - before;
  }
  tile = tile * CHUNK + turn_of_xcd % CHUNK;
  if (tile >= (cls ? ns : nl)) return;
  // the last group whose first tile is not past this one
  int n = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    n += __popcll(__ballot(lane + 64 * i < a.count && (cls ? first[i][1] : first[i][0]) <= tile));
  if (a.count > 128) {
    int more = 0;
    for (int q = lane + 128; q < a.count; q += 64) more += lists->start[cls][q] <= tile;
    for (int d = 1; d < 64; d <<= 1) more += __shfl_xor(more, d);
    n += __builtin_amdgcn_readfirstlane(more);
  }
  const int g = n - 1;
  if (g < 0) return;
  int lo, m, base;
  if (g < 128) {
    const int l = g & 63, i = g >> 6;
    base = __builtin_amdgcn_readlane(i ? (cls ? first[1][1] : first[1][0]) : (cls ? first[0][1] : first[0][0]), l);
    lo = __builtin_amdgcn_readlane(i ? row[1] : row[0], l);
    m = __builtin_amdgcn_readlane(i ? next[1] : next[0], l);
    clip_rows(a, lo, m);
  } else {
    group_rows(a, g, lo, m);
    base = lists->start[cls][g];
  }
  const int local = tile - base, tm = (m + G::UNIT - 1) / G::UNIT, tn = (a.N + G::UNIT - 1) / G::UNIT;
  if ((uint32_t)local >= (uint32_t)(tm * tn)) return;  // overlapping groups: the sums may not fit
  int mi, ni;
  raster(local, tm, tn, mi, ni, BAND);
  const int n0 = ni * G::UNIT, rows = m - mi * G::UNIT;
  const int64_t row0 = (int64_t)lo + (int64_t)mi * G::UNIT;
  const uint8_t* W = a.W + (int64_t)g * a.w_stride;
  const float* ws = a.ws + (int64_t)g * a.ws_stride;
  // Where a tile starts in K: rows a power of two apart keep all workgroups on
  // the same few memory channels while they walk K in step (64 rows each: 4.1
  // TB/s in step, 6.1 TB/s out of step).  Tiles that share a weight panel do
  // keep step, and the large ones that share rows.
  const int turn = 5 * g;
  if (rows > 128)
    f8_tile<typename G::Full>(lds, a, row0, rows, W, ws, n0, turn);
  else if (rows > 64)
    f8_tile<typename G::Half>(lds, a, row0, rows, W, ws, n0, turn + ni);
  else if (rows > 32)
    f8_tile<typename G::Short>(lds, a, row0, rows, W, ws, n0, turn + ni);
  else
    f8_tile<typename G::Tiny>(lds, a, row0, rows, W, ws, n0, turn + ni);
}

static hipError_t launch_skinny(const F8BlockLaunch& a, hipStream_t stream) {
  const dim3 grid((a.N + SK_N - 1) / SK_N, a.offsets ? a.count : 1, a.splits);
  // experts whose weights pass the 256 MB of the memory-side cache together are
  // not found there at the next call; a dense weight may be
  if (a.offsets && (int64_t)a.count * a.N * a.K > int64_t(256) << 20)
    hipLaunchKernelGGL((k_f8_skinny<2, true>), grid, dim3(SK_WAVES * 64), 0, stream, a);
  else if (a.offsets || a.M <= 32)
    hipLaunchKernelGGL((k_f8_skinny<2, false>), grid, dim3(SK_WAVES * 64), 0, stream, a);
  else
    hipLaunchKernelGGL((k_f8_skinny<4, false>), grid, dim3(SK_WAVES * 64), 0, stream, a);
  return hipGetLastError();
}

static int64_t tiles_of(int M, int N, int bm, int bn) {
  return ((int64_t)M + bm - 1) / bm * (((int64_t)N + bn - 1) / bn);
}

// How a dense call runs: the skinny kernel up to SK_ROWS rows, 256 x 256 tiles
// where they fill the device, else 128 x 128; and into how many parts K is
// split if there is a workspace.
struct F8Plan {
  int bm;  // 0: skinny
  int splits;
};
static F8Plan plan_dense(int M, int N, int K) {
  const int cus = device_cu_count();
  F8Plan p{0, 1};
  int64_t wgs = (N + SK_N - 1) / SK_N;
  if (M > SK_ROWS) {
    p.bm = tiles_of(M, N, 256, 256) >= cus ? 256 : 128;
    wgs = tiles_of(M, N, p.bm, p.bm);
  }
  // A split saves its share of the k-blocks, at what one costs a workgroup, and
  // adds a launch and the partial sums' way to memory and back (4 TB/s); it has
  // to save 3 us (128 x 512 x 8192: 46.6 to 16.5 us; 2048 x 1024 x 2048 would
  // go from 16.1 to 18.9 and stays whole).
  const int kb_n = (K + 127) / 128;
  const double us_per_block = p.bm ? 0.7 : M > 32 ? 0.45 : 0.19;
  double best = 3.0;
  for (int s = 2; s <= SPLIT_MOST && s * wgs <= cus && 4 * s <= kb_n; ++s) {
    const double save = us_per_block * kb_n * (1.0 - 1.0 / s) - 4.0 - 8e-6 / 4.0 * s * (double)M * (double)N;
    if (save > best) {
      best = save;
      p.splits = s;
    }
  }
  return p;
}
static int64_t part_ld(int N) { return ((int64_t)N + 7) / 8 * 8; }
size_t f8_block_workspace(int M, int N, int K) {
  const int splits = plan_dense(M, N, K).splits;
  return splits > 1 ? (size_t)splits * (size_t)M * (size_t)part_ld(N) * sizeof(float) : 0;
}
size_t f8_block_grouped_workspace(int) { return sizeof(F8Lists); }

hipError_t launch_f8_block(const F8BlockLaunch& rec, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  F8BlockLaunch a = rec;
  const F8Plan p = plan_dense(a.M, a.N, a.K);
  if (p.splits > 1 && workspace && workspace_bytes >= f8_block_workspace(a.M, a.N, a.K)) {
    a.splits = p.splits;
    a.part = (float*)workspace;
    a.ldp = part_ld(a.N);
  }
  hipError_t e;
  if (p.bm == 0) {
    e = launch_skinny(a, stream);
  } else {
    const unsigned tiles = (unsigned)((tiles_of(a.M, a.N, p.bm, p.bm) + XCDS - 1) / XCDS * XCDS);
    if (p.bm == 256)
      hipLaunchKernelGGL((k_f8_tiled<F8T256>), dim3(tiles, a.splits), dim3(F8T256::THREADS), 0, stream, a);
    else
      hipLaunchKernelGGL((k_f8_tiled<F8T128>), dim3(tiles, a.splits), dim3(F8T128::THREADS), 0, stream, a);
    e = hipGetLastError();
  }
  if (e != hipSuccess || a.splits <= 1) return e;
  hipLaunchKernelGGL(k_f8_join, dim3((unsigned)((a.M * (a.ldp / 8) + 255) / 256)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

// tiles of a grouped call at most (how many there are is known on the device
// only: every group may end in a partial unit)
static int64_t most_tiles(const F8BlockLaunch& a, int unit) {
  return ((int64_t)a.M / unit + std::min(a.count, a.M)) * (((int64_t)a.N + unit - 1) / unit);
}

template <class G>
static hipError_t launch_tiled_grouped(const F8BlockLaunch& a, F8Lists* lists, hipStream_t stream) {
  hipLaunchKernelGGL(k_f8_group_table, dim3(1), dim3(kMaxOffsetGroupCount), 0, stream, a, G::UNIT, G::LONG, lists);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t chunks = most_tiles(a, G::UNIT) / CHUNK + 2;  // each list's last one may be short
  const unsigned grid = (unsigned)((chunks + XCDS - 1) / XCDS * XCDS * CHUNK);
  hipLaunchKernelGGL(k_f8_tiled_grouped<G>, dim3(grid), dim3(G::THREADS), 0, stream, a, lists,
                     device_cu_count() / (2 * CHUNK));
  return hipGetLastError();
}

hipError_t launch_f8_block_grouped(const F8BlockLaunch& a, void* workspace, hipStream_t stream) {
  // Few rows in all, or two a group on average: weights alone.  How they are
  // spread is known on the device only; 128 groups, N 2048, K 4096, us here and in
  // tiles: 128 rows evenly 154 and 164, Zipf-skewed 66 and 69, in four groups 20
  // and 29, in one 36 and 40; 256 rows 155 and 166, 96 and 108, 37 and 32, 65 and
  // 54 (in two groups 66 and 40, the worst: a group's weights come once per 32
  // rows).  More rows than two a group: 16 groups, 256 rows 41 and 32.
  if (a.M <= SK_ROWS || (a.M <= 2 * a.count && a.M <= 256)) return launch_skinny(a, stream);
  if (most_tiles(a, F8Large::UNIT) < device_cu_count())
    return launch_tiled_grouped<F8Small>(a, (F8Lists*)workspace, stream);
  return launch_tiled_grouped<F8Large>(a, (F8Lists*)workspace, stream);
}

}  // namespace gmi
