// kernels_f8block.hip -- fp8 GEMM with block scales, dense and per group:
//   Y[m][n] = sum_b xs[m][b] ws[n / 128][b] sum_{k in block b} X[m][k] W[n][k]
// over blocks b of 128 k.  The matrix instruction forms each block's inner
// sum in fp32 (v_mfma_scale_f32_16x16x128_f8f6f4 with unit scales spans
// exactly one block), and one fp32 multiply-add per result folds it into the
// accumulator with the product of the two scales.  The result is rounded once,
// to bf16.
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

// grid.x: column blocks; grid.y: 64-row chunks (dense) or groups
__global__ __launch_bounds__(SK_WAVES * 64) void k_f8_skinny(F8BlockLaunch a) {
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
    lo = (int64_t)blockIdx.y * 64;
    hi = min((int64_t)a.M, lo + 64);
  }
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

static hipError_t launch_skinny(const F8BlockLaunch& a, hipStream_t stream) {
  const int nb = (a.N + SK_N - 1) / SK_N;
  const int gy = a.offsets ? a.count : (a.M + 63) / 64;
  hipLaunchKernelGGL(k_f8_skinny, dim3(nb, gy), dim3(SK_WAVES * 64), 0, stream, a);
  return hipGetLastError();
}

size_t f8_block_workspace(int, int, int) { return 0; }
size_t f8_block_grouped_workspace(int count) { return 16 + 16 * (size_t)count; }

hipError_t launch_f8_block(const F8BlockLaunch& a, void*, size_t, hipStream_t stream) {
  return launch_skinny(a, stream);
}

hipError_t launch_f8_block_grouped(const F8BlockLaunch& a, void*, hipStream_t stream) {
  return launch_skinny(a, stream);
}

}  // namespace gmi
