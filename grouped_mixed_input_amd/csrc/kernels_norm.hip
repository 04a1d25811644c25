// kernels_norm.hip -- root-mean-square norm with the residual's addition and
// an fp8 output with a scale per row and 128 columns, and its backward pass.
//
//   h = x + residual,  y = w h r,  r = 1 / sqrt(mean(h^2) + eps)
//   s = max(max |y| over the 128-column block, 448 * 2^-126) / 448,  q = e4m3(y / s)
// Backward, with n = h r and g = w dy:
//   dh = dres + r (g - n mean(g n)),  dw = sum over rows of dy n
//
// One pass over memory: a team of TPR threads holds one row in registers
// (each thread CPT chunks of 8 columns, 16-byte loads), reduces the sum of
// squares across the team and finishes the row from registers, so every input
// is read once and every output written once.  All sums and the norm itself
// are fp32; h, y and dh are rounded once to the 16-bit type.  y is formed
// from the unrounded fp32 sum x + residual.
//
// Bound by memory: 16384 x 4096 bf16 73 us forward (6.5 TB/s), 90 + 4.6 backward
// (6.0 TB/s in the main launch; a plain copy reaches 5.4).  One row of 4096:
// 2.5 us, an empty launch's time.
#include "gmi_device.hpp"
#include "gmi_internal.hpp"
#include "gmi_rows.hpp"

namespace gmi {

// Sum over the team of TPR threads that share a row.  `red` holds one float
// per wave of the workgroup; two barriers, so that the next call may reuse it.
template <int TPR>
__device__ __forceinline__ float team_sum(float v, float* red) {
  v = sum64(v);
  if constexpr (TPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    const int first = wave / (TPR / 64) * (TPR / 64);
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) v += red[first + i];
    __syncthreads();
  }
  return v;
}

// Workgroups of WG threads, WG / TPR rows at a time.
template <int DT, bool NT, int WG, int TPR, int CPT>
__global__ __launch_bounds__(WG) void k_rmsnorm_quant(NormLaunch a) {
  __shared__ float red[WG / 64];
  const int team = threadIdx.x / TPR, t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * (WG / TPR) + team;
  const bool live = row < a.rows;  // a team past the end still meets the barriers
  const int chunks = a.K / 8;
  const uint16_t* x = a.x + (live ? row * a.ldx : 0);
  const uint16_t* res = a.residual ? a.residual + (live ? row * a.ldr : 0) : nullptr;
  u32x4 xv[CPT], rv[CPT];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = t + i * TPR;
    const bool in = live && c < chunks;
    xv[i] = in ? load16<NT>(x + 8 * c) : u32x4{};
    rv[i] = in && res ? load16<NT>(res + 8 * c) : u32x4{};
  }
  float h[CPT][8];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    float r8[8];
    unpack8<DT>(xv[i], h[i]);
    unpack8<DT>(rv[i], r8);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[i][e] += r8[e];
      ss = __builtin_fmaf(h[i][e], h[i][e], ss);
    }
    const int c = t + i * TPR;
    if (a.h && live && c < chunks) store<NT>(a.h + row * a.ldh + 8 * c, pack8<DT>(h[i]));
  }
  ss = team_sum<TPR>(ss, red);
  const float r = 1.0f / sqrtf(ss / (float)a.K + a.eps);
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = t + i * TPR;
    const bool in = live && c < chunks;
    float w[8];
    unpack8<DT>(in ? *(const u32x4*)(a.weight + 8 * c) : u32x4{}, w);
    float amax = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[i][e] = h[i][e] * r * w[e];
      amax = fmaxf(amax, fabsf(h[i][e]));
    }
    if (a.y && in) store<false>(a.y + row * a.ldy + 8 * c, pack8<DT>(h[i]));
    if (!a.q) continue;
    // 16 neighbouring threads hold one block of 128 columns (those past K
    // hold zeros)
    const float s = block_scale(max16(amax));
    if (in) {
      store<false>(a.q + row * a.ldq + 8 * c, codes8(h[i], s));
      if (c % 16 == 0) a.scales[row * a.lds + c / 16] = s;
    }
  }
}

// Backward: a persistent grid; each team walks rows and keeps its share of the
// weight's gradient in registers, adds the teams of a workgroup in LDS (in a
// fixed order) and writes one fp32 row of partials per workgroup, which
// k_norm_dweight sums in workgroup order.
template <int DT, bool NT, int WG, int TPR, int CPT>
__global__ __launch_bounds__(WG) void k_rmsnorm_bwd(NormBwdLaunch a) {
  __shared__ float red[WG / 64];
  const int team = threadIdx.x / TPR, t = threadIdx.x % TPR;
  constexpr int TEAMS = WG / TPR;
  const int chunks = a.K / 8;
  u32x4 wv[CPT];
  float dw[CPT][8];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = t + i * TPR;
    wv[i] = c < chunks ? *(const u32x4*)(a.weight + 8 * c) : u32x4{};
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.0f;
  }
  const float inv_k = 1.0f / (float)a.K;
  for (int64_t base = (int64_t)blockIdx.x * TEAMS; base < a.rows; base += (int64_t)gridDim.x * TEAMS) {
    const int64_t row = base + team;
    const bool live = row < a.rows;
    u32x4 hv[CPT], gv[CPT], rv[CPT];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = t + i * TPR;
      const bool in = live && c < chunks;
      hv[i] = in ? load16<NT>(a.h + row * a.ldh + 8 * c) : u32x4{};
      gv[i] = in ? load16<NT>(a.dy + row * a.lddy + 8 * c) : u32x4{};
      rv[i] = in && a.dres ? load16<NT>(a.dres + row * a.lddr + 8 * c) : u32x4{};
    }
    float ss = 0.0f, gh = 0.0f;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      float h[8], g[8], w[8];
      unpack8<DT>(hv[i], h);
      unpack8<DT>(gv[i], g);
      unpack8<DT>(wv[i], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss = __builtin_fmaf(h[e], h[e], ss);
        gh = __builtin_fmaf(g[e] * w[e], h[e], gh);
      }
    }
    ss = team_sum<TPR>(ss, red);
    gh = team_sum<TPR>(gh, red);
    // a team without a row adds nothing, whatever eps is
    const float r = live ? 1.0f / sqrtf(ss * inv_k + a.eps) : 0.0f;
    const float m = gh * r * r * inv_k;  // mean(g n) / r * r^2: the factor of h inside r (g - h m)
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = t + i * TPR;
      float h[8], g[8], w[8], d[8];
      unpack8<DT>(hv[i], h);
      unpack8<DT>(gv[i], g);
      unpack8<DT>(wv[i], w);
      unpack8<DT>(rv[i], d);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d[e] = __builtin_fmaf(r, __builtin_fmaf(-h[e], m, g[e] * w[e]), d[e]);
        dw[i][e] = __builtin_fmaf(g[e], h[e] * r, dw[i][e]);
      }
      if (live && c < chunks) store<false>(a.dh + row * a.lddh + 8 * c, pack8<DT>(d));
    }
  }
  if (!a.partial) return;
  float* out = a.partial + (int64_t)blockIdx.x * a.K;
  if constexpr (TEAMS == 1) {
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = t + i * TPR;
      if (c < chunks) {
        *(f32x4*)(out + 8 * c) = f32x4{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
        *(f32x4*)(out + 8 * c + 4) = f32x4{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
      }
    }
  } else {
    // one chunk slice at a time through LDS, added over the teams in order
    __shared__ float sl[TEAMS][TPR * 8 + 8];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8; ++e) sl[team][t * 8 + e] = dw[i][e];
      __syncthreads();
      for (int j = threadIdx.x; j < TPR * 8; j += WG) {
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < TEAMS; ++k) v += sl[k][j];
        const int col = i * TPR * 8 + j;
        if (col < a.K) out[col] = v;
      }
    }
  }
}

// dweight[k] = sum of the partial rows in order: 32 columns a workgroup, four a
// thread, 32 threads over contiguous ranges of rows, added in a fixed order.
__global__ __launch_bounds__(256) void k_norm_dweight(const float* partial, int parts, int K, float* dweight) {
  __shared__ f32x4 red[32][8];
  const int cl = threadIdx.x & 7, rl = threadIdx.x >> 3;
  const int col = blockIdx.x * 32 + 4 * cl;  // K is a multiple of 8
  const int per = (parts + 31) / 32;
  f32x4 v{};
  if (col < K) {
    const int end = min(parts, (rl + 1) * per);
#pragma unroll 8
    for (int p = rl * per; p < end; ++p) v += *(const f32x4*)(partial + (int64_t)p * K + col);
  }
  red[rl][cl] = v;
  __syncthreads();
  if (threadIdx.x < 32 && blockIdx.x * 32 + (int)threadIdx.x < K) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += red[i][threadIdx.x >> 2][threadIdx.x & 3];
    dweight[blockIdx.x * 32 + threadIdx.x] = t;
  }
}

// Threads per row and chunks per thread.  Many rows: the fewest threads that
// hold a row in four chunks each (with eight the backward needs 378 registers
// a lane and one wave is left per SIMD: 104 us against 89 at 16384 x 4096 with
// two waves a row).  Few rows cannot fill the device that way, so the row is
// spread over 256 threads for latency.
// nt: from 2^25 elements on, where a call's tensors begin to push each other out
// of the 256 MB of the memory-side cache, inputs and h pass the caches.  What
// the next kernel reads (q, y, dh) does not.  4096 columns, us alone and with a
// product over 1024 columns that reads the result (all through the caches / all
// past them / this):
//   16384 rows, x, residual, h, q   86, 150    77.6, 144.5    72.7, 137
//    8192 rows, x, residual, h, q   46, 85     41.9, 85       40.4, 81
//    8192 rows, x and q alone       24.6, 65   22.2, 65       23.1, 64.4
//   16384 rows, the same and y      110, 194   104.8, 203     108.5, 191
//   16384 rows, backward            105, 195   92, 191        94.4, 185
struct NormShape {
  int tpr, cpt;
  bool nt;
};
static NormShape norm_shape(int64_t rows, int K) {
  const int chunks = K / 8;
  const int few = 4 * device_cu_count();
  int tpr = chunks <= 4 * 64 ? 64 : chunks <= 4 * 128 ? 128 : chunks <= 4 * 256 ? 256 : 512;
  if (rows < few && chunks > 64 && tpr < 256) tpr = 256;
  int cpt = 1;
  while (cpt * tpr < chunks) cpt *= 2;
  return {tpr, cpt, rows * K >= int64_t(1) << 25};
}

#define GMI_NORM_LAUNCH(KER, DT, NT, WG, TPR, CPT, grid, stream, args) \
  hipLaunchKernelGGL((KER<DT, NT, WG, TPR, CPT>), dim3(grid), dim3(WG), 0, stream, args)
#define GMI_NORM_CPT(KER, DT, NT, WG, TPR, cpt, grid, stream, args)               \
  do {                                                                            \
    if ((cpt) == 1) GMI_NORM_LAUNCH(KER, DT, NT, WG, TPR, 1, grid, stream, args); \
    else if ((cpt) == 2) GMI_NORM_LAUNCH(KER, DT, NT, WG, TPR, 2, grid, stream, args); \
    else GMI_NORM_LAUNCH(KER, DT, NT, WG, TPR, 4, grid, stream, args);            \
  } while (0)
#define GMI_NORM_TPR(KER, DT, NT, s, grid, stream, args)                                              \
  do {                                                                                                \
    if ((s).tpr == 64) GMI_NORM_CPT(KER, DT, NT, 256, 64, (s).cpt, grid, stream, args);               \
    else if ((s).tpr == 128) GMI_NORM_LAUNCH(KER, DT, NT, 256, 128, 4, grid, stream, args);           \
    else if ((s).tpr == 256) GMI_NORM_CPT(KER, DT, NT, 256, 256, (s).cpt, grid, stream, args);        \
    else if ((s).cpt <= 4) GMI_NORM_LAUNCH(KER, DT, NT, 512, 512, 4, grid, stream, args);             \
    else GMI_NORM_LAUNCH(KER, DT, NT, 512, 512, 8, grid, stream, args);                               \
  } while (0)
#define GMI_NORM_DISPATCH(KER, DT, s, grid, stream, args)                    \
  do {                                                                       \
    if ((s).nt) GMI_NORM_TPR(KER, DT, true, s, grid, stream, args);          \
    else GMI_NORM_TPR(KER, DT, false, s, grid, stream, args);                \
  } while (0)
static int norm_teams(const NormShape& s) { return s.tpr < 256 ? 256 / s.tpr : 1; }

hipError_t launch_rmsnorm_quant(const NormLaunch& all, int dtype, hipStream_t stream) {
  const NormShape s = norm_shape(all.rows, all.K);
  const int teams = norm_teams(s);
  constexpr int64_t most = int64_t(1) << 22;  // a launch's threads stay below 2^32
  NormLaunch a = all;
  for (int64_t row = 0; row < all.rows; row += most) {
    a.rows = all.rows - row < most ? all.rows - row : most;
    a.x = all.x + row * all.ldx;
    if (all.residual) a.residual = all.residual + row * all.ldr;
    if (all.h) a.h = all.h + row * all.ldh;
    if (all.y) a.y = all.y + row * all.ldy;
    if (all.q) {
      a.q = all.q + row * all.ldq;
      a.scales = all.scales + row * all.lds;
    }
    const unsigned grid = (unsigned)((a.rows + teams - 1) / teams);
    if (dtype == DT_F16)
      GMI_NORM_DISPATCH(k_rmsnorm_quant, DT_F16, s, grid, stream, a);
    else
      GMI_NORM_DISPATCH(k_rmsnorm_quant, DT_BF16, s, grid, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// workgroups of the backward: resident ones only, each adds one partial row
int norm_bwd_parts(int64_t rows, int K) {
  const NormShape s = norm_shape(rows, K);
  const int teams = norm_teams(s);
  const int64_t need = (rows + teams - 1) / teams, most = 2 * (int64_t)device_cu_count();
  return (int)(need < most ? need : most);
}

hipError_t launch_rmsnorm_bwd(const NormBwdLaunch& a, int dtype, float* dweight, hipStream_t stream) {
  const NormShape s = norm_shape(a.rows, a.K);
  const int grid = norm_bwd_parts(a.rows, a.K);
  if (grid == 0) {  // no rows: only the zero gradient of the weight
    hipLaunchKernelGGL(k_norm_dweight, dim3((a.K + 31) / 32), dim3(256), 0, stream, a.partial, 0, a.K, dweight);
    return hipGetLastError();
  }
  if (dtype == DT_F16)
    GMI_NORM_DISPATCH(k_rmsnorm_bwd, DT_F16, s, grid, stream, a);
  else
    GMI_NORM_DISPATCH(k_rmsnorm_bwd, DT_BF16, s, grid, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dweight) return e;
  hipLaunchKernelGGL(k_norm_dweight, dim3((a.K + 31) / 32), dim3(256), 0, stream, a.partial, grid, a.K, dweight);
  return hipGetLastError();
}

}  // namespace gmi
