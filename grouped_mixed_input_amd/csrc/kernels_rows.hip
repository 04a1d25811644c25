// kernels_rows.hip -- what a mixture-of-experts layer does to rows between its
// products: tokens to the rows of their experts and back with weights, the
// gated activation, and the gradients of these.
//
//   permute        out[slot_row[t][i]] = x[t]
//   unpermute      out[t] = add[t] + sum_i w[t][i] rows[slot_row[t][i]]
//   its gradient   drows[slot_row[t][i]] = w[t][i] dout[t],  dw[t][i] = <dout[t], rows[slot_row[t][i]]>
//   gate           v = g s u,  s = 1 / (1 + e^-g)
//   its gradient   dg = d u s (1 + g (1 - s)),  du = d g s
//
// A row number outside [0, rows) is a slot without an expert: nothing is read
// or written for it.  All are bound by memory: each input is read once and
// each output written once, 16 bytes a lane.  The walk is by token, so a
// token's row (or gradient) is fetched once for its k experts, and the sum over
// k has a fixed order.
#include "gmi_device.hpp"
#include "gmi_internal.hpp"
#include "gmi_rows.hpp"

namespace gmi {

// A wave serves part `part` of 2^shift of a token's columns: chunk
// 64 (part + j 2^shift) + lane for j = 0, 1, ...
struct TokenPart {
  int64_t t;
  int first, stride;  // chunks
};
__device__ __forceinline__ TokenPart token_part(int64_t w, int shift) {
  return {w >> shift, (int)(w & ((1 << shift) - 1)) * 64, 64 << shift};
}
// lane i: the row of the token's slot i, -1 without one
__device__ __forceinline__ int slot_of_lane(const int32_t* slot_row, int64_t t, int k, int rows, int lane) {
  const int r = lane < k ? slot_row[t * k + lane] : -1;
  return r < rows ? r : -1;
}

__global__ __launch_bounds__(256) void k_permute(PermuteLaunch a) {
  constexpr int CH = 4;
  const int lane = threadIdx.x & 63;
  for (int64_t w = (int64_t)blockIdx.x * 4 + wave_id(); w < a.waves; w += (int64_t)gridDim.x * 4) {
    const TokenPart p = token_part(w, a.shift);
    const int at = slot_of_lane(a.slot_row, p.t, a.k, a.rows, lane);
    const char* x = a.x + p.t * a.ldx;
    for (int c0 = p.first; c0 < a.chunks; c0 += CH * p.stride) {
      u32x4 v[CH];
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const int c = c0 + j * p.stride + lane;
        v[j] = c < a.chunks ? *(const u32x4*)(x + (int64_t)c * 16) : u32x4{};
      }
      for (int i = 0; i < a.k; ++i) {
        const int r = __builtin_amdgcn_readlane(at, i);
        if (r < 0) continue;
        char* o = a.out + r * a.ldo;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          const int c = c0 + j * p.stride + lane;
          if (c < a.chunks) *(u32x4*)(o + (int64_t)c * 16) = v[j];
        }
      }
    }
    for (int b = p.first + lane; b < a.blocks; b += p.stride) {
      const float s = a.x_scales[p.t * a.ldxs + b];
      for (int i = 0; i < a.k; ++i) {
        const int r = __builtin_amdgcn_readlane(at, i);
        if (r >= 0) a.out_scales[r * a.ldos + b] = s;
      }
    }
  }
}

// KT >= k slots a token: their rows are asked for together, CH chunks at a time
template <int DT, int KT>
__global__ __launch_bounds__(256) void k_unpermute(UnpermuteLaunch a) {
  constexpr int CH = KT >= 16 ? 1 : KT >= 8 ? 2 : 4;
  const int lane = threadIdx.x & 63;
  for (int64_t w = (int64_t)blockIdx.x * 4 + wave_id(); w < a.waves; w += (int64_t)gridDim.x * 4) {
    const TokenPart p = token_part(w, a.shift);
    const int at = slot_of_lane(a.slot_row, p.t, a.k, a.rows, lane);
    const float wt = a.weights && lane < a.k ? a.weights[p.t * a.k + lane] : 1.0f;
    int row[KT];
    float wi[KT];
#pragma unroll
    for (int i = 0; i < KT; ++i) {
      row[i] = __builtin_amdgcn_readlane(at, i);
      wi[i] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, wt), i));
    }
    for (int c0 = p.first; c0 < a.chunks; c0 += CH * p.stride) {
      u32x4 v[CH][KT], av[CH];
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const int c = c0 + j * p.stride + lane;
        const bool in = c < a.chunks;
#pragma unroll
        for (int i = 0; i < KT; ++i)
          v[j][i] = in && row[i] >= 0 ? *(const u32x4*)(a.y + row[i] * a.ldy + (int64_t)c * 8) : u32x4{};
        av[j] = in && a.add ? *(const u32x4*)(a.add + p.t * a.lda + (int64_t)c * 8) : u32x4{};
      }
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const int c = c0 + j * p.stride + lane;
        float acc[8], f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
#pragma unroll
        for (int i = 0; i < KT; ++i) {
          if (row[i] < 0) continue;  // its weight may be anything
          unpack8<DT>(v[j][i], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] = __builtin_fmaf(wi[i], f[e], acc[e]);
        }
        if (a.add) {
          unpack8<DT>(av[j], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] += f[e];
        }
        if (c < a.chunks) *(u32x4*)(a.out + p.t * a.ldo + (int64_t)c * 8) = pack8<DT>(acc);
      }
    }
  }
}

// WPT waves a token (1, or 4 where tokens are few).  With Q the rows leave as
// codes: the largest magnitude of w d over a block is |w| times that of d, to
// the bit (rounding keeps the order), so it is found once for all k.
template <int DT, bool Q, int KT, int WPT>
__global__ __launch_bounds__(256) void k_unpermute_bwd(UnpermuteBwdLaunch a) {
  __shared__ float red[4][KT];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int64_t step = (int64_t)gridDim.x * (4 / WPT);
  // (with four waves a token every wave of the workgroup makes the same turns, so all meet the barriers)
  for (int64_t t = (int64_t)blockIdx.x * (4 / WPT) + (WPT == 1 ? wave : 0); t < a.T; t += step) {
    const int at = slot_of_lane(a.slot_row, t, a.k, a.rows, lane);
    const float wt = a.weights && lane < a.k ? a.weights[t * a.k + lane] : 1.0f;
    int row[KT];
    float wi[KT], dot[KT];
#pragma unroll
    for (int i = 0; i < KT; ++i) {
      row[i] = __builtin_amdgcn_readlane(at, i);
      wi[i] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, wt), i));
      dot[i] = 0.0f;
    }
    for (int c0 = WPT == 1 ? 0 : wave * 64; c0 < a.chunks; c0 += 64 * WPT) {
      const int c = c0 + lane;
      const bool in = c < a.chunks;
      u32x4 v[KT];
      const u32x4 dv = in ? *(const u32x4*)(a.dout + t * a.ldd + (int64_t)c * 8) : u32x4{};
#pragma unroll
      for (int i = 0; i < KT; ++i)
        v[i] = in && a.y && row[i] >= 0 ? *(const u32x4*)(a.y + row[i] * a.ldy + (int64_t)c * 8) : u32x4{};
      float d[8], amax = 0.0f;
      unpack8<DT>(dv, d);
      if constexpr (Q) {
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(d[e]));
        amax = max16(amax);
      }
#pragma unroll
      for (int i = 0; i < KT; ++i) {
        if (row[i] < 0) continue;
        float f[8], g[8];
        unpack8<DT>(v[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dot[i] = __builtin_fmaf(d[e], f[e], dot[i]);
          g[e] = wi[i] * d[e];
        }
        if (!in) continue;
        if constexpr (Q) {
          const float s = block_scale(fabsf(wi[i]) * amax);
          *(u32x2*)(a.q + row[i] * a.ldq + (int64_t)c * 8) = codes8(g, s);
          if (c % 16 == 0) a.scales[row[i] * a.lds + c / 16] = s;
        } else {
          *(u32x4*)(a.drows + row[i] * a.lddr + (int64_t)c * 8) = pack8<DT>(g);
        }
      }
    }
    if (!a.dweights) continue;
    float mine = 0.0f;  // lane i: slot i
#pragma unroll
    for (int i = 0; i < KT; ++i) {
      const float s = sum64(dot[i]);
      if constexpr (WPT == 1)
        mine = lane == i ? s : mine;
      else if (lane == 0)
        red[wave][i] = s;
    }
    if constexpr (WPT > 1) {
      __syncthreads();
      if (lane < KT) mine = red[0][lane] + red[1][lane] + red[2][lane] + red[3][lane];
      __syncthreads();
    }
    if (lane < a.k && (WPT == 1 || wave == 0)) a.dweights[t * a.k + lane] = mine;
  }
}

// s = 1 / (1 + e^-g) and 1 - s, each to a few last bits: from e^-|g|, which
// cannot overflow, and without a difference
__device__ __forceinline__ void sigmoid2(float g, float& s, float& rest) {
  const float e = exp_le0(-fabsf(g));
  const float big = __builtin_amdgcn_rcpf(1.0f + e), small = e * big;
  s = g < 0.0f ? small : big;
  rest = g < 0.0f ? big : small;
}

// 16 lanes serve one block of 128 columns of a row; two blocks in flight.
template <int DT>
__global__ __launch_bounds__(256) void k_swiglu(SwigluLaunch a) {
  constexpr int U = 2;
  const int group = threadIdx.x >> 4, l16 = threadIdx.x & 15;
  const int nb = (a.N + 127) / 128, chunks = a.N / 8;
  const int64_t used = a.live ? max((int64_t)0, min(a.rows, (int64_t)*a.live - a.row0)) : a.rows;
  const uint32_t units = (uint32_t)(used * nb);
  u32x4 gv[U], uv[U];
  int64_t row[U];
  int c[U];
  bool in[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const uint32_t unit = (blockIdx.x * U + j) * 16 + group;
    row[j] = unit / (uint32_t)nb;
    c[j] = (int)(unit - (uint32_t)row[j] * nb) * 16 + l16;
    in[j] = unit < units && c[j] < chunks;
    const uint16_t* p = a.a + row[j] * a.lda + (int64_t)c[j] * 8;
    gv[j] = in[j] ? *(const u32x4*)p : u32x4{};
    uv[j] = in[j] ? *(const u32x4*)(p + a.N) : u32x4{};
  }
#pragma unroll
  for (int j = 0; j < U; ++j) {
    float g[8], u[8], amax = 0.0f;
    unpack8<DT>(gv[j], g);
    unpack8<DT>(uv[j], u);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float s, rest;
      sigmoid2(g[e], s, rest);
      g[e] = g[e] * s * u[e];
      amax = fmaxf(amax, fabsf(g[e]));
    }
    if (a.y && in[j]) *(u32x4*)(a.y + row[j] * a.ldy + (int64_t)c[j] * 8) = pack8<DT>(g);
    if (!a.q) continue;
    const float s = block_scale(max16(amax));
    if (in[j]) {
      *(u32x2*)(a.q + row[j] * a.ldq + (int64_t)c[j] * 8) = codes8(g, s);
      if (l16 == 0) a.scales[row[j] * a.lds + c[j] / 16] = s;
    }
  }
}

// PAIR: a thread makes the same columns of both halves of da, whose blocks of
// 128 do not mix (or which leaves in 16 bits).  Otherwise a block may hold the
// gate's last columns and the up projection's first: a thread makes eight
// columns of da, and the inputs are read twice.
template <int DT, bool Q, bool PAIR>
__global__ __launch_bounds__(256) void k_swiglu_bwd(SwigluLaunch a) {
  const int group = threadIdx.x >> 4, l16 = threadIdx.x & 15;
  const int cols = PAIR ? a.N : 2 * a.N;
  const int nb = (cols + 127) / 128, chunks = cols / 8, half = a.N / 8;
  const int64_t used = a.live ? max((int64_t)0, min(a.rows, (int64_t)*a.live - a.row0)) : a.rows;
  const uint32_t unit = blockIdx.x * 16 + group;
  const int64_t row = unit / (uint32_t)nb;
  const int c = (int)(unit - (uint32_t)row * nb) * 16 + l16;
  const bool in = row < used && c < chunks;
  const bool up = !PAIR && c >= half;
  const int cc = up ? c - half : c;
  const uint16_t* p = a.a + row * a.lda + (int64_t)cc * 8;
  float g[8], u[8], d[8], du[8];
  const u32x4 gv = in ? *(const u32x4*)p : u32x4{}, uv = in ? *(const u32x4*)(p + a.N) : u32x4{},
              dv = in ? *(const u32x4*)(a.dact + row * a.ldd + (int64_t)cc * 8) : u32x4{};
  unpack8<DT>(gv, g);
  unpack8<DT>(uv, u);
  unpack8<DT>(dv, d);
  float mg = 0.0f, mu = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float s, rest;
    sigmoid2(g[e], s, rest);
    du[e] = d[e] * g[e] * s;
    g[e] = d[e] * u[e] * s * __builtin_fmaf(g[e], rest, 1.0f);
    if (up) g[e] = du[e];
    mg = fmaxf(mg, fabsf(g[e]));
    mu = fmaxf(mu, fabsf(du[e]));
  }
  if constexpr (!Q) {
    if (!in) return;
    *(u32x4*)(a.y + row * a.ldy + (int64_t)c * 8) = pack8<DT>(g);
    *(u32x4*)(a.y + row * a.ldy + a.N + (int64_t)c * 8) = pack8<DT>(du);
  } else {
    const float sg = block_scale(max16(mg));
    const float su = PAIR ? block_scale(max16(mu)) : 0.0f;
    if (!in) return;
    *(u32x2*)(a.q + row * a.ldq + (int64_t)c * 8) = codes8(g, sg);
    if (l16 == 0) a.scales[row * a.lds + c / 16] = sg;
    if constexpr (PAIR) {
      *(u32x2*)(a.q + row * a.ldq + a.N + (int64_t)c * 8) = codes8(du, su);
      if (l16 == 0) a.scales[row * a.lds + a.N / 128 + c / 16] = su;
    }
  }
}

// Waves a token, as a power of two: one where tokens fill the device, up to one
// per 64 chunks where they do not.
static int part_shift(int64_t T, int chunks) {
  int s = 0;
  while (64 << s < chunks && T << s < 8 * (int64_t)device_cu_count()) ++s;
  return s;
}
// workgroups of four waves; a kernel's waves walk on past 2^20 of them
static unsigned wave_grid(int64_t waves) {
  const int64_t need = (waves + 3) / 4, most = int64_t(1) << 20;
  return (unsigned)(need < most ? need : most);
}

hipError_t launch_permute(const PermuteLaunch& args, hipStream_t stream) {
  PermuteLaunch a = args;
  a.shift = part_shift(a.T, a.chunks);
  a.waves = a.T << a.shift;
  hipLaunchKernelGGL(k_permute, dim3(wave_grid(a.waves)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

#define GMI_ROWS_K(KER, k, grid, stream, a, ...)                                                              \
  do {                                                                                                        \
    if ((k) <= 1) hipLaunchKernelGGL((KER(1)), dim3(grid), dim3(256), 0, stream, a);                          \
    else if ((k) <= 2) hipLaunchKernelGGL((KER(2)), dim3(grid), dim3(256), 0, stream, a);                     \
    else if ((k) <= 4) hipLaunchKernelGGL((KER(4)), dim3(grid), dim3(256), 0, stream, a);                     \
    else if ((k) <= 8) hipLaunchKernelGGL((KER(8)), dim3(grid), dim3(256), 0, stream, a);                     \
    else hipLaunchKernelGGL((KER(16)), dim3(grid), dim3(256), 0, stream, a);                                  \
  } while (0)

hipError_t launch_unpermute(const UnpermuteLaunch& args, int dtype, hipStream_t stream) {
  UnpermuteLaunch a = args;
  a.shift = part_shift(a.T, a.chunks);
  a.waves = a.T << a.shift;
  const unsigned grid = wave_grid(a.waves);
#define GMI_F16_K(KT) k_unpermute<DT_F16, KT>
#define GMI_BF16_K(KT) k_unpermute<DT_BF16, KT>
  if (dtype == DT_F16)
    GMI_ROWS_K(GMI_F16_K, a.k, grid, stream, a);
  else
    GMI_ROWS_K(GMI_BF16_K, a.k, grid, stream, a);
#undef GMI_F16_K
#undef GMI_BF16_K
  return hipGetLastError();
}

template <int DT, bool Q, int WPT>
static void launch_unpermute_bwd_as(const UnpermuteBwdLaunch& a, unsigned grid, hipStream_t stream) {
#define GMI_BWD_K(KT) k_unpermute_bwd<DT, Q, KT, WPT>
  GMI_ROWS_K(GMI_BWD_K, a.k, grid, stream, a);
#undef GMI_BWD_K
}
template <int DT, bool Q>
static void launch_unpermute_bwd_by(const UnpermuteBwdLaunch& a, hipStream_t stream) {
  // four waves a token where one each would leave SIMDs without a wave
  if (a.chunks > 64 && a.T < 8 * (int64_t)device_cu_count())
    launch_unpermute_bwd_as<DT, Q, 4>(a, wave_grid(4 * a.T), stream);
  else
    launch_unpermute_bwd_as<DT, Q, 1>(a, wave_grid(a.T), stream);
}
hipError_t launch_unpermute_bwd(const UnpermuteBwdLaunch& a, int dtype, hipStream_t stream) {
  if (dtype == DT_F16) {
    if (a.q) launch_unpermute_bwd_by<DT_F16, true>(a, stream);
    else launch_unpermute_bwd_by<DT_F16, false>(a, stream);
  } else {
    if (a.q) launch_unpermute_bwd_by<DT_BF16, true>(a, stream);
    else launch_unpermute_bwd_by<DT_BF16, false>(a, stream);
  }
  return hipGetLastError();
}

// rows of one launch: block numbers and threads stay below 2^32
static int64_t swiglu_rows(int cols) { return (int64_t(1) << 27) / ((cols + 127) / 128); }
static SwigluLaunch swiglu_from(const SwigluLaunch& all, int64_t row, int64_t most) {
  SwigluLaunch a = all;
  a.row0 = row;
  a.rows = all.rows - row < most ? all.rows - row : most;
  a.a = all.a + row * all.lda;
  if (all.dact) a.dact = all.dact + row * all.ldd;
  if (all.y) a.y = all.y + row * all.ldy;
  if (all.q) {
    a.q = all.q + row * all.ldq;
    a.scales = all.scales + row * all.lds;
  }
  return a;
}

hipError_t launch_swiglu(const SwigluLaunch& all, int dtype, hipStream_t stream) {
  const int64_t most = swiglu_rows(all.N);
  for (int64_t row = 0; row < all.rows; row += most) {
    const SwigluLaunch a = swiglu_from(all, row, most);
    const unsigned grid = (unsigned)((a.rows * ((a.N + 127) / 128) + 31) / 32);
    if (dtype == DT_F16)
      hipLaunchKernelGGL(k_swiglu<DT_F16>, dim3(grid), dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL(k_swiglu<DT_BF16>, dim3(grid), dim3(256), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT>
static void launch_swiglu_bwd_as(const SwigluLaunch& a, hipStream_t stream) {
  const bool pair = !a.q || a.N % 128 == 0;
  const int64_t nb = ((pair ? a.N : 2 * (int64_t)a.N) + 127) / 128;
  const unsigned grid = (unsigned)((a.rows * nb + 15) / 16);
  if (!a.q)
    hipLaunchKernelGGL((k_swiglu_bwd<DT, false, true>), dim3(grid), dim3(256), 0, stream, a);
  else if (pair)
    hipLaunchKernelGGL((k_swiglu_bwd<DT, true, true>), dim3(grid), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((k_swiglu_bwd<DT, true, false>), dim3(grid), dim3(256), 0, stream, a);
}
hipError_t launch_swiglu_bwd(const SwigluLaunch& all, int dtype, hipStream_t stream) {
  const int64_t most = swiglu_rows(2 * all.N);
  for (int64_t row = 0; row < all.rows; row += most) {
    const SwigluLaunch a = swiglu_from(all, row, most);
    if (dtype == DT_F16)
      launch_swiglu_bwd_as<DT_F16>(a, stream);
    else
      launch_swiglu_bwd_as<DT_BF16>(a, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace gmi
