// kernels_lora.hip -- low-rank adapters of many requests beside one dense
// product: Y[m] = base[m] + s_a (X[m] A_a^T) B_a^T with the row's own adapter a.
//
// Two launches: T = X A^T over runs of K (fp32 partial sums), then Y from T.
// Both walk tiles of 64 rows in the order of the call.  Neighbouring rows of
// one adapter form a run, and a run is the unit of work: its rows are the
// columns of 16 x 16 x 32 matrix instructions, 16 at a time, and a lane past
// the run's end repeats its last row and is not written, so no row's values
// (an infinity, a NaN) can reach another's.  Sorted rows make long runs; rows
// in any order give the same results from shorter ones.
#include <algorithm>

#include "gmi_device.hpp"
#include "gmi_internal.hpp"

namespace gmi {

constexpr int LO_ROWS = 64;  // rows a tile: a wave's lanes hold their row and adapter numbers

// The tile's rows: lane l holds row and adapter of position 64 tile + l (-1:
// no adapter, -2: no row), and `starts` marks the positions where a run begins.
struct LoraTile {
  int row, id;
  uint64_t starts;
};
__device__ __forceinline__ LoraTile lora_tile(const LoraLaunch& a, int tile) {
  const int lane = threadIdx.x & 63, pos = tile * LO_ROWS + lane;
  LoraTile t;
  t.row = pos < a.M ? a.order ? a.order[pos] : pos : -1;
  if ((uint32_t)t.row >= (uint32_t)a.M) t.row = -1;
  t.id = t.row >= 0 ? a.index[t.row] : -2;
  if (t.row >= 0 && (uint32_t)t.id >= (uint32_t)a.adapters) t.id = -1;
  const int prev = __shfl_up(t.id, 1);
  t.starts = __ballot(lane == 0 || t.id != prev);
  return t;
}
__device__ __forceinline__ int run_end(uint64_t starts, int p0) {
  const uint64_t later = p0 < 63 ? starts >> (p0 + 1) : 0;
  return later ? p0 + 1 + __builtin_ctzll(later) : LO_ROWS;
}

// 16 bytes, or zeros
__device__ __forceinline__ u32x4 load_if(const uint16_t* p, bool in) { return in ? *(const u32x4*)p : u32x4{}; }

// T of one run, its rows p0 .. p1 - 1 of the tile, over k0 .. k1 - 1.  The four
// waves take 64 k in turn, two instructions each way; their sums meet in LDS,
// a rank tile at a time, and are added in wave order.
template <int DT, int RT, int NS>
__device__ __forceinline__ void lora_down(const LoraLaunch& a, const LoraTile& t, int tile, int p0, int p1, int k0,
                                          int k1, float* part, f32x4 (*red)[4][64]) {
  const int lane = threadIdx.x & 63, wave = wave_id(), i16 = lane & 15, kg = lane >> 4;
  const int id = __builtin_amdgcn_readlane(t.id, p0);
  const uint16_t* xp[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) xp[s] = a.X + __shfl(t.row, min(p0 + 16 * s + i16, p1 - 1)) * a.ldx + kg * 8;
  const uint16_t* ap[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) ap[r] = a.A + id * a.a_stride + min(16 * r + i16, a.rank - 1) * a.lda + kg * 8;
  f32x4 acc[RT][NS];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int s = 0; s < NS; ++s) acc[r][s] = f32x4{};
  for (int k = k0 + 64 * wave; k < k1; k += 256) {
    u32x4 xv[2][NS], av[2][RT];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = k + 32 * h + kg * 8 < k1;
#pragma unroll
      for (int s = 0; s < NS; ++s) xv[h][s] = load_if(xp[s] + k + 32 * h, in);
#pragma unroll
      for (int r = 0; r < RT; ++r) av[h][r] = load_if(ap[r] + k + 32 * h, in);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int s = 0; s < NS; ++s) acc[r][s] = mfma16<DT>(av[h][r], xv[h][s], acc[r][s]);
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    __syncthreads();
#pragma unroll
    for (int s = 0; s < NS; ++s) red[wave][s][lane] = acc[r][s];
    __syncthreads();
    if (wave < NS) {
      const f32x4 v = red[0][wave][lane] + red[1][wave][lane] + red[2][wave][lane] + red[3][wave][lane];
      const int p = p0 + 16 * wave + i16, col = 16 * r + 4 * kg;
      if (p < p1 && col < a.rank) *(f32x4*)(part + ((int64_t)tile * LO_ROWS + p) * a.rank + col) = v;
    }
  }
}

// grid: tiles x run slots x runs of K
template <int DT, int RT>
__global__ __launch_bounds__(256) void k_lora_down(LoraLaunch a, int k_per) {
  __shared__ f32x4 red[4][4][64];
  const int tile = blockIdx.x;
  const LoraTile t = lora_tile(a, tile);
  uint64_t runs = t.starts & __ballot(t.id >= 0);
  const int k0 = blockIdx.z * k_per, k1 = min(a.K, k0 + k_per);
  float* part = a.part + (int64_t)blockIdx.z * a.M * a.rank;
  for (int n = 0; runs; ++n, runs &= runs - 1) {
    if (n % (int)gridDim.y != (int)blockIdx.y) continue;
    const int p0 = __builtin_ctzll(runs), p1 = run_end(t.starts, p0);
    if (p1 - p0 <= 16)
      lora_down<DT, RT, 1>(a, t, tile, p0, p1, k0, k1, part, red);
    else if (p1 - p0 <= 32)
      lora_down<DT, RT, 2>(a, t, tile, p0, p1, k0, k1, part, red);
    else
      lora_down<DT, RT, 4>(a, t, tile, p0, p1, k0, k1, part, red);
  }
}

// T as operand of the second product.  A 16-bit T would cost the result as much
// again as its own rounding, so T goes in as two terms, t = hi + lo, whose
// products with B are summed: what is lost is 2^-17 (bf16) or 2^-22 (fp16) of
// t.  fp16 cannot hold every t: a row is scaled by the power of two that brings
// its largest to [1, 2), and `f` takes it back.  Up to rank 16 both terms fit
// one instruction (k 0..15 hi, 16..31 lo, against B twice).
template <int DT, int RS, bool ONE>
struct LoraT {
  u32x4 hi[RS], lo[ONE ? 1 : RS];
  float f;
};
__device__ __forceinline__ float max4(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
template <int DT, int RS, bool ONE>
__device__ __forceinline__ void load_t(const LoraLaunch& a, int64_t pos, bool in, LoraT<DT, RS, ONE>& t) {
  const int lane = threadIdx.x & 63, kg = lane >> 4;
  float v[RS][8];
#pragma unroll
  for (int r = 0; r < RS; ++r) {
    const int col = ONE ? 8 * (kg & 1) : 32 * r + 8 * kg;
    f32x4 s0{}, s1{};
    if (in && col < a.rank) {
      const float* p = a.part + pos * a.rank + col;
#pragma unroll 4
      for (int q = 0; q < a.splits; ++q) {
        s0 += *(const f32x4*)p;
        s1 += *(const f32x4*)(p + 4);
        p += (int64_t)a.M * a.rank;
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[r][e] = s0[e];
      v[r][4 + e] = s1[e];
    }
  }
  t.f = 1.0f;
  if constexpr (DT == DT_F16) {
    float m = 0.0f;
#pragma unroll
    for (int r = 0; r < RS; ++r)
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[r][e]));
    m = max4(m);
    // 2^(exponent of m), inside the normal range with its reciprocal; rows that
    // hold an infinity stay as they are
    const uint32_t ex = min(max(__builtin_bit_cast(uint32_t, m) >> 23, 2u), 252u);
    const bool scale = m < __builtin_inff();
    t.f = scale ? __builtin_bit_cast(float, ex << 23) : 1.0f;
    const float inv = scale ? __builtin_bit_cast(float, (254u - ex) << 23) : 1.0f;
#pragma unroll
    for (int r = 0; r < RS; ++r)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[r][e] *= inv;
  }
#pragma unroll
  for (int r = 0; r < RS; ++r) {
    u32x4 hi, lo;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      hi[e] = pack2<DT>(v[r][2 * e], v[r][2 * e + 1]);
      const float h0 = from_bits<DT>(hi[e] & 0xffffu), h1 = from_bits<DT>(hi[e] >> 16);
      // (no rest beside an infinity)
      lo[e] = pack2<DT>(fabsf(h0) < __builtin_inff() ? v[r][2 * e] - h0 : 0.0f,
                        fabsf(h1) < __builtin_inff() ? v[r][2 * e + 1] - h1 : 0.0f);
    }
    if constexpr (ONE) {
      t.hi[0] = kg < 2 ? hi : lo;
    } else {
      t.hi[r] = hi;
      t.lo[r] = lo;
    }
  }
}

// Y of one run: a wave makes 64 columns of up to 64 rows at a time.  B is the
// instruction's first operand, its rows dealt so that a lane ends with 16
// neighbouring columns of one row of Y: row i of instruction m is column
// 16 (i / 4) + 4 m + i % 4, and a lane's results are columns 16 (l / 16) + 4 m + j.
template <int DT, int RS, bool ONE, int NS>
__device__ __forceinline__ void lora_up(const LoraLaunch& a, const LoraTile& t, int tile, int p0, int p1, int n0,
                                        int n1) {
  const int lane = threadIdx.x & 63, i16 = lane & 15, kg = lane >> 4;
  const int id = __builtin_amdgcn_readlane(t.id, p0);
  const uint16_t* b = a.B + id * a.b_stride;
  const float scale = a.scales ? a.scales[id] : 1.0f;
  LoraT<DT, RS, ONE> tv[NS];
  int64_t row[NS];
  bool in[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int p = p0 + 16 * s + i16;
    in[s] = p < p1;
    row[s] = __shfl(t.row, min(p, p1 - 1));
    load_t<DT, RS, ONE>(a, (int64_t)tile * LO_ROWS + p, in[s], tv[s]);
    tv[s].f *= scale;
  }
  for (int c0 = n0 + 64 * wave_id(); c0 < n1; c0 += 256) {
    const int col = c0 + 16 * kg;
    u32x4 bv[4][RS], base[NS][2];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int n = c0 + 16 * (i16 >> 2) + 4 * m + (i16 & 3);
#pragma unroll
      for (int r = 0; r < RS; ++r) {
        const int k = ONE ? 8 * (kg & 1) : 32 * r + 8 * kg;
        bv[m][r] = load_if(b + n * a.ldb + k, n < a.N && k < a.rank);
      }
    }
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        base[s][h] = load_if(a.base + row[s] * a.ldbase + col + 8 * h, a.base && in[s] && col + 8 * h < a.N);
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      f32x4 acc[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        acc[m] = f32x4{};
#pragma unroll
        for (int r = 0; r < RS; ++r) {
          acc[m] = mfma16<DT>(bv[m][r], tv[s].hi[r], acc[m]);
          if constexpr (!ONE) acc[m] = mfma16<DT>(bv[m][r], tv[s].lo[r], acc[m]);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f32x4 v = acc[2 * h + e / 2];
          o[e] = pack2<DT>(__builtin_fmaf(tv[s].f, v[2 * (e % 2)], from_bits<DT>(base[s][h][e] & 0xffffu)),
                           __builtin_fmaf(tv[s].f, v[2 * (e % 2) + 1], from_bits<DT>(base[s][h][e] >> 16)));
        }
        if (in[s] && col + 8 * h < a.N) *(u32x4*)(a.Y + row[s] * a.ldy + col + 8 * h) = o;
      }
    }
  }
}

// rows without an adapter: base, or zeros
__device__ __forceinline__ void lora_copy(const LoraLaunch& a, const LoraTile& t, int p0, int p1, int n0, int n1) {
  if (a.base == a.Y) return;
  const int lane = threadIdx.x & 63;
  for (int p = p0 + wave_id(); p < p1; p += 4) {
    const int64_t row = __builtin_amdgcn_readlane(t.row, p);
    for (int c = n0 + 8 * lane; c < n1; c += 512)
      *(u32x4*)(a.Y + row * a.ldy + c) = load_if(a.base + row * a.ldbase + c, a.base != nullptr);
  }
}

// grid: tiles x run slots x column blocks
template <int DT, int RS, bool ONE>
__global__ __launch_bounds__(256) void k_lora_up(LoraLaunch a, int n_per) {
  const int tile = blockIdx.x;
  const LoraTile t = lora_tile(a, tile);
  uint64_t runs = t.starts & __ballot(t.id > -2);
  const int n0 = blockIdx.z * n_per, n1 = min(a.N, n0 + n_per);
  for (int n = 0; runs; ++n, runs &= runs - 1) {
    if (n % (int)gridDim.y != (int)blockIdx.y) continue;
    const int p0 = __builtin_ctzll(runs), p1 = run_end(t.starts, p0);
    if (__builtin_amdgcn_readlane(t.id, p0) < 0)
      lora_copy(a, t, p0, p1, n0, n1);
    else if (p1 - p0 <= 16)
      lora_up<DT, RS, ONE, 1>(a, t, tile, p0, p1, n0, n1);
    else if (p1 - p0 <= 32)
      lora_up<DT, RS, ONE, 2>(a, t, tile, p0, p1, n0, n1);
    else
      lora_up<DT, RS, ONE, 4>(a, t, tile, p0, p1, n0, n1);
  }
}

// Workgroups for the runs of a tile: as many as runs may be while tiles are
// few; long batches have long runs.
static int lora_slots(int M) {
  const int tiles = (M + LO_ROWS - 1) / LO_ROWS;
  return std::max(1, std::min(std::min(M, LO_ROWS), LO_ROWS / tiles));
}
// Runs of K: two workgroups a CU for the tiles, none below 256 k.
static int lora_splits(int M, int K) {
  const int tiles = (M + LO_ROWS - 1) / LO_ROWS;
  return std::max(1, std::min({K / 256, 512 / tiles, 16}));
}
size_t lora_workspace(int M, int K, int rank) { return (size_t)lora_splits(M, K) * M * rank * sizeof(float); }

template <int DT>
static hipError_t launch_lora_as(const LoraLaunch& args, hipStream_t stream) {
  LoraLaunch a = args;
  a.splits = lora_splits(a.M, a.K);
  const int tiles = (a.M + LO_ROWS - 1) / LO_ROWS, slots = lora_slots(a.M);
  const int k_per = ((a.K + a.splits - 1) / a.splits + 63) / 64 * 64;
  const dim3 down(tiles, slots, a.splits);
  if (a.rank <= 16) hipLaunchKernelGGL((k_lora_down<DT, 1>), down, dim3(256), 0, stream, a, k_per);
  else if (a.rank <= 32) hipLaunchKernelGGL((k_lora_down<DT, 2>), down, dim3(256), 0, stream, a, k_per);
  else if (a.rank <= 64) hipLaunchKernelGGL((k_lora_down<DT, 4>), down, dim3(256), 0, stream, a, k_per);
  else hipLaunchKernelGGL((k_lora_down<DT, 8>), down, dim3(256), 0, stream, a, k_per);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // columns: 256 a workgroup, more where that gives two workgroups a CU
  const int64_t blocks = (a.N + 255) / 256;
  const int64_t want = std::min<int64_t>(blocks, std::max<int64_t>(1, std::min<int64_t>(512 / tiles, 65535)));
  const int n_per = (int)((blocks + want - 1) / want * 256);
  const dim3 up(tiles, slots, (unsigned)((a.N + n_per - 1) / n_per));
  if (a.rank <= 16) hipLaunchKernelGGL((k_lora_up<DT, 1, true>), up, dim3(256), 0, stream, a, n_per);
  else if (a.rank <= 32) hipLaunchKernelGGL((k_lora_up<DT, 1, false>), up, dim3(256), 0, stream, a, n_per);
  else if (a.rank <= 64) hipLaunchKernelGGL((k_lora_up<DT, 2, false>), up, dim3(256), 0, stream, a, n_per);
  else hipLaunchKernelGGL((k_lora_up<DT, 4, false>), up, dim3(256), 0, stream, a, n_per);
  return hipGetLastError();
}
hipError_t launch_lora(const LoraLaunch& a, int dtype, hipStream_t stream) {
  return dtype == DT_F16 ? launch_lora_as<DT_F16>(a, stream) : launch_lora_as<DT_BF16>(a, stream);
}

}  // namespace gmi
