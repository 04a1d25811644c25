// kernels_lora.hip -- low-rank adapters of many requests beside one dense
// product: Y[m] = base[m] + s_a (X[m] A_a^T) B_a^T with the row's own adapter a.
//
// Two launches: T = X A^T over runs of K (fp32 partial sums, added in one order),
// then Y from T.  Both walk tiles of 64 rows in the order of the call.
// Neighbouring rows of one adapter form a run, and a run is the unit of work:
// its rows are the columns of 16 x 16 x 32 matrix instructions, 16 at a time,
// and a lane past the run's end repeats its last row and is not written, so no
// row's values (an infinity, a NaN) can reach another's.  Sorted rows make long
// runs; rows in any order give the same results, to the bit, from shorter ones.
//
// Up to 511 rows the operands go straight into registers (a decode step's runs
// have a row or two: latency counts); from 512 on through rings in LDS, copied
// in whole lines.  8192 x 8192, rank 64, 8 adapters, us of both kernels, through
// registers / through LDS: 256 rows (rank 16) 13.2 / 16.2, 512 rows 35 / 28, 1024
// rows 38 / 26, 4096 rows 90 / 60.
//
// Bound by memory and by what a launch takes to start (a first copy waits for
// the row's place, then for its adapter's number): 4096 rows 22.9 + 37.4 us, the
// second at 5.0 TB/s past the 7 us that it needs for any size; 16 rows of 16
// adapters, rank 16, 4.3 + 5.4.
#include <algorithm>

#include "gmi_device.hpp"
#include "gmi_internal.hpp"
#include "gmi_rows.hpp"

namespace gmi {

constexpr int LO_WAVES = 4;
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

// Where four columns of T of one place stand.  LONG: places side by side, as the
// lanes that write and read them are; a run of one or two rows has its row's
// columns together instead.
template <bool LONG>
__device__ __forceinline__ int64_t part_at(const LoraLaunch& a, int64_t pos, int col) {
  return LONG ? ((int64_t)(col >> 2) * a.M + pos) * 4 : pos * a.rank + col;
}

// Runs of K at most; fewer past rank 16 in the kernels for long runs, where the
// second kernel's waves sum all runs each, which costs more than shorter runs
// save (8 runs / 16, both kernels: 700 rows 1024 x 8192, rank 32, 16.2 / 23.4 us;
// 1024 rows 8192 x 8192, rank 128, 36 / 42, rank 64 25.8 / 27.7).  Up to rank 16
// half the lanes take half of them (512 rows 18.1 / 16.4).
constexpr int kMostSplits = 16, kLongSplits = 8;
// 16 bytes, or zeros
__device__ __forceinline__ u32x4 load_if(const uint16_t* p, bool in) { return in ? *(const u32x4*)p : u32x4{}; }

// The workgroup's share: a tile, a part (of K, or of the columns), and one of the
// places that take turns at the tile's runs.  Consecutive tiles, which share
// adapters, lie on one XCD, whose L2 then holds an adapter once.  First places
// come first, so that they spread over the CUs; the others, which often find no
// run, come behind them.
struct LoraShare {
  int tile, slot, part;
};
__device__ __forceinline__ bool lora_share(int tiles, int parts, LoraShare& s) {
  const int each = (tiles * parts + XCDS - 1) / XCDS * XCDS;
  s.slot = blockIdx.x / each;
  const int id = remap_slot(blockIdx.x - s.slot * each, each);
  s.tile = id / parts;
  s.part = id - s.tile * parts;
  return s.tile < tiles;
}

// T of one run, its rows p0 .. p1 - 1 of the tile, over k0 .. k1 - 1.  The four
// waves take 64 k in turn, two instructions each way, the next 64 on their way
// while these multiply; their sums meet in LDS, a rank tile at a time, and are
// added in wave order.
template <int DT, int RT, int NS>
__device__ __forceinline__ void lora_down(const LoraLaunch& a, const LoraTile& t, int tile, int p0, int p1, int k0,
                                          int k1, float* part, f32x4 (*red)[4][4][64]) {
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
  struct Step {
    u32x4 x[2][NS], a[2][RT];
  };
  const auto fetch = [&](Step& f, int k) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int s = 0; s < NS; ++s) f.x[h][s] = *(const u32x4*)(xp[s] + k + 32 * h);
#pragma unroll
      for (int r = 0; r < RT; ++r) f.a[h][r] = *(const u32x4*)(ap[r] + k + 32 * h);
    }
  };
  const auto multiply = [&](const Step& f) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int s = 0; s < NS; ++s) acc[r][s] = mfma16<DT>(f.a[h][r], f.x[h][s], acc[r][s]);
  };
  int k = k0 + 64 * wave;
  const int whole = k0 + (k1 - k0) / 64 * 64;
  if (k < whole) {
    Step f;
    fetch(f, k);
    for (k += 256; k < whole; k += 256) {
      Step next;
      fetch(next, k);
      multiply(f);
      f = next;
    }
    multiply(f);
  }
  if (k < k1) {  // the rest of K, less than 64
    Step f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = k + 32 * h + kg * 8 < k1;
#pragma unroll
      for (int s = 0; s < NS; ++s) f.x[h][s] = load_if(xp[s] + k + 32 * h, in);
#pragma unroll
      for (int r = 0; r < RT; ++r) f.a[h][r] = load_if(ap[r] + k + 32 * h, in);
    }
    multiply(f);
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    // two buffers: a wave may write the next rank tile while others add this one
#pragma unroll
    for (int s = 0; s < NS; ++s) red[r & 1][wave][s][lane] = acc[r][s];
    __syncthreads();
    if (wave < NS) {
      const auto& w = red[r & 1];
      const f32x4 v = w[0][wave][lane] + w[1][wave][lane] + w[2][wave][lane] + w[3][wave][lane];
      const int p = p0 + 16 * wave + i16, col = 16 * r + 4 * kg;
      if (p < p1 && col < a.rank) *(f32x4*)(part + part_at<false>(a, tile * LO_ROWS + p, col)) = v;
    }
  }
  __syncthreads();
}

template <int DT, int RT>
__global__ __launch_bounds__(256) void k_lora_down(LoraLaunch a, int tiles, int slots, int k_per) {
  __shared__ f32x4 red[2][4][4][64];
  LoraShare sh;
  if (!lora_share(tiles, a.splits, sh)) return;
  const LoraTile t = lora_tile(a, sh.tile);
  uint64_t runs = t.starts & __ballot(t.id >= 0);
  const int k0 = min(a.K, sh.part * k_per), k1 = min(a.K, k0 + k_per);
  float* part = a.part + (int64_t)sh.part * a.M * a.rank;
  for (int n = 0; runs; ++n, runs &= runs - 1) {
    if (n % slots != sh.slot) continue;
    const int p0 = __builtin_ctzll(runs), p1 = run_end(t.starts, p0);
    if (p1 - p0 <= 16)
      lora_down<DT, RT, 1>(a, t, sh.tile, p0, p1, k0, k1, part, red);
    else if (p1 - p0 <= 32)
      lora_down<DT, RT, 2>(a, t, sh.tile, p0, p1, k0, k1, part, red);
    else
      lora_down<DT, RT, 4>(a, t, sh.tile, p0, p1, k0, k1, part, red);
  }
}

// Long runs go through LDS.  With a row a lane, as the matrix instruction wants
// it, each of a load's 64 lanes is an access of its own (61 an instruction
// measured); copies whose neighbouring lanes take a row's neighbouring 16 bytes
// make 17.  Row n of 128 bytes has its eight 16-byte chunks c in slots c ^ (n % 8),
// so that what a matrix operand reads lies in different banks.
typedef __attribute__((address_space(1))) void global_void;
template <bool NT>
__device__ __forceinline__ void copy16(const void* p, char* dst) {
  __builtin_amdgcn_global_load_lds((const global_void*)(uint64_t)p, (lds_void*)dst, 16, 0, NT ? CPOL_NT : 0);
}
__device__ __forceinline__ void group_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
// T of one run as above, each wave 16 of its rows: a ring of stages of 64 k, X's
// 64 rows and RT x 16 rows of A, that the waves fill and read together.
template <int RT>
constexpr int kDownStage = (LO_ROWS + 16 * RT) * 128;
constexpr int kDownRing = 4;
template <int DT, int RT>
__device__ __forceinline__ void lora_down_long(const LoraLaunch& a, const LoraTile& t, int tile, int p0, int p1, int k0,
                                               int k1, int r0, float* part, char* lds) {
  constexpr int COPIES = (8 + 2 * RT + 3) / 4;  // of 8 rows, a wave and stage; some may be made twice
  const int lane = threadIdx.x & 63, wave = wave_id(), i16 = lane & 15, kg = lane >> 4;
  const int id = __builtin_amdgcn_readlane(t.id, p0);
  const int sub = lane >> 3, chunk = (lane & 7) ^ sub;  // this lane's row of a copy, and the chunk its slot holds
  const uint16_t* src[COPIES];
  int dst[COPIES];
#pragma unroll
  for (int j = 0; j < COPIES; ++j) {
    const int c = min(wave + 4 * j, 7 + 2 * RT);
    dst[j] = c * 1024;
    src[j] = c < 8 ? a.X + __shfl(t.row, min(p0 + 8 * c + sub, p1 - 1)) * a.ldx
                   : a.A + id * a.a_stride + min(r0 + 8 * (c - 8) + sub, a.rank - 1) * a.lda;
  }
  const int units = (k1 - k0 + 63) / 64;  // of 64 k
  // adapters start at different k, so that rows a power of two apart do not send
  // all tiles to the same few memory channels at a time (4096 rows x 8192, 128
  // adapters of rank 64: 57 us without, 49 with); not tiles, since a row's sums
  // would then depend on its place
  const int rot = units > 0 ? (int)((uint32_t)id % (uint32_t)units) : 0;
  const auto start = [&](int i) { return k0 + 64 * (i + rot < units ? i + rot : i + rot - units); };
  const auto fetch = [&](int i) {
    // (a chunk past K is not multiplied: any address in the row will do)
    const int k = min(start(min(i, units - 1)) + 8 * chunk, a.K - 8);
    char* stage = lds + (i % kDownRing) * kDownStage<RT>;
#pragma unroll
    for (int j = 0; j < COPIES; ++j) {
      if (j < 2)  // X's eight copies
        copy16<true>(src[j] + k, stage + dst[j]);
      else
        copy16<false>(src[j] + k, stage + dst[j]);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  f32x4 acc[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) acc[r] = f32x4{};
  const bool busy = p0 + 16 * wave < p1;
  const int f0 = i16 * 128 + ((kg ^ (i16 & 7)) << 4), f1 = i16 * 128 + (((kg + 4) ^ (i16 & 7)) << 4);
  if (units > 0) {
#pragma unroll
    for (int i = 0; i < kDownRing - 1; ++i) fetch(i);
    for (int i = 0; i < units; ++i) {
      wait_vm_le<(kDownRing - 2) * COPIES>();
      group_barrier();
      fetch(i + kDownRing - 1);
      if (!busy) continue;
      const char* stage = lds + (i % kDownRing) * kDownStage<RT>;
      u32x4 x[2], w[2][RT];
      x[0] = *(const u32x4*)(stage + wave * 2048 + f0);
      x[1] = *(const u32x4*)(stage + wave * 2048 + f1);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        w[0][r] = *(const u32x4*)(stage + LO_ROWS * 128 + r * 2048 + f0);
        w[1][r] = *(const u32x4*)(stage + LO_ROWS * 128 + r * 2048 + f1);
      }
      __builtin_amdgcn_sched_barrier(0);  // all on their way before the first is waited for
      const int k = start(i);
      if (k + 64 > k1) {  // the end of K: zeros from there on
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool in = k + 32 * h + kg * 8 < k1;
          x[h] = in ? x[h] : u32x4{};
#pragma unroll
          for (int r = 0; r < RT; ++r) w[h][r] = in ? w[h][r] : u32x4{};
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[r] = mfma16<DT>(w[h][r], x[h], acc[r]);
      wait_lgkm();  // read before the barrier that frees the stage
    }
  }
  wait_vm_le<0>();  // nothing lands any more
  group_barrier();
  const int p = p0 + 16 * wave + i16;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int col = r0 + 16 * r + 4 * kg;
    if (p < p1 && col < a.rank) *(f32x4*)(part + part_at<true>(a, tile * LO_ROWS + p, col)) = acc[r];
  }
}
template <int DT, int RT>
__global__ __launch_bounds__(256) void k_lora_down_long(LoraLaunch a, int tiles, int slots, int k_per, int halves) {
  __shared__ __align__(16) char lds[kDownRing * kDownStage<RT>];
  LoraShare sh;
  if (!lora_share(tiles, a.splits * halves, sh)) return;
  const LoraTile t = lora_tile(a, sh.tile);
  uint64_t runs = t.starts & __ballot(t.id >= 0);
  const int split = sh.part / halves, r0 = (sh.part - split * halves) * 16 * RT;
  const int k0 = min(a.K, split * k_per), k1 = min(a.K, k0 + k_per);
  float* part = a.part + (int64_t)split * a.M * a.rank;
  for (int n = 0; runs; ++n, runs &= runs - 1) {
    if (n % slots != sh.slot) continue;
    const int p0 = __builtin_ctzll(runs), p1 = run_end(t.starts, p0);
    lora_down_long<DT, RT>(a, t, sh.tile, p0, p1, k0, k1, r0, part, lds);
  }
}

// T as operand of the second product.  A 16-bit T would cost the result as much
// again as its own rounding, so T goes in as two terms, t = hi + lo, whose
// products with B are summed: what is lost is 2^-17 (bf16) or 2^-22 (fp16) of
// t.  fp16 cannot hold every t: a row is scaled by the power of two that brings
// its largest, infinities aside, to [1, 2), and `f` takes it back.  Up to rank 16
// both terms fit one instruction (k 0..15 hi, 16..31 lo, against B twice).
template <int DT, int RS, bool ONE>
struct LoraT {
  u32x4 hi[RS], lo[ONE ? 1 : RS];
  float f;
};
__device__ __forceinline__ float max4(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
// C quarters of the sum over the runs of K from the j-th on; quarter q holds the
// runs q, q + 4, ..., at most R of them, and two quarters are added before two
// pairs are.  With ONE lanes 32 apart hold the same columns, and each sums every
// other run of a quarter.  Loads are on their way together; past the last run it
// is read again and not added.
template <bool LONG, int RS, bool ONE, int C, int R>
__device__ __forceinline__ void sum_rounds(const LoraLaunch& a, int64_t pos, bool in, int j, float (&v)[RS][8]) {
  // places of a lane on their way (128 rows, rank 128, the second kernel: 17.1 us, with
  // four 18.4; long runs with 16: 512 rows, rank 64, 17.9 for 18.4, 1024, rank 128, 22.5 for 21.4)
  constexpr int MOST = 8;
  constexpr int AT = C * R <= MOST ? R : MOST / C, RG = C * AT * RS <= MOST ? RS : MOST / (C * AT);  // runs, rank tiles
  const int kg = (threadIdx.x & 63) >> 4, every = ONE ? 8 : 4;
  const int64_t run = (int64_t)a.M * a.rank, beside = LONG ? 4 * (int64_t)a.M : 4;
  j += ONE ? 4 * (kg >> 1) : 0;
#pragma unroll
  for (int r0 = 0; r0 < RS; r0 += RG) {
    float sum[RG][C][8];
    bool there[RG];
    const float* p[RG];
#pragma unroll
    for (int r = 0; r < RG; ++r) {
      const int col = ONE ? 8 * (kg & 1) : 32 * (r0 + r) + 8 * kg;
      there[r] = in && col < a.rank;
      p[r] = there[r] ? a.part + part_at<LONG>(a, pos, col) : a.part;
    }
#pragma unroll
    for (int q0 = 0; q0 < R; q0 += AT) {
      f32x4 s[RG][C][AT][2];
#pragma unroll
      for (int r = 0; r < RG; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int q = 0; q < AT; ++q) {
            const int64_t at = min(j + c + (q0 + q) * every, a.splits - 1) * run;
            s[r][c][q][0] = *(const f32x4*)(p[r] + at);
            s[r][c][q][1] = *(const f32x4*)((there[r] ? p[r] + beside : p[r]) + at);
          }
#pragma unroll
      for (int r = 0; r < RG; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (q0 == 0) sum[r][c][e] = 0.0f;
#pragma unroll
            for (int q = 0; q < AT; ++q)
              sum[r][c][e] += there[r] && j + c + (q0 + q) * every < a.splits ? s[r][c][q][e / 4][e % 4] : 0.0f;
          }
    }
#pragma unroll
    for (int r = 0; r < RG; ++r)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (ONE) {
#pragma unroll
          for (int c = 0; c < C; ++c) sum[r][c][e] += __shfl_xor(sum[r][c][e], 32);
        }
        if constexpr (C == 1) v[r0 + r][e] = sum[r][0][e];
        else if constexpr (C == 2) v[r0 + r][e] = sum[r][0][e] + sum[r][1][e];
        else v[r0 + r][e] = (sum[r][0][e] + sum[r][1][e]) + (sum[r][2][e] + sum[r][3][e]);
      }
    __builtin_amdgcn_sched_barrier(0);  // the next ranks' loads would spill
  }
}
template <bool LONG, int RS, bool ONE, int C>
__device__ __forceinline__ void sum_t(const LoraLaunch& a, int64_t pos, bool in, int j, float (&v)[RS][8]) {
  const int rounds = (a.splits + (ONE ? 7 : 3)) / (ONE ? 8 : 4);
  static_assert(kLongSplits <= 8 && kMostSplits <= 16);
  if (C > 1 && a.splits == 1) sum_rounds<LONG, RS, ONE, 1, 1>(a, pos, in, j, v);
  else if (rounds <= 1) sum_rounds<LONG, RS, ONE, C, 1>(a, pos, in, j, v);
  else if (ONE || rounds <= 2) sum_rounds<LONG, RS, ONE, C, 2>(a, pos, in, j, v);
  else if constexpr (!LONG && !ONE) sum_rounds<LONG, RS, ONE, C, kMostSplits / 4>(a, pos, in, j, v);
}
template <int DT, int RS, bool ONE>
__device__ __forceinline__ void split_t(float (&v)[RS][8], LoraT<DT, RS, ONE>& t) {
  const int kg = (threadIdx.x & 63) >> 4;
  t.f = 1.0f;
  if constexpr (DT == DT_F16) {
    float m = 0.0f;
#pragma unroll
    for (int r = 0; r < RS; ++r)
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[r][e]) < __builtin_inff() ? fabsf(v[r][e]) : 0.0f);
    m = max4(m);
    // 2^(exponent of m), inside the normal range with its reciprocal
    const uint32_t ex = min(max(__builtin_bit_cast(uint32_t, m) >> 23, 2u), 252u);
    t.f = __builtin_bit_cast(float, ex << 23);
    const float inv = __builtin_bit_cast(float, (254u - ex) << 23);
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

// column of row i of instruction m among the 64 of a wave
__device__ __forceinline__ int dealt_column(int m, int i) {
  return 32 * (m >> 1) + 8 * (i >> 2) + 4 * (m & 1) + (i & 3);
}
// 16 rows of 64 columns: B's operands times T, on base
template <int DT, int RS, bool ONE>
__device__ __forceinline__ void lora_columns(const u32x4 (&b)[RS][4], const LoraT<DT, RS, ONE>& t,
                                             const u32x4 (&base)[2], u32x4 (&out)[2]) {
  f32x4 acc[4];
#pragma unroll
  for (int m = 0; m < 4; ++m) acc[m] = f32x4{};
#pragma unroll
  for (int r = 0; r < RS; ++r) {
#pragma unroll
    for (int m = 0; m < 4; ++m) acc[m] = mfma16<DT>(b[r][m], t.hi[r], acc[m]);
    if constexpr (!ONE) {
#pragma unroll
      for (int m = 0; m < 4; ++m) acc[m] = mfma16<DT>(b[r][m], t.lo[r], acc[m]);
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const f32x4 v = acc[2 * h + e / 2];
      out[h][e] = pack2<DT>(__builtin_fmaf(t.f, v[2 * (e % 2)], from_bits<DT>(base[h][e] & 0xffffu)),
                            __builtin_fmaf(t.f, v[2 * (e % 2) + 1], from_bits<DT>(base[h][e] >> 16)));
    }
  }
}

template <int DT, int RS, bool ONE>
union LoraUpLds {
  LoraT<DT, RS, ONE> t[4][64];  // past 16 rows
  f32x4 part[4][RS][2][64];     // up to 16
};
// Y of one short run: a wave makes 64 columns of up to 64 rows at a time.  B is
// the instruction's first operand, its rows dealt so that a lane ends with eight
// neighbouring columns of one row of Y twice: row i of instruction m is column
// 32 (m / 2) + 8 (i / 4) + 4 (m % 2) + i % 4, and a lane's results are columns
// 32 (m / 2) + 8 (l / 16) + 4 (m % 2) + j.  B and base are asked for before T,
// which comes of the longer way: up to 16 rows a wave sums a quarter of the runs of
// K and the quarters meet in LDS, so that 16 runs cost one trip to memory (78 rows
// 1432 x 4296, rank 64: 11.4 us with four trips, 8.3; 128 rows 8192 x 8192, rank
// 128: 21 and 17).  Past 16 rows each wave makes T of 16 of them for all, in the
// same order of the sum.
template <int DT, int RS, bool ONE, int NS>
__device__ __forceinline__ void lora_up(const LoraLaunch& a, const LoraTile& t, int tile, int p0, int p1, int n0,
                                        int n1, LoraUpLds<DT, RS, ONE>& lds) {
  const int lane = threadIdx.x & 63, wave = wave_id(), i16 = lane & 15, kg = lane >> 4;
  const int id = __builtin_amdgcn_readlane(t.id, p0);
  const uint16_t* b = a.B + id * a.b_stride;
  const uint16_t* from[NS];
  uint16_t* to[NS];
  bool in[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int p = p0 + 16 * s + i16;
    in[s] = p < p1;
    const int64_t row = __shfl(t.row, min(p, p1 - 1));
    from[s] = a.base + row * a.ldbase + 8 * kg;
    to[s] = a.Y + row * a.ldy + 8 * kg;
  }
  u32x4 bv[RS][4], base[NS][2];
  const auto fetch = [&](int c0) {
#pragma unroll
    for (int r = 0; r < RS; ++r) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int n = c0 + dealt_column(m, i16), k = ONE ? 8 * (kg & 1) : 32 * r + 8 * kg;
        bv[r][m] = load_if(b + n * a.ldb + k, n < a.N && k < a.rank);
      }
    }
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        base[s][h] = load_if(from[s] + c0 + 32 * h, a.base && in[s] && c0 + 8 * kg + 32 * h < a.N);
  };
  int c0 = n0 + 64 * wave;
  if (c0 < n1) fetch(c0);
  const float scale = a.scales ? a.scales[id] : 1.0f;
  const int p = p0 + (NS == 1 ? 0 : 16 * wave) + i16;
  const int64_t pos = (int64_t)tile * LO_ROWS + p;
  float v[RS][8];
  LoraT<DT, RS, ONE> t0;
  if constexpr (NS == 1) {
    sum_t<false, RS, ONE, 1>(a, pos, p < p1, wave, v);
#pragma unroll
    for (int r = 0; r < RS; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        lds.part[wave][r][h][lane] = f32x4{v[r][4 * h], v[r][4 * h + 1], v[r][4 * h + 2], v[r][4 * h + 3]};
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RS; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 s = (lds.part[0][r][h][lane] + lds.part[1][r][h][lane]) +
                        (lds.part[2][r][h][lane] + lds.part[3][r][h][lane]);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[r][4 * h + e] = s[e];
      }
    split_t(v, t0);
    t0.f *= scale;
  } else {
    if (wave < NS) {
      // (two quarters at a time: with four the kernel takes the registers of two waves)
      float w[RS][8];
      sum_t<false, RS, ONE, 2>(a, pos, p < p1, 0, v);
      sum_t<false, RS, ONE, 2>(a, pos, p < p1, 2, w);
#pragma unroll
      for (int r = 0; r < RS; ++r)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[r][e] += w[r][e];
      split_t(v, t0);
      t0.f *= scale;
      lds.t[wave][lane] = t0;
    }
    __syncthreads();
  }
  while (c0 < n1) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      LoraT<DT, RS, ONE> tv;
      if constexpr (NS == 1)
        tv = t0;
      else
        tv = lds.t[s][lane];
      u32x4 o[2];
      lora_columns(bv, tv, base[s], o);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (in[s] && c0 + 8 * kg + 32 * h < a.N) *(u32x4*)(to[s] + c0 + 32 * h) = o[h];
    }
    c0 += 256;
    if (c0 < n1) fetch(c0);
  }
  __syncthreads();  // the next run's T may come
}

// rows without an adapter: base, or zeros
__device__ __forceinline__ void lora_copy(const LoraLaunch& a, const LoraTile& t, int p0, int p1, int n0, int n1) {
  if (a.base == a.Y) return;
  const int lane = threadIdx.x & 63;
  constexpr int ROWS = 8;  // of a wave on their way at a time
  for (int c = n0 + 8 * lane; c < n1; c += 512) {
    for (int p = p0 + wave_id(); p < p1; p += LO_WAVES * ROWS) {
      u32x4 v[ROWS];
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        const int64_t row = __builtin_amdgcn_readlane(t.row, min(p + LO_WAVES * j, p1 - 1));
        v[j] = load_if(a.base + row * a.ldbase + c, a.base != nullptr);
      }
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        const int64_t row = __builtin_amdgcn_readlane(t.row, min(p + LO_WAVES * j, p1 - 1));
        if (p + LO_WAVES * j < p1) *(u32x4*)(a.Y + row * a.ldy + c) = v[j];
      }
    }
  }
}

// Slots of B's 16-byte chunks c in a row n of 64 RS bytes (32 with ONE): c ^
// b_turn(n), which spreads the rows that one matrix operand reads over the banks.
template <int RS, bool ONE>
__device__ __forceinline__ int b_turn(int n) {
  if constexpr (ONE) return n >> 4 & 1;
  if constexpr (RS == 1) return (4 - (n >> 3)) & 3;
  if constexpr (RS == 2) return (n >> 1 & 1) | (n >> 3 & 3) << 1;
  return (n & 3) | (n >> 3 & 3) << 2;
}
// Y of one long run: 64 columns at a time, each wave 16 rows of all of them.  B's
// 64 rows are a stage of a ring that the waves fill and read together; base's
// rows come beside it, for the wave alone, Y's take their place and leave in
// whole lines.
template <int RS, bool ONE>
constexpr int kUpB = 64 * (ONE ? 32 : 64 * RS);
template <int RS, bool ONE>
constexpr int kUpStage = kUpB<RS, ONE> + LO_ROWS * 128;
template <int RS>
constexpr int kUpRing = RS > 2 ? 3 : 4;
template <int DT, int RS, bool ONE>
__device__ __forceinline__ void lora_up_long(const LoraLaunch& a, const LoraTile& t, int tile, int p0, int p1, int n0,
                                             int n1, char* lds) {
  constexpr int CH = ONE ? 2 : 4 * RS, PITCH = 16 * CH, D = kUpRing<RS>;
  constexpr int BC = (CH + 3) / 4, COPIES = BC + 2;  // copies a wave and stage
  const int lane = threadIdx.x & 63, wave = wave_id(), i16 = lane & 15, kg = lane >> 4;
  const int id = __builtin_amdgcn_readlane(t.id, p0);
  const uint16_t* b = a.B + id * a.b_stride;
  // B: copy c holds 64 / CH rows
  int brow[BC], bdst[BC];
  const uint16_t* bsrc[BC];
#pragma unroll
  for (int j = 0; j < BC; ++j) {
    const int c = min(wave + 4 * j, CH - 1);
    brow[j] = c * (64 / CH) + lane / CH;
    bsrc[j] = b + min(((lane % CH) ^ b_turn<RS, ONE>(brow[j])) * 8, a.rank - 8);  // (past the rank: not multiplied)
    bdst[j] = c * 1024;
  }
  // base and Y: copy q of this wave holds 8 of its 16 rows
  const int sub = lane >> 3, chunk = (lane & 7) ^ sub;
  const uint16_t* from[2];
  uint16_t* to[2];
  bool in[2];
  const uint16_t* base = a.base ? a.base : a.Y;  // without a base anything is read and nothing added
  const int64_t ldbase = a.base ? a.ldbase : a.ldy;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int p = p0 + 16 * wave + 8 * q + sub;
    const int64_t row = __shfl(t.row, min(p, p1 - 1));
    in[q] = p < p1;
    from[q] = base + row * ldbase;
    to[q] = a.Y + row * a.ldy;
  }
  const int steps = (n1 - n0 + 63) / 64;  // of 64 columns
  const int rot = tile % steps;
  const auto start = [&](int i) { return n0 + 64 * (i + rot < steps ? i + rot : i + rot - steps); };
  const auto fetch = [&](int i) {
    const int c0 = start(min(i, steps - 1));
    char* stage = lds + (i % D) * kUpStage<RS, ONE>;
    const int left = a.N - c0;  // columns; past the last one anything is read
#pragma unroll
    for (int j = 0; j < BC; ++j)
      copy16<false>(bsrc[j] + c0 * a.ldb + (left < 64 ? min(brow[j], left - 1) : brow[j]) * a.ldb, stage + bdst[j]);
#pragma unroll
    for (int q = 0; q < 2; ++q)
      copy16<true>(from[q] + c0 + (left < 64 ? min(8 * chunk, left - 8) : 8 * chunk),
                  stage + kUpB<RS, ONE> + wave * 2048 + q * 1024);
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int i = 0; i < D - 1; ++i) fetch(i);
  LoraT<DT, RS, ONE> tv;
  float tsum[RS][8];
  sum_t<true, RS, ONE, 4>(a, (int64_t)tile * LO_ROWS + p0 + 16 * wave + i16, p0 + 16 * wave + i16 < p1, 0, tsum);
  split_t(tsum, tv);
  tv.f *= a.scales ? a.scales[id] : 1.0f;
  const bool busy = p0 + 16 * wave < p1;
  // all of the wave's stores are made: they count among what a stage is waited for
  const bool whole = p0 + 16 * wave + 16 <= p1 && a.N % 64 == 0;
  const int bf = i16 * 128 + ((kg ^ (i16 & 7)) << 4), bg = i16 * 128 + (((kg + 4) ^ (i16 & 7)) << 4);
  int bfrag[RS][4];
#pragma unroll
  for (int r = 0; r < RS; ++r)
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int n = dealt_column(m, i16);
      bfrag[r][m] = n * PITCH + (((ONE ? kg & 1 : 4 * r + kg) ^ b_turn<RS, ONE>(n)) << 4);
    }
  const bool ragged = a.rank % (8 * CH) != 0;
  for (int i = 0; i < steps; ++i) {
    if (whole && i >= D - 2)
      wait_vm_le<(D - 2) * (COPIES + 2)>();
    else
      wait_vm_le<(D - 2) * COPIES>();
    group_barrier();
    fetch(i + D - 1);
    if (!busy) continue;
    char* stage = lds + (i % D) * kUpStage<RS, ONE>;
    char* own = stage + kUpB<RS, ONE> + wave * 2048;
    u32x4 v[RS][4], z[2];
#pragma unroll
    for (int r = 0; r < RS; ++r)
#pragma unroll
      for (int m = 0; m < 4; ++m) v[r][m] = *(const u32x4*)(stage + bfrag[r][m]);
    z[0] = *(const u32x4*)(own + bf);
    z[1] = *(const u32x4*)(own + bg);
    __builtin_amdgcn_sched_barrier(0);  // all on their way before the first is waited for
    if (ragged) {
#pragma unroll
      for (int r = 0; r < RS; ++r)
#pragma unroll
        for (int m = 0; m < 4; ++m)
          if (8 * (ONE ? kg & 1 : 4 * r + kg) >= a.rank) v[r][m] = u32x4{};
    }
    if (!a.base) z[0] = z[1] = u32x4{};
    u32x4 o[2];
    lora_columns(v, tv, z, o);
    *(u32x4*)(own + bf) = o[0];
    *(u32x4*)(own + bg) = o[1];
    asm volatile("" ::: "memory");  // (the LDS serves a wave in order)
    const int col = start(i) + 8 * chunk;
    const u32x4 y0 = *(const u32x4*)(own + lane * 16), y1 = *(const u32x4*)(own + 1024 + lane * 16);
    wait_lgkm();  // read before the barrier that frees the stage
    if (whole) {
      store<true>(to[0] + col, y0);
      store<true>(to[1] + col, y1);
    } else if (col < a.N) {
      if (in[0]) store<true>(to[0] + col, y0);
      if (in[1]) store<true>(to[1] + col, y1);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  wait_vm_le<0>();  // nothing lands any more
  group_barrier();
}

template <int DT, int RS, bool ONE>
__global__ __launch_bounds__(256) void k_lora_up_long(LoraLaunch a, int tiles, int slots, int n_per, int parts) {
  __shared__ __align__(16) char lds[kUpRing<RS> * kUpStage<RS, ONE>];
  LoraShare sh;
  if (!lora_share(tiles, parts, sh)) return;
  const LoraTile t = lora_tile(a, sh.tile);
  uint64_t runs = t.starts & __ballot(t.id > -2);
  const int n0 = sh.part * n_per, n1 = min(a.N, n0 + n_per);
  for (int n = 0; runs; ++n, runs &= runs - 1) {
    if (n % slots != sh.slot) continue;
    const int p0 = __builtin_ctzll(runs), p1 = run_end(t.starts, p0);
    if (__builtin_amdgcn_readlane(t.id, p0) < 0)
      lora_copy(a, t, p0, p1, n0, n1);
    else
      lora_up_long<DT, RS, ONE>(a, t, sh.tile, p0, p1, n0, n1, lds);
  }
}

template <int DT, int RS, bool ONE>
__global__ __launch_bounds__(256) void k_lora_up(LoraLaunch a, int tiles, int slots, int n_per, int parts) {
  __shared__ LoraUpLds<DT, RS, ONE> lds;
  LoraShare sh;
  if (!lora_share(tiles, parts, sh)) return;
  const LoraTile t = lora_tile(a, sh.tile);
  uint64_t runs = t.starts & __ballot(t.id > -2);
  const int n0 = sh.part * n_per, n1 = min(a.N, n0 + n_per);
  for (int n = 0; runs; ++n, runs &= runs - 1) {
    if (n % slots != sh.slot) continue;
    const int p0 = __builtin_ctzll(runs), p1 = run_end(t.starts, p0);
    if (__builtin_amdgcn_readlane(t.id, p0) < 0)
      lora_copy(a, t, p0, p1, n0, n1);
    else if (p1 - p0 <= 16)
      lora_up<DT, RS, ONE, 1>(a, t, sh.tile, p0, p1, n0, n1, lds);
    else if (p1 - p0 <= 32)
      lora_up<DT, RS, ONE, 2>(a, t, sh.tile, p0, p1, n0, n1, lds);
    else
      lora_up<DT, RS, ONE, 4>(a, t, sh.tile, p0, p1, n0, n1, lds);
  }
}

// How a call is dealt out.
struct LoraPlan {
  int tiles, slots;          // slots: workgroups that take turns at a tile's runs
  int splits, k_per;         // runs of K
  int64_t parts, n_per;      // column blocks
  bool wide;                 // through LDS, for long runs
};
// The border is that of 8 adapters (the figures at the head): with hundreds of
// them runs stay short from 512 rows on too, which was not timed.
static bool lora_wide(int M) { return M >= 512; }
// runs of K at most, which the workspace has room for: none below 256 k
static int lora_most_splits(int M, int K, int rank) {
  const int tiles = (M + LO_ROWS - 1) / LO_ROWS, most = lora_wide(M) && rank > 16 ? kLongSplits : kMostSplits;
  return std::max(1, std::min({K / 256, (lora_wide(M) ? 256 : 512) / tiles, most}));
}
size_t lora_workspace(int M, int K, int rank) {
  return (size_t)lora_most_splits(M, K, rank) * M * rank * sizeof(float);
}

static LoraPlan lora_plan(const LoraLaunch& a) {
  LoraPlan p;
  p.tiles = (a.M + LO_ROWS - 1) / LO_ROWS;
  p.wide = lora_wide(a.M);
  // twice the runs that sorted rows make of a tile on average, and one without an
  // adapter: a workgroup with two runs takes them one after the other (4096 rows
  // with tiles of two runs: 89 us for 60), one with none still has to find that
  // out (64 rows of 32 adapters with a workgroup per row: 16 us for 7.4)
  const int64_t runs = std::min<int64_t>(LO_ROWS, 1 + 2 * (((int64_t)a.adapters * LO_ROWS + a.M - 1) / a.M));
  int64_t down, up;  // parts wanted: one workgroup a CU beside the further slots, or two
  if (p.wide) {
    p.slots = (int)std::min<int64_t>(4, runs);
    down = up = 256 / p.tiles;
  } else {
    p.slots = (int)std::min<int64_t>({32, a.M, LO_ROWS / p.tiles, runs});
    p.slots = std::max(p.slots, 1);
    down = up = 512 / (p.tiles * p.slots);
  }
  p.splits = std::max<int>(1, std::min<int64_t>(lora_most_splits(a.M, a.K, a.rank), down));
  p.k_per = ((a.K + p.splits - 1) / p.splits + 63) / 64 * 64;
  p.splits = (a.K + p.k_per - 1) / p.k_per;  // (the rounding may leave none for the last)
  const int64_t blocks = ((int64_t)a.N + 255) / 256, want = std::max<int64_t>(1, std::min(blocks, up));
  p.n_per = (blocks + want - 1) / want * 256;
  p.parts = (a.N + p.n_per - 1) / p.n_per;
  return p;
}

// workgroups, in whole rounds of the XCDs for each slot
static dim3 lora_grid(const LoraPlan& p, int64_t parts) {
  return dim3((unsigned)((p.tiles * parts + XCDS - 1) / XCDS * XCDS * p.slots));
}

template <int DT, int RT>
static void launch_lora_down(const LoraLaunch& a, const LoraPlan& p, hipStream_t stream) {
  hipLaunchKernelGGL((k_lora_down<DT, RT>), lora_grid(p, p.splits), dim3(256), 0, stream, a, p.tiles, p.slots, p.k_per);
}
// ranks above 64 in two halves, each a part
template <int DT, int RT>
static void launch_lora_down_long(const LoraLaunch& a, const LoraPlan& p, int halves, hipStream_t stream) {
  hipLaunchKernelGGL((k_lora_down_long<DT, RT>), lora_grid(p, p.splits * halves), dim3(256), 0, stream, a, p.tiles,
                     p.slots, p.k_per, halves);
}
template <int DT, int RS, bool ONE>
static void launch_lora_up(const LoraLaunch& a, const LoraPlan& p, hipStream_t stream) {
  if (p.wide)
    hipLaunchKernelGGL((k_lora_up_long<DT, RS, ONE>), lora_grid(p, p.parts), dim3(256), 0, stream, a, p.tiles, p.slots,
                       (int)p.n_per, (int)p.parts);
  else
    hipLaunchKernelGGL((k_lora_up<DT, RS, ONE>), lora_grid(p, p.parts), dim3(256), 0, stream, a, p.tiles, p.slots,
                       (int)p.n_per, (int)p.parts);
}

template <int DT>
static hipError_t launch_lora_as(const LoraLaunch& args, hipStream_t stream) {
  LoraLaunch a = args;
  const LoraPlan p = lora_plan(a);
  a.splits = p.splits;
  if (p.wide) {
    if (a.rank <= 16) launch_lora_down_long<DT, 1>(a, p, 1, stream);
    else if (a.rank <= 32) launch_lora_down_long<DT, 2>(a, p, 1, stream);
    else launch_lora_down_long<DT, 4>(a, p, a.rank > 64 ? 2 : 1, stream);
  } else {
    if (a.rank <= 16) launch_lora_down<DT, 1>(a, p, stream);
    else if (a.rank <= 32) launch_lora_down<DT, 2>(a, p, stream);
    else if (a.rank <= 64) launch_lora_down<DT, 4>(a, p, stream);
    else launch_lora_down<DT, 8>(a, p, stream);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.rank <= 16) launch_lora_up<DT, 1, true>(a, p, stream);
  else if (a.rank <= 32) launch_lora_up<DT, 1, false>(a, p, stream);
  else if (a.rank <= 64) launch_lora_up<DT, 2, false>(a, p, stream);
  else launch_lora_up<DT, 4, false>(a, p, stream);
  return hipGetLastError();
}
hipError_t launch_lora(const LoraLaunch& a, int dtype, hipStream_t stream) {
  return dtype == DT_F16 ? launch_lora_as<DT_F16>(a, stream) : launch_lora_as<DT_BF16>(a, stream);
}

}  // namespace gmi
