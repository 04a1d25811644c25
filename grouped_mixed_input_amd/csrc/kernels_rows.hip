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
//
// 16384 tokens, top 8, 4096 columns: permute (fp8) 106 to 111 us (5.6 to 5.9
// TB/s), unpermute (bf16, with add) 242 (5.55), its gradient as codes 334 (5.3);
// 131072 x 2 x 1024 bf16: gate 111 us (6.1 TB/s), its gradient 168 (6.3), where
// arithmetic takes as long as memory.  Rows of 4 KB far apart cost 15% over a
// contiguous walk.  Few tokens: 3.6 us a launch, of which an empty one takes 2.5.
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

// chunks that a lane asks for at once: of a token's row, and of its k rows
constexpr int kPermuteChunks = 4;
template <int KT>
constexpr int kUnpermuteChunks = KT >= 16 ? 1 : KT >= 8 ? 2 : 4;

// NT: the copies go past the caches (the token's own row does not: 106 us of
// 124 with it, at 16384 x 8 x 4096 fp8).
template <bool NT>
__global__ __launch_bounds__(256) void k_permute(PermuteLaunch a) {
  constexpr int CH = kPermuteChunks;
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
        v[j] = c < a.chunks ? load16<false>(x + (int64_t)c * 16) : u32x4{};
      }
      for (int i = 0; i < a.k; ++i) {
        const int r = __builtin_amdgcn_readlane(at, i);
        if (r < 0) continue;
        char* o = a.out + r * a.ldo;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          const int c = c0 + j * p.stride + lane;
          if (c < a.chunks) store<NT>(o + (int64_t)c * 16, v[j]);
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
template <int DT, bool NT, int KT>
__global__ __launch_bounds__(256) void k_unpermute(UnpermuteLaunch a) {
  constexpr int CH = kUnpermuteChunks<KT>;
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
          v[j][i] = in && row[i] >= 0 ? load16<NT>(a.y + row[i] * a.ldy + (int64_t)c * 8) : u32x4{};
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

// sum + <a, b> over eight columns, each product of two 16-bit values added with
// one fp32 rounding.  (The instructions for product pairs round otherwise: bf16's
// is off by more where terms cancel, fp16's drops bits of subnormal operands.)
template <int DT>
__device__ __forceinline__ float dot8(u32x4 a, u32x4 b, float sum) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sum = __builtin_fmaf(from_bits<DT>(a[i] & 0xffffu), from_bits<DT>(b[i] & 0xffffu), sum);
    sum = __builtin_fmaf(from_bits<DT>(a[i] >> 16), from_bits<DT>(b[i] >> 16), sum);
  }
  return sum;
}

// A slot's row out of lane i, a scalar.  The walk over columns asks anew each
// time: kept, the 2 k row addresses would take more scalar registers than there
// are, and their spills cost vector instructions.
__device__ __forceinline__ int again(int at) {
  asm volatile("" : "+v"(at));
  return at;
}

// WPT waves a token (1, or 4 for longer rows), CH chunks at a time.  With Q the
// rows leave as codes: (w d) / (|w| m / 448), m the block's largest |d|, is
// 448 d / m with w's sign, so the codes are found once for all k slots, and the
// slots' scales by one lane each.  Where |w| m or m leaves the range that the
// scale's bound and infinity cut, w does not cancel and the slot's codes are
// its own.
template <int DT, bool Q, bool NT, int KT, int WPT>
__global__ __launch_bounds__(256) void k_unpermute_bwd(UnpermuteBwdLaunch a) {
  constexpr int CH = KT > 8 ? 1 : 2;
  __shared__ float red[4][KT];
  const int lane = threadIdx.x & 63, wave = wave_id(), l16 = lane & 15;
  const int64_t step = (int64_t)gridDim.x * (4 / WPT);
  // (with four waves a token every wave of the workgroup makes the same turns, so all meet the barriers)
  for (int64_t t = (int64_t)blockIdx.x * (4 / WPT) + (WPT == 1 ? wave : 0); t < a.T; t += step) {
    const int slots = slot_of_lane(a.slot_row, t, a.k, a.rows, lane);
    const float wt = a.weights && lane < a.k ? a.weights[t * a.k + lane] : 1.0f;
    // every 16 lanes hold the slots once
    const int slot16 = __shfl(slots, l16);
    const float w16 = __shfl(wt, l16);
    float dot[KT];
#pragma unroll
    for (int i = 0; i < KT; ++i) dot[i] = 0.0f;
    for (int c0 = WPT == 1 ? 0 : wave * 64; c0 < a.chunks; c0 += 64 * WPT * CH) {
      const int at = again(slots);
      u32x4 v[CH][KT], dv[CH];
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const int c = c0 + 64 * WPT * j + lane;
        dv[j] = u32x4{};
        if (c >= a.chunks) continue;
        dv[j] = load16<NT>(a.dout + t * a.ldd + (int64_t)c * 8);
        if (!a.y) continue;
#pragma unroll
        for (int i = 0; i < KT; ++i) {
          const int r = __builtin_amdgcn_readlane(at, i);
          if (r >= 0) v[j][i] = load16<NT>(a.y + r * a.ldy + (int64_t)c * 8);
        }
      }
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const int to = again(slots);
        const int c = c0 + 64 * WPT * j + lane;
        float d[8], m = 0.0f;
        unpack8<DT>(dv[j], d);
        u32x2 codes{};
        uint64_t own = 0;  // bit 16 b + i: slot i's codes of block b are its own
        if constexpr (Q) {
#pragma unroll
          for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(d[e]));
          m = max16(m);
          codes = codes8(d, block_scale(m));
          const float am = fabsf(w16) * m;
          if (slot16 >= 0 && c - l16 < a.chunks) a.scales[slot16 * a.lds + c / 16] = block_scale(am);
          own = __ballot(!(fminf(am, m) >= kF8Max * 0x1p-126f && am < __builtin_inff()));
        }
        if (c >= a.chunks) continue;
#pragma unroll
        for (int i = 0; i < KT; ++i) {
          const int r = __builtin_amdgcn_readlane(to, i);
          if (r < 0) continue;
          const float wi = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, wt), i));
          if (a.y) dot[i] = dot8<DT>(dv[j], v[j][i], dot[i]);
          float g[8];
          if constexpr (Q) {
            const uint32_t sign = (__builtin_bit_cast(uint32_t, wi) >> 31) * 0x80808080u;
            u32x2 q{codes[0] ^ sign, codes[1] ^ sign};
            if (own >> i & 0x0001000100010001ull) {
#pragma unroll
              for (int e = 0; e < 8; ++e) g[e] = wi * d[e];
              if (own >> ((lane & 48) + i) & 1) q = codes8(g, block_scale(fabsf(wi) * m));
            }
            store<NT>(a.q + r * a.ldq + (int64_t)c * 8, q);
          } else if (a.drows) {
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = wi * d[e];
            store<NT>(a.drows + r * a.lddr + (int64_t)c * 8, pack8<DT>(g));
          }
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

constexpr int kSwigluUnits = 2;

// s = 1 / (1 + e^-g), and 1 - s as e^-g s, which cancels nothing.  e^-g as 2^t
// with t = -g log2 e rounded, times e^r = 1 + r with r = -g - t ln 2: 2^t alone
// would carry t's rounding, |g| 2^-24 of it.  What is left of that is |g| 2^-28,
// ln 2 in fp32; exponential and reciprocal bring a last bit each.  From 88.5 on
// e^-g would pass the fp32 range: the bound keeps it finite there, s is below
// 2^-126, for which the reciprocal gives 0, and 1 - s comes out 0 with it, where
// only its product with s is wanted; infinities would leave NaN in r.
// (131072 x 2 x 1024, without r and with 1 - s as a difference: 110 us for 111 in
// the forward call, 164 for 168 in its gradient.)
struct Sigmoid {
  float s, rest;
};
__device__ __forceinline__ Sigmoid sigmoid(float g) {
  constexpr float LOG2E = 1.44269504f, LN2 = 0.693147182f;
  g = __builtin_amdgcn_fmed3f(g, -88.5f, 128.0f);
  const float t = g * -LOG2E;
  float e = __builtin_amdgcn_exp2f(t);
  e = __builtin_fmaf(e, __builtin_fmaf(-LN2, t, -g), e);
  const float s = __builtin_amdgcn_rcpf(1.0f + e);
  return {s, e * s};
}

// unit / nb and the rest, by the multiplier that the launch brings
struct RowBlock {
  uint32_t row, block;
};
__device__ __forceinline__ RowBlock row_block(const SwigluLaunch& a, uint32_t unit, uint32_t nb) {
  const uint32_t row = nb == 1 ? unit : __umulhi(unit, a.magic) >> a.magic_shift;
  return {row, unit - row * nb};
}

// 16 lanes serve one block of 128 columns of a row, U blocks in flight (131072 x
// 2 x 1024: 126 us with one, 120 with two, 122 with four).
template <int DT, bool NT>
__global__ __launch_bounds__(256) void k_swiglu(SwigluLaunch a) {
  constexpr int U = kSwigluUnits;
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
    const RowBlock rb = row_block(a, unit, nb);
    row[j] = rb.row;
    c[j] = (int)rb.block * 16 + l16;
    in[j] = unit < units && c[j] < chunks;
    const uint16_t* p = a.a + row[j] * a.lda + (int64_t)c[j] * 8;
    gv[j] = in[j] ? load16<NT>(p) : u32x4{};
    uv[j] = in[j] ? load16<NT>(p + a.N) : u32x4{};
  }
#pragma unroll
  for (int j = 0; j < U; ++j) {
    float g[8], u[8], amax = 0.0f;
    unpack8<DT>(gv[j], g);
    unpack8<DT>(uv[j], u);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      g[e] = g[e] * sigmoid(g[e]).s * u[e];
      amax = fmaxf(amax, fabsf(g[e]));
    }
    if (a.y && in[j]) store<NT>(a.y + row[j] * a.ldy + (int64_t)c[j] * 8, pack8<DT>(g));
    if (!a.q) continue;
    const float s = block_scale(max16(amax));
    if (in[j]) {
      store<NT>(a.q + row[j] * a.ldq + (int64_t)c[j] * 8, codes8(g, s));
      if (l16 == 0) a.scales[row[j] * a.lds + c[j] / 16] = s;
    }
  }
}

// PAIR: a thread makes the same columns of both halves of da, whose blocks of
// 128 do not mix (or which leaves in 16 bits).  Otherwise a block may hold the
// gate's last columns and the up projection's first: a thread makes eight
// columns of da, and the inputs are read twice.
template <int DT, bool Q, bool PAIR, bool NT>
__global__ __launch_bounds__(256) void k_swiglu_bwd(SwigluLaunch a) {
  const int group = threadIdx.x >> 4, l16 = threadIdx.x & 15;
  const int cols = PAIR ? a.N : 2 * a.N;
  const int nb = (cols + 127) / 128, chunks = cols / 8, half = a.N / 8;
  const int64_t used = a.live ? max((int64_t)0, min(a.rows, (int64_t)*a.live - a.row0)) : a.rows;
  const RowBlock rb = row_block(a, blockIdx.x * 16 + group, nb);
  const int64_t row = rb.row;
  const int c = (int)rb.block * 16 + l16;
  const bool in = row < used && c < chunks;
  const bool up = !PAIR && c >= half;
  const int cc = up ? c - half : c;
  const uint16_t* p = a.a + row * a.lda + (int64_t)cc * 8;
  float g[8], u[8], d[8], du[8];
  unpack8<DT>(in ? load16<NT>(p) : u32x4{}, g);
  unpack8<DT>(in ? load16<NT>(p + a.N) : u32x4{}, u);
  unpack8<DT>(in ? load16<NT>(a.dact + row * a.ldd + (int64_t)cc * 8) : u32x4{}, d);
  float mg = 0.0f, mu = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const Sigmoid sg = sigmoid(g[e]);
    du[e] = d[e] * g[e] * sg.s;
    g[e] = d[e] * u[e] * sg.s * __builtin_fmaf(g[e], sg.rest, 1.0f);
    if (up) g[e] = du[e];
    mg = fmaxf(mg, fabsf(g[e]));
    mu = fmaxf(mu, fabsf(du[e]));
  }
  if constexpr (!Q) {
    if (!in) return;
    uint16_t* o = a.y + row * a.ldy + (int64_t)c * 8;
    store<NT>(o, pack8<DT>(g));
    store<NT>(o + a.N, pack8<DT>(du));
  } else {
    const float sg = block_scale(max16(mg));
    const float su = PAIR ? block_scale(max16(mu)) : 0.0f;
    if (!in) return;
    uint8_t* o = a.q + row * a.ldq + (int64_t)c * 8;
    float* os = a.scales + row * a.lds + c / 16;
    store<NT>(o, codes8(g, sg));
    if (l16 == 0) *os = sg;
    if constexpr (PAIR) {
      store<NT>(o + a.N, codes8(du, su));
      if (l16 == 0) os[a.N / 128] = su;
    }
  }
}

// Waves a token, as a power of two: enough that a wave asks for its columns at
// once, `ch` chunks a lane (16384 x 8 x 4096 unpermuted with four waves a token
// 242 us, with two 248, with one 257), and more, down to one chunk, where
// tokens do not fill the device.
static int part_shift(int64_t T, int chunks, int ch) {
  int s = 0;
  while (int64_t(64) * ch << s < chunks) ++s;
  while (int64_t(64) << s < chunks && T << s < 8 * (int64_t)device_cu_count()) ++s;
  return s;
}
// workgroups of four waves; a kernel's waves walk on past 2^20 of them
static unsigned wave_grid(int64_t waves) {
  const int64_t need = (waves + 3) / 4, most = int64_t(1) << 20;
  return (unsigned)(need < most ? need : most);
}

// Accesses past the caches (loads of what is read once, stores), by the bytes
// of the largest tensor.  One border for all: the gate and its gradient would gain
// half a microsecond at 4 MB, alone, and nothing with the product beside them.
// 4096 columns, top 8, inner 1024, us alone and with the grouped product that
// writes the input or reads the result (through / past; the gates' with a sigmoid
// that was three instructions shorter):
//                 64 tokens (4 MB)         256 (17 MB)             4096 (268 MB)         16384
//   permute       5.2, 171 / 5.7, 169      5.8, 186 / 5.9, 182     32.7, 478 / 28.7, 450  124 / 107
//   unpermute     5.3, 99 / 5.5, 99        6.9, 112 / 6.0, 112     61, 335 / 53.5, 322    239 / 211
//   its gradient  6.4, 96 / 7.5, 96        9.1, 105 / 8.3, 102     93, 343 / 85, 307      351 / 328
//   gate          5.6, 263 / 5.1, 263      5.7, 286 / 5.1, 286     31.6, 755 / 28.4, 717  121 / 110
//   its gradient  5.6, 91 / 4.9, 90        6.4, 97 / 5.4, 97       48, 296 / 43, 259      187 / 172
static bool past_caches(int64_t bytes) { return bytes >= int64_t(1) << 23; }

hipError_t launch_permute(const PermuteLaunch& args, hipStream_t stream) {
  PermuteLaunch a = args;
  a.shift = part_shift(a.T, a.chunks, kPermuteChunks);
  a.waves = a.T << a.shift;
  const unsigned grid = wave_grid(a.waves);
  if (past_caches(a.T * a.k * a.chunks * 16))
    hipLaunchKernelGGL(k_permute<true>, dim3(grid), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL(k_permute<false>, dim3(grid), dim3(256), 0, stream, a);
  return hipGetLastError();
}

// f with the smallest of 1, 2, 4, 8, 16 that holds k, as a type
template <int KT>
struct SlotCount {
  static constexpr int value = KT;
};
template <class F>
static void by_slots(int k, F f) {
  if (k <= 1) f(SlotCount<1>{});
  else if (k <= 2) f(SlotCount<2>{});
  else if (k <= 4) f(SlotCount<4>{});
  else if (k <= 8) f(SlotCount<8>{});
  else f(SlotCount<16>{});
}

template <int DT, bool NT>
static void launch_unpermute_as(UnpermuteLaunch a, hipStream_t stream) {
  by_slots(a.k, [&](auto n) {
    constexpr int KT = decltype(n)::value;
    a.shift = part_shift(a.T, a.chunks, kUnpermuteChunks<KT>);
    a.waves = a.T << a.shift;
    hipLaunchKernelGGL((k_unpermute<DT, NT, KT>), dim3(wave_grid(a.waves)), dim3(256), 0, stream, a);
  });
}
hipError_t launch_unpermute(const UnpermuteLaunch& a, int dtype, hipStream_t stream) {
  const bool nt = past_caches(a.T * a.k * a.chunks * 16);
  if (dtype == DT_F16)
    nt ? launch_unpermute_as<DT_F16, true>(a, stream) : launch_unpermute_as<DT_F16, false>(a, stream);
  else
    nt ? launch_unpermute_as<DT_BF16, true>(a, stream) : launch_unpermute_as<DT_BF16, false>(a, stream);
  return hipGetLastError();
}

template <int DT, bool Q, bool NT>
static void launch_unpermute_bwd_as(const UnpermuteBwdLaunch& a, hipStream_t stream) {
  by_slots(a.k, [&](auto n) {
    constexpr int KT = decltype(n)::value;
    if (a.chunks > 64)
      hipLaunchKernelGGL((k_unpermute_bwd<DT, Q, NT, KT, 4>), dim3(wave_grid(4 * a.T)), dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL((k_unpermute_bwd<DT, Q, NT, KT, 1>), dim3(wave_grid(a.T)), dim3(256), 0, stream, a);
  });
}
template <int DT>
static void launch_unpermute_bwd_by(const UnpermuteBwdLaunch& a, hipStream_t stream) {
  const bool nt = past_caches(a.T * a.k * a.chunks * 16);
  if (a.q)
    nt ? launch_unpermute_bwd_as<DT, true, true>(a, stream) : launch_unpermute_bwd_as<DT, true, false>(a, stream);
  else
    nt ? launch_unpermute_bwd_as<DT, false, true>(a, stream) : launch_unpermute_bwd_as<DT, false, false>(a, stream);
}
hipError_t launch_unpermute_bwd(const UnpermuteBwdLaunch& a, int dtype, hipStream_t stream) {
  if (dtype == DT_F16)
    launch_unpermute_bwd_by<DT_F16>(a, stream);
  else
    launch_unpermute_bwd_by<DT_BF16>(a, stream);
  return hipGetLastError();
}

// rows of one launch: block numbers stay below 2^27
static int64_t swiglu_rows(int64_t nb) { return (int64_t(1) << 27) / nb; }
// From row `row` on, at most `most`, with nb blocks a row.  The quotient of a
// block number b < 2^27 stands above bit p of b m, m = ceil(2^p / nb) = (2^p + e)
// / nb with e < nb <= 2^(p - 27): b m / 2^p is past b / nb by b e / (2^p nb), less
// than the 1 / nb that the next whole number is away.
static SwigluLaunch swiglu_from(const SwigluLaunch& all, int64_t row, int64_t most, int64_t nb) {
  SwigluLaunch a = all;
  int p = 32;
  while (int64_t(1) << (p - 27) < nb) ++p;
  a.magic = (uint32_t)(((int64_t(1) << p) + nb - 1) / nb);  // (nb == 1 does without)
  a.magic_shift = p - 32;
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

template <int DT>
static void launch_swiglu_as(const SwigluLaunch& a, bool nt, dim3 grid, hipStream_t stream) {
  if (nt)
    hipLaunchKernelGGL((k_swiglu<DT, true>), grid, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((k_swiglu<DT, false>), grid, dim3(256), 0, stream, a);
}
hipError_t launch_swiglu(const SwigluLaunch& all, int dtype, hipStream_t stream) {
  const int64_t nb = ((int64_t)all.N + 127) / 128, most = swiglu_rows(nb);
  const bool nt = past_caches(all.rows * all.N * 4);
  for (int64_t row = 0; row < all.rows; row += most) {
    const SwigluLaunch a = swiglu_from(all, row, most, nb);
    constexpr int per = 16 * kSwigluUnits;
    const dim3 grid((unsigned)((a.rows * nb + per - 1) / per));
    if (dtype == DT_F16)
      launch_swiglu_as<DT_F16>(a, nt, grid, stream);
    else
      launch_swiglu_as<DT_BF16>(a, nt, grid, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT, bool NT>
static void launch_swiglu_bwd_as(const SwigluLaunch& a, bool pair, dim3 grid, hipStream_t stream) {
  if (!a.q) hipLaunchKernelGGL((k_swiglu_bwd<DT, false, true, NT>), grid, dim3(256), 0, stream, a);
  else if (pair) hipLaunchKernelGGL((k_swiglu_bwd<DT, true, true, NT>), grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((k_swiglu_bwd<DT, true, false, NT>), grid, dim3(256), 0, stream, a);
}
hipError_t launch_swiglu_bwd(const SwigluLaunch& all, int dtype, hipStream_t stream) {
  const bool pair = !all.q || all.N % 128 == 0, nt = past_caches(all.rows * all.N * 4);
  const int64_t nb = ((pair ? 1 : 2) * (int64_t)all.N + 127) / 128, most = swiglu_rows(nb);
  for (int64_t row = 0; row < all.rows; row += most) {
    const SwigluLaunch a = swiglu_from(all, row, most, nb);
    const dim3 grid((unsigned)((a.rows * nb + 15) / 16));
    if (dtype == DT_F16)
      nt ? launch_swiglu_bwd_as<DT_F16, true>(a, pair, grid, stream)
         : launch_swiglu_bwd_as<DT_F16, false>(a, pair, grid, stream);
    else
      nt ? launch_swiglu_bwd_as<DT_BF16, true>(a, pair, grid, stream)
         : launch_swiglu_bwd_as<DT_BF16, false>(a, pair, grid, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace gmi
