// kernels_route.hip -- expert routing: the top-k experts of every token, their
// weights, rows per expert with the row order the grouped GEMM calls take, and
// the balance loss; and the gradient of the logits.
//
//   p = softmax(logits) over the E experts of a live token
//   weights: p of the k largest logits (equal ones: lowest expert first), divided by their sum on request
//   loss = E sum_e f_e P_e, f_e = counts_e / sum counts, P_e = mean of p_e over the live tokens
// A token is live if the mask keeps it and some logit lies above -infinity;
// an expert whose logit is -infinity (or NaN) is never taken.  Missing slots
// hold expert -1 and weight 0 and are not counted.
//
// A group of L lanes (16, or 64 past 256 experts) holds one token's logits in
// registers, V per lane, expert e = j L + lane.  Each of the k picks is a
// maximum over V registers and four (six) lane exchanges; for 16-bit logits
// value and expert share one 32-bit key, so that the exchange settles ties.
// Order within an expert: a bitmask per expert over the 64 tokens of a pass
// gives each slot its rank by counting the bits below it -- no sort, and the
// same result on every run.
//
// Bound by latency, not by bytes or arithmetic: 16384 tokens x 128 bf16 experts,
// top 8, 7.8 us and 8.6 for the second launch (4 MB read in 0.8 at copy rate);
// 16 tokens fp32 5.5 in one launch; backward 6.3 and, 777 x 60, 3.5 (an empty
// launch takes 2.5).
#include <algorithm>

#include "gmi_device.hpp"
#include "gmi_internal.hpp"
#include "gmi_rows.hpp"

namespace gmi {

constexpr int RT_F32 = 3;       // GMI_F32
constexpr int RT_PASS = 64;     // tokens per pass of a workgroup
constexpr int RT_THREADS = 1024;

template <int DT>
__device__ __forceinline__ float logit_at(const void* p, int64_t i) {
  if constexpr (DT == RT_F32)
    return ((const float*)p)[i];
  else
    return from_bits<DT>(((const uint16_t*)p)[i]);
}

template <int CTRL>
__device__ __forceinline__ int dpp_i(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
}
// v of this lane combined with that of the lane 16 (32) further or back, by
// swapping rows (halves) of two copies: no trip through the LDS crossbar
template <class T, class F>
__device__ __forceinline__ T across16(T v, F f) {
  const uint32_t bits = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane16_swap(bits, bits, false, false);
  const uint32_t lo = r[0], hi = r[1];  // (a bit cast of a vector's element takes its first)
  return f(__builtin_bit_cast(T, lo), __builtin_bit_cast(T, hi));
}
template <class T, class F>
__device__ __forceinline__ T across32(T v, F f) {
  const uint32_t bits = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane32_swap(bits, bits, false, false);
  const uint32_t lo = r[0], hi = r[1];  // (a bit cast of a vector's element takes its first)
  return f(__builtin_bit_cast(T, lo), __builtin_bit_cast(T, hi));
}
// reduction over a group of L = 16 or 64 lanes, result in every lane
template <int L, class T, class F>
__device__ __forceinline__ T group_reduce(T v, F f) {
  v = f(v, __builtin_bit_cast(T, dpp_i<0xB1>(__builtin_bit_cast(int, v))));
  v = f(v, __builtin_bit_cast(T, dpp_i<0x4E>(__builtin_bit_cast(int, v))));
  v = f(v, __builtin_bit_cast(T, dpp_i<0x141>(__builtin_bit_cast(int, v))));
  v = f(v, __builtin_bit_cast(T, dpp_i<0x140>(__builtin_bit_cast(int, v))));
  if constexpr (L == 64) {
    v = across16(v, f);
    v = across32(v, f);
  }
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  return group_reduce<L>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int L>
__device__ __forceinline__ uint32_t group_min(uint32_t v) {
  return group_reduce<L>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
  return group_reduce<L>(v, [](float a, float b) { return a + b; });
}

// Order-preserving key of a logit: larger value, larger key; 0 for values that
// are never taken (-infinity, NaN).  -0 and +0 get the same key.
__device__ __forceinline__ uint32_t order_key(float f) {
  if (!(f > -__builtin_inff())) return 0u;
  const uint32_t u = __builtin_bit_cast(uint32_t, f + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
// 16-bit logits: value in the upper half, the expert's complement below it
// (the lowest expert wins a tie); E <= 1024
template <int DT>
__device__ __forceinline__ uint32_t packed_key(float f, int e) {
  if (!(f > -__builtin_inff())) return 0u;
  uint32_t u;
  if constexpr (DT == DT_F16)
    u = __builtin_bit_cast(uint16_t, (_Float16)(f + 0.0f));
  else
    u = __builtin_bit_cast(uint32_t, f + 0.0f) >> 16;
  u = u & 0x8000u ? (~u & 0xffffu) : u | 0x8000u;
  return u << 16 | (0xffffu - (uint32_t)e);
}

// Exclusive prefix sum over n <= 1024 values, one per thread of a
// RT_THREADS workgroup; returns this thread's, and the total in `total`.
__device__ __forceinline__ int block_scan(int v, int* wave_sums, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // inside rows of 16 lanes, then the last lane of a row onto the next one and
  // that of the lower half onto the upper
  int s = v;
  s += __builtin_amdgcn_update_dpp(0, s, 0x111, 0xF, 0xF, false);
  s += __builtin_amdgcn_update_dpp(0, s, 0x112, 0xF, 0xF, false);
  s += __builtin_amdgcn_update_dpp(0, s, 0x114, 0xF, 0xF, false);
  s += __builtin_amdgcn_update_dpp(0, s, 0x118, 0xF, 0xF, false);
  s += __builtin_amdgcn_update_dpp(0, s, 0x142, 0xA, 0xF, false);
  s += __builtin_amdgcn_update_dpp(0, s, 0x143, 0xC, 0xF, false);
  __syncthreads();
  if (lane == 63) wave_sums[wave] = s;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < RT_THREADS / 64; ++i) {
    const int w = wave_sums[i];
    before += i < wave ? w : 0;
    total += w;
  }
  return before + s - v;
}

// loss from the per-expert sums of p and counts (one expert per thread)
__device__ __forceinline__ void write_loss(const RouteLaunch& a, float psum, int count, int total, int live,
                                           float* wave_part) {
  float v = (float)count * psum;
  v = group_sum<64>(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) wave_part[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.0f;
    for (int i = 0; i < RT_THREADS / 64; ++i) s += wave_part[i];
    *a.loss = total > 0 ? (float)a.E * s / ((float)total * (float)live) : 0.0f;
    *a.live = live;
  }
}

// row length of the workgroups' counts and sums: 16-byte loads
__device__ __forceinline__ int route_ld(int E) { return (E + 7) & ~7; }
// Routing of a contiguous range of tokens per workgroup.  Writes indices,
// weights and each slot's rank among the workgroup's slots of its expert
// (into slot_row), and the workgroup's counts and sums of p per expert.  With
// a single workgroup the rest follows at once.
template <int DT, int L, int V>
__global__ __launch_bounds__(RT_THREADS) void k_route(RouteLaunch a) {
  constexpr int GROUPS = RT_THREADS / L, EP = L * V;
  __shared__ uint32_t mask[RT_PASS / 32][EP];
  __shared__ int base[EP];
  __shared__ float psum_lds[RT_THREADS / 64][EP];
  __shared__ int wave_i[RT_THREADS / 64];
  __shared__ float wave_f[RT_THREADS / 64];
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  for (int e = threadIdx.x; e < EP; e += RT_THREADS) {
    base[e] = 0;
    for (int w = 0; w < RT_PASS / 32; ++w) mask[w][e] = 0u;
  }
  float psum[V];
#pragma unroll
  for (int j = 0; j < V; ++j) psum[j] = 0.0f;
  int live_here = 0;
  // a single workgroup with a group per token keeps slot and rank at hand
  int my_sel = -1, my_rank = -1;
  const bool direct = GROUPS == RT_PASS && gridDim.x == 1;
  const int first = blockIdx.x * a.tokens_per_wg, end = min(a.T, first + a.tokens_per_wg);
  __syncthreads();
  for (int t0 = first; t0 < end; t0 += RT_PASS) {
#pragma unroll
    for (int sub = 0; sub < RT_PASS; sub += GROUPS) {
      const int tl = sub + group, t = t0 + tl;
      const bool in = t < end && (!a.mask || a.mask[t]);
      float x[V];
      uint32_t key[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int e = j * L + lane;
        x[j] = in && e < a.E ? logit_at<DT>(a.logits, (int64_t)t * a.ld + e) : -__builtin_inff();
        key[j] = DT == RT_F32 ? order_key(x[j]) : packed_key<DT>(x[j], e);
      }
      int sel = -1;
      float top = 0.0f, val = 0.0f;
      for (int i = 0; i < a.k; ++i) {
        uint32_t m = key[0];
#pragma unroll
        for (int j = 1; j < V; ++j) m = m > key[j] ? m : key[j];
        m = group_max<L>(m);
        int e;
        float f;
        if constexpr (DT == RT_F32) {
          uint32_t at = 0xffffffffu;
#pragma unroll
          for (int j = V - 1; j >= 0; --j) at = key[j] == m ? (uint32_t)(j * L + lane) : at;
          e = (int)group_min<L>(at);
#pragma unroll
          for (int j = 0; j < V; ++j) key[j] = j * L + lane == e ? 0u : key[j];
          f = __builtin_bit_cast(float, m & 0x80000000u ? m & 0x7fffffffu : ~m);
        } else {
          e = (int)(0xffffu - (m & 0xffffu));
#pragma unroll
          for (int j = 0; j < V; ++j) key[j] = key[j] == m ? 0u : key[j];
          const uint32_t u = m >> 16;
          f = from_bits<DT>(u & 0x8000u ? u & 0x7fffu : ~u & 0xffffu);
        }
        if (i == 0) {
          top = f;
          if (m == 0u) break;  // nothing to take: the token is not live
        }
        if (lane == i && m != 0u) {
          sel = e;
          val = f;
        }
      }
      // not-a-number only where a live token holds one (or +infinity)
      const bool live = group_max<L>((uint32_t)(sel >= 0)) != 0u;
      float sum = 0.0f;
      float p[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int e = j * L + lane;
        p[j] = live && e < a.E ? exp_le0(x[j] - top) : 0.0f;
        sum += p[j];
      }
      sum = group_sum<L>(sum);
      const float inv = live ? 1.0f / sum : 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) psum[j] += p[j] * inv;
      live_here += live && lane == 0;
      float w = sel >= 0 ? exp_le0(val - top) : 0.0f;
      const float wsum = a.renorm ? group_sum<L>(w) + (sum - sum) : sum;  // a NaN of the row reaches the weights
      w = sel >= 0 ? w / wsum : 0.0f;
      if (t < end && lane < a.k) {
        a.indices[(int64_t)t * a.k + lane] = sel;
        a.weights[(int64_t)t * a.k + lane] = w;
      }
      if (sel >= 0) atomicOr(&mask[tl >> 5][sel], 1u << (tl & 31));
      if constexpr (GROUPS == RT_PASS) {
        __syncthreads();
        if (t < end && lane < a.k) {
          int r = -1;
          if (sel >= 0) {
            r = base[sel] + __popc(mask[tl >> 5][sel] & ((1u << (tl & 31)) - 1u));
            for (int q = 0; q < tl >> 5; ++q) r += __popc(mask[q][sel]);
          }
          if (direct) {
            my_sel = sel;
            my_rank = r;
          } else {
            a.slot_row[(int64_t)t * a.k + lane] = r;
          }
        }
      }
    }
    if constexpr (GROUPS != RT_PASS) {
      // several passes filled the masks: the ranks in a second walk
      __syncthreads();
      const int n = min(RT_PASS, end - t0) * a.k;
      for (int s = threadIdx.x; s < n; s += RT_THREADS) {
        const int tl = s / a.k;
        const int64_t slot = (int64_t)t0 * a.k + s;
        const int sel = a.indices[slot];
        int r = -1;
        if (sel >= 0) {
          r = base[sel] + __popc(mask[tl >> 5][sel] & ((1u << (tl & 31)) - 1u));
          for (int q = 0; q < tl >> 5; ++q) r += __popc(mask[q][sel]);
        }
        a.slot_row[slot] = r;
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < EP; e += RT_THREADS) {
      int c = base[e];
      for (int w = 0; w < RT_PASS / 32; ++w) {
        c += __popc(mask[w][e]);
        mask[w][e] = 0u;
      }
      base[e] = c;
    }
    __syncthreads();
  }
  // sums of p over the workgroup: the wave's groups, then the waves in order
  // (those that had a token)
  const auto add = [](float x, float y) { return x + y; };
  const int waves = min(RT_THREADS / 64, (end - first + 64 / L - 1) / (64 / L));
  if ((int)threadIdx.x < 64 * waves) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float v = psum[j];
      if constexpr (L == 16) v = across32(across16(v, add), add);
      if ((threadIdx.x & 63) < L) psum_lds[threadIdx.x >> 6][j * L + lane] = v;
    }
    const float lf = group_sum<64>((float)live_here);
    if ((threadIdx.x & 63) == 0) wave_i[threadIdx.x >> 6] = (int)lf;
  }
  __syncthreads();
  int live_wg = 0;
  for (int i = 0; i < waves; ++i) live_wg += wave_i[i];
  const int e = threadIdx.x;
  float ps = 0.0f;
  if (e < a.E)
    for (int i = 0; i < waves; ++i) ps += psum_lds[i][e];
  if (gridDim.x > 1) {
    const int ld = route_ld(a.E);
    if (e < ld) {
      a.wg_counts[(int64_t)blockIdx.x * ld + e] = (uint16_t)base[e];
      a.wg_psum[(int64_t)blockIdx.x * ld + e] = ps;
    }
    if (e == 0) a.wg_live[blockIdx.x] = live_wg;
    return;
  }
  const int cnt = e < a.E ? base[e] : 0;
  int total;
  const int off = block_scan(cnt, wave_i, total);
  if (e < a.E) {
    a.counts[e] = cnt;
    a.offsets[e] = off;
    base[e] = off;
  }
  if (e == 0) a.offsets[a.E] = total;
  __syncthreads();  // base now holds the offsets; ranks were written by this workgroup
  const int slots = a.T * a.k;
  if (direct) {
    if (lane < a.k && group < a.T) {
      const int s = group * a.k + lane, r = my_sel >= 0 ? base[my_sel] + my_rank : -1;
      a.slot_row[s] = r;
      if (r >= 0) a.row_slot[r] = s;
    }
    for (int s = total + threadIdx.x; s < slots; s += RT_THREADS) a.row_slot[s] = -1;
  } else {
    for (int s = threadIdx.x; s < slots; s += RT_THREADS) {
      const int x = a.indices[s];
      if (x >= 0) {
        const int r = base[x] + a.slot_row[s];
        a.slot_row[s] = r;
        a.row_slot[r] = s;
      }
      if (s >= total) a.row_slot[s] = -1;
    }
  }
  write_loss(a, ps, cnt, total, live_wg, wave_f);
}

// Column sums of the workgroups' 16-bit count matrix for expert tid: over all
// workgroups and over those before b.  `part` is 2 x 8 RT_THREADS integers.
__device__ __forceinline__ void sum_counts(const uint16_t* counts, int ld, int E, int wgs, int b,
                                           int32_t (*part)[8 * RT_THREADS], int& st, int& sp) {
  const int tid = threadIdx.x;
  // a team of `team` threads (a power of two) reads one row of the matrix
  int team = 1;
  while (team < ld / 8) team *= 2;
  const int slices = RT_THREADS / team, c = tid % team, sl = tid / team;
  int tot[8], pre[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) tot[i] = pre[i] = 0;
  if (c < ld / 8) {
#pragma unroll 4
    for (int q = sl; q < wgs; q += slices) {
      const u32x4 v = *(const u32x4*)(counts + (int64_t)q * ld + 8 * c);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int n = (int)(i & 1 ? v[i / 2] >> 16 : v[i / 2] & 0xffffu);
        tot[i] += n;
        pre[i] += q < b ? n : 0;
      }
    }
  }
  // the teams of a wave, then the waves (or slices, of teams wider than a wave)
  for (int d = team; d < 64; d *= 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      tot[i] += __shfl_xor(tot[i], d);
      pre[i] += __shfl_xor(pre[i], d);
    }
  }
  const int wide = max(team, 64), groups = RT_THREADS / wide;
  if (tid % wide < team) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      part[0][(tid / wide) * team * 8 + c * 8 + i] = tot[i];
      part[1][(tid / wide) * team * 8 + c * 8 + i] = pre[i];
    }
  }
  __syncthreads();
  st = sp = 0;
  if (tid < E) {
    for (int g = 0; g < groups; ++g) {
      st += part[0][g * team * 8 + tid];
      sp += part[1][g * team * 8 + tid];
    }
  }
}

// Second launch: every workgroup sums the count matrix for itself (totals, and
// what lies before its own tokens), turns the ranks of its slots into rows and
// writes both orders.  One further workgroup writes counts, offsets and loss;
// it has the longest way and so asks for the sums of p before all else.
// Latency is what it costs, so the slots are fetched before the matrix, the
// matrix is 16 bits wide and read eight experts a load: with 256 workgroups and
// 128 experts four loads a thread (32-bit, one expert a load: 15.9 us).
// Eight waves a SIMD: the further workgroup has to find room beside another one
// on a device that the rest fill (with 79 registers and so one workgroup a CU
// the call of 16384 tokens x 128 took 18.8 us for 17.0).
__global__ __launch_bounds__(RT_THREADS, 8) void k_route_place(RouteLaunch a, int wgs) {
  __shared__ int32_t part[2][8 * RT_THREADS];  // partial totals and prefixes, then floats of the sums of p
  __shared__ int row0[RT_THREADS];
  __shared__ int wave_i[RT_THREADS / 64];
  __shared__ float wave_f[RT_THREADS / 64];
  const int b = blockIdx.x, tid = threadIdx.x, ld = route_ld(a.E);
  const bool last = b == wgs;
  const int64_t s0 = (int64_t)b * a.tokens_per_wg * a.k;
  const int64_t s1 = last ? s0 : min((int64_t)a.T * a.k, s0 + (int64_t)a.tokens_per_wg * a.k);
  int x = -1, r = 0;
  if (s0 + tid < s1) {
    x = a.indices[s0 + tid];
    r = a.slot_row[s0 + tid];
  }
  // sums of p: a team of `four` threads reads one row, four experts a load
  int four = 1, live = 0;
  while (four < ld / 4) four *= 2;
  const int fc = tid % four;
  f32x4 ps{};
  if (last) {
    if (fc < ld / 4) {
#pragma unroll 8
      for (int q = tid / four; q < wgs; q += RT_THREADS / four) ps += *(const f32x4*)(a.wg_psum + (int64_t)q * ld + 4 * fc);
    }
    for (int q = tid; q < wgs; q += RT_THREADS) live += a.wg_live[q];
  }
  int st, sp;
  sum_counts(a.wg_counts, ld, a.E, wgs, b, part, st, sp);
  int total;
  const int off = block_scan(st, wave_i, total);
  row0[tid] = off + sp;
  __syncthreads();
  if (last) {
    if (tid < a.E) {
      a.counts[tid] = st;
      a.offsets[tid] = off;
    }
    if (tid == 0) a.offsets[a.E] = total;
    // the lanes of a wave that hold the same experts, then the waves
    float* fp = (float*)part[0];
    for (int d = four; d < 64; d *= 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) ps[i] += __shfl_xor(ps[i], d);
    }
    const int wide4 = max(four, 64);
    if (tid % wide4 < four) *(f32x4*)(fp + (tid / wide4) * four * 4 + fc * 4) = ps;
    int live_all;
    block_scan(live, wave_i, live_all);  // its barriers publish the sums too
    float sf = 0.0f;
    if (tid < a.E)
      for (int g = 0; g < RT_THREADS / wide4; ++g) sf += fp[g * four * 4 + tid];
    write_loss(a, sf, st, total, live_all, wave_f);
    return;
  }
  for (int64_t s = s0 + tid; s < s1;) {
    if (x >= 0) {
      r += row0[x];
      a.slot_row[s] = r;
      a.row_slot[r] = (int)s;
    }
    if (s >= total) a.row_slot[s] = -1;  // rows past the last one; s runs over every row number too
    s += RT_THREADS;
    if (s < s1) {
      x = a.indices[s];
      r = a.slot_row[s];
    }
  }
}

// Rows ordered by a number each carries.  A pass of a workgroup takes one row
// per thread: the lanes of a wave that hold the same group find each other by
// ballots over the number's bits, so a row's rank is a count of bits below its
// lane, plus what earlier waves and passes put into the group.  Rows of no
// group are a group of their own behind the others, whose counts go nowhere.
// With one workgroup the places follow at once; otherwise the ranks wait in
// `place` for k_group_place.
// Latency bounds it: 64 rows 2.8 us (an empty launch 2.5), 131072 rows into 128
// groups 4.0 and 6.6 in the second launch.
__global__ __launch_bounds__(RT_THREADS) void k_group(GroupLaunch a) {
  __shared__ uint16_t hist[RT_THREADS / 64][kMaxGroups + 8];
  __shared__ int base[kMaxGroups + 8];
  __shared__ int wave_i[RT_THREADS / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int first = blockIdx.x * a.rows_per_wg, end = min(a.n, first + a.rows_per_wg);
  for (int g = tid; g <= a.G; g += RT_THREADS) {
    base[g] = 0;
    for (int w = 0; w < RT_THREADS / 64; ++w) hist[w][g] = 0;
  }
  __syncthreads();
  for (int s0 = first; s0 < end; s0 += RT_THREADS) {
    const int s = s0 + tid;
    const bool in = s < end;
    int g = in ? a.index[s] : 0;
    if ((uint32_t)g >= (uint32_t)a.G) g = a.G;
    uint64_t same = __ballot(in);
    for (int bit = 0; 1 << bit <= a.G; ++bit) {
      const uint64_t set = __ballot(g >> bit & 1);
      same &= g >> bit & 1 ? set : ~set;
    }
    const int before = __popcll(same & ((1ull << lane) - 1ull));
    if (in && before == 0) hist[wave][g] = (uint16_t)__popcll(same);
    __syncthreads();
    if (in) {
      int r = base[g] + before;
      for (int w = 0; w < wave; ++w) r += hist[w][g];
      a.place[s] = r;
    }
    __syncthreads();
    for (int q = tid; q <= a.G; q += RT_THREADS) {
      int c = base[q];
      for (int w = 0; w < RT_THREADS / 64; ++w) {
        c += hist[w][q];
        hist[w][q] = 0;
      }
      base[q] = c;
    }
    __syncthreads();
  }
  if (gridDim.x > 1) {
    const int ld = route_ld(a.G);
    if (tid < ld) a.wg_counts[(int64_t)blockIdx.x * ld + tid] = tid < a.G ? (uint16_t)base[tid] : 0;
    return;
  }
  int total;
  const int off = block_scan(tid < a.G ? base[tid] : 0, wave_i, total);
  if (tid < a.G) {
    a.offsets[tid] = off;
    base[tid] = off;
  }
  if (tid == 0) {
    a.offsets[a.G] = total;
    base[a.G] = total;
  }
  __syncthreads();
  for (int s = tid; s < a.n; s += RT_THREADS) {
    int g = a.index[s];
    if ((uint32_t)g >= (uint32_t)a.G) g = a.G;
    const int r = base[g] + a.place[s];  // this thread's own rank
    a.order[r] = s;
    a.place[s] = g < a.G ? r : -1;
  }
}

// Every workgroup sums the count matrix for itself, as k_route_place does, and
// turns its rows' ranks into places.
__global__ __launch_bounds__(RT_THREADS) void k_group_place(GroupLaunch a, int wgs) {
  __shared__ int32_t part[2][8 * RT_THREADS];
  __shared__ int row0[kMaxGroups + 1];
  __shared__ int wave_i[RT_THREADS / 64];
  const int b = blockIdx.x, tid = threadIdx.x;
  const int first = b * a.rows_per_wg, end = min(a.n, first + a.rows_per_wg);
  int s = first + tid;
  int g = 0, r = 0;
  if (s < end) {
    g = a.index[s];
    r = a.place[s];
  }
  int st, sp;
  sum_counts(a.wg_counts, route_ld(a.G), a.G, wgs, b, part, st, sp);
  int total, before;
  const int off = block_scan(st, wave_i, total);
  block_scan(sp, wave_i, before);
  if (tid < a.G) row0[tid] = off + sp;
  if (tid == 0) row0[a.G] = total + first - before;  // rows of no group before this workgroup
  if (b == 0) {
    if (tid < a.G) a.offsets[tid] = off;
    if (tid == 0) a.offsets[a.G] = total;
  }
  __syncthreads();
  while (s < end) {
    if ((uint32_t)g >= (uint32_t)a.G) g = a.G;
    r += row0[g];
    a.order[r] = s;
    a.place[s] = g < a.G ? r : -1;
    s += RT_THREADS;
    if (s < end) {
      g = a.index[s];
      r = a.place[s];
    }
  }
}

// LDS written by one lane of a wave and read by another: the LDS serves a
// wave's accesses in order, so only the compiler has to keep it
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Gradient of the logits.  dp_e = dloss E f_e / live is the loss's, the
// weights' comes in at the taken experts: before the softmax's own derivative
// without renormalisation, after it as that of a softmax over the taken ones
// with it.  The k scattered values of a token go through a row of LDS that its
// lanes share (a wave keeps its rows to itself, so no barrier).
template <int DT, int L, int V>
__global__ __launch_bounds__(256) void k_route_bwd(RouteBwdLaunch a) {
  constexpr int GROUPS = 256 / L, EP = L * V;
  __shared__ float row_lds[GROUPS][EP];
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  float* row = row_lds[group];
  float dp0[V];
  const int total = a.offsets[a.E], live_n = *a.live;
  const float g = total > 0 && live_n > 0 ? *a.dloss * (float)a.E / ((float)total * (float)live_n) : 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = j * L + lane;
    dp0[j] = e < a.E ? g * (float)(a.offsets[e + 1] - a.offsets[e]) : 0.0f;
    row[e] = 0.0f;
  }
  wave_fence();
  for (int64_t t0 = (int64_t)blockIdx.x * GROUPS; t0 < a.T; t0 += (int64_t)gridDim.x * GROUPS) {
    const int64_t t = t0 + group;
    const bool in = t < a.T && (!a.mask || a.mask[t]);
    float x[V];
    float top = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = j * L + lane;
      x[j] = in && e < a.E ? logit_at<DT>(a.logits, t * a.ld + e) : -__builtin_inff();
      top = fmaxf(top, x[j]);
    }
    int sel = -1;
    float dw = 0.0f, w = 0.0f;
    if (in && lane < a.k) {
      sel = a.indices[t * a.k + lane];
      if (sel >= a.E) sel = -1;
      if (sel >= 0) {
        dw = a.dweights[t * a.k + lane];
        w = a.weights[t * a.k + lane];
      }
    }
    top = group_reduce<L>(top, [](float p, float q) { return fmaxf(p, q); });
    const bool live = top > -__builtin_inff();
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = j * L + lane;
      x[j] = live && e < a.E ? exp_le0(x[j] - top) : 0.0f;
      sum += x[j];
    }
    sum = group_sum<L>(sum);
    const float inv = live ? 1.0f / sum : 0.0f;
    float add = dw;
    if (a.renorm) add = w * (dw - group_sum<L>(w * dw));
    if (sel >= 0) row[sel] = add;
    wave_fence();
    float sc[V], dot = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      sc[j] = row[j * L + lane];
      x[j] *= inv;
      dot = __builtin_fmaf(x[j], a.renorm ? dp0[j] : dp0[j] + sc[j], dot);
    }
    dot = group_sum<L>(dot);
    wave_fence();
    if (sel >= 0) row[sel] = 0.0f;
    wave_fence();
    if (t < a.T) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int e = j * L + lane;
        float d = a.renorm ? __builtin_fmaf(x[j], dp0[j] - dot, sc[j]) : x[j] * (dp0[j] + sc[j] - dot);
        if (!live) d = 0.0f;
        if (e < a.E) {
          if constexpr (DT == RT_F32)
            ((float*)a.dlogits)[t * a.ldd + e] = d;
          else
            ((uint16_t*)a.dlogits)[t * a.ldd + e] = (uint16_t)to_bits<DT>(d);
        }
      }
    }
  }
}

// lanes per token and experts per lane: 16 lanes up to 256 experts, then 64
#define GMI_ROUTE_V(KER, DT, E, grid, wg, stream, ...)                                              \
  do {                                                                                              \
    if ((E) <= 64) hipLaunchKernelGGL((KER<DT, 16, 4>), dim3(grid), dim3(wg), 0, stream, __VA_ARGS__);       \
    else if ((E) <= 128) hipLaunchKernelGGL((KER<DT, 16, 8>), dim3(grid), dim3(wg), 0, stream, __VA_ARGS__); \
    else if ((E) <= 256) hipLaunchKernelGGL((KER<DT, 16, 16>), dim3(grid), dim3(wg), 0, stream, __VA_ARGS__); \
    else if ((E) <= 512) hipLaunchKernelGGL((KER<DT, 64, 8>), dim3(grid), dim3(wg), 0, stream, __VA_ARGS__); \
    else hipLaunchKernelGGL((KER<DT, 64, 16>), dim3(grid), dim3(wg), 0, stream, __VA_ARGS__);       \
  } while (0)
#define GMI_ROUTE(KER, dtype, E, grid, wg, stream, ...)                                  \
  do {                                                                                   \
    if ((dtype) == DT_F16) GMI_ROUTE_V(KER, DT_F16, E, grid, wg, stream, __VA_ARGS__);   \
    else if ((dtype) == DT_BF16) GMI_ROUTE_V(KER, DT_BF16, E, grid, wg, stream, __VA_ARGS__); \
    else GMI_ROUTE_V(KER, RT_F32, E, grid, wg, stream, __VA_ARGS__);                     \
  } while (0)

RoutePlan plan_route(int T, int E) {
  RoutePlan p;
  const int64_t passes = ((int64_t)T + RT_PASS - 1) / RT_PASS;
  // 256 workgroups: the second launch reads every workgroup's counts, which
  // have 16 bits (one workgroup for no tokens at all: it writes the zero counts)
  const int64_t per = std::min<int64_t>((passes + 255) / 256, 65535 / RT_PASS);
  p.tokens_per_wg = (int)(std::max<int64_t>(per, 1) * RT_PASS);
  p.wgs = passes > 0 ? (int)((passes + per - 1) / per) : 1;
  p.bytes = p.wgs > 1 ? (size_t)p.wgs * ((size_t)((E + 7) / 8 * 8) * 6 + 4) : 0;
  return p;
}

hipError_t launch_route(const RouteLaunch& args, int dtype, void* workspace, hipStream_t stream) {
  RouteLaunch a = args;
  const RoutePlan p = plan_route(a.T, a.E);
  a.tokens_per_wg = p.tokens_per_wg;
  if (p.wgs > 1) {
    const size_t ld = (size_t)(a.E + 7) / 8 * 8;
    a.wg_psum = (float*)workspace;
    a.wg_counts = (uint16_t*)(a.wg_psum + p.wgs * ld);
    a.wg_live = (int32_t*)(a.wg_counts + p.wgs * ld);
  }
  GMI_ROUTE(k_route, dtype, a.E, p.wgs, RT_THREADS, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.wgs == 1) return e;
  hipLaunchKernelGGL(k_route_place, dim3(p.wgs + 1), dim3(RT_THREADS), 0, stream, a, p.wgs);
  return hipGetLastError();
}

hipError_t launch_route_bwd(const RouteBwdLaunch& a, int dtype, hipStream_t stream) {
  const int groups = a.E <= 256 ? 16 : 4;
  const int64_t need = ((int64_t)a.T + groups - 1) / groups, most = 4 * (int64_t)device_cu_count();
  const unsigned grid = (unsigned)(need < most ? need : most);
  GMI_ROUTE(k_route_bwd, dtype, a.E, grid, 256, stream, a);
  return hipGetLastError();
}

GroupPlan plan_group(int n, int G) {
  GroupPlan p;
  // One launch up to two passes of a workgroup (2048 rows into 128 groups 6.4 us,
  // two launches 8.5; four passes, 4096 rows, 10.8 against 8.6); then 256
  // workgroups, whose counts have 16 bits
  const int64_t passes = ((int64_t)n + RT_THREADS - 1) / RT_THREADS;
  const int64_t per = passes <= 2 ? std::max<int64_t>(passes, 1)
                                  : std::min<int64_t>((passes + 255) / 256, 65535 / RT_THREADS);
  p.rows_per_wg = (int)(per * RT_THREADS);
  p.wgs = (int)std::max<int64_t>((passes + per - 1) / per, 1);
  p.bytes = p.wgs > 1 ? (size_t)p.wgs * ((G + 7) / 8 * 8) * 2 : 0;
  return p;
}

hipError_t launch_group(const GroupLaunch& args, void* workspace, hipStream_t stream) {
  GroupLaunch a = args;
  const GroupPlan p = plan_group(a.n, a.G);
  a.rows_per_wg = p.rows_per_wg;
  a.wg_counts = (uint16_t*)workspace;
  hipLaunchKernelGGL(k_group, dim3(p.wgs), dim3(RT_THREADS), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.wgs == 1) return e;
  hipLaunchKernelGGL(k_group_place, dim3(p.wgs), dim3(RT_THREADS), 0, stream, a, p.wgs);
  return hipGetLastError();
}

}  // namespace gmi
