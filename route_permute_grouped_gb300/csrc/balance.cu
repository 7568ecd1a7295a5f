// The router's auxiliary losses from its logits and the selected experts: the
// sequence-wise balance loss and the z-loss with the expert counts of every
// sequence (forward), and the gradient of the logits (backward).
#include <math.h>

#include <algorithm>

#include "host_util.h"
#include "mma.cuh"

namespace moe {

// Rows are handled by groups of G lanes, each lane holding NV sets of four
// consecutive experts (set j: experts 4 (lane + G j) ..): 4 G NV >= E. A group
// takes kBalUnroll rows at a time, so that their loads and the latencies of
// their reductions overlap.
constexpr int kBalThreads = 256;
constexpr int kBalWarps = kBalThreads / 32;
constexpr int kBalUnroll = 2;

// The forward's blocks take equal runs of CH rows, whatever sequences lie in
// them (their partial sums would otherwise come from as many short blocks as
// there are ends of sequences). Block b's part of sequence s goes to slot b + s:
// along the rows the pairs (b, s) step up one at a time in b or s, so each has a
// slot of its own and those of a sequence are neighbours.
__device__ __forceinline__ int seq_begin(const int32_t* off, int s, int S, int T) {
  if (off == nullptr) return s == 0 ? 0 : T;
  const int v = off[s];
  return v < 0 ? 0 : (v > T ? T : v);
}

// number of s in [0, S) with key(s) <= c, by the whole block
template <class F>
__device__ __forceinline__ int count_le(int S, F key, int c) {
  int n = 0;
  for (int s0 = 0; s0 < S; s0 += static_cast<int>(blockDim.x)) {
    const int s = s0 + static_cast<int>(threadIdx.x);
    n += __syncthreads_count(s < S && key(s) <= c);
  }
  return n;
}

// Two floats in one 64-bit register and the packed arithmetic on them (one
// instruction for two elements).
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ f2 both(float a) { return pack2(a, a); }
__device__ __forceinline__ float2 unpack2(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float side_sum(f2 v) {
  const float2 x = unpack2(v);
  return x.x + x.y;
}

// Rows of whole 16-byte pieces (VEC) come through shared memory, two passes of a
// warp ahead: each lane copies the pieces that it will hold, so no other thread's
// copies are waited for, and its registers stay free for the rows at hand (loads to
// registers: 131021 x 256 sigmoid both ways 90.5 us for 83, 65536 x 256 softmax 43
// for 39).
constexpr int kAhead = 2;
template <int NV>
using RowRing = float4[kAhead][kBalUnroll][NV][kBalThreads];
template <int G, int NV, bool VEC>
__device__ __forceinline__ void ask_row(RowRing<NV>& ring, int slot, int u, const float* row, int E, int gl) {
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = 4 * (gl + G * j);
      if (e < E) cp_async16(smem_u32(&ring[slot][u][j][threadIdx.x]), row + e, true);
    }
  }
}
// `top`: the largest |logit| this lane has loaded so far. Places behind the last
// expert hold a finite value whose exponential is 0 (row_scores).
constexpr float kNoExpert = -1e30f;
template <int G, int NV, bool VEC>
__device__ __forceinline__ void load_row(const RowRing<NV>& ring, int slot, int u, const float* row, int E, int gl,
                                         f2 (&v)[2 * NV], float& top) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = 4 * (gl + G * j);
    float x[4] = {kNoExpert, kNoExpert, kNoExpert, kNoExpert};
    if constexpr (VEC) {
      if (e < E) {
        const float4 q = ring[slot][u][j][threadIdx.x];
        x[0] = q.x; x[1] = q.y; x[2] = q.z; x[3] = q.w;
        top = fmaxf(fmaxf(top, fmaxf(fabsf(x[0]), fabsf(x[1]))), fmaxf(fabsf(x[2]), fabsf(x[3])));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e + i < E) {
          x[i] = row[e + i];
          top = fmaxf(top, fabsf(x[i]));
        }
    }
    v[2 * j] = pack2(x[0], x[1]);
    v[2 * j + 1] = pack2(x[2], x[3]);
  }
}
template <int G>
__device__ __forceinline__ float group_max(float x) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
// The sums of a and of b over the lanes of a group: the halves of the group
// exchange one of the two first, so each reduces one value (G = 32: 6 shuffles
// for two sums instead of 10). half_sum leaves the sum of b in the group's upper
// half and that of a in the lower one, swap_halves gives both to every lane.
template <int G>
__device__ __forceinline__ float half_sum(float a, float b, int gl) {
  const bool up = (gl & (G / 2)) != 0;
  float keep = (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, G / 2);
#pragma unroll
  for (int o = G / 4; o > 0; o >>= 1) keep += __shfl_xor_sync(0xffffffffu, keep, o);
  return keep;
}
template <int G>
__device__ __forceinline__ void swap_halves(float keep, float& a, float& b, int gl) {
  const bool up = (gl & (G / 2)) != 0;
  const float other = __shfl_xor_sync(0xffffffffu, keep, G / 2);
  a = up ? other : keep;
  b = up ? keep : other;
}
template <int G>
__device__ __forceinline__ void group_sum2(float& a, float& b, int gl) {
  swap_halves<G>(half_sum<G>(a, b, gl), a, b, gl);
}

// The score functions of the kBalUnroll = 2 rows of a group. On return v holds
// exp(l - m), `inv` the inverse of their sum and `lse` the log-sum-exp; for
// sigmoid scores s holds the sigmoids and `sinv` the inverse of their sum. The
// backward (BWD) has in s the slopes sigmoid (1 - sigmoid) instead, and in `dot`
// the sum of the unnormalised scores times w.
//
// What bounds a row beside its bytes is its instructions (the first kernels: 36
// an element, 113 us for 131021 x 256 sigmoid scores; these: 36 us) and the
// special functions among them (16 a clock and SM). So m is 0 (NEAR) as long as no
// logit of the warp's rows is beyond 40 in magnitude: no maximum is reduced, one
// exponential x = exp(l) serves both scores, sigmoid(l) = x / (1 + x) and
// 1 - sigmoid(l) = 1 / (1 + x) without cancellation, and the sum stays below
// 256 e^40. Rows with larger logits take m = max l and exp(-|l|); where m < 0 their
// sigmoids exp(l) / (1 + exp(l)) come without the factor exp(m), which their sum
// has too: below -88 it leaves fp32's range.
// exp(l) is 2^h (1 + c) with h = round(l log2 e) and c = l - h ln 2, what the
// rounding of h has left (one fused product; c^2 is below 2^-38): without c every
// row that lies around 35 would be off by half a step of 50, 7.5e-7 of its
// probabilities in the mean. Behind a subtracted maximum c is not needed: h is off
// by half a step of itself, as l - m is. The logarithm and the reciprocal of a
// row's sum are taken once for each half of the group's lanes, a row for each.
constexpr float kNear = 40.0f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float ex2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
template <int G, int NV, bool SIG, bool BWD, bool NEAR, class Weights>
__device__ __forceinline__ void row_scores(int gl, int E, bool need_lse, f2 (&v)[kBalUnroll][2 * NV],
                                           f2 (&s)[kBalUnroll][2 * NV], const f2 (&w)[2 * NV], Weights weights_of,
                                           float (&inv)[kBalUnroll], float (&lse)[kBalUnroll],
                                           float (&sinv)[kBalUnroll], float (&dot)[kBalUnroll]) {
  static_assert(kBalUnroll == 2, "the sums are reduced in pairs");
  float sum[2], ssum[2], m[2] = {0.0f, 0.0f};
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    if constexpr (!NEAR) {
      m[u] = -INFINITY;
#pragma unroll
      for (int i = 0; i < 2 * NV; ++i) {
        const int e = 4 * (gl + G * (i >> 1)) + 2 * (i & 1);
        const float2 l = unpack2(v[u][i]);
        v[u][i] = pack2(e < E ? l.x : -INFINITY, e + 1 < E ? l.y : -INFINITY);
        const float2 k = unpack2(v[u][i]);
        m[u] = fmaxf(m[u], fmaxf(k.x, k.y));
      }
      m[u] = group_max<G>(m[u]);
    }
    weights_of(u);  // into w
    f2 sum2 = both(0.0f), ssum2 = both(0.0f), dot2 = both(0.0f);
#pragma unroll
    for (int i = 0; i < 2 * NV; ++i) {
      const f2 l2 = v[u][i];
      const f2 h2 = mul2(NEAR ? l2 : add2(l2, both(-m[u])), both(kLog2e));
      const float2 x = unpack2(h2);
      v[u][i] = pack2(ex2_approx(x.x), ex2_approx(x.y));
      if constexpr (NEAR) v[u][i] = fma2(v[u][i], fma2(h2, both(-kLn2), l2), v[u][i]);
      sum2 = add2(sum2, v[u][i]);
      if constexpr (SIG) {
        f2 a, b;
        if constexpr (NEAR) {
          const float2 o = unpack2(add2(v[u][i], both(1.0f)));
          b = pack2(rcp_approx(o.x), rcp_approx(o.y));
          a = mul2(v[u][i], b);
        } else {
          const float2 l = unpack2(l2);
          const float tx = expf(-fabsf(l.x)), ty = expf(-fabsf(l.y));
          const float rx = rcp_approx(1.0f + tx), ry = rcp_approx(1.0f + ty);
          const float2 q = unpack2(v[u][i]);  // (m < 0: no l is above 0)
          a = pack2(l.x >= 0.0f ? rx : (m[u] < 0.0f ? q.x : tx) * rx, l.y >= 0.0f ? ry : (m[u] < 0.0f ? q.y : ty) * ry);
          b = pack2(l.x >= 0.0f ? tx * rx : rx, l.y >= 0.0f ? ty * ry : ry);
        }
        s[u][i] = BWD ? mul2(a, b) : a;
        // the softmax of a row with a logit of +inf is no number, but only the z-loss wants it
        if (!NEAR && !need_lse) v[u][i] = both(0.0f);
        ssum2 = add2(ssum2, a);
        if constexpr (BWD) dot2 = fma2(a, w[i], dot2);
      } else if constexpr (BWD) {
        dot2 = fma2(v[u][i], w[i], dot2);
      }
    }
    sum[u] = side_sum(sum2);
    ssum[u] = SIG ? side_sum(ssum2) : 0.0f;
    dot[u] = BWD ? side_sum(dot2) : 0.0f;
  }
  const float half = half_sum<G>(sum[0], sum[1], gl);
  swap_halves<G>(rcp_approx(half), inv[0], inv[1], gl);
  lse[0] = lse[1] = 0.0f;
  if (need_lse) {
    swap_halves<G>(logf(half), lse[0], lse[1], gl);
    lse[0] += m[0];
    lse[1] += m[1];
  }
  if constexpr (SIG) swap_halves<G>(rcp_approx(half_sum<G>(ssum[0], ssum[1], gl)), sinv[0], sinv[1], gl);
  if constexpr (BWD) group_sum2<G>(dot[0], dot[1], gl);
}

// A sum in two floats: s + e is the exact sum so far but for the roundings of e.
// For sums of many partial sums in a fixed order (fp64 additions run at about two
// a clock and SM: a block-wide fp64 tree took 36 us where this takes one).
struct Sum2 {
  float s = 0.0f, e = 0.0f;
  __device__ __forceinline__ void add(float x) {
    const float t = s + x, b = t - s;
    e += (s - (t - b)) + (x - b);
    s = t;
  }
  __device__ __forceinline__ void add(const Sum2& o) {
    add(o.s);
    e += o.e;
  }
  // e of an infinite sum is not a number
  __device__ __forceinline__ float value() const { return isfinite(s) ? s + e : s; }
};
__device__ __forceinline__ Sum2 warp_sum(Sum2 x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sum2 y;
    y.s = __shfl_xor_sync(0xffffffffu, x.s, o);
    y.e = __shfl_xor_sync(0xffffffffu, x.e, o);
    x.add(y);
  }
  return x;
}
__device__ __forceinline__ int warp_sum(int x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

struct BalParams {
  const float* logits;
  const int32_t* topk;
  const int32_t* off;
  const uint8_t* mask;
  int T, E, k, S, CH, slots;
  int sigmoid, need_lse;  // need_lse: z_coeff is not 0
  float balance_coeff, z_coeff;
  // workspace
  float* part_p;      // [slots][E] sums of p
  int32_t* part_c;    // [slots][E] counts
  float* part_z;      // [slots] sums of lse^2
  int32_t* part_n;    // [slots] valid rows
  float2* seq_b;      // [S][32-expert groups] balance loss of each sequence (before the mean over sequences)
  float2* seq_z;      // [S] sum of lse^2
  int32_t* seq_n;     // [S]
  int* ticket;
  // outputs
  int32_t* counts;
  float* losses;
  float* stats;
  DevStatus* st;
};

// Forward, first pass: each block's sums of p, counts, sum of lse^2 and number
// of valid rows for every sequence in its rows. Bound by HBM and, beside it, its
// instructions (131021 x 256 sigmoid: 134 MB in 36 us, 3.7 TB/s; 65536 x 256
// softmax: 67 MB in 18). The sums over rows stay in registers, one set per lane
// group, and are joined over the groups and warps in a fixed order.
struct BalChunk {
  int lo, hi;
};
template <int G, int NV, bool VEC, bool SIG>
__device__ __forceinline__ void part_of_sequence(const BalParams& p, const BalChunk ch, int slot) {
  __shared__ int s_cnt[256];
  __shared__ float s_sum[kBalWarps][256];
  __shared__ float s_z[kBalWarps];
  __shared__ int s_n[kBalWarps];
  __shared__ RowRing<NV> s_rows;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gl = lane & (G - 1), grp = lane / G;
  constexpr int RPW = 32 / G, U = kBalUnroll, kPass = U * kBalWarps * RPW;
  const auto row_of = [&](int t0, int u) { return t0 + u * kBalWarps * RPW + grp; };
  const auto valid = [&](int t) { return t < ch.hi && (p.mask == nullptr || p.mask[t] != 0); };
  const auto ask = [&](int t0, int slot) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = row_of(t0, u);
      if (VEC && valid(t)) ask_row<G, NV, VEC>(s_rows, slot, u, p.logits + static_cast<size_t>(t) * p.E, p.E, gl);
    }
    if (VEC) cp_async_commit();
  };
  const int first = ch.lo + warp * RPW;
  for (int i = 0; i < kAhead; ++i) ask(first + i * kPass, i);
  __syncthreads();  // the last sequence's sums have been read
  s_cnt[tid] = 0;
  __syncthreads();
  // the selected experts of the valid rows
  const int slots = (ch.hi - ch.lo) * p.k;
  const int32_t* idx = p.topk + static_cast<size_t>(ch.lo) * p.k;
  for (int i = tid; i < slots; i += kBalThreads) {
    if (p.mask != nullptr && p.mask[ch.lo + i / p.k] == 0) continue;
    const int e = __ldcg(idx + i);
    if (e < 0 || e >= p.E) set_status(p.st, MOE_ERR_DEVICE_INDEX, 50);
    else atomicAdd(&s_cnt[e], 1);
  }
  f2 acc2[2 * NV];
#pragma unroll
  for (int i = 0; i < 2 * NV; ++i) acc2[i] = both(0.0f);
  float z = 0.0f;
  int n = 0;
  for (int t0 = first, slot = 0; t0 < ch.hi; t0 += kPass, slot ^= 1) {
    f2 v[U][2 * NV];
    float top = 0.0f;
    bool ok[U];
    if (VEC) cp_async_wait<kAhead - 1>();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = row_of(t0, u);
      ok[u] = valid(t);
      if (ok[u]) {
        load_row<G, NV, VEC>(s_rows, slot, u, p.logits + static_cast<size_t>(t) * p.E, p.E, gl, v[u], top);
      } else {
#pragma unroll
        for (int i = 0; i < 2 * NV; ++i) v[u][i] = both(0.0f);
      }
    }
    const bool near = __all_sync(0xffffffffu, top <= kNear);
    ask(t0 + kAhead * kPass, slot);  // (what the slot held has been read: `near` needed it)
    f2 s[U][2 * NV];
    float inv[U], lse[U], sinv[U], dot[U];
    const auto none = [](int) {};
    if (near) row_scores<G, NV, SIG, false, true>(gl, p.E, p.need_lse, v, s, acc2, none, inv, lse, sinv, dot);
    else row_scores<G, NV, SIG, false, false>(gl, p.E, p.need_lse, v, s, acc2, none, inv, lse, sinv, dot);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (ok[u]) {
        const f2 scale = both(SIG ? sinv[u] : inv[u]);
#pragma unroll
        for (int i = 0; i < 2 * NV; ++i) acc2[i] = fma2(SIG ? s[u][i] : v[u][i], scale, acc2[i]);
        if (gl == 0) {
          z += lse[u] * lse[u];
          ++n;
        }
      }
    }
  }
  float acc[4 * NV];
#pragma unroll
  for (int i = 0; i < 2 * NV; ++i) {
    const float2 x = unpack2(acc2[i]);
    acc[2 * i] = x.x;
    acc[2 * i + 1] = x.y;
  }
  // groups of a warp, then warps
#pragma unroll
  for (int o = G; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    z += __shfl_xor_sync(0xffffffffu, z, o);
    n += __shfl_xor_sync(0xffffffffu, n, o);
  }
  if (lane < G) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) s_sum[warp][4 * (gl + G * j) + i] = acc[4 * j + i];
  }
  if (lane == 0) {
    s_z[warp] = z;
    s_n[warp] = n;
  }
  __syncthreads();
  if (tid < p.E) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kBalWarps; ++w) s += s_sum[w][tid];
    p.part_p[static_cast<size_t>(slot) * p.E + tid] = s;
    p.part_c[static_cast<size_t>(slot) * p.E + tid] = s_cnt[tid];
  }
  if (tid == 0) {
    for (int w = 1; w < kBalWarps; ++w) {
      z += s_z[w];
      n += s_n[w];
    }
    p.part_z[slot] = z;
    p.part_n[slot] = n;
  }
}

template <int G, int NV, bool VEC, bool SIG>
__global__ void __launch_bounds__(kBalThreads, 4) balance_part_kernel(const BalParams p) {
  chain_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0;
  const int lo = blockIdx.x * p.CH, hi = min(p.T, lo + p.CH);
  // the first sequence that ends behind the first row
  int s = p.off == nullptr ? 0 : count_le(p.S, [&](int i) { return seq_begin(p.off, i + 1, p.S, p.T); }, lo);
  for (; s < p.S; ++s) {
    const int begin = seq_begin(p.off, s, p.S, p.T);
    if (begin >= hi) break;
    BalChunk ch;
    ch.lo = max(lo, begin);
    ch.hi = min(hi, seq_begin(p.off, s + 1, p.S, p.T));
    if (ch.lo < ch.hi) part_of_sequence<G, NV, VEC, SIG>(p, ch, blockIdx.x + s);
  }
  chain_release();
}

// Forward, second pass: a block for each sequence and 32 experts adds their
// slots (a lane an expert, the warps sharing the slots; fixed order), writes
// the counts and the weight row of the backward; the block that finishes last
// adds the sequences. Latency: 9 to 13 us from a cold L2.
template <int kBalJoinWarps>
__global__ void __launch_bounds__(32 * kBalJoinWarps) balance_join_kernel(const BalParams p) {
  constexpr int kBalJoin = 32 * kBalJoinWarps, kBatch = 10;
  __shared__ Sum2 s_p[kBalJoinWarps][32];
  __shared__ int s_c[kBalJoinWarps][32];
  __shared__ Sum2 s_z[kBalJoinWarps], s_b[kBalJoinWarps];
  __shared__ int s_n[kBalJoinWarps], s_f[kBalJoinWarps];
  __shared__ int s_last;
  const int s = blockIdx.x, cg = blockIdx.y, groups = gridDim.y, E = p.E;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  chain_wait();
  const int b = seq_begin(p.off, s, p.S, p.T), e = seq_begin(p.off, s + 1, p.S, p.T);
  if (tid == 0 && p.off != nullptr) {
    const int rb = p.off[s], re = p.off[s + 1];
    if (rb < 0 || re < rb || re > p.T) set_status(p.st, MOE_ERR_DEVICE_INDEX, 51);
  }
  const int first = b / p.CH + s, x = 32 * cg + lane;
  const int nch = e > b ? min((e - 1) / p.CH - b / p.CH + 1, p.slots - first) : 0;
  Sum2 P, z;
  int c = 0, n = 0;
  if (x < E) {
    // kBatch loads in flight: the sums wait for memory once a batch
    for (int i0 = warp; i0 < nch; i0 += kBatch * kBalJoinWarps) {
      float pv[kBatch];
      int cv[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = i0 + j * kBalJoinWarps;
        const size_t at = static_cast<size_t>(first + i) * E + x;
        pv[j] = i < nch ? p.part_p[at] : 0.0f;
        cv[j] = i < nch ? p.part_c[at] : 0;
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        P.add(pv[j]);
        c += cv[j];
      }
    }
  }
  for (int i = tid; i < nch; i += kBalJoin) {
    z.add(p.part_z[first + i]);
    n += p.part_n[first + i];
  }
  n = warp_sum(n);
  z = warp_sum(z);
  s_p[warp][lane] = P;
  s_c[warp][lane] = c;
  if (lane == 0) {
    s_z[warp] = z;
    s_n[warp] = n;
  }
  __syncthreads();
  if (warp == 0) {
    n = 0;
    P = Sum2();
    c = 0;
    z = Sum2();
#pragma unroll
    for (int w = 0; w < kBalJoinWarps; ++w) {
      n += s_n[w];
      z.add(s_z[w]);
      P.add(s_p[w][lane]);
      c += s_c[w][lane];
    }
    float w = 0.0f;
    if (x < E) {
      // in the order that keeps the factors near 1: f, then the two means
      if (n > 0) w = p.balance_coeff * (static_cast<float>(E) / p.k * (static_cast<float>(c) / n)) / n;
      p.counts[static_cast<size_t>(s) * E + x] = c;
      p.stats[static_cast<size_t>(s) * E + x] = w;
    }
    Sum2 term;
    term.add(w * P.value());
    term = warp_sum(term);
    if (lane == 0) {
      p.seq_b[static_cast<size_t>(s) * groups + cg] = make_float2(term.s, term.e);
      if (cg == 0) {
        p.seq_z[s] = make_float2(z.s, z.e);
        p.seq_n[s] = n;
      }
      __threadfence();
      s_last = atomicAdd(p.ticket, 1) == p.S * groups - 1;
      __threadfence();
    }
  }
  __syncthreads();
  if (!s_last) return;
  Sum2 lb, lz;
  int cnt = 0, filled = 0;
  for (int i = tid; i < p.S * groups; i += kBalJoin) {
    const float2 v = __ldcg(p.seq_b + i);
    lb.add(v.x);
    lb.e += v.y;
  }
  for (int i = tid; i < p.S; i += kBalJoin) {
    const float2 v = __ldcg(p.seq_z + i);
    lz.add(v.x);
    lz.e += v.y;
    const int m = __ldcg(p.seq_n + i);
    cnt += m;
    filled += m > 0;
  }
  lb = warp_sum(lb);
  lz = warp_sum(lz);
  cnt = warp_sum(cnt);
  filled = warp_sum(filled);
  if (lane == 0) {
    s_b[warp] = lb;
    s_z[warp] = lz;
    s_n[warp] = cnt;
    s_f[warp] = filled;
  }
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kBalJoinWarps; ++w) {
      lb.add(s_b[w]);
      lz.add(s_z[w]);
      cnt += s_n[w];
      filled += s_f[w];
    }
    const float share = filled > 0 ? 1.0f / filled : 0.0f, per = cnt > 0 ? p.z_coeff / cnt : 0.0f;
    p.losses[0] = filled > 0 ? lb.value() * share : 0.0f;
    p.losses[1] = per != 0.0f ? lz.value() * per : 0.0f;
    float* tail = p.stats + static_cast<size_t>(p.S) * E;
    tail[0] = share;
    tail[1] = 2.0f * per;
    *p.ticket = 0;  // the workspace as it was found: other calls count from 0 in the same word
  }
}

// Backward: one pass over the logits, each block's rows from the last one up: of
// the rows that the forward's pass read, the later ones are still in L2. w is the sequence's weight row
// alpha E c / (k n^2); the mean over the sequences and the losses' own
// gradients scale it. Bound by HBM (131021 x 256 sigmoid: 268 MB in 48 us, 5.6 TB/s).
constexpr int kBalBwdThreads = 256;
// Resident blocks on an SM: sigmoid scores need more than 64 registers (131021 x 256
// both ways, inputs not in L2: four blocks 91.3 us, three 88.8; 65536 x 256 softmax:
// four 38.5, three 40.6)
constexpr int bal_bwd_blocks(bool sigmoid) { return sigmoid ? 3 : 4; }
constexpr int kBalBwdWarps = kBalBwdThreads / 32;
template <int G, int NV, bool VEC, bool SIG>
__global__ void __launch_bounds__(kBalBwdThreads, bal_bwd_blocks(SIG))
    balance_bwd_kernel(const BalParams p, const float* dlosses, int rows_per_block, float* dlogits) {
  __shared__ RowRing<NV> s_rows;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  chain_wait();
  const int lo = static_cast<int>(min(static_cast<long long>(blockIdx.x) * rows_per_block, static_cast<long long>(p.T)));
  const int hi = static_cast<int>(min(static_cast<long long>(lo) + rows_per_block, static_cast<long long>(p.T)));
  const int gl = lane & (G - 1), grp = lane / G;
  constexpr int RPW = 32 / G, U = kBalUnroll, kPass = U * kBalBwdWarps * RPW;
  const auto ask = [&](int t0, int slot) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * kBalBwdWarps * RPW + grp;
      if (VEC && t0 >= lo && t < hi && (p.mask == nullptr || p.mask[t] != 0))
        ask_row<G, NV, VEC>(s_rows, slot, u, p.logits + static_cast<size_t>(t) * p.E, p.E, gl);
    }
    if (VEC) cp_async_commit();
  };
  const int first = lo + warp * RPW + (hi - lo - 1) / kPass * kPass;
  for (int i = 0; i < kAhead; ++i) ask(first - i * kPass, i);
  // the last sequence that begins at or before the block's last row
  const int s0 = p.off == nullptr ? 0 : count_le(p.S, [&](int i) { return seq_begin(p.off, i, p.S, p.T); }, hi - 1) - 1;
  const float* tail = p.stats + static_cast<size_t>(p.S) * p.E;
  const float gb = (dlosses != nullptr ? dlosses[0] : 1.0f) * tail[0];
  const float gz = (dlosses != nullptr ? dlosses[1] : 1.0f) * tail[1];
  int s = s0, have = -1;  // the sequence of the row at hand, and the one whose weights w holds
  int begin = s >= 0 ? seq_begin(p.off, s, p.S, p.T) : 0, end = s >= 0 ? seq_begin(p.off, s + 1, p.S, p.T) : 0;
  f2 w[2 * NV];
#pragma unroll
  for (int i = 0; i < 2 * NV; ++i) w[i] = both(0.0f);
  for (int t0 = first, slot = 0; t0 >= lo; t0 -= kPass, slot ^= 1) {
    f2 v[U][2 * NV];
    float top = 0.0f;
    int seq[U];  // -1: no valid row
    if (VEC) cp_async_wait<kAhead - 1>();
#pragma unroll
    for (int u = U - 1; u >= 0; --u) {
      const int t = t0 + u * kBalBwdWarps * RPW + grp;
      seq[u] = -1;
      if (t < hi) {
        if (t < begin && s >= 0) {  // rows come in descending order
          while (s >= 0 && seq_begin(p.off, s, p.S, p.T) > t) --s;
          begin = s >= 0 ? seq_begin(p.off, s, p.S, p.T) : 0;
          end = s >= 0 ? seq_begin(p.off, s + 1, p.S, p.T) : 0;
        }
        if (s >= 0 && t >= begin && t < end && (p.mask == nullptr || p.mask[t] != 0)) seq[u] = s;
      }
      if (seq[u] >= 0) {
        load_row<G, NV, VEC>(s_rows, slot, u, p.logits + static_cast<size_t>(t) * p.E, p.E, gl, v[u], top);
      } else {
#pragma unroll
        for (int i = 0; i < 2 * NV; ++i) v[u][i] = both(0.0f);
      }
    }
    const bool near = __all_sync(0xffffffffu, top <= kNear);
    ask(t0 - kAhead * kPass, slot);
    const auto weights_of = [&](int u) {
      if (seq[u] < 0 || seq[u] == have) return;
      have = seq[u];
#pragma unroll
      for (int i = 0; i < 2 * NV; ++i) {
        const int e = 4 * (gl + G * (i >> 1)) + 2 * (i & 1);
        const float* row = p.stats + static_cast<size_t>(have) * p.E;
        w[i] = pack2(e < p.E ? gb * row[e] : 0.0f, e + 1 < p.E ? gb * row[e + 1] : 0.0f);
      }
    };
    f2 q[U][2 * NV];
    float inv[U], lse[U], sinv[U], dot[U];
    if (near) row_scores<G, NV, SIG, true, true>(gl, p.E, p.need_lse, v, q, w, weights_of, inv, lse, sinv, dot);
    else row_scores<G, NV, SIG, true, false>(gl, p.E, p.need_lse, v, q, w, weights_of, inv, lse, sinv, dot);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * kBalBwdWarps * RPW + grp;
      if (t >= hi) continue;
      weights_of(u);
      const bool live = seq[u] >= 0;
      const f2 mean = both(-dot[u] * (SIG ? sinv[u] : inv[u]));
      const f2 zz = both(p.need_lse ? gz * lse[u] * inv[u] : 0.0f);
      const f2 scale = both(SIG ? sinv[u] : inv[u]);
      float* out = dlogits + static_cast<size_t>(t) * p.E;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float d[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int i = 2 * j + h;
          const f2 away = mul2(add2(w[i], mean), scale);
          const float2 x = unpack2(SIG ? fma2(q[u][i], away, mul2(v[u][i], zz)) : mul2(v[u][i], add2(away, zz)));
          d[2 * h] = live ? x.x : 0.0f;
          d[2 * h + 1] = live ? x.y : 0.0f;
        }
        const int e = 4 * (gl + G * j);
        if constexpr (VEC) {
          if (e < p.E) __stcs(reinterpret_cast<float4*>(out + e), make_float4(d[0], d[1], d[2], d[3]));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (e + i < p.E) out[e + i] = d[i];
        }
      }
    }
  }
}

// Lanes of a row (below) and rows that a lane group may add up in fp32
constexpr int kBalRun = 64;
static int balance_lanes(int E) { return E <= 16 ? 2 : (E <= 32 ? 4 : (E <= 64 ? 8 : (E <= 128 ? 16 : 32))); }

// Lanes of a row by E: the smallest group whose lanes hold eight experts each, so
// that a warp's shuffles serve several rows (72025 x 128: 31.8 us with four experts
// a lane, 26.9 with eight); four each for up to 8 experts.
template <class F>
static cudaError_t balance_dispatch(int E, bool sigmoid, F f) {
  const bool vec = E % 4 == 0;
  cudaError_t e = cudaSuccess;
#define MOE_BAL_SIG(G, NV, VEC)                                                                                  \
  do {                                                                                                           \
    if (sigmoid) e = f(std::integral_constant<int, G>{}, std::integral_constant<int, NV>{}, VEC{}, std::true_type{}); \
    else e = f(std::integral_constant<int, G>{}, std::integral_constant<int, NV>{}, VEC{}, std::false_type{});       \
  } while (0)
#define MOE_BAL(G, NV)                               \
  do {                                               \
    if (vec) MOE_BAL_SIG(G, NV, std::true_type);     \
    else MOE_BAL_SIG(G, NV, std::false_type);        \
  } while (0)
  if (E <= 8) MOE_BAL(2, 1);
  else if (E <= 16) MOE_BAL(2, 2);
  else if (E <= 32) MOE_BAL(4, 2);
  else if (E <= 64) MOE_BAL(8, 2);
  else if (E <= 128) MOE_BAL(16, 2);
  else MOE_BAL(32, 2);  // (balance_lanes gives the same)
#undef MOE_BAL
#undef MOE_BAL_SIG
  return e;
}

static int check_balance(const moe_balance_config* c) {
  if (c == nullptr) return MOE_ERR_INVALID_ARG;
  if (c->T < 1 || c->E < 1 || c->k < 1 || c->n_seqs < 1 || c->k > c->E) return MOE_ERR_INVALID_ARG;
  if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (!isfinite(c->balance_coeff) || !isfinite(c->z_coeff)) return MOE_ERR_INVALID_ARG;
  if (c->E > 256 || c->k > 16 || c->n_seqs > (1 << 16)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (static_cast<long long>(c->T) * c->k >= (1ll << 30)) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

// Rows of a block: one wave of `resident` blocks for each SM (half a wave more than
// that took 70 us where one wave took 36)
static int balance_block_rows(int T, int S, int resident) {
  const int want = (T + resident * 152 - 1) / (resident * 152);
  // a block takes its sequences one after the other: short ones in smaller blocks
  const int least = std::min(32, std::max(4, T / S));
  return std::max(least, want);
}

struct BalWs {
  size_t part_p, part_c, part_z, part_n, seq_b, seq_z, seq_n, total;
  int CH, blocks, slots;
};
static BalWs balance_ws(const moe_balance_config& c) {
  BalWs w{};
  size_t o = 256;  // the status word; its chunk counter is the ticket
  auto take = [&](size_t b) {
    const size_t at = o;
    o += (b + 255) & ~size_t(255);
    return at;
  };
  w.CH = balance_block_rows(c.T, c.n_seqs, 4);
  // The sums over a block's rows are fp32 in its lane groups: of a longer batch (from
  // 311297 rows of more than 128 experts on) as many whole waves of blocks as keep a
  // group's run at kBalRun rows.
  const int most = kBalRun * kBalWarps * (32 / balance_lanes(c.E));
  if (w.CH > most) {
    const int blocks = 4 * 152 * ((w.CH + most - 1) / most);
    w.CH = (c.T + blocks - 1) / blocks;
  }
  w.blocks = (c.T + w.CH - 1) / w.CH;
  w.slots = w.blocks + c.n_seqs;
  const size_t n = w.slots, S = c.n_seqs;
  w.part_p = take(4 * n * c.E);
  w.part_c = take(4 * n * c.E);
  w.part_z = take(4 * n);
  w.part_n = take(4 * n);
  w.seq_b = take(8 * S * ((c.E + 31) / 32));
  w.seq_z = take(8 * S);
  w.seq_n = take(4 * S);
  w.total = o;
  return w;
}

static BalParams balance_params(const moe_balance_config& c, const float* logits, const int32_t* off,
                                const uint8_t* mask) {
  BalParams p{};
  p.logits = logits;
  p.off = off;
  p.mask = mask;
  p.T = c.T;
  p.E = c.E;
  p.k = c.k;
  p.S = c.n_seqs;
  p.sigmoid = c.score == MOE_SCORE_SIGMOID;
  p.need_lse = c.z_coeff != 0.0f;
  p.balance_coeff = c.balance_coeff;
  p.z_coeff = c.z_coeff;
  return p;
}

static bool misaligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_balance_workspace_bytes(const moe_balance_config* cfg) {
  return check_balance(cfg) != MOE_OK ? 0 : balance_ws(*cfg).total;
}

size_t moe_balance_stats_floats(const moe_balance_config* cfg) {
  return check_balance(cfg) != MOE_OK ? 0 : static_cast<size_t>(cfg->n_seqs) * cfg->E + 2;
}

int moe_balance_loss_fwd(const moe_balance_config* cfg, const float* logits, const int32_t* topk_idx,
                         const int32_t* seq_offsets, const uint8_t* token_mask, float* losses, int32_t* counts,
                         float* stats, void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nvtx("moe_balance_loss_fwd");
  const int st = check_balance(cfg);
  if (st != MOE_OK) return st;
  const moe_balance_config& c = *cfg;
  if (!logits || !topk_idx || !losses || !counts || !stats || !ws) return MOE_ERR_INVALID_ARG;
  if (seq_offsets == nullptr && c.n_seqs != 1) return MOE_ERR_INVALID_ARG;
  for (const void* q : {static_cast<const void*>(logits), static_cast<const void*>(topk_idx),
                        static_cast<const void*>(seq_offsets), static_cast<const void*>(token_mask),
                        static_cast<const void*>(losses), static_cast<const void*>(counts),
                        static_cast<const void*>(stats), static_cast<const void*>(ws)})
    if (misaligned16(q)) return MOE_ERR_INVALID_ARG;
  const BalWs L = balance_ws(c);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  BalParams p = balance_params(c, logits, seq_offsets, token_mask);
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.topk = topk_idx;
  p.CH = L.CH;
  p.slots = L.slots;
  p.part_p = reinterpret_cast<float*>(w + L.part_p);
  p.part_c = reinterpret_cast<int32_t*>(w + L.part_c);
  p.part_z = reinterpret_cast<float*>(w + L.part_z);
  p.part_n = reinterpret_cast<int32_t*>(w + L.part_n);
  p.seq_b = reinterpret_cast<float2*>(w + L.seq_b);
  p.seq_z = reinterpret_cast<float2*>(w + L.seq_z);
  p.seq_n = reinterpret_cast<int32_t*>(w + L.seq_n);
  p.st = reinterpret_cast<DevStatus*>(w);
  p.ticket = &p.st->chunk_counter;
  p.counts = counts;
  p.losses = losses;
  p.stats = stats;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = balance_dispatch(c.E, p.sigmoid, [&](auto g, auto nv, auto vec, auto sig) {
    return launch_chained(
        balance_part_kernel<decltype(g)::value, decltype(nv)::value, decltype(vec)::value, decltype(sig)::value>,
        L.blocks, kBalThreads, 0, s, p);
  });
  if (e != cudaSuccess) return status_from_cuda(e);
  // a large block for each of few, long sequences, small blocks for many short ones. Both ways in us
  // with large blocks, small, by slots a sequence: equal sequences of 16384 x 128, 513 17.9, 20.4; 257
  // 17.1, 17.7; 171 17.4, 16.8; 103 17.4, 15.8; 65 16.5, 14.1; of 131072 x 256, 304 79.4, 81.4; 152
  // 80.7, 79.8; 61 80.6, 78.2; cut at random, where the longest is two to three times the mean, 16384 x
  // 128, 129 17.8, 18.3; 86 17.6, 17.7; 65 17.8, 17.3; 131072 x 256, 152 82.0, 83.0; 76 82.4, 82.4; 41
  // 82.0, 81.3. The border lies between the two kinds' own, 200 and 70: neither loses much.
  const dim3 grid(c.n_seqs, (c.E + 31) / 32);
  e = L.slots / c.n_seqs > 100 ? launch_chained(balance_join_kernel<32>, grid, 1024, 0, s, p)
                              : launch_chained(balance_join_kernel<4>, grid, 128, 0, s, p);
  record_stage(s, 43, 2);
  return status_from_cuda(e);
}

int moe_balance_loss_bwd(const moe_balance_config* cfg, const float* logits, const float* stats, const float* dlosses,
                         const int32_t* seq_offsets, const uint8_t* token_mask, float* dlogits, void* stream) {
  NvtxRange nvtx("moe_balance_loss_bwd");
  const int st = check_balance(cfg);
  if (st != MOE_OK) return st;
  const moe_balance_config& c = *cfg;
  if (!logits || !stats || !dlogits) return MOE_ERR_INVALID_ARG;
  if (seq_offsets == nullptr && c.n_seqs != 1) return MOE_ERR_INVALID_ARG;
  for (const void* q : {static_cast<const void*>(logits), static_cast<const void*>(stats),
                        static_cast<const void*>(dlosses), static_cast<const void*>(seq_offsets),
                        static_cast<const void*>(token_mask), static_cast<const void*>(dlogits)})
    if (misaligned16(q)) return MOE_ERR_INVALID_ARG;
  // in place a thread writes what it has read itself; shifted, what another block has still to read
  const size_t lb = 4 * static_cast<size_t>(c.T) * c.E, sb = 4 * (static_cast<size_t>(c.n_seqs) * c.E + 2);
  if ((dlogits != logits && overlap(logits, lb, dlogits, lb)) || overlap(stats, sb, dlogits, lb))
    return MOE_ERR_INVALID_ARG;
  BalParams p = balance_params(c, logits, seq_offsets, token_mask);
  p.stats = const_cast<float*>(stats);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int rows = balance_block_rows(c.T, 1, bal_bwd_blocks(p.sigmoid != 0));
  const int grid = (c.T + rows - 1) / rows;
  const cudaError_t e = balance_dispatch(c.E, p.sigmoid, [&](auto g, auto nv, auto vec, auto sig) {
    return launch_chained(
        balance_bwd_kernel<decltype(g)::value, decltype(nv)::value, decltype(vec)::value, decltype(sig)::value>, grid,
        kBalBwdThreads, 0, s, p, dlosses, rows, dlogits);
  });
  record_stage(s, 44, 1);
  return status_from_cuda(e);
}

}  // extern "C"
