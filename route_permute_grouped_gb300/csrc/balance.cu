// The router's auxiliary losses from its logits and the selected experts: the
// sequence-wise balance loss and the z-loss with the expert counts of every
// sequence (forward), and the gradient of the logits (backward).
#include <math.h>

#include <algorithm>

#include "host_util.h"

namespace moe {

// Rows are handled by groups of G lanes, each lane holding NV sets of four
// consecutive experts (set j: experts 4 (lane + G j) ..): 4 G NV >= E.
constexpr int kBalThreads = 256;
constexpr int kBalWarps = kBalThreads / 32;

// Chunks of the token axis: sequence s takes the chunk numbers from
// base(s) = off[s] / CH + s on, ceil(len / CH) of them, which is less than
// base(s + 1) - base(s) + 1, so each chunk number belongs to one sequence at
// most and nothing has to be scanned.
struct BalChunk {
  int s, lo, hi;  // rows [lo, hi) of sequence s; lo == hi: no rows
};

__device__ __forceinline__ int seq_begin(const int32_t* off, int s, int S, int T) {
  if (off == nullptr) return s == 0 ? 0 : T;
  const int v = off[s];
  return v < 0 ? 0 : (v > T ? T : v);
}

// number of s in [0, S) with key(s) <= c, by the whole block
template <class F>
__device__ __forceinline__ int count_le(int S, F key, int c) {
  int n = 0;
  for (int s0 = 0; s0 < S; s0 += kBalThreads) {
    const int s = s0 + static_cast<int>(threadIdx.x);
    n += __syncthreads_count(s < S && key(s) <= c);
  }
  return n;
}

__device__ __forceinline__ BalChunk chunk_of(const int32_t* off, int S, int T, int CH, int c) {
  const int s = count_le(S, [&](int i) { return seq_begin(off, i, S, T) / CH + i; }, c) - 1;
  BalChunk r{-1, 0, 0};
  if (s < 0) return r;
  const int b = seq_begin(off, s, S, T), e = seq_begin(off, s + 1, S, T);
  const long long lo = b + static_cast<long long>(c - (b / CH + s)) * CH;
  r.s = s;
  if (lo >= b && lo < e) {  // offsets that descend give chunks without rows
    r.lo = static_cast<int>(lo);
    r.hi = static_cast<int>(min(static_cast<long long>(e), lo + CH));
  }
  return r;
}

template <int G, int NV, bool VEC>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int gl, float (&v)[4 * NV]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = 4 * (gl + G * j);
    if constexpr (VEC) {
      if (e < E) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(row + e));
        v[4 * j] = x.x; v[4 * j + 1] = x.y; v[4 * j + 2] = x.z; v[4 * j + 3] = x.w;
      } else {
        v[4 * j] = v[4 * j + 1] = v[4 * j + 2] = v[4 * j + 3] = -INFINITY;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * j + i] = e + i < E ? __ldg(row + e + i) : -INFINITY;
    }
  }
}
template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
template <int G>
__device__ __forceinline__ float group_max(float x) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// softmax of a row: v -> exp(v - max), returns 1 / sum and the row's
// log-sum-exp
template <int G, int NV>
__device__ __forceinline__ float row_softmax(float (&v)[4 * NV], float& lse) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < 4 * NV; ++i) m = fmaxf(m, v[i]);
  m = group_max<G>(m);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 4 * NV; ++i) {
    v[i] = expf(v[i] - m);
    sum += v[i];
  }
  sum = group_sum<G>(sum);
  lse = m + logf(sum);
  return 1.0f / sum;
}

// sigmoid and 1 - sigmoid without cancellation: t = exp(-|l|)
__device__ __forceinline__ float2 sigmoid2(float l) {
  const float t = expf(-fabsf(l));
  const float a = 1.0f / (1.0f + t), b = t * a;
  return l >= 0.0f ? make_float2(a, b) : make_float2(b, a);
}

struct BalParams {
  const float* logits;
  const int32_t* topk;
  const int32_t* off;
  const uint8_t* mask;
  int T, E, k, S, CH, chunks;
  int sigmoid, need_lse;
  float balance_coeff, z_coeff;
  // workspace
  float* part_p;      // [chunks][E] sums of p
  int32_t* part_c;    // [chunks][E] counts
  float* part_z;      // [chunks] sums of lse^2
  int32_t* part_n;    // [chunks] valid rows
  double* seq_b;      // [S] balance loss of each sequence (before the mean over sequences)
  double* seq_z;      // [S] sum of lse^2
  int32_t* seq_n;     // [S]
  int* ticket;
  // outputs
  int32_t* counts;
  float* losses;
  float* stats;
  DevStatus* st;
};

// Forward, first pass: every chunk's sums of p, counts, sum of lse^2 and
// number of valid rows. The sums over rows stay in registers, one set per lane
// group, and are joined over the groups and warps in a fixed order.
template <int G, int NV, bool VEC>
__global__ void __launch_bounds__(kBalThreads) balance_part_kernel(const BalParams p) {
  __shared__ int s_cnt[256];
  __shared__ float s_sum[kBalWarps][256];
  __shared__ float s_z[kBalWarps];
  __shared__ int s_n[kBalWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (blockIdx.x == 0 && tid == 0) *p.ticket = 0;
  const BalChunk ch = chunk_of(p.off, p.S, p.T, p.CH, blockIdx.x);
  if (ch.s < 0 || ch.lo >= ch.hi) return;
  s_cnt[tid] = 0;
  __syncthreads();
  const int gl = lane & (G - 1), grp = lane / G;
  constexpr int RPW = 32 / G;
  float acc[4 * NV];
#pragma unroll
  for (int i = 0; i < 4 * NV; ++i) acc[i] = 0.0f;
  float z = 0.0f;
  int n = 0;
  for (int t0 = ch.lo + warp * RPW; t0 < ch.hi; t0 += kBalWarps * RPW) {
    const int t = t0 + grp;
    const bool ok = t < ch.hi && (p.mask == nullptr || p.mask[t] != 0);
    float v[4 * NV];
    if (ok) {
      load_row<G, NV, VEC>(p.logits + static_cast<size_t>(t) * p.E, p.E, gl, v);
    } else {
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i) v[i] = 0.0f;
    }
    if (p.sigmoid) {
      float s[4 * NV], sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i) {
        s[i] = sigmoid2(v[i]).x;
        sum += s[i];
      }
      const float inv = 1.0f / group_sum<G>(sum);
      if (ok) {
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) acc[i] += s[i] * inv;
      }
    }
    float lse = 0.0f;
    if (!p.sigmoid || p.need_lse) {
      const float inv = row_softmax<G, NV>(v, lse);
      if (!p.sigmoid && ok) {
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) acc[i] += v[i] * inv;
      }
    }
    if (ok && gl == 0) {
      z += lse * lse;
      ++n;
    }
  }
  // the selected experts of the valid rows
  const int slots = (ch.hi - ch.lo) * p.k;
  const int32_t* idx = p.topk + static_cast<size_t>(ch.lo) * p.k;
  for (int i = tid; i < slots; i += kBalThreads) {
    if (p.mask != nullptr && p.mask[ch.lo + i / p.k] == 0) continue;
    const int e = __ldg(idx + i);
    if (e < 0 || e >= p.E) set_status(p.st, MOE_ERR_DEVICE_INDEX, 50);
    else atomicAdd(&s_cnt[e], 1);
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
      for (int i = 0; i < 4; ++i) {
        const int e = 4 * (gl + G * j) + i;
        if (e < 256) s_sum[warp][e] = acc[4 * j + i];
      }
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
    p.part_p[static_cast<size_t>(blockIdx.x) * p.E + tid] = s;
    p.part_c[static_cast<size_t>(blockIdx.x) * p.E + tid] = s_cnt[tid];
  }
  if (tid == 0) {
    for (int w = 1; w < kBalWarps; ++w) {
      z += s_z[w];
      n += s_n[w];
    }
    p.part_z[blockIdx.x] = z;
    p.part_n[blockIdx.x] = n;
  }
}

// Forward, second pass: one block per sequence adds its chunks (fp64, fixed
// order), writes its counts and the weight row of the backward; the block that
// finishes last adds the sequences.
constexpr int kBalJoin = 1024;
__global__ void __launch_bounds__(kBalJoin) balance_join_kernel(const BalParams p) {
  __shared__ double s_p[kBalJoin];
  __shared__ int s_c[kBalJoin];
  __shared__ double s_z[32];
  __shared__ int s_n[32];
  __shared__ int s_last;
  const int s = blockIdx.x, tid = threadIdx.x, E = p.E;
  const int b = seq_begin(p.off, s, p.S, p.T), e = seq_begin(p.off, s + 1, p.S, p.T);
  if (tid == 0 && p.off != nullptr) {
    const int rb = p.off[s], re = p.off[s + 1];
    if (rb < 0 || re < rb || re > p.T) set_status(p.st, MOE_ERR_DEVICE_INDEX, 51);
  }
  const int first = b / p.CH + s;
  const int nch = e > b ? min((e - b + p.CH - 1) / p.CH, p.chunks - first) : 0;
  // thread (g, x): expert x, chunks g, g + groups, ...
  const int Eb = (E + 31) & ~31, groups = kBalJoin / Eb, x = tid % Eb, g = tid / Eb;
  double P = 0.0;
  int c = 0;
  if (x < E && g < groups) {
    for (int i = g; i < nch; i += groups) {
      P += p.part_p[static_cast<size_t>(first + i) * E + x];
      c += p.part_c[static_cast<size_t>(first + i) * E + x];
    }
  }
  double z = 0.0;
  int n = 0;
  for (int i = tid; i < nch; i += kBalJoin) {
    z += p.part_z[first + i];
    n += p.part_n[first + i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    z += __shfl_xor_sync(0xffffffffu, z, o);
    n += __shfl_xor_sync(0xffffffffu, n, o);
  }
  if ((tid & 31) == 0) {
    s_z[tid >> 5] = z;
    s_n[tid >> 5] = n;
  }
  s_p[tid] = P;
  s_c[tid] = c;
  __syncthreads();
  z = 0.0;
  n = 0;
  for (int w = 0; w < 32; ++w) {
    z += s_z[w];
    n += s_n[w];
  }
  double term = 0.0;
  if (tid < E) {
    P = 0.0;
    c = 0;
    for (int i = 0; i < groups; ++i) {
      P += s_p[i * Eb + tid];
      c += s_c[i * Eb + tid];
    }
    p.counts[static_cast<size_t>(s) * E + tid] = c;
    double w = 0.0;
    if (n > 0) {
      w = static_cast<double>(p.balance_coeff) * E * c / (static_cast<double>(p.k) * n * n);
      term = w * P;
    }
    p.stats[static_cast<size_t>(s) * E + tid] = static_cast<float>(w);
  }
  __syncthreads();
  s_p[tid] = term;
  __syncthreads();
  for (int st = kBalJoin / 2; st > 0; st >>= 1) {
    if (tid < st) s_p[tid] += s_p[tid + st];
    __syncthreads();
  }
  if (tid == 0) {
    p.seq_b[s] = s_p[0];
    p.seq_z[s] = z;
    p.seq_n[s] = n;
    __threadfence();
    s_last = atomicAdd(p.ticket, 1) == p.S - 1;
    __threadfence();
  }
  __syncthreads();
  if (!s_last) return;
  double lb = 0.0, lz = 0.0, cnt = 0.0, filled = 0.0;
  for (int i = tid; i < p.S; i += kBalJoin) {
    lb += __ldcg(p.seq_b + i);
    lz += __ldcg(p.seq_z + i);
    const int m = __ldcg(p.seq_n + i);
    cnt += m;
    filled += m > 0 ? 1.0 : 0.0;
  }
  double* vals[4] = {&lb, &lz, &cnt, &filled};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    __syncthreads();
    s_p[tid] = *vals[j];
    __syncthreads();
    for (int st = kBalJoin / 2; st > 0; st >>= 1) {
      if (tid < st) s_p[tid] += s_p[tid + st];
      __syncthreads();
    }
    *vals[j] = s_p[0];
  }
  if (tid == 0) {
    const double share = filled > 0 ? 1.0 / filled : 0.0, per = cnt > 0 ? p.z_coeff / cnt : 0.0;
    p.losses[0] = static_cast<float>(lb * share);
    p.losses[1] = per != 0.0 ? static_cast<float>(lz * per) : 0.0f;
    float* tail = p.stats + static_cast<size_t>(p.S) * E;
    tail[0] = static_cast<float>(share);
    tail[1] = static_cast<float>(2.0 * per);
  }
}

// Backward: one pass over the logits. w is the sequence's weight row
// alpha E c / (k n^2); the mean over the sequences and the losses' own
// gradients scale it.
template <int G, int NV, bool VEC>
__global__ void __launch_bounds__(kBalThreads) balance_bwd_kernel(const BalParams p, const float* __restrict__ dlosses,
                                                                  int rows_per_block, float* __restrict__ dlogits) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int lo = static_cast<int>(min(static_cast<long long>(blockIdx.x) * rows_per_block, static_cast<long long>(p.T)));
  const int hi = static_cast<int>(min(static_cast<long long>(lo) + rows_per_block, static_cast<long long>(p.T)));
  // the last sequence that begins at or before the block's first row
  const int s0 = p.off == nullptr ? 0 : count_le(p.S, [&](int i) { return seq_begin(p.off, i, p.S, p.T); }, lo) - 1;
  const float* tail = p.stats + static_cast<size_t>(p.S) * p.E;
  const float gb = (dlosses != nullptr ? dlosses[0] : 1.0f) * tail[0];
  const float gz = (dlosses != nullptr ? dlosses[1] : 1.0f) * tail[1];
  const int gl = lane & (G - 1), grp = lane / G;
  constexpr int RPW = 32 / G;
  int s = s0, have = -1;
  float w[4 * NV];
  for (int t0 = lo + warp * RPW; t0 < hi; t0 += kBalWarps * RPW) {
    const int t = t0 + grp;
    bool ok = t < hi;
    if (ok) {
      while (s + 1 < p.S && seq_begin(p.off, s + 1, p.S, p.T) <= t) ++s;
      ok = s >= 0 && t >= seq_begin(p.off, s, p.S, p.T) && t < seq_begin(p.off, s + 1, p.S, p.T) &&
           (p.mask == nullptr || p.mask[t] != 0);
    }
    float v[4 * NV], sg[4 * NV], d[4 * NV];
    if (ok) {
      load_row<G, NV, VEC>(p.logits + static_cast<size_t>(t) * p.E, p.E, gl, v);
      if (have != s) {
        have = s;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = 4 * (gl + G * j) + i;
            w[4 * j + i] = e < p.E ? gb * p.stats[static_cast<size_t>(s) * p.E + e] : 0.0f;
          }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i) v[i] = 0.0f;
      have = -1;
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i) w[i] = 0.0f;
    }
    if (p.sigmoid) {
      float sum = 0.0f, dot = 0.0f;
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i) {
        const float2 q = sigmoid2(v[i]);
        sg[i] = q.x;
        d[i] = q.x * q.y;
        sum += q.x;
        dot += q.x * w[i];
      }
      const float inv = 1.0f / group_sum<G>(sum);
      const float mean = group_sum<G>(dot) * inv;
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i) d[i] = d[i] * inv * (w[i] - mean);
    }
    if (!p.sigmoid || p.need_lse) {
      float lse;
      const float inv = row_softmax<G, NV>(v, lse);
      const float zz = gz * lse;
      if (!p.sigmoid) {
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) dot += v[i] * w[i];
        const float mean = group_sum<G>(dot) * inv;
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) d[i] = v[i] * inv * (p.need_lse ? w[i] - mean + zz : w[i] - mean);
      } else {
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) d[i] += v[i] * inv * zz;
      }
    }
    if (t < hi) {
      float* out = dlogits + static_cast<size_t>(t) * p.E;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int e = 4 * (gl + G * j);
        if constexpr (VEC) {
          if (e < p.E)
            *reinterpret_cast<float4*>(out + e) = ok ? make_float4(d[4 * j], d[4 * j + 1], d[4 * j + 2], d[4 * j + 3])
                                                     : make_float4(0.f, 0.f, 0.f, 0.f);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (e + i < p.E) out[e + i] = ok ? d[4 * j + i] : 0.0f;
        }
      }
    }
  }
}

// Lanes of a row by E: the smallest group whose lanes hold four experts each,
// two sets of four from 129 experts on.
template <class F>
static cudaError_t balance_dispatch(int E, bool vec, F f) {
#define MOE_BAL(G, NV)                                                            \
  do {                                                                            \
    if (vec) f(std::integral_constant<int, G>{}, std::integral_constant<int, NV>{}, std::true_type{}); \
    else f(std::integral_constant<int, G>{}, std::integral_constant<int, NV>{}, std::false_type{});    \
  } while (0)
  if (E <= 8) MOE_BAL(2, 1);
  else if (E <= 16) MOE_BAL(4, 1);
  else if (E <= 32) MOE_BAL(8, 1);
  else if (E <= 64) MOE_BAL(16, 1);
  else if (E <= 128) MOE_BAL(32, 1);
  else MOE_BAL(32, 2);
#undef MOE_BAL
  return cudaGetLastError();
}

static int check_balance(const moe_balance_config* c) {
  if (c == nullptr) return MOE_ERR_INVALID_ARG;
  if (c->T < 1 || c->E < 1 || c->k < 1 || c->n_seqs < 1 || c->k > c->E) return MOE_ERR_INVALID_ARG;
  if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (!isfinite(c->balance_coeff) || !isfinite(c->z_coeff)) return MOE_ERR_INVALID_ARG;
  if (c->E > 256 || c->k > 16 || c->n_seqs > (1 << 20)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (static_cast<long long>(c->T) * c->k >= (1ll << 30)) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

// Rows of a chunk: about two chunks for each SM, whole passes of the block
static int balance_chunk_rows(int T) {
  const int want = (T + 303) / 304;
  return std::max(64, (want + 31) / 32 * 32);
}

struct BalWs {
  size_t part_p, part_c, part_z, part_n, seq_b, seq_z, seq_n, total;
  int CH, chunks;
};
static BalWs balance_ws(const moe_balance_config& c) {
  BalWs w{};
  size_t o = 256;  // the status word; its chunk counter is the ticket
  auto take = [&](size_t b) {
    const size_t at = o;
    o += (b + 255) & ~size_t(255);
    return at;
  };
  w.CH = balance_chunk_rows(c.T);
  w.chunks = c.T / w.CH + c.n_seqs + 1;
  const size_t n = w.chunks, S = c.n_seqs;
  w.part_p = take(4 * n * c.E);
  w.part_c = take(4 * n * c.E);
  w.part_z = take(4 * n);
  w.part_n = take(4 * n);
  w.seq_b = take(8 * S);
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
  p.chunks = L.chunks;
  p.part_p = reinterpret_cast<float*>(w + L.part_p);
  p.part_c = reinterpret_cast<int32_t*>(w + L.part_c);
  p.part_z = reinterpret_cast<float*>(w + L.part_z);
  p.part_n = reinterpret_cast<int32_t*>(w + L.part_n);
  p.seq_b = reinterpret_cast<double*>(w + L.seq_b);
  p.seq_z = reinterpret_cast<double*>(w + L.seq_z);
  p.seq_n = reinterpret_cast<int32_t*>(w + L.seq_n);
  p.st = reinterpret_cast<DevStatus*>(w);
  p.ticket = &p.st->chunk_counter;
  p.counts = counts;
  p.losses = losses;
  p.stats = stats;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = balance_dispatch(c.E, c.E % 4 == 0, [&](auto g, auto nv, auto vec) {
    balance_part_kernel<decltype(g)::value, decltype(nv)::value, decltype(vec)::value>
        <<<L.chunks, kBalThreads, 0, s>>>(p);
  });
  if (e != cudaSuccess) return status_from_cuda(e);
  balance_join_kernel<<<c.n_seqs, kBalJoin, 0, s>>>(p);
  e = cudaGetLastError();
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
  BalParams p = balance_params(c, logits, seq_offsets, token_mask);
  p.stats = const_cast<float*>(stats);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int grid_max = 8 * num_sms();
  const int rows = std::max(32, (c.T + grid_max - 1) / grid_max);
  const int grid = (c.T + rows - 1) / rows;
  const cudaError_t e = balance_dispatch(c.E, c.E % 4 == 0, [&](auto g, auto nv, auto vec) {
    balance_bwd_kernel<decltype(g)::value, decltype(nv)::value, decltype(vec)::value>
        <<<grid, kBalThreads, 0, s>>>(p, dlosses, rows, dlogits);
  });
  record_stage(s, 44, 1);
  return status_from_cuda(e);
}

}  // extern "C"
