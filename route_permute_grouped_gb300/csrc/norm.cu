// Norms before and after a block with its gate and the scaled residual, and their
// backward (moe_block_norm_fwd, moe_block_norm_bwd):
//   u = post ? y ry wp : y,  h = a r + g u,  n = h rh wn,
//   ry = 1 / sqrt(mean(y^2) + eps),  rh = 1 / sqrt(mean(h^2) + eps).
// Both directions move each tensor once and are bound by that (forward y, r in, h, n
// out; backward y, r, dh, dn in, dy, dr out): a block of threads holds a row in
// registers from its loads to its stores, and h is computed again in the backward
// rather than kept. With dnw = dn wn the backward is
//   dH = A + S1 hh,  A = dh + rh dnw,  hh = h rh,  S1 = -rh / H sum dnw hh,
//   dr = a dH,  dy = ry (g dH wp - yy / H S2),  yy = y ry,  S2 = sum g dH wp yy,
// and since dH is linear in S1, S2 = SA + S1 SB with sums of A and hh alone: one
// reduction over the block for a row. No power of rh or ry above the first is formed: a
// row is right wherever the forward's sum of squares is (rh^3 leaves fp32 at rows of 1e13
// and of 1e-13). The gradients of the weights and of a channel
// gate are sums over rows, dpre's of dn h rh and one more for both others,
//   D = sum g_t dH y ry  (g_t: a token's gate),  dpost = g D,  dgate = wp D:
// a thread adds its columns' in fp32 over at most 64 rows, then in two floats in the
// workspace; a second kernel joins the blocks' in order.
// Measured: 16384 x 4096 in bf16 (residual and norm) forward 86 us, 6.2 TB/s, backward 140, 5.8 TB/s,
// 8 of it the join; 5003 x 7168 with both norms, a channel gate and an fp32 stream 78 us, 5.5 TB/s, and
// 119, 5.4 TB/s: what is lost there are the rows' one (forward two) sums over a block that has an SM
// nearly to itself. y and dn fp32 too: 8192 x 4096 without post norm and gate 80 us, 5.9 TB/s, and 112, 6.6 TB/s,
// with them 90 and 169, 4.4 TB/s; 16384 x 2048 with them 84 and 134, 5.5 TB/s. Longer rows: 4096 x 8192 in bf16 49 us,
// 5.5 TB/s, and 68, 5.9 TB/s, with both norms, gate and fp32 stream 71 and 128, 4.7 TB/s (registers held to 64 of
// 1024 threads); 2048 x 16384 59 us, 4.5 TB/s, and 124, 3.3 TB/s, with all of it 101 and 192, 3.1 TB/s (two runs a
// thread in those registers, up to 1.4 KB a thread spilled, and no row ahead in shared memory).
#include <atomic>
#include <type_traits>

#include "host_util.h"
#include "mma.cuh"

namespace moe {

constexpr int kNormFlush = 64;   // rows added in fp32 alone (16: backward of 16384 x 4096 150 us for 137)
constexpr int kNormMaxH = 16384;

struct NormParams {
  int T, H;
  float eps, a;
  int res, gate, post, pre;
  const void *y, *r, *dh, *dn;
  const float *wp, *g, *wn;
  void *h, *dr;
  __nv_bfloat16 *n, *dy;
  float *stats, *dgate, *part;
  int lo;                    // a block has more than kNormFlush rows: sums in two floats
  const float* cstats;
};

// A thread's 8 columns of a row (run i of n8): with bf16 streams alone 8i .. 8i + 7, one
// 16-byte access; where a stream is fp32 (SP) four in each half of the row, quads i and n8 + i,
// so that a warp's 16-byte accesses of either half are one run of bytes (8i .. 8i + 7 in fp32
// would be two accesses that touch every sector by half: 5003 x 7168 with an fp32 stream,
// forward 88 us and backward 179 against 78 and 121).
template <bool SP>
__device__ __forceinline__ int quad(int i, int n8, int k) {
  return SP ? i + k * n8 : 2 * i + k;
}
template <bool F32, bool SP>
struct Vec8 {
  static_assert(SP || !F32, "fp32 streams are split");
  uint4 a, b;
  __device__ __forceinline__ void load(const void* base, size_t row, int i, int n8) {
    if constexpr (F32) {
      const uint4* p = static_cast<const uint4*>(base) + 2 * row * n8;
      a = __ldcs(p + quad<SP>(i, n8, 0));
      b = __ldcs(p + quad<SP>(i, n8, 1));
    } else if constexpr (SP) {
      const uint2* p = static_cast<const uint2*>(base) + 2 * row * n8;
      const uint2 u = __ldcs(p + quad<SP>(i, n8, 0)), v = __ldcs(p + quad<SP>(i, n8, 1));
      a = make_uint4(u.x, u.y, v.x, v.y);
    } else {
      a = __ldcs(static_cast<const uint4*>(base) + row * n8 + i);
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
    if constexpr (F32) {
      const uint32_t x[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = __uint_as_float(w[j]);
        v[4 + j] = __uint_as_float(x[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = bf16_lo(w[j]);
        v[2 * j + 1] = bf16_hi(w[j]);
      }
    }
  }
};
template <bool F32, bool SP>
__device__ __forceinline__ void store8(void* base, size_t row, int i, int n8, const float (&v)[8]) {
  if constexpr (F32) {
    uint4* p = static_cast<uint4*>(base) + 2 * row * n8;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      p[quad<SP>(i, n8, k)] = make_uint4(__float_as_uint(v[4 * k]), __float_as_uint(v[4 * k + 1]),
                                         __float_as_uint(v[4 * k + 2]), __float_as_uint(v[4 * k + 3]));
  } else if constexpr (SP) {
    uint2* p = static_cast<uint2*>(base) + 2 * row * n8;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      p[quad<SP>(i, n8, k)] = make_uint2(pack_bf16x2(v[4 * k], v[4 * k + 1]), pack_bf16x2(v[4 * k + 2], v[4 * k + 3]));
  } else {
    static_cast<uint4*>(base)[row * n8 + i] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                         pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
}
template <bool SP>
__device__ __forceinline__ void weights8(const float* w, int i, int n8, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float4 a = reinterpret_cast<const float4*>(w)[quad<SP>(i, n8, k)];
    v[4 * k] = a.x; v[4 * k + 1] = a.y; v[4 * k + 2] = a.z; v[4 * k + 3] = a.w;
  }
}

// Sum of one value over the warp, of three: a lane of the k-th run of eight leaves with the k-th's
// (six exchanges for fifteen: the exchanges' pipe takes one a cycle and SM)
__device__ __forceinline__ float warp_sum(const float (&v)[1], int) {
  float s = v[0];
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  return s;
}
__device__ __forceinline__ float warp_sum(const float (&v)[3], int lane) {
  const bool up = lane & 16, odd = lane & 8;
  float a = up ? v[2] : v[0], b = up ? 0.0f : v[1];
  a += __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 16);
  b += __shfl_xor_sync(0xffffffffu, up ? v[1] : 0.0f, 16);
  float s = odd ? b : a;
  s += __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
#pragma unroll
  for (int d = 4; d >= 1; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  return s;
}
// Sums of N values over the block, in every thread; `s` alternates between two halves, so
// that one barrier a sum is enough
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* s, int& turn) {
  const int warp = warp_id(), lane = lane_id(), nw = blockDim.x >> 5;
  float* b = s + (turn & 1) * 96;
  ++turn;
  const float mine = warp_sum(v, lane);
  if ((lane & 7) == 0 && (lane >> 3) < N) b[(lane >> 3) * 32 + warp] = mine;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane < nw ? b[i * 32 + lane] : 0.0f;
  const float all = warp_sum(v, lane);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = N == 1 ? all : __shfl_sync(0xffffffffu, all, 8 * i);
}

// RF: residual stream fp32, OF: y (and dn) fp32; NC runs of 8 columns a thread
template <bool RF, bool OF, int NC>
__global__ void __launch_bounds__(512) norm_fwd_kernel(const __grid_constant__ NormParams p) {
  __shared__ float red[2 * 96];
  chain_wait();
  int turn = 0;
  constexpr bool SP = RF || OF;
  const int n8 = p.H >> 3;
  const float inv = 1.0f / static_cast<float>(p.H);
  for (int row = blockIdx.x; row < p.T; row += gridDim.x) {
    Vec8<OF, SP> yv[NC];
    Vec8<RF, SP> rv[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      if (i < n8) {
        yv[c].load(p.y, row, i, n8);
        if (p.res) rv[c].load(p.r, row, i, n8);
      }
    }
    float ry = 1.0f, h[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (static_cast<int>(threadIdx.x + c * blockDim.x) < n8) yv[c].get(h[c]);
      else {
#pragma unroll
        for (int j = 0; j < 8; ++j) h[c][j] = 0.0f;
      }
    }
    if (p.post) {
      float s[1] = {0.0f};
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[0] = fmaf(h[c][j], h[c][j], s[0]);
      block_sum(s, red, turn);
      ry = __frsqrt_rn(fmaf(s[0], inv, p.eps));
    }
    const float gt = p.gate == MOE_GATE_TOKEN ? p.g[row] : 1.0f;
    float s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      if (i < n8) {
        if (p.post) {
          float w[8];
          weights8<SP>(p.wp, i, n8, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[c][j] = h[c][j] * ry * w[j];
        }
        if (p.gate == MOE_GATE_CHANNEL) {
          float w[8];
          weights8<SP>(p.g, i, n8, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[c][j] *= w[j];
        } else if (p.gate == MOE_GATE_TOKEN) {
#pragma unroll
          for (int j = 0; j < 8; ++j) h[c][j] *= gt;
        }
        if (p.res) {
          float r[8];
          rv[c].get(r);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[c][j] = fmaf(p.a, r[j], h[c][j]);
        }
        if (p.h != nullptr) store8<RF, SP>(p.h, row, i, n8, h[c]);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[0] = fmaf(h[c][j], h[c][j], s[0]);
      }
    }
    if (p.pre) {
      block_sum(s, red, turn);
      const float rh = __frsqrt_rn(fmaf(s[0], inv, p.eps));
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int i = threadIdx.x + c * blockDim.x;
        if (i < n8) {
          float w[8];
          weights8<SP>(p.wn, i, n8, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[c][j] = h[c][j] * rh * w[j];
          store8<false, SP>(p.n, row, i, n8, h[c]);
        }
      }
      if (threadIdx.x == 0) p.stats[2 * static_cast<size_t>(row) + 1] = rh;
    } else if (threadIdx.x == 0) {
      p.stats[2 * static_cast<size_t>(row) + 1] = 0.0f;
    }
    if (threadIdx.x == 0) p.stats[2 * static_cast<size_t>(row)] = ry;
  }
}

// hi + lo += v without losing what v leaves below hi's last bit
__device__ __forceinline__ void two_add(float& hi, float& lo, float v) {
  const float s = hi + v, b = s - hi;
  lo += (hi - (s - b)) + (v - b);
  hi = s;
}

// A thread's 16-byte copies of its columns of the rows ahead, `S` rows deep in shared
// memory; it waits for its own copies alone. Rows of four tensors lie behind one another,
// fp32 ones in two planes of 16 bytes a thread.
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

template <bool RF, bool OF, int NC, int S>
struct NormRing {
  static constexpr int kY = OF ? 2 : 1, kR = RF ? 2 : 1;  // planes
  static constexpr bool SP = RF || OF;
  uint8_t* base;
  int n8;
  __device__ __forceinline__ uint8_t* at(int stage, int plane, int i) const {
    return base + ((static_cast<size_t>(stage) * (2 * kY + 2 * kR) + plane) * n8 + i) * 16;
  }
  template <int P>
  __device__ __forceinline__ void put(int stage, int plane, int i, const void* src, size_t row) const {
    const uint8_t* q = static_cast<const uint8_t*>(src) + row * n8 * (16 * P);
    const uint32_t dst = smem_u32(at(stage, plane, i));
    if constexpr (P == 2) {
      cp_async16(dst, q + 16 * quad<SP>(i, n8, 0), true);
      cp_async16(dst + 16 * n8, q + 16 * quad<SP>(i, n8, 1), true);
    } else if constexpr (SP) {
      cp_async8(dst, q + 8 * quad<SP>(i, n8, 0));
      cp_async8(dst + 8, q + 8 * quad<SP>(i, n8, 1));
    } else {
      cp_async16(dst, q + 16 * i, true);
    }
  }
  // y, the residual, dn, dh of a row (those that there are)
  __device__ __forceinline__ void load(const NormParams& p, int stage, int row) const {
    if (row < p.T) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int i = threadIdx.x + c * blockDim.x;
        if (i < n8) {
          put<kY>(stage, 0, i, p.y, row);
          if (p.pre) put<kY>(stage, kY, i, p.dn, row);
          if (p.res) put<kR>(stage, 2 * kY, i, p.r, row);
          if (p.dh != nullptr) put<kR>(stage, 2 * kY + kR, i, p.dh, row);
        }
      }
    }
    cp_async_commit();
  }
  template <bool F32>
  __device__ __forceinline__ void get(int stage, int plane, int i, float (&v)[8]) const {
    Vec8<F32, SP> x;
    x.a = *reinterpret_cast<const uint4*>(at(stage, plane, i));
    if constexpr (F32) x.b = *reinterpret_cast<const uint4*>(at(stage, plane + 1, i));
    x.get(v);
  }
};

// FULL: with a post norm or a gate, whose gradients are another sum a column. A thread
// holds a column's sums, its weights, A and h: 64 registers for 8 columns, two blocks of
// 512 threads an SM or one of MAXT (72 registers up to 896 threads: the 64 of 1024 spill,
// into an L1 that shared memory has left small). S: rows on their way in shared memory; 0: straight from
// global memory (rows too long for it).
template <bool RF, bool OF, bool FULL, int NC, int S, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 512 ? 2 : 1) norm_bwd_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float red[2 * 96];
  using Ring = NormRing<RF, OF, NC, S>;
  constexpr bool SP = RF || OF;
  chain_wait();
  chain_release();
  int turn = 0;
  const int n8 = p.H >> 3;
  const float inv = 1.0f / static_cast<float>(p.H);
  const bool token = FULL && p.gate == MOE_GATE_TOKEN, post = FULL && p.post;
  const bool sum_d = FULL && (p.post || p.gate == MOE_GATE_CHANNEL);
  float an[NC][8], ad[FULL ? NC : 1][8];  // the sums of dpre and D
  float wn[NC][8], gw[FULL ? NC : 1][8];  // pre weight, gate x post weight
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      an[c][j] = wn[c][j] = 0.0f;
      if constexpr (FULL) {
        ad[c][j] = 0.0f;
        gw[c][j] = 1.0f;
      }
    }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = threadIdx.x + c * blockDim.x;
    if (i < n8) {
      if (p.pre) weights8<SP>(p.wn, i, n8, wn[c]);
      if constexpr (FULL) {
        if (p.post) weights8<SP>(p.wp, i, n8, gw[c]);
        if (p.gate == MOE_GATE_CHANNEL) {
          float g[8];
          weights8<SP>(p.g, i, n8, g);
#pragma unroll
          for (int j = 0; j < 8; ++j) gw[c][j] *= g[j];
        }
      }
    }
  }
  // a block's sums: [2][H], then what two floats keep beyond
  float* hi = p.part + static_cast<size_t>(blockIdx.x) * 4 * p.H;
  auto flush = [&](bool first) {
    const size_t beyond = 2 * static_cast<size_t>(p.H);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
#pragma unroll
      for (int k = 0; k < (FULL ? 2 : 1); ++k) {
        float(&v)[8] = k == 0 ? an[c] : ad[FULL ? c : 0];
        if (i < n8 && (k == 0 ? p.pre != 0 : sum_d)) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float4* d = reinterpret_cast<float4*>(hi + static_cast<size_t>(k) * p.H) + quad<SP>(i, n8, q);
            float4* e = reinterpret_cast<float4*>(hi + static_cast<size_t>(k) * p.H + beyond) + quad<SP>(i, n8, q);
            float4 s = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
            float4 lo = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (!first) {
              const float4 w = s;
              s = *d;
              lo = *e;
              two_add(s.x, lo.x, w.x);
              two_add(s.y, lo.y, w.y);
              two_add(s.z, lo.z, w.z);
              two_add(s.w, lo.w, w.w);
            }
            *d = s;
            if (p.lo) *e = lo;
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
      }
    }
  };
  const Ring ring{smem, n8};
  if constexpr (S > 0)
    for (int k = 0; k + 1 < S; ++k) ring.load(p, k, blockIdx.x + k * gridDim.x);
  // a row's scalars, asked for a row ahead
  float ry1 = 1.0f, rh1 = 0.0f, gt1 = 1.0f;
  auto scalars = [&](int row) {
    if (row < p.T) {
      if (post) ry1 = p.cstats[2 * static_cast<size_t>(row)];
      if (p.pre) rh1 = p.cstats[2 * static_cast<size_t>(row) + 1];
      if (token) gt1 = p.g[row];
    }
  };
  scalars(blockIdx.x);
  int rows = 0, stage = 0;
  bool first = true;
  for (int row = blockIdx.x; row < p.T; row += gridDim.x) {
    if constexpr (S > 0) {
      // (a thread reads and writes its own places only)
      ring.load(p, stage == 0 ? S - 1 : stage - 1, row + (S - 1) * gridDim.x);
      cp_async_wait<S - 1>();
    }
    const float ry = ry1, rh = rh1, gt = gt1;
    scalars(row + gridDim.x);
    auto get_own = [&](int i, auto f32, const void* src, int plane, float(&v)[8]) {
      constexpr bool F32 = decltype(f32)::value;
      if constexpr (S > 0) {
        ring.template get<F32>(stage, plane, i, v);
      } else {
        Vec8<F32, SP> x;
        x.load(src, row, i, n8);
        x.get(v);
      }
    };
    constexpr std::bool_constant<RF> rf{};
    constexpr std::bool_constant<OF> of{};
    float s0 = 0.0f, sa = 0.0f, sb = 0.0f;
    float A[NC][8], h[NC][8];  // h: with pre, h rh from the sums on
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      if (i < n8) {
        float t[8], x[8];  // x: what the sums for dy (or a token's gate) take A and hh with
        get_own(i, of, p.y, 0, x);
        if constexpr (FULL) {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = x[j] * ry * gw[c][j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) h[c][j] = token ? gt * x[j] : x[j];
        if (p.res) {
          get_own(i, rf, p.r, 2 * Ring::kY, t);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[c][j] = fmaf(p.a, t[j], h[c][j]);
        }
        if (p.dh != nullptr) {
          get_own(i, rf, p.dh, 2 * Ring::kY + Ring::kR, A[c]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) A[c][j] = 0.0f;
        }
        if (p.pre) {
          get_own(i, of, p.dn, Ring::kY, t);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            h[c][j] *= rh;
            an[c][j] = fmaf(t[j], h[c][j], an[c][j]);
            const float d = t[j] * wn[c][j];
            s0 = fmaf(d, h[c][j], s0);
            A[c][j] = fmaf(rh, d, A[c][j]);
          }
        }
        if constexpr (FULL) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            sa = fmaf(A[c][j], x[j], sa);
            sb = fmaf(h[c][j], x[j], sb);
          }
        }
      }
    }
    float s1 = 0.0f, s2 = 0.0f;
    if constexpr (FULL) {
      float s[3] = {s0, sa, sb};
      block_sum(s, red, turn);
      s1 = s[0] * -rh * inv;
      s2 = p.pre ? fmaf(s1, s[2], s[1]) : s[1];  // (without pre h is as large as it is)
    } else {
      float s[1] = {s0};
      block_sum(s, red, turn);
      s1 = s[0] * -rh * inv;
    }
    if (token && threadIdx.x == 0) p.dgate[row] = s2;
    // dy = ry (g dH wp) - (y ry) ry / H (ry S2); a token's sums are without its g
    const float yf = post ? (token ? gt : 1.0f) * s2 * ry * inv : 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      if (i < n8) {
        float (&d)[8] = A[c];
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = fmaf(s1, h[c][j], d[j]);
        if (p.res) {
          float t[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) t[j] = p.a * d[j];
          store8<RF, SP>(p.dr, row, i, n8, t);
        }
        if constexpr (FULL) {
          float t[8];
          get_own(i, of, p.y, 0, t);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            t[j] *= ry;
            d[j] *= gt;
            ad[c][j] = fmaf(d[j], t[j], ad[c][j]);
            d[j] = ry * (d[j] * gw[c][j]) - t[j] * yf;
          }
        }
        store8<false, SP>(p.dy, row, i, n8, d);
      }
    }
    if (p.part != nullptr && ++rows == kNormFlush) {
      flush(first);
      first = false;
      rows = 0;
    }
    if (++stage == S) stage = 0;
  }
  if (p.part != nullptr && (rows > 0 || first)) flush(first);
  if constexpr (S > 0) cp_async_wait_all();
}

// dpre (blockIdx.y 0), or dpost and dgate from D (1): sums over the blocks of hi + lo, in two
// floats; a thread a column and a sixteenth of the blocks, four of them on their way at a
// time
__global__ void __launch_bounds__(512) norm_join_kernel(const float* part, int blocks, int H, int lo, const float* wp,
                                                        const float* g, float* dpre, float* dpost, float* dgate) {
  __shared__ float s[2][16][33];
  chain_wait();
  const int lane = threadIdx.x & 31, col = blockIdx.x * 32 + lane, k = blockIdx.y, q = threadIdx.x >> 5;
  if (k == 0 ? dpre == nullptr : dpost == nullptr && dgate == nullptr) return;
  float hi = 0.0f, rest = 0.0f;
  if (col < H) {
    const float* src = part + static_cast<size_t>(k) * H + col;
    const size_t step = 4 * static_cast<size_t>(H);
    for (int b = q; b < blocks; b += 64) {
      float v[4], w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* r = src + (b + 16 * i) * step;
        v[i] = b + 16 * i < blocks ? __ldcg(r) : 0.0f;
        w[i] = lo && b + 16 * i < blocks ? __ldcg(r + 2 * static_cast<size_t>(H)) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        two_add(hi, rest, v[i]);
        rest += w[i];
      }
    }
  }
  s[0][q][lane] = hi;
  s[1][q][lane] = rest;
  __syncthreads();
  if (q == 0 && col < H) {
#pragma unroll
    for (int i = 1; i < 16; ++i) {
      two_add(hi, rest, s[0][i][lane]);
      rest += s[1][i][lane];
    }
    const float d = hi + rest;
    if (k == 0) dpre[col] = d;
    if (k == 1 && dpost != nullptr) dpost[col] = g != nullptr ? g[col] * d : d;
    if (k == 1 && dgate != nullptr) dgate[col] = wp != nullptr ? wp[col] * d : d;
  }
}

static int check_norm(const moe_norm_config* c) {
  if (c == nullptr) return MOE_ERR_INVALID_ARG;
  if (c->T < 1 || c->H < 1 || !(c->eps >= 0.0f)) return MOE_ERR_INVALID_ARG;
  if (c->gate < MOE_GATE_NONE || c->gate > MOE_GATE_TOKEN) return MOE_ERR_INVALID_ARG;
  for (int v : {c->residual, c->post, c->pre, c->residual_fp32, c->out_fp32})
    if (v != 0 && v != 1) return MOE_ERR_INVALID_ARG;
  if (c->residual_scale != c->residual_scale) return MOE_ERR_INVALID_ARG;
  // (a row index and a stride of blocks beyond it stay within 32 bits)
  if (c->H % 8 || c->H > kNormMaxH || c->T > (1 << 30)) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}
// runs of 8 columns a thread in the backward
static int norm_runs(int H) { return H <= 8192 ? 1 : 2; }
static dim3 norm_threads(int H, int nc) { return dim3(((H / 8 + nc - 1) / nc + 31) / 32 * 32); }
constexpr size_t kNormSmem = 230400;      // of a block, at most
constexpr size_t kNormSmemSM = 233472;    // of an SM
constexpr size_t kNormSmemOther = 1792;   // a block's sums and what the system keeps

// bytes of a row of y, dn, the residual and dh
static size_t norm_row_bytes(const moe_norm_config& c) {
  return static_cast<size_t>(c.H) * 2 * ((c.out_fp32 ? 4 : 2) + (c.residual_fp32 ? 4 : 2));
}
// rows on their way in shared memory in the backward: none where rows are too long for two
static int norm_ring(const moe_norm_config& c) { return c.H <= 8192 && 2 * norm_row_bytes(c) <= kNormSmem ? 2 : 0; }
// blocks of the backward: those that an SM holds at once, at 64 registers a thread and with their rows (counted
// by threads alone: 32768 x 1024 fp32 in and out, gate and both norms, 8 blocks for 6, 162 us for 133; 16384 x 2048 164 for 134)
static int norm_per_sm(const moe_norm_config& c) {
  int per = 1024 / static_cast<int>(norm_threads(c.H, norm_runs(c.H)).x);
  const int hold = static_cast<int>(kNormSmemSM / (norm_ring(c) * norm_row_bytes(c) + kNormSmemOther));
  if (per > hold) per = hold;
  return per < 16 ? per : 16;
}
static int norm_blocks(const moe_norm_config& c) {
  const int most = norm_per_sm(c) * num_sms();
  return c.T < most ? c.T : most;
}
static bool norm_sums(const moe_norm_config& c) { return c.pre || c.post || c.gate == MOE_GATE_CHANNEL; }

template <bool RF, bool OF, int NC>
static cudaError_t launch_fwd(const moe_norm_config& c, const NormParams& p, int grid, cudaStream_t s) {
  return launch_chained(norm_fwd_kernel<RF, OF, NC>, dim3(grid), norm_threads(c.H, NC), 0, s, p);
}
template <bool RF, bool OF, bool FULL, int NC, int S, int MAXT>
static cudaError_t launch_bwd(const moe_norm_config& c, const NormParams& p, int grid, cudaStream_t s) {
  const size_t bytes = S * norm_row_bytes(c);
  const auto kernel = norm_bwd_kernel<RF, OF, FULL, NC, S, MAXT>;
  if constexpr (S > 0) {
    static std::atomic<unsigned long long> set{0};  // devices whose kernel has its shared memory
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!(set.load() & (1ull << (dev & 63)))) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem);
      if (e != cudaSuccess) return e;
      set.fetch_or(1ull << (dev & 63));
    }
  }
  return launch_chained(kernel, dim3(grid), norm_threads(c.H, NC), bytes, s, p);
}
// One row on its way beside the row at work (two, where they fit: 16384 x 4096 138 us for 137), none where two
// rows pass the shared memory. Up to 7168 columns 896 threads of 72 registers (1024 of 64: 5003 x 7168
// with an fp32 stream 147 us for 117, 4096 x 7168 106 for 85); up to 4096 blocks of at most 512 threads,
// several an SM.
template <bool RF, bool OF, bool FULL>
static cudaError_t launch_bwd(const moe_norm_config& c, const NormParams& p, int grid, cudaStream_t s) {
  if (c.H > 8192) return launch_bwd<RF, OF, FULL, 2, 0, 1024>(c, p, grid, s);
  if (c.H > 7168)
    return norm_ring(c) ? launch_bwd<RF, OF, FULL, 1, 2, 1024>(c, p, grid, s)
                                : launch_bwd<RF, OF, FULL, 1, 0, 1024>(c, p, grid, s);
  if (c.H > 4096) return launch_bwd<RF, OF, FULL, 1, 2, 896>(c, p, grid, s);  // (at most 224 KB)
  return launch_bwd<RF, OF, FULL, 1, 2, 512>(c, p, grid, s);
}
template <bool RF, bool OF>
static cudaError_t launch_norm(bool bwd, const moe_norm_config& c, const NormParams& p, int grid, cudaStream_t s) {
  const int n8 = c.H / 8;
  if (!bwd) {
    // runs of 8 columns a thread, in blocks of at most 512 threads (16384 x 4096: one run 93 us, two 86, four
    // 90; 5003 x 7168 two 77, four 84)
    if (n8 <= 128) return launch_fwd<RF, OF, 1>(c, p, grid, s);
    return n8 <= 1024 ? launch_fwd<RF, OF, 2>(c, p, grid, s) : launch_fwd<RF, OF, 4>(c, p, grid, s);
  }
  return c.post || c.gate ? launch_bwd<RF, OF, true>(c, p, grid, s) : launch_bwd<RF, OF, false>(c, p, grid, s);
}
static cudaError_t launch_norm(bool bwd, const moe_norm_config& c, const NormParams& p, int grid, cudaStream_t s) {
  if (c.residual_fp32) return c.out_fp32 ? launch_norm<true, true>(bwd, c, p, grid, s) : launch_norm<true, false>(bwd, c, p, grid, s);
  return c.out_fp32 ? launch_norm<false, true>(bwd, c, p, grid, s) : launch_norm<false, false>(bwd, c, p, grid, s);
}

struct NormArray {
  const void* p;
  size_t bytes;
};

}  // namespace moe

using namespace moe;

static bool norm_misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
static bool norm_clash(const NormArray& a, const NormArray& b) { return overlap(a.p, a.bytes, b.p, b.bytes); }

extern "C" {

int moe_block_norm_fwd(const moe_norm_config* cfg, const void* y, const void* residual, const float* post_weight,
                       const float* gate, const float* pre_weight, void* h, moe_bf16* n, float* stats, void* stream) {
  NvtxRange nvtx("moe_block_norm_fwd");
  int r = check_norm(cfg);
  if (r != MOE_OK) return r;
  const moe_norm_config& c = *cfg;
  if (!c.residual) residual = nullptr;
  if (!c.post) post_weight = nullptr;
  if (!c.gate) gate = nullptr;
  if (!c.pre) pre_weight = nullptr, n = nullptr;
  if (!y || !stats || (c.residual && !residual) || (c.post && !post_weight) || (c.gate && !gate) ||
      (c.pre && (!pre_weight || !n)) || (!h && !n))
    return MOE_ERR_INVALID_ARG;
  for (const void* p : {y, residual, static_cast<const void*>(post_weight), static_cast<const void*>(gate),
                        static_cast<const void*>(pre_weight), static_cast<const void*>(h),
                        static_cast<const void*>(n), static_cast<const void*>(stats)})
    if (norm_misaligned(p)) return MOE_ERR_INVALID_ARG;
  const size_t N = static_cast<size_t>(c.T) * c.H, sb = c.residual_fp32 ? 4 : 2, yb = c.out_fp32 ? 4 : 2;
  const NormArray Y{y, N * yb}, R{residual, N * sb}, Hh{h, N * sb}, Nn{n, N * 2}, S{stats, 8ull * c.T};
  const NormArray small[3] = {{post_weight, 4ull * c.H}, {gate, 4ull * (c.gate == MOE_GATE_TOKEN ? c.T : c.H)}, {pre_weight, 4ull * c.H}};
  // a thread reads its part of a row before it writes it: one of the same shape and type may be written over
  if ((norm_clash(Hh, Y) && !(h == y && sb == yb)) || (norm_clash(Hh, R) && h != residual) ||
      (norm_clash(Nn, Y) && !(n == y && yb == 2)) || norm_clash(Nn, R) || norm_clash(Hh, Nn) || norm_clash(S, Y) ||
      norm_clash(S, R) || norm_clash(S, Hh) || norm_clash(S, Nn))
    return MOE_ERR_INVALID_ARG;
  for (const NormArray& w : small)
    if (norm_clash(w, Hh) || norm_clash(w, Nn) || norm_clash(w, S)) return MOE_ERR_INVALID_ARG;
  NormParams p{};
  p.T = c.T; p.H = c.H; p.eps = c.eps; p.a = c.residual_scale;
  p.res = c.residual; p.gate = c.gate; p.post = c.post; p.pre = c.pre;
  p.y = y; p.r = residual; p.wp = post_weight; p.g = gate; p.wn = pre_weight;
  p.h = h; p.n = reinterpret_cast<__nv_bfloat16*>(n); p.stats = stats;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int most = 16 * num_sms();
  r = status_from_cuda(launch_norm(false, c, p, c.T < most ? c.T : most, s));
  if (r == MOE_OK) record_stage(s, 53, 1);
  return r;
}

size_t moe_norm_workspace_bytes(const moe_norm_config* cfg) {
  if (check_norm(cfg) != MOE_OK) return 0;
  return sizeof(DevStatus) + 16ull * cfg->H * norm_blocks(*cfg);
}

int moe_block_norm_bwd(const moe_norm_config* cfg, const void* dh, const void* dn, const void* y,
                       const void* residual, const float* post_weight, const float* gate, const float* pre_weight,
                       const float* stats, moe_bf16* dy, void* dresidual, float* dpost_weight, float* dgate,
                       float* dpre_weight, void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nvtx("moe_block_norm_bwd");
  int r = check_norm(cfg);
  if (r != MOE_OK) return r;
  const moe_norm_config& c = *cfg;
  if (!c.residual) residual = nullptr, dresidual = nullptr;
  if (!c.post) post_weight = nullptr, dpost_weight = nullptr;
  if (!c.gate) gate = nullptr, dgate = nullptr;
  if (!c.pre) pre_weight = nullptr, dn = nullptr, dpre_weight = nullptr;
  if (!y || !stats || !dy || !ws || (!dh && !dn) || (c.residual && (!residual || !dresidual)) ||
      (c.post && (!post_weight || !dpost_weight)) || (c.gate && (!gate || !dgate)) ||
      (c.pre && (!pre_weight || !dn || !dpre_weight)))
    return MOE_ERR_INVALID_ARG;
  const size_t N = static_cast<size_t>(c.T) * c.H, sb = c.residual_fp32 ? 4 : 2, yb = c.out_fp32 ? 4 : 2;
  const size_t gb = 4ull * (c.gate == MOE_GATE_TOKEN ? c.T : c.H), hb = 4ull * c.H;
  const size_t need = moe_norm_workspace_bytes(cfg);
  const NormArray in[8] = {{dh, N * sb}, {dn, N * yb}, {y, N * yb}, {residual, N * sb}, {post_weight, hb},
                           {gate, gb}, {pre_weight, hb}, {stats, 8ull * c.T}};
  const NormArray out[6] = {{dy, N * 2}, {dresidual, N * sb}, {dpost_weight, hb}, {dgate, gb}, {dpre_weight, hb},
                            {ws, need}};
  for (const NormArray& a : in)
    if (norm_misaligned(a.p)) return MOE_ERR_INVALID_ARG;
  for (const NormArray& a : out)
    if (norm_misaligned(a.p)) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < 6; ++i) {
    for (int j = 0; j < 8; ++j) {
      const bool same = out[i].p == in[j].p && ((i == 1 && j == 0) || (i == 0 && j == 1 && yb == 2));
      if (norm_clash(out[i], in[j]) && !same) return MOE_ERR_INVALID_ARG;
    }
    for (int j = 0; j < i; ++j)
      if (norm_clash(out[i], out[j])) return MOE_ERR_INVALID_ARG;
  }
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  NormParams p{};
  p.T = c.T; p.H = c.H; p.eps = c.eps; p.a = c.residual_scale;
  p.res = c.residual; p.gate = c.gate; p.post = c.post; p.pre = c.pre;
  p.y = y; p.r = residual; p.dh = dh; p.dn = dn; p.wp = post_weight; p.g = gate; p.wn = pre_weight;
  p.dr = dresidual; p.dy = reinterpret_cast<__nv_bfloat16*>(dy); p.cstats = stats; p.dgate = dgate;
  p.part = norm_sums(c) ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + sizeof(DevStatus)) : nullptr;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int blocks = norm_blocks(c);
  p.lo = c.T > kNormFlush * blocks ? 1 : 0;
  r = status_from_cuda(launch_norm(true, c, p, blocks, s));
  if (r != MOE_OK) return r;
  record_stage(s, 54, 1);
  if (!norm_sums(c)) return MOE_OK;
  const float* part = p.part;
  const bool channel = c.gate == MOE_GATE_CHANNEL;
  float* dg = channel ? dgate : nullptr;
  const float* cg = channel ? gate : nullptr;
  r = status_from_cuda(launch_chained(norm_join_kernel, dim3((c.H + 31) / 32, 2), dim3(512), 0, s, part, blocks, c.H,
                                      p.lo, post_weight, cg, dpre_weight, dpost_weight, dg));
  if (r == MOE_OK) record_stage(s, 55, 1);
  return r;
}

}  // extern "C"
