// Norms before and after a block with its gate and the scaled residual, and their
// backward (moe_block_norm_fwd, moe_block_norm_bwd):
//   u = post ? y ry wp : y,  h = a r + g u,  n = h rh wn,
//   ry = 1 / sqrt(mean(y^2) + eps),  rh = 1 / sqrt(mean(h^2) + eps).
// Both directions move each tensor once and are bound by that (forward y, r in, h, n
// out; backward y, r, dh, dn in, dy, dr out): a block of threads holds a row in
// registers from its loads to its stores, and h is computed again in the backward
// rather than kept. With dnw = dn wn the backward is
//   dH = A + S1 B,  A = dh + rh dnw,  B = -h rh^3 / H,  S1 = sum dnw h,
//   dr = a dH,  dy = ry (g dH wp - y ry^2 / H S2),  S2 = sum g dH wp y,
// and since dH is linear in S1, S2 = SA + S1 SB with sums of A and B alone: one
// reduction over the block for a row. The gradients of the weights and of a channel
// gate are sums over rows: a thread adds its columns' in fp32 over at most 64 rows,
// then in two floats in the workspace; a second kernel joins the blocks' in order.
#include "host_util.h"

namespace moe {

constexpr int kNormFlush = 64;   // rows added in fp32 alone
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
  const float* cstats;
};

// 8 elements of a row, from bf16 or fp32
template <bool F32>
struct Vec8 {
  uint4 a, b;
  __device__ __forceinline__ void load(const void* base, size_t i8) {
    const uint4* p = static_cast<const uint4*>(base) + (F32 ? 2 : 1) * i8;
    a = __ldcs(p);
    if constexpr (F32) b = __ldcs(p + 1);
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
template <bool F32>
__device__ __forceinline__ void store8(void* base, size_t i8, const float (&v)[8]) {
  uint4* p = static_cast<uint4*>(base) + (F32 ? 2 : 1) * i8;
  if constexpr (F32) {
    p[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    p[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
  } else {
    p[0] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
}
__device__ __forceinline__ void weights8(const float* w, int i8, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(w)[2 * i8], b = reinterpret_cast<const float4*>(w)[2 * i8 + 1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Sums of N values over the block, in every thread; `s` alternates between two halves, so
// that one barrier a sum is enough
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* s, int& turn) {
  const int warp = warp_id(), lane = lane_id(), nw = blockDim.x >> 5;
  float* b = s + (turn & 1) * 96;
  ++turn;
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) b[i * 32 + warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane < nw ? b[i * 32 + lane] : 0.0f;
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
}

// RF: residual stream fp32, OF: y (and dn) fp32; NC runs of 8 columns a thread
template <bool RF, bool OF, int NC>
__global__ void __launch_bounds__(512) norm_fwd_kernel(const __grid_constant__ NormParams p) {
  __shared__ float red[2 * 96];
  chain_wait();
  int turn = 0;
  const int n8 = p.H >> 3;
  const float inv = 1.0f / static_cast<float>(p.H);
  for (int row = blockIdx.x; row < p.T; row += gridDim.x) {
    const size_t r8 = static_cast<size_t>(row) * n8;
    Vec8<OF> yv[NC];
    Vec8<RF> rv[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      if (i < n8) {
        yv[c].load(p.y, r8 + i);
        if (p.res) rv[c].load(p.r, r8 + i);
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
          weights8(p.wp, i, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[c][j] = h[c][j] * ry * w[j];
        }
        if (p.gate == MOE_GATE_CHANNEL) {
          float w[8];
          weights8(p.g, i, w);
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
        if (p.h != nullptr) store8<RF>(p.h, r8 + i, h[c]);
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
          weights8(p.wn, i, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[c][j] = h[c][j] * rh * w[j];
          store8<false>(p.n, r8 + i, h[c]);
        }
      }
      if (threadIdx.x == 0) p.stats[2 * static_cast<size_t>(row) + 1] = rh;
    }
    if (threadIdx.x == 0 && p.post) p.stats[2 * static_cast<size_t>(row)] = ry;
  }
}

// hi + lo += v without losing what v leaves below hi's last bit
__device__ __forceinline__ void two_add(float& hi, float& lo, float v) {
  const float s = hi + v, b = s - hi;
  lo += (hi - (s - b)) + (v - b);
  hi = s;
}

template <bool RF, bool OF, int NC>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const __grid_constant__ NormParams p) {
  __shared__ float red[2 * 96];
  chain_wait();
  chain_release();
  int turn = 0;
  const int n8 = p.H >> 3;
  const float inv = 1.0f / static_cast<float>(p.H);
  const bool channel = p.gate == MOE_GATE_CHANNEL, token = p.gate == MOE_GATE_TOKEN;
  const bool second = p.post || token;  // a sum for dy or for the token's gate
  float an[NC][8], ap[NC][8], ag[NC][8];  // of dpre, dpost, dgate
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) an[c][j] = ap[c][j] = ag[c][j] = 0.0f;
  // a block's sums: [3][H], then what two floats keep beyond
  float* hi = p.part + static_cast<size_t>(blockIdx.x) * 6 * p.H;
  auto flush = [&](bool first) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      if (i >= n8) continue;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        if (!(k == 0 ? p.pre : k == 1 ? p.post : channel)) continue;
        float* d = hi + static_cast<size_t>(k) * p.H + 8 * i;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float v = k == 0 ? an[c][j] : k == 1 ? ap[c][j] : ag[c][j], lo = 0.0f;
          if (!first) {
            float s = d[j];
            lo = d[3 * static_cast<size_t>(p.H) + j];
            two_add(s, lo, v);
            v = s;
          }
          d[j] = v;
          d[3 * static_cast<size_t>(p.H) + j] = lo;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) an[c][j] = ap[c][j] = ag[c][j] = 0.0f;
    }
  };
  int rows = 0;
  bool first = true;
  for (int row = blockIdx.x; row < p.T; row += gridDim.x) {
    const size_t r8 = static_cast<size_t>(row) * n8;
    Vec8<OF> yv[NC], nv[NC];
    Vec8<RF> rv[NC], hv[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      if (i < n8) {
        yv[c].load(p.y, r8 + i);
        if (p.res) rv[c].load(p.r, r8 + i);
        if (p.pre) nv[c].load(p.dn, r8 + i);
        if (p.dh != nullptr) hv[c].load(p.dh, r8 + i);
      }
    }
    const float ry = p.post ? p.cstats[2 * static_cast<size_t>(row)] : 1.0f;
    const float rh = p.pre ? p.cstats[2 * static_cast<size_t>(row) + 1] : 0.0f;
    const float gt = token ? p.g[row] : 1.0f;
    const float bf = -rh * rh * rh * inv;
    float s[3] = {0.0f, 0.0f, 0.0f};
    float A[NC][8], h[NC][8], u[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      if (i < n8) {
        float w[8], g[8], t[8];
        yv[c].get(u[c]);
        if (p.post) {
          weights8(p.wp, i, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) u[c][j] = u[c][j] * ry * w[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = gt;
        if (channel) weights8(p.g, i, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[c][j] = g[j] * u[c][j];
        if (p.res) {
          rv[c].get(t);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[c][j] = fmaf(p.a, t[j], h[c][j]);
        }
        if (p.dh != nullptr) hv[c].get(A[c]);
        else {
#pragma unroll
          for (int j = 0; j < 8; ++j) A[c][j] = 0.0f;
        }
        if (p.pre) {
          nv[c].get(t);
          weights8(p.wn, i, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            an[c][j] = fmaf(t[j], h[c][j] * rh, an[c][j]);
            const float d = t[j] * w[j];
            s[0] = fmaf(d, h[c][j], s[0]);
            A[c][j] = fmaf(rh, d, A[c][j]);
          }
        }
        if (second) {
          // g u = g y ry wp: the sums are of ry S2; a token's gate wants them without g
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float x = (token ? 1.0f : g[j]) * u[c][j];
            s[1] = fmaf(A[c][j], x, s[1]);
            s[2] = fmaf(bf * h[c][j], x, s[2]);
          }
        }
      }
    }
    float s1 = 0.0f, s2 = 0.0f;
    if (p.pre || second) {
      block_sum(s, red, turn);
      s1 = s[0] * bf;
      s2 = fmaf(s[0], s[2], s[1]);
    }
    if (token && threadIdx.x == 0) p.dgate[row] = s2;
    // dy = ry (g dH wp) - y ry^2 / H (ry S2)
    const float yf = p.post ? (token ? gt : 1.0f) * s2 * ry * ry * inv : 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      if (i < n8) {
        float w[8], g[8], t[8], d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = fmaf(s1, h[c][j], A[c][j]);
        if (p.res) {
#pragma unroll
          for (int j = 0; j < 8; ++j) t[j] = p.a * d[j];
          store8<RF>(p.dr, r8 + i, t);
        }
        if (channel) {
          weights8(p.g, i, g);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            ag[c][j] = fmaf(d[j], u[c][j], ag[c][j]);
            d[j] *= g[j];
          }
        } else if (token) {
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] *= gt;
        }
        if (p.post) {
          weights8(p.wp, i, w);
          yv[c].get(t);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            ap[c][j] = fmaf(d[j], t[j] * ry, ap[c][j]);
            d[j] = fmaf(d[j] * w[j], ry, -t[j] * yf);
          }
        }
        store8<false>(p.dy, r8 + i, d);
      }
    }
    if (++rows == kNormFlush) {
      flush(first);
      first = false;
      rows = 0;
    }
  }
  if (p.part != nullptr && (rows > 0 || first)) flush(first);
}

// out[k][j] = sum over the blocks of hi + lo; a thread a column and a sixteenth of the blocks
__global__ void __launch_bounds__(512) norm_join_kernel(const float* part, int blocks, int H, float* dpre, float* dpost,
                                                        float* dgate) {
  __shared__ double s[16][33];
  chain_wait();
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), k = blockIdx.y, q = threadIdx.x >> 5;
  float* out = k == 0 ? dpre : k == 1 ? dpost : dgate;
  if (out == nullptr) return;
  double v = 0.0;
  if (col < H) {
    const float* src = part + static_cast<size_t>(k) * H + col;
    for (int b = q; b < blocks; b += 16) {
      const float* r = src + static_cast<size_t>(b) * 6 * H;
      v += static_cast<double>(__ldcg(r)) + static_cast<double>(__ldcg(r + 3 * static_cast<size_t>(H)));
    }
  }
  s[q][threadIdx.x & 31] = v;
  __syncthreads();
  if (q == 0 && col < H) {
    double t = 0.0;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += s[i][threadIdx.x];
    out[col] = static_cast<float>(t);
  }
}

static int check_norm(const moe_norm_config* c) {
  if (c == nullptr) return MOE_ERR_INVALID_ARG;
  if (c->T < 1 || c->H < 1 || !(c->eps >= 0.0f)) return MOE_ERR_INVALID_ARG;
  if (c->gate < MOE_GATE_NONE || c->gate > MOE_GATE_TOKEN) return MOE_ERR_INVALID_ARG;
  for (int v : {c->residual, c->post, c->pre, c->residual_fp32, c->out_fp32})
    if (v != 0 && v != 1) return MOE_ERR_INVALID_ARG;
  if (c->residual_scale != c->residual_scale) return MOE_ERR_INVALID_ARG;
  if (c->H % 8 || c->H > kNormMaxH) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}
static int norm_blocks(const moe_norm_config& c) { return c.T < 2 * num_sms() ? c.T : 2 * num_sms(); }
static bool norm_sums(const moe_norm_config& c) { return c.pre || c.post || c.gate == MOE_GATE_CHANNEL; }

// runs of 8 columns a thread: 512 threads at most
static int norm_runs(int H) { return H <= 1024 ? 1 : H <= 8192 ? 2 : 4; }
static dim3 norm_threads(int H) {
  const int nc = norm_runs(H), n = (H / 8 + nc - 1) / nc;
  return dim3((n + 31) / 32 * 32);
}

template <bool BWD>
static cudaError_t launch_norm(const moe_norm_config& c, const NormParams& p, int grid, cudaStream_t s) {
  const int nc = norm_runs(c.H);
  auto go = [&](auto kern) { return launch_chained(kern, dim3(grid), norm_threads(c.H), 0, s, p); };
#define MOE_NORM(RF, OF)                                                                       \
  (nc == 1   ? go(BWD ? norm_bwd_kernel<RF, OF, 1> : norm_fwd_kernel<RF, OF, 1>)               \
   : nc == 2 ? go(BWD ? norm_bwd_kernel<RF, OF, 2> : norm_fwd_kernel<RF, OF, 2>)               \
             : go(BWD ? norm_bwd_kernel<RF, OF, 4> : norm_fwd_kernel<RF, OF, 4>))
  if (c.residual_fp32) return c.out_fp32 ? MOE_NORM(true, true) : MOE_NORM(true, false);
  return c.out_fp32 ? MOE_NORM(false, true) : MOE_NORM(false, false);
#undef MOE_NORM
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
  r = status_from_cuda(launch_norm<false>(c, p, c.T < most ? c.T : most, s));
  if (r == MOE_OK) record_stage(s, 53, 1);
  return r;
}

size_t moe_norm_workspace_bytes(const moe_norm_config* cfg) {
  if (check_norm(cfg) != MOE_OK) return 0;
  return sizeof(DevStatus) + 24ull * cfg->H * norm_blocks(*cfg);
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
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + sizeof(DevStatus));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int blocks = norm_blocks(c);
  r = status_from_cuda(launch_norm<true>(c, p, blocks, s));
  if (r != MOE_OK) return r;
  record_stage(s, 54, 1);
  if (!norm_sums(c)) return MOE_OK;
  const float* part = p.part;
  float* dg = c.gate == MOE_GATE_CHANNEL ? dgate : nullptr;
  r = status_from_cuda(launch_chained(norm_join_kernel, dim3((c.H + 31) / 32, 3), dim3(512), 0, s, part, blocks, c.H,
                                      dpre_weight, dpost_weight, dg));
  if (r == MOE_OK) record_stage(s, 55, 1);
  return r;
}

}  // extern "C"
