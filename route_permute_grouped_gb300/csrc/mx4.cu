// MXFP4 (OCP Microscaling Formats v1.0, MXFP4): blocks of 32 consecutive elements
// along the contraction share a power of two 2^s, s = floor(log2 max|v|) - 2 clamped to
// [-127, 127] (-127 for a block of zeros), kept as the E8M0 byte s + 127; an element is
// v / 2^s rounded to E2M1 (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6; to nearest, ties to the
// even code, saturating at 6). A block with an infinity or a NaN has the byte 255: all of
// it stands for NaN.
//
// All kernels here move bytes: per element 2 of bf16 one way and 17/32 of codes and
// scales the other (16384 x 4096 rows 28 us either way, 6.1 TB/s; 32 experts of 4096 x 1536
// 260 us, 5.9 TB/s). Rows: four lanes a block, so that every access of a warp is
// contiguous. Weights: a block of threads turns a tile of 128 k x 128 columns, its
// loads 128 bytes of a weight row a warp, and stages the codes in shared memory, from
// where they leave in the layout that few.cuh's copies read.
#include <cuda_fp4.h>

#include <initializer_list>

#include "host_util.h"

namespace moe {

constexpr int kMx4Tile = 16384 + 1024;  // codes and scales of 128 columns x 256 elements

// Arithmetic in pairs of bf16, which hold every step exactly: magnitudes and their
// maximum (a NaN stays one), the division by the block's power of two, and back the
// values times it. About four instructions an element either way; decoding each code in
// fp32 took twelve and bound the way back (16384 x 4096 rows 46 us).
__device__ __forceinline__ uint32_t bf162_max_abs(uint32_t m, uint32_t v) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(v & 0x7fff7fffu));
  return r;
}
__device__ __forceinline__ uint32_t bf162_mul(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
// scale byte of a block of maximum magnitude `amax` (bf16 bits): its exponent less 2;
// 255 where it is an infinity or a NaN
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax) {
  const uint32_t e = amax >> 7;
  return e >= 255u ? 255u : e > 2u ? e - 2u : 0u;
}
// 2^-s twice: s + 127 = sb <= 252, so that it is a normal bf16 number (255: zero)
__device__ __forceinline__ uint32_t mx4_inverse(uint32_t sb) { return sb == 255u ? 0u : (254u - sb) * 0x00800080u; }
// 2^s twice (a subnormal number for sb = 0), NaN for 255
__device__ __forceinline__ uint32_t mx4_scale(uint32_t sb) {
  return sb == 255u ? 0x7fc07fc0u : sb == 0u ? 0x00400040u : sb * 0x00800080u;
}
// codes of a pair, the lower half's in the low four bits
__device__ __forceinline__ uint32_t mx4_pair(uint32_t v) {
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(make_float2(bf16_lo(v), bf16_hi(v)), __NV_E2M1, cudaRoundNearest));
}
// four codes (the low 16 bits) as two pairs: their magnitudes' bytes looked up four at a time
__device__ __forceinline__ void mx4_values4(uint32_t c, uint32_t scale, uint32_t& a, uint32_t& b) {
  const uint32_t sel = c & 0x7777u;
  const uint32_t hi = __byte_perm(0x3f3f3f00u, 0x40404040u, sel), lo = __byte_perm(0xc0800000u, 0xc0804000u, sel);
  a = bf162_mul(__byte_perm(lo, hi, 0x5140) | ((c << 12) & 0x8000u) | ((c << 24) & 0x80000000u), scale);
  b = bf162_mul(__byte_perm(lo, hi, 0x7362) | ((c << 4) & 0x8000u) | ((c << 16) & 0x80000000u), scale);
}

// x [M, K] -> q [M, K/2], s [M, K/32]; a thread 8 elements, four threads a block of 32,
// two blocks on their way
__global__ void __launch_bounds__(256) mx4_quantize_kernel(const __nv_bfloat16* x, long long n8, uint8_t* q,
                                                           uint8_t* s) {
  chain_wait();
  const long long step = static_cast<long long>(gridDim.x) * 256;
  const unsigned group = 0xFu << (threadIdx.x & 28);
  // (whole groups of four lanes run or skip: n8 is a multiple of 4)
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < n8; i += 2 * step) {
    uint4 w[2];
    w[0] = __ldcs(reinterpret_cast<const uint4*>(x) + i);
    const bool two = i + step < n8;
    if (two) w[1] = __ldcs(reinterpret_cast<const uint4*>(x) + i + step);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (u == 1 && !two) break;
      const long long at = i + u * step;
      uint32_t m = bf162_max_abs(bf162_max_abs(bf162_max_abs(bf162_max_abs(0u, w[u].x), w[u].y), w[u].z), w[u].w);
      m = bf162_max_abs(m, __shfl_xor_sync(group, m, 1));
      m = bf162_max_abs(m, __shfl_xor_sync(group, m, 2));
      m = bf162_max_abs(m, m >> 16);
      const uint32_t sb = mx4_scale_byte(m & 0xffffu), inv = mx4_inverse(sb);
      const uint32_t c = mx4_pair(bf162_mul(w[u].x, inv)) | (mx4_pair(bf162_mul(w[u].y, inv)) << 8) |
                         (mx4_pair(bf162_mul(w[u].z, inv)) << 16) | (mx4_pair(bf162_mul(w[u].w, inv)) << 24);
      reinterpret_cast<uint32_t*>(q)[at] = sb == 255u ? 0u : c;
      if ((threadIdx.x & 3) == 0) s[at >> 2] = static_cast<uint8_t>(sb);
    }
  }
}

// the way back, exact (every value is a bf16 number); a thread 8 elements, four on their way
__global__ void __launch_bounds__(256) mx4_dequantize_kernel(const uint8_t* q, const uint8_t* s, long long n8,
                                                             __nv_bfloat16* x) {
  chain_wait();
  const long long step = static_cast<long long>(gridDim.x) * 256;
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < n8; i += 4 * step) {
    uint32_t c[4], sb[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const long long at = i + u * step;
      c[u] = at < n8 ? __ldcg(reinterpret_cast<const uint32_t*>(q) + at) : 0u;
      sb[u] = at < n8 ? __ldcg(s + (at >> 2)) : 0u;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (i + u * step >= n8) break;
      uint4 v;
      const uint32_t f = mx4_scale(sb[u]);
      mx4_values4(c[u], f, v.x, v.y);
      mx4_values4(c[u] >> 16, f, v.z, v.w);
      reinterpret_cast<uint4*>(x)[i + u * step] = v;
    }
  }
}

// A weight [E][K][N] bf16 and where its tiles go. A tile holds 128 columns x 256 elements
// of k as the few-token kernel's shared memory has them: a column's 128 bytes of codes
// with their 16-byte chunks swizzled (chunk c of column r at c ^ (r % 8)), 16 KB, then two
// times 512 scale bytes, byte 16 (r % 32) + 4 (r / 32) + b of half h that of column r's
// block 4 h + b. Tile (e, column block nb, k block kb) is number ((e nnb + nb) nkb + kb)
// `tiles` + `which` (W1 and W3 alternate: tiles = 2); k beyond K is zeros.
struct Mx4Weight {
  const __nv_bfloat16* w;
  __nv_bfloat16* out;  // the way back
  uint8_t* q;
  int K, N, tiles, which;
  long long first;     // its first half tile among all of the launch
};
struct Mx4Weights {
  Mx4Weight w[6];
  int n;
  long long total;
};

// half a tile at a time: 128 elements of k
template <bool BACK>
__global__ void __launch_bounds__(256) mx4_weights_kernel(const __grid_constant__ Mx4Weights a) {
  __shared__ __align__(16) uint8_t codes[128 * 64];
  __shared__ __align__(16) uint8_t scales[512];
  chain_wait();
  const int warp = warp_id(), lane = lane_id();
  const int b = warp & 3, col = (warp >> 2) * 64 + 2 * lane;  // the thread's block along k and its two columns
  for (long long t = blockIdx.x; t < a.total; t += gridDim.x) {
    int i = 0;
    while (i + 1 < a.n && t >= a.w[i + 1].first) ++i;
    const Mx4Weight& w = a.w[i];
    const int nkb = (w.K + 255) >> 8, nnb = w.N >> 7;
    const long long r = t - w.first;
    // columns innermost: neighbouring blocks read neighbouring parts of the weight's rows
    const int nb = static_cast<int>(r % nnb);
    const long long r2 = r / nnb;
    const int k2 = static_cast<int>(r2 % (2 * nkb)), half = k2 & 1;
    const long long e = r2 / (2 * nkb);
    uint8_t* tile = w.q + (((e * nnb + nb) * nkb + (k2 >> 1)) * w.tiles + w.which) * kMx4Tile;
    const bool in = 128 * k2 < w.K;  // (beyond: the last tile's second half)
    const size_t at = (static_cast<size_t>(e) * w.K + 128 * k2 + 32 * b) * w.N + 128 * nb + col;
    // 16-byte chunk i of the half: column i / 4, block i % 4
    auto chunk = [&](int i) { return reinterpret_cast<uint4*>(tile + (i >> 2) * 128 + (((4 * half + (i & 3)) ^ ((i >> 2) & 7)) << 4)); };
    uint4* sf = reinterpret_cast<uint4*>(tile + 16384 + 512 * half);
    if constexpr (!BACK) {
      uint32_t v[32];
      const uint32_t* src = reinterpret_cast<const uint32_t*>(w.w + at);
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = in ? __ldcs(src + static_cast<size_t>(j) * (w.N >> 1)) : 0u;
      uint32_t mx = 0u;
#pragma unroll
      for (int j = 0; j < 32; ++j) mx = bf162_max_abs(mx, v[j]);
      const uint32_t s0 = mx4_scale_byte(mx & 0xffffu), s1 = mx4_scale_byte(mx >> 16);
      const uint32_t inv = (mx4_inverse(s0) & 0xffffu) | (mx4_inverse(s1) & 0xffff0000u);
      uint32_t c0[4] = {0, 0, 0, 0}, c1[4] = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const uint32_t a = bf162_mul(v[2 * j], inv), d = bf162_mul(v[2 * j + 1], inv);
        c0[j >> 2] |= mx4_pair(__byte_perm(a, d, 0x5410)) << (8 * (j & 3));
        c1[j >> 2] |= mx4_pair(__byte_perm(a, d, 0x7632)) << (8 * (j & 3));
      }
      if (s0 == 255u) c0[0] = c0[1] = c0[2] = c0[3] = 0u;
      if (s1 == 255u) c1[0] = c1[1] = c1[2] = c1[3] = 0u;
      __syncthreads();  // the half before has left
      *reinterpret_cast<uint4*>(codes + col * 64 + b * 16) = make_uint4(c0[0], c0[1], c0[2], c0[3]);
      *reinterpret_cast<uint4*>(codes + (col + 1) * 64 + b * 16) = make_uint4(c1[0], c1[1], c1[2], c1[3]);
      scales[16 * (col & 31) + 4 * (col >> 5) + b] = static_cast<uint8_t>(s0);
      scales[16 * ((col + 1) & 31) + 4 * (col >> 5) + b] = static_cast<uint8_t>(s1);
      __syncthreads();
      for (int i = threadIdx.x; i < 512; i += 256) *chunk(i) = reinterpret_cast<const uint4*>(codes)[i];
      if (threadIdx.x < 32) sf[threadIdx.x] = reinterpret_cast<const uint4*>(scales)[threadIdx.x];
    } else {
      __syncthreads();
      for (int i = threadIdx.x; i < 512; i += 256) reinterpret_cast<uint4*>(codes)[i] = __ldcg(chunk(i));
      if (threadIdx.x < 32) reinterpret_cast<uint4*>(scales)[threadIdx.x] = __ldcg(sf + threadIdx.x);
      __syncthreads();
      if (!in) continue;
      const uint4 a0 = *reinterpret_cast<const uint4*>(codes + col * 64 + b * 16);
      const uint4 a1 = *reinterpret_cast<const uint4*>(codes + (col + 1) * 64 + b * 16);
      const uint32_t c0[4] = {a0.x, a0.y, a0.z, a0.w}, c1[4] = {a1.x, a1.y, a1.z, a1.w};
      const uint32_t f0 = mx4_scale(scales[16 * (col & 31) + 4 * (col >> 5) + b]);
      const uint32_t f1 = mx4_scale(scales[16 * ((col + 1) & 31) + 4 * (col >> 5) + b]);
      uint32_t* dst = reinterpret_cast<uint32_t*>(w.out + at);
      const size_t ld = w.N >> 1;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // four elements of either column, then of each k both columns'
        uint32_t a01, a23, d01, d23;
        mx4_values4(c0[j >> 1] >> (16 * (j & 1)), f0, a01, a23);
        mx4_values4(c1[j >> 1] >> (16 * (j & 1)), f1, d01, d23);
        dst[(4 * j) * ld] = __byte_perm(a01, d01, 0x5410);
        dst[(4 * j + 1) * ld] = __byte_perm(a01, d01, 0x7632);
        dst[(4 * j + 2) * ld] = __byte_perm(a23, d23, 0x5410);
        dst[(4 * j + 3) * ld] = __byte_perm(a23, d23, 0x7632);
      }
    }
  }
}

static int check_mx4(const moe_config* cfg) {
  const int s = validate_config(cfg);
  if (s != MOE_OK) return s;
  if (cfg->H % 128 || cfg->F % 128 || cfg->F_shared % 128) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

static bool mx4_aligned(std::initializer_list<const void*> ps, uintptr_t to) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) & (to - 1)) return false;
  return true;
}

static int mx4_weights(const moe_config* cfg, const void* const (&bf)[6], const moe_mx4_weights* w, bool back,
                       void* stream) {
  const int st = check_mx4(cfg);
  if (st != MOE_OK) return st;
  const moe_config& c = *cfg;
  const int n = c.F_shared ? 6 : 3;
  if (!w || !w->w13 || !w->w2 || (c.F_shared && (!w->w13s || !w->w2s))) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (!bf[i] || !mx4_aligned({bf[i]}, 16)) return MOE_ERR_INVALID_ARG;
  if (!mx4_aligned({w->w13, w->w2, w->w13s, w->w2s}, 16)) return MOE_ERR_INVALID_ARG;
  const uint8_t* q[4] = {w->w13, w->w2, w->w13s, w->w2s};
  const int nq = c.F_shared ? 4 : 2;
  auto bf_bytes = [&](int j) { return 2ull * (j >= 3 ? c.F_shared : static_cast<size_t>(c.E) * c.F) * c.H; };
  for (int i = 0; i < nq; ++i) {
    const size_t bytes = moe_mx4_weight_bytes(cfg, i);
    for (int j = 0; j < n; ++j)
      if (overlap(q[i], bytes, bf[j], bf_bytes(j))) return MOE_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(q[i], bytes, q[j], moe_mx4_weight_bytes(cfg, j))) return MOE_ERR_INVALID_ARG;
  }
  for (int i = 0; back && i < n; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(bf[i], bf_bytes(i), bf[j], bf_bytes(j))) return MOE_ERR_INVALID_ARG;
  Mx4Weights a{};
  a.n = n;
  for (int i = 0; i < n; ++i) {
    Mx4Weight& m = a.w[i];
    const bool sh = i >= 3, down = i % 3 == 2;
    const int F = sh ? c.F_shared : c.F;
    m.w = static_cast<const __nv_bfloat16*>(bf[i]);
    m.out = static_cast<__nv_bfloat16*>(const_cast<void*>(bf[i]));
    m.q = down ? (sh ? w->w2s : w->w2) : (sh ? w->w13s : w->w13);
    m.K = down ? F : c.H;
    m.N = down ? c.H : F;
    m.tiles = down ? 1 : 2;
    m.which = down ? 0 : i % 3;
    m.first = a.total;
    a.total += static_cast<long long>(sh ? 1 : c.E) * ((m.K + 255) / 256 * 2) * (m.N / 128);
  }
  const long long most = 8ll * num_sms();
  const int grid = static_cast<int>(a.total < most ? a.total : most);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = back ? launch_chained(mx4_weights_kernel<true>, dim3(grid), dim3(256), 0, s, a)
                             : launch_chained(mx4_weights_kernel<false>, dim3(grid), dim3(256), 0, s, a);
  const int r = status_from_cuda(e);
  if (r == MOE_OK) record_stage(s, back ? 52 : 51, 1);
  return r;
}

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_mx4_weight_bytes(const moe_config* cfg, int which) {
  if (check_mx4(cfg) != MOE_OK || which < 0 || which > 3) return 0;
  const bool shared = which >= 2, down = which & 1;
  const size_t F = shared ? cfg->F_shared : cfg->F, H = cfg->H, E = shared ? 1 : cfg->E;
  const size_t tiles = down ? (H / 128) * ((F + 255) / 256) : 2 * (F / 128) * ((H + 255) / 256);
  return F == 0 ? 0 : E * tiles * kMx4Tile;
}

int moe_mx4_quantize_weights(const moe_config* cfg, const moe_bf16* W1, const moe_bf16* W3, const moe_bf16* W2,
                             const moe_bf16* Ws1, const moe_bf16* Ws3, const moe_bf16* Ws2, const moe_mx4_weights* w,
                             void* stream) {
  NvtxRange nvtx("moe_mx4_quantize_weights");
  const void* bf[6] = {W1, W3, W2, Ws1, Ws3, Ws2};
  return mx4_weights(cfg, bf, w, false, stream);
}

int moe_mx4_dequantize_weights(const moe_config* cfg, const moe_mx4_weights* w, moe_bf16* W1, moe_bf16* W3,
                               moe_bf16* W2, moe_bf16* Ws1, moe_bf16* Ws3, moe_bf16* Ws2, void* stream) {
  NvtxRange nvtx("moe_mx4_dequantize_weights");
  const void* bf[6] = {W1, W3, W2, Ws1, Ws3, Ws2};
  return mx4_weights(cfg, bf, w, true, stream);
}

static int mx4_rows_check(const void* x, long long M, int K, const uint8_t* q, const uint8_t* s) {
  if (!x || !q || !s || M < 1 || K < 1) return MOE_ERR_INVALID_ARG;
  if (!mx4_aligned({x, q, s}, 16)) return MOE_ERR_INVALID_ARG;
  if (K % 32 || M > (1ll << 60) / K) return MOE_ERR_UNSUPPORTED_SHAPE;
  const size_t n = static_cast<size_t>(M) * K;
  if (overlap(x, 2 * n, q, n / 2) || overlap(x, 2 * n, s, n / 32) || overlap(q, n / 2, s, n / 32)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

int moe_mx4_quantize(const moe_bf16* x, long long M, int K, uint8_t* q, uint8_t* scales, void* stream) {
  NvtxRange nvtx("moe_mx4_quantize");
  int r = mx4_rows_check(x, M, K, q, scales);
  if (r != MOE_OK) return r;
  const long long n8 = M * K / 8, blocks = (n8 + 255) / 256, most = 16ll * num_sms();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  r = status_from_cuda(launch_chained(mx4_quantize_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)),
                                      dim3(256), 0, s, reinterpret_cast<const __nv_bfloat16*>(x), n8, q, scales));
  if (r == MOE_OK) record_stage(s, 51, 1);
  return r;
}

int moe_mx4_dequantize(const uint8_t* q, const uint8_t* scales, long long M, int K, moe_bf16* x, void* stream) {
  NvtxRange nvtx("moe_mx4_dequantize");
  int r = mx4_rows_check(x, M, K, q, scales);
  if (r != MOE_OK) return r;
  const long long n8 = M * K / 8, blocks = (n8 + 255) / 256, most = 16ll * num_sms();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  r = status_from_cuda(launch_chained(mx4_dequantize_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)),
                                      dim3(256), 0, s, q, scales, n8, reinterpret_cast<__nv_bfloat16*>(x)));
  if (r == MOE_OK) record_stage(s, 52, 1);
  return r;
}

}  // extern "C"
