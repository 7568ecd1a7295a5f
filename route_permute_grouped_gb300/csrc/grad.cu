// Global norm of a list of gradients and its clipping: one pass that sums the
// squares (or takes the maximum) of every tensor, one that scales.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <type_traits>
#include <vector>

#include "host_util.h"

namespace moe {

// A tensor list as the kernels take it: the tensors of one launch by value in
// the kernel's parameters, so a call copies nothing to the device and captures
// into a graph as it is. A chunk is kChunkVecs 16-byte vectors of one tensor;
// `first` holds each tensor's first chunk.
constexpr int kListTensors = 768;
constexpr int kGradThreads = 512;
constexpr int kVecsPerThread = 4;
constexpr int kChunkVecs = kGradThreads * kVecsPerThread;  // 32 KB
constexpr int kMaxLaunches = 64;                           // 49152 tensors
constexpr int kMaxPartials = 2048;                         // CTAs of one launch

struct GradItem {
  const void* in;
  void* out;
  long long n;
};
template <int N>
struct GradBlock {
  int count;    // tensors
  int chunks;   // chunks of all of them
  int apart;    // some tensor has an output of its own
  int first[N];
  uint8_t dtype[N];
  GradItem item[N];
};
struct GradList {
  uint32_t magic;
  int n, launches, pad;
  GradBlock<kListTensors> block[1];  // `launches` of them
};
constexpr uint32_t kListMagic = 0x6d6f6c31u;

static size_t list_bytes(int n) {
  const int launches = (n + kListTensors - 1) / kListTensors;
  return offsetof(GradList, block) + sizeof(GradBlock<kListTensors>) * static_cast<size_t>(launches > 0 ? launches : 1);
}
static int elem_bytes(int dtype) { return dtype == MOE_FP32 ? 4 : 2; }

// Where the 16-byte vectors of a tensor begin: elements before the first
// aligned address (at most n), the vectors, and the elements after them.
struct Span {
  int head;
  long long vecs;
  int tail;
};
__host__ __device__ inline Span span_of(const void* p, long long n, int eb) {
  Span s;
  const int per = 16 / eb;
  const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u);
  long long head = mis == 0 ? 0 : (16 - mis) / eb;
  if (head > n) head = n;
  s.head = static_cast<int>(head);
  s.vecs = (n - head) / per;
  s.tail = static_cast<int>(n - head - s.vecs * per);
  return s;
}

template <int N>
__device__ __forceinline__ int find_tensor(const GradBlock<N>& b, int chunk) {
  int lo = 0, hi = b.count;  // the last tensor whose first chunk is <= chunk
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.first[mid] <= chunk) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ float elem_f32(const void* p, long long i, int dtype) {
  if (dtype == MOE_FP32) return static_cast<const float*>(p)[i];
  if (dtype == MOE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void store_elem(void* p, long long i, int dtype, float v) {
  if (dtype == MOE_FP32) static_cast<float*>(p)[i] = v;
  else if (dtype == MOE_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}
// the 4 or 8 values of a 16-byte vector
template <int DT>
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[DT == MOE_FP32 ? 4 : 8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (DT == MOE_FP32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == MOE_BF16) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
      } else {
        const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[2 * i] = h.x;
        f[2 * i + 1] = h.y;
      }
    }
  }
}
template <int DT>
__device__ __forceinline__ uint4 pack(const float (&f)[DT == MOE_FP32 ? 4 : 8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == MOE_FP32) w[i] = __float_as_uint(f[i]);
    else if constexpr (DT == MOE_BF16) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    else {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The squares of a thread's values: a sum in two floats (s + e: the exact sum but
// for the roundings of e), and beside it one in fp64 for values whose squares
// leave fp32. A square leaves its range for |g| above 2^64 and loses its bits
// below 2^-63, so a group (the 16 or 32 values of a pass) whose largest magnitude
// lies outside [2^-60, 2^40] and is not 0 is squared in fp64; NaN and infinities
// take that way too. Elsewhere the group's squares are added in fp32 and the
// groups in two floats: 2^85 a group leaves room for 2^42 of them. fp64 runs at
// about two additions a clock and SM, which even the blocks' own reductions felt
// (norm of 123 MB: 32 us with fp64 throughout).
constexpr uint32_t kSquareLo = (127u - 60u) << 23, kSquareHi = (127u + 40u) << 23;
struct Squares {
  float s = 0.0f, e = 0.0f;
  uint32_t top = 0;  // largest magnitude, as fp32 bits: NaN above infinity above the finite values
  double far = 0.0;
  __device__ __forceinline__ void add(float x) {
    const float t = s + x, b = t - s;
    e += (s - (t - b)) + (x - b);
    s = t;
  }
  template <int NV>
  __device__ __forceinline__ void group(const float (&f)[NV]) {
    float q = 0.0f;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      q = fmaf(f[i], f[i], q);
      m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
    }
    top = max(top, m);
    if (m <= kSquareHi && (m >= kSquareLo || m == 0)) {
      add(q);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) far += static_cast<double>(f[i]) * f[i];
    }
  }
};

template <int DT>
__device__ __forceinline__ void norm_chunk(const uint4* v, long long vecs, long long at, Squares& sq) {
  constexpr int PER = DT == MOE_FP32 ? 4 : 8;
  uint4 w[kVecsPerThread];
#pragma unroll
  for (int j = 0; j < kVecsPerThread; ++j) {
    const long long i = at + j * kGradThreads + threadIdx.x;
    w[j] = i < vecs ? __ldcg(v + i) : make_uint4(0, 0, 0, 0);
  }
  float f[kVecsPerThread * PER];
#pragma unroll
  for (int j = 0; j < kVecsPerThread; ++j) {
    float g[PER];
    unpack<DT>(w[j], g);
#pragma unroll
    for (int i = 0; i < PER; ++i) f[j * PER + i] = g[i];
  }
  sq.group(f);
}

// A CTA takes the chunks first, first + blocks, ... (neighbouring CTAs on
// neighbouring chunks: runs of chunks for each CTA took 10% longer to scale
// 2.4 GB). The tensor of the first one is searched, later ones lie further on.
template <int N>
struct ChunkWalk {
  int c, t;
  __device__ __forceinline__ ChunkWalk(const GradBlock<N>& b, int first) : c(first) {
    t = c < b.chunks ? find_tensor(b, c) : 0;
  }
  __device__ __forceinline__ void next(const GradBlock<N>& b, int blocks) {
    c += blocks;
    if (c >= b.chunks) return;
    if (t + 1 < b.count && b.first[t + 1] <= c) {
      ++t;
      if (t + 1 < b.count && b.first[t + 1] <= c) t = find_tensor(b, c);
    }
  }
};

// Each CTA's sum (fp64) and largest magnitude go to its partial; the CTA that
// arrives last, over all launches of a list, adds them in a fixed order, writes
// the norm and puts the ticket back to 0. Bound by HBM: 2.42 GB in 350 us, 6.9 TB/s;
// 35 MB in 18 us from a cold L2, where the launch, the first loads and the join weigh as much.
struct NormPartial {
  double sum;
  unsigned long long top;
};
constexpr int kGradWarps = kGradThreads / 32;
template <int N>
__global__ void __launch_bounds__(kGradThreads)
    norm_kernel(const __grid_constant__ GradBlock<N> b, NormPartial* __restrict__ partials, int at_partial, int all,
                int kind, int* __restrict__ ticket, float* __restrict__ norm) {
  Squares sq;
  chain_wait();
  for (ChunkWalk<N> run(b, blockIdx.x); run.c < b.chunks; run.next(b, gridDim.x)) {
    const int c = run.c, t = run.t;
    const int dt = b.dtype[t];
    const GradItem it = b.item[t];
    const int eb = dt == MOE_FP32 ? 4 : 2;
    const Span sp = span_of(it.in, it.n, eb);
    const uint4* v = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(it.in) + static_cast<size_t>(sp.head) * eb);
    const long long at = static_cast<long long>(c - b.first[t]) * kChunkVecs;
    if (dt == MOE_FP32) norm_chunk<MOE_FP32>(v, sp.vecs, at, sq);
    else if (dt == MOE_BF16) norm_chunk<MOE_BF16>(v, sp.vecs, at, sq);
    else norm_chunk<MOE_FP16>(v, sp.vecs, at, sq);
    if (at == 0 && threadIdx.x < static_cast<unsigned>(sp.head + sp.tail)) {
      const long long i = threadIdx.x < static_cast<unsigned>(sp.head) ? threadIdx.x : it.n - sp.tail + (threadIdx.x - sp.head);
      const float f[1] = {elem_f32(it.in, i, dt)};
      sq.group(f);
    }
  }
  __shared__ float2 s_sum[kGradWarps];
  __shared__ uint32_t s_top[kGradWarps];
  __shared__ double s_far[kGradThreads];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  chain_release();
  const bool any_far = __syncthreads_or(sq.far != 0.0) != 0;  // true for NaN
  if (any_far) s_far[tid] = sq.far;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float os = __shfl_xor_sync(0xffffffffu, sq.s, o), oe = __shfl_xor_sync(0xffffffffu, sq.e, o);
    sq.add(os);
    sq.e += oe;
    sq.top = max(sq.top, __shfl_xor_sync(0xffffffffu, sq.top, o));
  }
  if (lane == 0) {
    s_sum[warp] = make_float2(sq.s, sq.e);
    s_top[warp] = sq.top;
  }
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kGradWarps; ++w) {
      sq.add(s_sum[w].x);
      sq.e += s_sum[w].y;
      sq.top = max(sq.top, s_top[w]);
    }
    double sum = static_cast<double>(sq.s) + sq.e;
    if (any_far)
      for (int i = 0; i < kGradThreads; ++i) sum += s_far[i];
    partials[at_partial + blockIdx.x].sum = sum;
    partials[at_partial + blockIdx.x].top = sq.top;
    __threadfence();
    s_last = atomicAdd(ticket, 1) == all - 1;
    __threadfence();
  }
  __syncthreads();
  if (!s_last) return;
  // a warp's worth of fp64 additions: the block's threads add what lies
  // kGradThreads apart (rarely more than two), lane l those of threads l, l + 32, ...
  double sum = 0.0;
  uint32_t top = 0;
  for (int i = tid; i < all; i += kGradThreads) {
    sum += __ldcg(&partials[i].sum);
    top = max(top, static_cast<uint32_t>(__ldcg(&partials[i].top)));
  }
  s_far[tid] = sum;
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) s_top[warp] = top;
  __syncthreads();
  if (warp != 0) return;
  sum = 0.0;
#pragma unroll
  for (int w = 0; w < kGradWarps; ++w) {
    sum += s_far[32 * w + lane];
    top = max(top, s_top[w]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) {
    *norm = kind == MOE_NORM_MAX ? __uint_as_float(top) : static_cast<float>(sqrt(sum));
    *ticket = 0;
  }
}

// A chunk of a tensor in the thread's registers
struct Chunk {
  GradItem it;
  Span sp;
  int dt, eb;
  long long at;  // first vector
  uint4 w[kVecsPerThread];
};
template <int N>
__device__ __forceinline__ void fetch(const GradBlock<N>& b, int c, Chunk& k) {
  const int t = find_tensor(b, c);
  k.it = b.item[t];
  k.dt = b.dtype[t];
  k.eb = k.dt == MOE_FP32 ? 4 : 2;
  k.sp = span_of(k.it.in, k.it.n, k.eb);
  k.at = static_cast<long long>(c - b.first[t]) * kChunkVecs;
  const uint4* v = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(k.it.in) +
                                                  static_cast<size_t>(k.sp.head) * k.eb);
#pragma unroll
  for (int j = 0; j < kVecsPerThread; ++j) {
    const long long i = k.at + j * kGradThreads + threadIdx.x;
    if (i < k.sp.vecs) k.w[j] = __ldcg(v + i);
  }
}
template <int DT>
__device__ __forceinline__ void scale_chunk(const Chunk& k, uint4* __restrict__ o, float coef) {
  constexpr int PER = DT == MOE_FP32 ? 4 : 8;
#pragma unroll
  for (int j = 0; j < kVecsPerThread; ++j) {
    const long long i = k.at + j * kGradThreads + threadIdx.x;
    if (i < k.sp.vecs) {
      float f[PER];
      unpack<DT>(k.w[j], f);
#pragma unroll
      for (int e = 0; e < PER; ++e) f[e] *= coef;
      o[i] = pack<DT>(f);
    }
  }
}

// g = round(g * coef), coef = min(1, max_norm / (norm + 1e-6)) (NaN for a NaN
// norm, 1 for an infinite max_norm and any other norm). coef = 1 leaves every bit as it is, so tensors scaled in place are
// then neither read further nor written. The chunks go from the last one down:
// what the norm's pass read last is what L2 still holds. A block's first chunk is
// on its way while the norm's last block still adds up: the norm's kernel only
// reads it, and has waited for all ahead of it. Bound by HBM: 2.42 GB scaled in
// 690 us, 7.0 TB/s; norm and scaling of 35 MB, the second out of L2, 20 us.
template <int N>
__global__ void __launch_bounds__(kGradThreads) clip_kernel(const __grid_constant__ GradBlock<N> b,
                                                            const float* __restrict__ norm, float max_norm, int resident) {
  const int grid = static_cast<int>(gridDim.x), first = static_cast<int>(blockIdx.x);
  const bool any = first < b.chunks;
  int i = any ? (b.chunks - 1 - first) / grid : 0;
  Chunk k;
  if (any && first < resident) fetch(b, first + i * grid, k);
  chain_wait();
  const float n = __ldcg(norm);
  float coef = max_norm / (n + 1e-6f);
  if (coef > 1.0f || (isinf(max_norm) && !isnan(n))) coef = 1.0f;
  if (!any || (coef == 1.0f && !b.apart)) return;
  if (first >= resident) fetch(b, first + i * grid, k);
  while (true) {
    if (coef != 1.0f || k.it.in != k.it.out) {
      uint8_t* ob = static_cast<uint8_t*>(k.it.out) + static_cast<size_t>(k.sp.head) * k.eb;
      if ((reinterpret_cast<uintptr_t>(ob) & 15u) == 0) {
        uint4* o = reinterpret_cast<uint4*>(ob);
        if (k.dt == MOE_FP32) scale_chunk<MOE_FP32>(k, o, coef);
        else if (k.dt == MOE_BF16) scale_chunk<MOE_BF16>(k, o, coef);
        else scale_chunk<MOE_FP16>(k, o, coef);
      } else {
        // the output is aligned otherwise than the input: element by element
        const int per = 16 / k.eb;
        const long long end = min(k.sp.vecs, k.at + kChunkVecs) * per;
        for (long long e = k.at * per + threadIdx.x; e < end; e += kGradThreads)
          store_elem(k.it.out, k.sp.head + e, k.dt, elem_f32(k.it.in, k.sp.head + e, k.dt) * coef);
      }
      const unsigned head = static_cast<unsigned>(k.sp.head);
      if (k.at == 0 && threadIdx.x < head + k.sp.tail) {
        const long long e = threadIdx.x < head ? threadIdx.x : k.it.n - k.sp.tail + (threadIdx.x - head);
        store_elem(k.it.out, e, k.dt, elem_f32(k.it.in, e, k.dt) * coef);
      }
    }
    if (--i < 0) return;
    fetch(b, first + i * grid, k);
  }
}

template <int N>
static auto clip_kernel_of(const GradBlock<N>*) {
  return clip_kernel<N>;
}
template <int N>
static auto norm_kernel_of(const GradBlock<N>*) {
  return norm_kernel<N>;
}
// Blocks of the norm: what is resident at a time (twice that, 123 MB: 32.1 us for
// norm and clipping below the threshold, 27.4 so)
static int norm_grid(int chunks) { return std::max(1, std::min({chunks, 2 * num_sms(), kMaxPartials})); }
// Blocks of the clipping: the resident ones while those have up to 16 chunks, more
// beyond: blocks that go through hundreds of chunks drift apart (norm and clipping in
// us with two chunks a block, 16, and resident blocks alone: 140 MB 70, 66, 66; 560
// MB 254, 259, 267; 2400 MB 1019, 1036, 1091; but with two chunks a block 37000
// blocks start for nothing where nothing is scaled).
static int clip_grid(int chunks) { return std::max(1, std::min(chunks, std::max(2 * num_sms(), chunks / 16))); }

// launches `f` with the block in the smallest parameter size that holds it
template <class F>
static cudaError_t with_block(const GradBlock<kListTensors>& b, F f) {
  auto copy = [&](auto& small) {
    small.count = b.count;
    small.chunks = b.chunks;
    small.apart = b.apart;
    memcpy(small.first, b.first, sizeof(int) * b.count);
    memcpy(small.dtype, b.dtype, b.count);
    memcpy(small.item, b.item, sizeof(GradItem) * b.count);
    f(small);
  };
  if (b.count <= 16) {
    GradBlock<16> s;
    copy(s);
  } else if (b.count <= 128) {
    GradBlock<128> s;
    copy(s);
  } else {
    f(b);
  }
  return cudaGetLastError();
}

static const GradList* as_list(const void* list) {
  const GradList* l = static_cast<const GradList*>(list);
  return l != nullptr && (reinterpret_cast<uintptr_t>(list) & 7u) == 0 && l->magic == kListMagic ? l : nullptr;
}

static int run_norm(const GradList& l, int kind, float* norm, void* ws, cudaStream_t s) {
  int* ticket = &static_cast<DevStatus*>(ws)->chunk_counter;
  NormPartial* partials = reinterpret_cast<NormPartial*>(static_cast<uint8_t*>(ws) + sizeof(DevStatus));
  int all = 0;
  for (int i = 0; i < l.launches; ++i) all += norm_grid(l.block[i].chunks);
  int at = 0;
  for (int i = 0; i < l.launches; ++i) {
    const int grid = norm_grid(l.block[i].chunks);
    cudaError_t e2 = cudaSuccess;
    const cudaError_t e = with_block(l.block[i], [&](const auto& b) {
      using Block = std::remove_cv_t<std::remove_reference_t<decltype(b)>>;
      e2 = launch_chained(norm_kernel_of(static_cast<const Block*>(nullptr)), grid, kGradThreads, 0, s, b, partials, at,
                          all, kind, ticket, norm);
    });
    if (e2 != cudaSuccess) return status_from_cuda(e2);
    if (e != cudaSuccess) return status_from_cuda(e);
    record_stage(s, 40, 1);
    at += grid;
  }
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_tensor_list_bytes(int n) { return n < 0 || n > kMaxLaunches * kListTensors ? 0 : list_bytes(n); }

int moe_tensor_list_build(const moe_tensor* ts, int n, void* list, size_t list_size) {
  if (n < 0 || (ts == nullptr && n > 0) || list == nullptr || (reinterpret_cast<uintptr_t>(list) & 7u) != 0)
    return MOE_ERR_INVALID_ARG;
  if (n > kMaxLaunches * kListTensors) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (list_size < list_bytes(n)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  struct Range {
    uintptr_t lo, hi;
    int id;
    bool write;
  };
  std::vector<Range> ranges;
  try {
    ranges.reserve(2 * static_cast<size_t>(n));
  } catch (...) {
    return MOE_ERR_INVALID_ARG;
  }
  GradList* l = static_cast<GradList*>(list);
  l->magic = 0;
  l->n = n;
  l->pad = 0;
  l->launches = std::max(1, (n + kListTensors - 1) / kListTensors);
  for (int i = 0; i < l->launches; ++i) l->block[i].count = l->block[i].chunks = l->block[i].apart = 0;
  for (int i = 0; i < n; ++i) {
    const moe_tensor& t = ts[i];
    if (t.dtype != MOE_FP32 && t.dtype != MOE_BF16 && t.dtype != MOE_FP16) return MOE_ERR_INVALID_ARG;
    if (t.n < 0 || (t.n > 0 && t.data == nullptr)) return MOE_ERR_INVALID_ARG;
    const int eb = elem_bytes(t.dtype);
    void* out = t.out != nullptr ? t.out : t.data;
    if (reinterpret_cast<uintptr_t>(t.data) % eb != 0 || reinterpret_cast<uintptr_t>(out) % eb != 0)
      return MOE_ERR_INVALID_ARG;
    if (t.n >= (1ll << 42)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (t.n == 0) continue;
    const uintptr_t a = reinterpret_cast<uintptr_t>(t.data), o = reinterpret_cast<uintptr_t>(out);
    const size_t bytes = static_cast<size_t>(t.n) * eb;
    if (out != t.data) ranges.push_back({a, a + bytes, i, false});
    ranges.push_back({o, o + bytes, i, true});
    GradBlock<kListTensors>& b = l->block[i / kListTensors];
    const Span sp = span_of(t.data, t.n, eb);
    const long long chunks = std::max(1ll, (sp.vecs + kChunkVecs - 1) / kChunkVecs);
    if (b.chunks + chunks > (1ll << 30)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (out != t.data) b.apart = 1;
    b.first[b.count] = b.chunks;
    b.dtype[b.count] = static_cast<uint8_t>(t.dtype);
    b.item[b.count] = {t.data, out, t.n};
    b.chunks += static_cast<int>(chunks);
    ++b.count;
  }
  // what is written must not be read or written for another tensor: two CTAs
  // would race, and a tensor listed twice would be scaled twice
  std::sort(ranges.begin(), ranges.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t read_end = 0, write_end = 0;
  for (const Range& r : ranges) {
    if (r.lo < write_end || (r.write && r.lo < read_end)) return MOE_ERR_INVALID_ARG;
    (r.write ? write_end : read_end) = std::max(r.write ? write_end : read_end, r.hi);
  }
  l->magic = kListMagic;
  return MOE_OK;
}

size_t moe_grad_norm_workspace_bytes(void) {
  return sizeof(DevStatus) + sizeof(NormPartial) * static_cast<size_t>(kMaxLaunches) * kMaxPartials;
}

int moe_grad_norm(const void* list, int kind, float* norm, void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nvtx("moe_grad_norm");
  const GradList* l = as_list(list);
  if (l == nullptr || norm == nullptr || ws == nullptr || (kind != MOE_NORM_L2 && kind != MOE_NORM_MAX))
    return MOE_ERR_INVALID_ARG;
  if (((reinterpret_cast<uintptr_t>(norm) | reinterpret_cast<uintptr_t>(ws)) & 15u) != 0)
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < moe_grad_norm_workspace_bytes()) return MOE_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return run_norm(*l, kind, norm, ws, s);
}

int moe_clip_grad_norm(const void* list, int kind, float max_norm, float* norm, void* ws, size_t ws_bytes,
                       void* stream) {
  NvtxRange nvtx("moe_clip_grad_norm");
  const GradList* l = as_list(list);
  if (l == nullptr || norm == nullptr || ws == nullptr || (kind != MOE_NORM_L2 && kind != MOE_NORM_MAX) ||
      !(max_norm >= 0.0f))
    return MOE_ERR_INVALID_ARG;
  if (((reinterpret_cast<uintptr_t>(norm) | reinterpret_cast<uintptr_t>(ws)) & 15u) != 0)
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < moe_grad_norm_workspace_bytes()) return MOE_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int st = run_norm(*l, kind, norm, ws, s);
  if (st != MOE_OK) return st;
  for (int i = 0; i < l->launches; ++i) {
    cudaError_t e2 = cudaSuccess;
    const cudaError_t e = with_block(l->block[i], [&](const auto& b) {
      using Block = std::remove_cv_t<std::remove_reference_t<decltype(b)>>;
      e2 = launch_chained(clip_kernel_of(static_cast<const Block*>(nullptr)), clip_grid(b.chunks), kGradThreads, 0, s,
                          b, static_cast<const float*>(norm), max_norm, 2 * num_sms());
    });
    if (e2 != cudaSuccess) return status_from_cuda(e2);
    if (e != cudaSuccess) return status_from_cuda(e);
    record_stage(s, 41, 1);
  }
  return MOE_OK;
}

}  // extern "C"
