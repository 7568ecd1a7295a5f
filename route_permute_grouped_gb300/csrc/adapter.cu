// Low-rank adapters of many requests beside a shared projection: row t of a
// batch gets base[t] + s_a (x[t] A_a) B_a of its own adapter a, and the
// backward of that. Rows are ordered by adapter once for a batch (the plan);
// every product then works on tiles of one adapter's rows: up to 64 of them on
// mma.sync for small batches (here), up to 128 on tcgen05 for large ones
// (adapter_tc.cuh).
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <atomic>

#include "adapter_tc.cuh"

namespace moe {

constexpr int kTileRows = 64;
constexpr int kPlanThreads = 1024;
// Chunks up to which the placing blocks count all rows themselves; beyond, a launch
// of its own counts first (random rows of 40 adapters: 2000 rows 5.7 us both ways,
// 8192 rows 10.6 us and 5.8)
constexpr int kPlanChunks = 2;
constexpr int kMaxAdapters = 1024;
constexpr int kAdSMs = 152;

// ---------------------------------------------------------------------------
// the plan
// ---------------------------------------------------------------------------
struct PlanLayout {
  size_t hdr, seg, tiles, big, order, hist, total;
  int max_tiles, max_big, chunks;
};
static PlanLayout plan_layout(const moe_adapter_config& c) {
  PlanLayout p{};
  size_t o = 256;  // the status word
  auto take = [&](size_t b) {
    const size_t at = o;
    o += (b + 255) & ~size_t(255);
    return at;
  };
  p.max_tiles = c.T / kTileRows + std::min(c.T, c.L + 1);
  p.max_big = c.T / 128 + std::min(c.T, c.L + 1);
  p.chunks = (c.T + kPlanThreads - 1) / kPlanThreads;
  p.hdr = take(64);
  p.seg = take(4 * (static_cast<size_t>(c.L) + 2));
  p.tiles = take(16 * static_cast<size_t>(p.max_tiles));
  p.big = take(16 * static_cast<size_t>(p.max_big));
  p.order = take(4 * static_cast<size_t>(c.T));
  p.hist = take(4 * static_cast<size_t>(p.chunks) * (c.L + 2));
  p.total = o;
  return p;
}
static PlanView plan_view(const moe_adapter_config& c, const void* plan, const PlanLayout& p, void* ws) {
  const uint8_t* b = static_cast<const uint8_t*>(plan);
  return {reinterpret_cast<const int4*>(b + p.hdr), reinterpret_cast<const int32_t*>(b + p.seg),
          reinterpret_cast<const int4*>(b + p.tiles), reinterpret_cast<const int4*>(b + p.big),
          reinterpret_cast<const int32_t*>(b + p.order), c.T, c.L,
          static_cast<DevStatus*>(ws)};
}

// The key of a row: its adapter, or L for none. An index >= L counts as none and
// is reported through `bad`.
__device__ __forceinline__ int plan_key(int a, int L, bool& bad) {
  bad = a >= L;
  return a < 0 || bad ? L : a;
}

// counts of each key in a chunk of 1024 rows, and whether it has a bad index
__global__ void __launch_bounds__(kPlanThreads) plan_hist_kernel(const int32_t* __restrict__ idx, int T, int L,
                                                                 int32_t* __restrict__ hist) {
  __shared__ int s_h[kMaxAdapters + 1];
  for (int i = threadIdx.x; i <= L; i += kPlanThreads) s_h[i] = 0;
  __syncthreads();
  const int t = blockIdx.x * kPlanThreads + threadIdx.x;
  bool bad = false;
  chain_wait();
  chain_release();
  const int key = t < T ? plan_key(__ldcg(idx + t), L, bad) : -1;
  const unsigned peers = __match_any_sync(0xffffffffu, key);  // one addition for a warp's equal keys
  if (key >= 0 && (threadIdx.x & 31) == __ffs(peers) - 1) atomicAdd(&s_h[key], __popc(peers));
  bad = __syncthreads_or(bad);
  int32_t* row = hist + static_cast<size_t>(blockIdx.x) * (L + 2);
  for (int i = threadIdx.x; i <= L; i += kPlanThreads) row[i] = s_h[i];
  if (threadIdx.x == 0) row[L + 1] = bad;
}

// exclusive scan of two values per key over s_a and s_b ([L + 1], in place) by
// the whole block: each warp scans 32 keys, one warp the warps' sums
__device__ __forceinline__ void scan_keys(int* s_a, int* s_b, int n, int* s_w) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int carry_a = 0, carry_b = 0;
  for (int k0 = 0; k0 < n; k0 += kPlanThreads) {
    const int i = k0 + threadIdx.x;
    const int a = i < n ? s_a[i] : 0, b = i < n ? s_b[i] : 0;
    int xa = a, xb = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int ya = __shfl_up_sync(0xffffffffu, xa, o), yb = __shfl_up_sync(0xffffffffu, xb, o);
      if (lane >= o) {
        xa += ya;
        xb += yb;
      }
    }
    if (lane == 31) {
      s_w[warp] = xa;
      s_w[32 + warp] = xb;
    }
    __syncthreads();
    if (warp == 0) {
      int wa = s_w[lane], wb = s_w[32 + lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int ya = __shfl_up_sync(0xffffffffu, wa, o), yb = __shfl_up_sync(0xffffffffu, wb, o);
        if (lane >= o) {
          wa += ya;
          wb += yb;
        }
      }
      s_w[lane] = wa;
      s_w[32 + lane] = wb;
    }
    __syncthreads();
    const int pa = warp > 0 ? s_w[warp - 1] : 0, pb = warp > 0 ? s_w[32 + warp - 1] : 0;
    if (i < n) {
      s_a[i] = carry_a + pa + xa - a;
      s_b[i] = carry_b + pb + xb - b;
    }
    const int ta = s_w[31], tb = s_w[63];
    __syncthreads();
    carry_a += ta;
    carry_b += tb;
  }
}

// Positions of a chunk's rows (rows of an adapter stay in token order: a
// stable counting sort), and from the first chunk the segments, the tiles of both
// sizes and the status.
__global__ void __launch_bounds__(kPlanThreads)
    plan_place_kernel(const int32_t* __restrict__ idx, int T, int L, int chunks, const int32_t* __restrict__ hist,
                      int4* __restrict__ hdr, int32_t* __restrict__ seg, int4* __restrict__ tiles, int max_tiles,
                      int4* __restrict__ big, int max_big, int32_t* __restrict__ order, DevStatus* st) {
  __shared__ int s_first[kMaxAdapters + 1];   // first position of each key
  __shared__ int s_tile[kMaxAdapters + 1];    // first tile of each key: 64 rows in the low half, 128 in the high
  __shared__ int s_before[kMaxAdapters + 1];  // rows of each key in earlier chunks
  __shared__ __align__(4) uint8_t s_warp[32][kMaxAdapters + 1];
  __shared__ int s_w[64];
  const int keys = L + 1, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, me = blockIdx.x;
  for (int i = tid; i < 32 * (kMaxAdapters + 1) / 4; i += kPlanThreads) reinterpret_cast<int*>(&s_warp[0][0])[i] = 0;
  for (int i = tid; i < keys; i += kPlanThreads) s_first[i] = s_before[i] = 0;
  __syncthreads();
  const int t = me * kPlanThreads + tid;
  bool bad = false;
  if (hist == nullptr) chain_wait();  // the call's first kernel; else hist's launch is, which has waited
  const int key = t < T ? plan_key(__ldcg(idx + t), L, bad) : -1;
  const unsigned peers = __match_any_sync(0xffffffffu, key);
  const int rank = __popc(peers & ((1u << lane) - 1u));
  if (key >= 0 && rank == 0) s_warp[warp][key] = static_cast<uint8_t>(__popc(peers));
  if (hist == nullptr) {
    // few chunks: every block counts them all (s_first holds counts until the scan)
    int a[kPlanChunks];
#pragma unroll
    for (int c = 0; c < kPlanChunks; ++c) {
      const int tc = c * kPlanThreads + tid;
      a[c] = tc < T ? __ldcg(idx + tc) : INT_MIN;
    }
#pragma unroll
    for (int c = 0; c < kPlanChunks; ++c) {
      bool b = false;
      const int k = c * kPlanThreads + tid < T ? plan_key(a[c], L, b) : -1;
      bad |= b;
      const unsigned same = __match_any_sync(0xffffffffu, k);
      if (k >= 0 && lane == __ffs(same) - 1) {
        atomicAdd(&s_first[k], __popc(same));
        if (c < me) atomicAdd(&s_before[k], __popc(same));
      }
    }
  } else {
    chain_wait();
    for (int i = tid; i < keys; i += kPlanThreads) {
      int n = 0, before = 0;
#pragma unroll 8
      for (int c = 0; c < chunks; ++c) {
        const int h = __ldcg(hist + static_cast<size_t>(c) * (keys + 1) + i);
        before += c < me ? h : 0;
        n += h;
      }
      s_first[i] = n;
      s_before[i] = before;
    }
  }
  __syncthreads();
  for (int i = tid; i < keys; i += kPlanThreads)
    s_tile[i] = (s_first[i] + kTileRows - 1) / kTileRows | ((s_first[i] + 127) / 128) << 16;
  __syncthreads();
  scan_keys(s_first, s_tile, keys, s_w);
  __syncthreads();
  if (key >= 0) {
    int pos = s_first[key] + s_before[key] + rank;
#pragma unroll 8
    for (int w = 0; w < warp; ++w) pos += s_warp[w][key];
    order[pos] = t;
  }
  if (me == 0) {
    for (int i = tid; i < keys; i += kPlanThreads) {
      seg[i] = s_first[i];
      const int n = (i < L ? s_first[i + 1] : T) - s_first[i], a = i < L ? i : -1;
      const int nt = (n + kTileRows - 1) / kTileRows, t0 = s_tile[i] & 0xffff;
      const int nb = (n + 127) / 128, b0 = static_cast<int>(static_cast<uint32_t>(s_tile[i]) >> 16);
      for (int j = 0; j < nt; ++j)
        if (t0 + j < max_tiles)
          tiles[t0 + j] = make_int4(a, s_first[i] + j * kTileRows, min(kTileRows, n - j * kTileRows), 0);
      for (int j = 0; j < nb; ++j)
        if (b0 + j < max_big) big[b0 + j] = make_int4(a, s_first[i] + j * 128, min(128, n - j * 128), 0);
      if (i == L) {
        seg[L + 1] = T;
        hdr[0] = make_int4(min(t0 + nt, max_tiles), T, L, kPlanMagic);
        hdr[1] = make_int4(min(b0 + nb, max_big), 0, 0, 0);
      }
    }
    if (hist != nullptr)
      for (int c = tid; c < chunks; c += kPlanThreads) bad |= __ldcg(hist + static_cast<size_t>(c) * (keys + 1) + L + 1) != 0;
    bad = __syncthreads_or(bad);
    if (tid == 0) st->status = bad ? MOE_ERR_DEVICE_INDEX : MOE_OK;
  }
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------
constexpr int kAdThreads = 128;
constexpr int kBlockK = 64;

// Shared-memory rows are padded by 16 bytes: the eight rows of an 8x8 matrix
// then lie in different banks.
template <int RP, bool WT>
struct ShrinkSmem {
  static constexpr int kXRow = kBlockK + 8;
  static constexpr int kWRow = WT ? kBlockK + 8 : RP + 8;
  static constexpr int kX = kTileRows * kXRow * 2;
  static constexpr int kW = (WT ? RP : kBlockK) * kWRow * 2;
  static constexpr int kStage = kX + kW;
  // three blocks of an SM with as many stages as fit: at small ranks a block of 64
  // is gone in less than a load takes
  static constexpr int kStages = RP <= 32 ? 5 : (RP == 64 ? 4 : 3);
  static constexpr int kTotal = kStages * kStage;
};

// parts[split][position][j] = sum over the split's part of C of X[t][c] W_a[c][j].
// W_a is [C][r] (WT = false: A of the forward) or [r][C] (WT = true: B of the
// backward). fp32 accumulation, joined every 64 products in ordinary fp32 adds.
// Bound by latency: a block's few dozen loads and the launch itself (64 rows of 48
// adapters, K = 7168, rank 16: 10 MB in 9.0 us; 1 row: 6.1 us).
template <int RP, bool WT>
__global__ void __launch_bounds__(kAdThreads)
    adapter_shrink_kernel(const __nv_bfloat16* __restrict__ X, const __nv_bfloat16* __restrict__ W, PlanView plan,
                          int T, int C, int r, int splits, float* __restrict__ parts) {
  extern __shared__ __align__(16) uint8_t smem[];
  using S = ShrinkSmem<RP, WT>;
  chain_wait();
  chain_release();
  const int4 tile = __ldcg(plan.tiles + blockIdx.x);  // (in bounds for every block, of use to the first ones)
  if (static_cast<int>(blockIdx.x) >= plan_tiles(plan)) return;
  if (tile.x < 0) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nkb = (C + kBlockK - 1) / kBlockK, per = (nkb + splits - 1) / splits;
  const int kb0 = blockIdx.y * per, kb1 = min(nkb, kb0 + per);
  const __nv_bfloat16* Wa = W + static_cast<size_t>(tile.x) * C * r;
  const uint32_t base = smem_u32(smem);

  // this thread's 16-byte pieces of a stage's rows: piece tid % 8 of rows
  // tid / 8 + 16 i
  const __nv_bfloat16* xrow[4];
  bool xok[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = (tid >> 3) + 16 * i;
    xok[i] = row < tile.z;
    xrow[i] = X + (xok[i] ? static_cast<size_t>(plan.order[tile.y + row]) * C : 0);
  }
  auto load = [&](int kb, int slot) {
    const uint32_t sx = base + slot * S::kStage, sw = sx + S::kX;
    const int c0 = kb * kBlockK;
    const int c = c0 + (tid & 7) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool ok = xok[i] && c < C;
      cp_async16(sx + (((tid >> 3) + 16 * i) * S::kXRow + (tid & 7) * 8) * 2, ok ? xrow[i] + c : X, ok);
    }
    if constexpr (WT) {
      for (int i = tid; i < RP * 8; i += kAdThreads) {
        const int j = i >> 3, cc = c0 + (i & 7) * 8;
        const bool ok = j < r && cc < C;
        cp_async16(sw + (j * S::kWRow + (i & 7) * 8) * 2, ok ? Wa + static_cast<size_t>(j) * C + cc : W, ok);
      }
    } else {
      for (int i = tid; i < kBlockK * (RP / 8); i += kAdThreads) {
        const int cc = i / (RP / 8), j = (i % (RP / 8)) * 8;
        const bool ok = j < r && c0 + cc < C;
        cp_async16(sw + (cc * S::kWRow + j) * 2, ok ? Wa + static_cast<size_t>(c0 + cc) * r + j : W, ok);
      }
    }
  };

  float acc[RP / 8][4];
#pragma unroll
  for (int n = 0; n < RP / 8; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
#pragma unroll
  for (int s = 0; s < S::kStages - 1; ++s) {
    if (kb0 + s < kb1) load(kb0 + s, s);
    cp_async_commit();
  }
  int slot = 0;
  for (int kb = kb0; kb < kb1; ++kb) {
    cp_async_wait<S::kStages - 2>();
    __syncthreads();
    {
      const int nxt = kb + S::kStages - 1;
      if (nxt < kb1) load(nxt, (slot + S::kStages - 1) % S::kStages);
      cp_async_commit();
    }
    if (warp * 16 < tile.z) {
      const uint32_t sx = base + slot * S::kStage, sw = sx + S::kX;
      float part[RP / 8][4];
#pragma unroll
      for (int n = 0; n < RP / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[n][i] = 0.0f;
#pragma unroll
      for (int k = 0; k < kBlockK; k += 16) {
        uint32_t a[4];
        ldmatrix_x4(a, sx + ((warp * 16 + (lane & 15)) * S::kXRow + k + 8 * (lane >> 4)) * 2);
#pragma unroll
        for (int n = 0; n < RP; n += 16) {
          uint32_t b[4];
          if constexpr (WT)
            ldmatrix_x4(b, sw + ((n + (lane & 7) + 8 * (lane >> 4)) * S::kWRow + k + 8 * ((lane >> 3) & 1)) * 2);
          else
            ldmatrix_x4_trans(b, sw + ((k + (lane & 15)) * S::kWRow + n + 8 * (lane >> 4)) * 2);
          mma_bf16(part[n / 8], a, b[0], b[1]);
          mma_bf16(part[n / 8 + 1], a, b[2], b[3]);
        }
      }
#pragma unroll
      for (int n = 0; n < RP / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] += part[n][i];
    }
    slot = (slot + 1) % S::kStages;
  }
  cp_async_wait<0>();
  float* out = parts + (static_cast<size_t>(blockIdx.y) * T + tile.y) * RP;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = warp * 16 + (lane >> 2) + 8 * h;
    if (row < tile.z) {
#pragma unroll
      for (int n = 0; n < RP / 8; ++n)
        *reinterpret_cast<float2*>(out + static_cast<size_t>(row) * RP + 8 * n + 2 * (lane & 3)) =
            make_float2(acc[n][2 * h], acc[n][2 * h + 1]);
    }
  }
}

// Columns of a block's step: four warps as 2 x 2, each 32 rows x 64 columns.
constexpr int kTileCols = 128;
template <int RP, bool WT, bool F32>
struct ExpandSmem {
  // parts of u that the product takes: two (16 bits) leave an error of 2^-17 of
  // u, far below the rounding of a bf16 result; fp32 results take all three
  static constexpr int kParts = F32 ? 3 : 2;
  static constexpr bool kRegs = kParts * RP <= 128;  // u's fragments stay in registers
  static constexpr int kURow = RP + 8;
  static constexpr int kU = kTileRows * kURow * 2;  // one part
  static constexpr int kWRow = WT ? RP + 8 : kTileCols + 8;
  static constexpr int kW = (WT ? kTileCols : RP) * kWRow * 2;
  static constexpr int kYRow = 64 * (F32 ? 4 : 2) + 16;  // bytes of a row of a warp's 32 x 64 block
  static constexpr int kY = 32 * kYRow;
  static constexpr int kBufs = RP <= 32 && !F32 ? 3 : 2;  // tiles of W and of the base on hand
  static constexpr int kTotal = kParts * kU + kBufs * (kW + 4 * kY) + 4 * kTileRows;
};

// out[t][c] = base[t][c] + sum_j u[position][j] W_a[j][c], u = s_a sum over the
// splits of parts. W_a is [r][C] (WT = false: B of the forward) or [C][r]
// (WT = true: A of the backward). A block takes 64 rows of one adapter and runs
// over its share of the columns, u's bf16 parts in registers (shared memory at
// the largest ranks), the next step's tiles of W and of the base on their way
// while this step's are multiplied; each warp brings, completes and stores its
// own 32 x 64 piece of the output in whole 128-byte lines. The blocks of the
// first columns keep u's three parts for the weight gradients (u_keep:
// [3][T][RP]).
// W and base are asked for before the wait for the shrink, whose call's first kernel
// has waited for them. Base and out pass once, W_a comes from L2 once for every 64
// rows; what bounds the batches it serves is latency (64 rows of 48 adapters, N =
// 4096, rank 16: 7 MB in 8.9 us; 1 row: 6.0 us).
template <int RP, bool WT, bool F32>
__global__ void __launch_bounds__(kAdThreads, RP <= 64 && !F32 ? 3 : 2)
    adapter_expand_kernel(const float* __restrict__ parts, int splits, const float* __restrict__ scale,
                          const __nv_bfloat16* __restrict__ W, PlanView plan, int T, int C, int r, int steps,
                          const void* base_in, void* out, __nv_bfloat16* __restrict__ u_keep) {
  extern __shared__ __align__(16) uint8_t smem[];
  using S = ExpandSmem<RP, WT, F32>;
  constexpr int EB = F32 ? 4 : 2, PER = 16 / EB, PIECES = 64 / PER, PARTS = S::kParts;
  chain_release();
  const int4 tile = __ldcg(plan.tiles + blockIdx.x);  // (in bounds for every block, of use to the first ones)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int first = blockIdx.y * steps * kTileCols, last = min(C, first + steps * kTileCols);
  if (static_cast<int>(blockIdx.x) >= plan_tiles(plan) || first >= last) return chain_leave();
  int* s_tok = reinterpret_cast<int*>(smem + PARTS * S::kU + S::kBufs * (S::kW + 4 * S::kY));
  if (tid < tile.z) s_tok[tid] = plan.order[tile.y + tid];
  __syncthreads();
  if (tile.x < 0) {
    // rows without an adapter: the base as it is
    if (base_in == out) return chain_leave();
    chain_wait();
    const int vecs = (last - first) / PER;
    for (int row = warp; row < tile.z; row += kAdThreads / 32) {
      const size_t at = (static_cast<size_t>(s_tok[row]) * C + first) * EB;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base_in) + at);
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(out) + at);
      for (int i = lane; i < vecs; i += 32) dst[i] = base_in != nullptr ? src[i] : make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const __nv_bfloat16* Wa = W + static_cast<size_t>(tile.x) * C * r;
  const uint32_t sb = smem_u32(smem);
  const int wm = (warp & 1) * 32, wn = (warp >> 1) * 64;
  const bool mine = wm < tile.z;  // this warp has rows
  uint8_t* sy0 = smem + PARTS * S::kU + S::kBufs * S::kW + warp * S::kY;
  auto load = [&](int c0, int slot) {
    const uint32_t sw = sb + PARTS * S::kU + slot * S::kW;
    if constexpr (WT) {
#pragma unroll
      for (int k = 0; k < kTileCols * (RP / 8) / kAdThreads; ++k) {
        const int i = tid + k * kAdThreads, c = i / (RP / 8), j = (i % (RP / 8)) * 8;
        const bool ok = j < r && c0 + c < last;
        cp_async16(sw + (c * S::kWRow + j) * 2, ok ? Wa + static_cast<size_t>(c0 + c) * r + j : W, ok);
      }
    } else {
#pragma unroll
      for (int k = 0; k < RP * (kTileCols / 8) / kAdThreads; ++k) {
        const int i = tid + k * kAdThreads, j = i / (kTileCols / 8), c = (i % (kTileCols / 8)) * 8;
        const bool ok = j < r && c0 + c < last;
        cp_async16(sw + (j * S::kWRow + c) * 2, ok ? Wa + static_cast<size_t>(j) * C + c0 + c : W, ok);
      }
    }
    if (mine && base_in != nullptr) {
      const uint32_t sy = smem_u32(sy0 + slot * 4 * S::kY);
#pragma unroll
      for (int k = 0; k < PIECES; ++k) {
        const int i = lane + 32 * k, row = i / PIECES, c = (i % PIECES) * PER;
        const bool ok = wm + row < tile.z && c0 + wn + c < last;
        if (ok)
          cp_async16(sy + row * S::kYRow + c * EB,
                     static_cast<const uint8_t*>(base_in) + (static_cast<size_t>(s_tok[wm + row]) * C + c0 + wn + c) * EB,
                     true);
      }
    }
  };
#pragma unroll
  for (int b = 0; b < S::kBufs - 1; ++b) {
    if (first + b * kTileCols < last) load(first + b * kTileCols, b);
    cp_async_commit();
  }
  // u of the tile's rows
  const float sc = scale[tile.x];
  chain_wait();
  for (int i = tid; i < kTileRows * (RP / 4); i += kAdThreads) {
    const int row = i / (RP / 4), j = (i % (RP / 4)) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < tile.z) {
      const float* p = parts + static_cast<size_t>(tile.y + row) * RP + j;
      // six splits in flight: one load after the other took half of a small call
      for (int s0 = 0; s0 < splits; s0 += 6) {
        float4 w[6];
#pragma unroll
        for (int q = 0; q < 6; ++q)
          w[q] = s0 + q < splits ? __ldcg(reinterpret_cast<const float4*>(p + static_cast<size_t>(s0 + q) * T * RP))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int q = 0; q < 6; ++q) {
          v.x += w[q].x; v.y += w[q].y; v.z += w[q].z; v.w += w[q].w;
        }
      }
    }
    const float f[4] = {v.x * sc, v.y * sc, v.z * sc, v.w * sc};
    __nv_bfloat16 part[3][4];
#pragma unroll
    for (int q = 0; q < 4; ++q) split_bf16(f[q], part[0][q], part[1][q], part[2][q]);
#pragma unroll
    for (int h = 0; h < 3; ++h) {
      const uint2 v2 = *reinterpret_cast<const uint2*>(part[h]);
      if (h < PARTS) *reinterpret_cast<uint2*>(smem + h * S::kU + (row * S::kURow + j) * 2) = v2;
      if (u_keep != nullptr && blockIdx.y == 0 && row < tile.z)
        *reinterpret_cast<uint2*>(u_keep + (static_cast<size_t>(h) * T + tile.y + row) * RP + j) = v2;
    }
  }
  __syncthreads();
  auto u_frag = [&](uint32_t (&a)[4], int h, int m, int k) {
    ldmatrix_x4(a, sb + h * S::kU + ((wm + 16 * m + (lane & 15)) * S::kURow + k + 8 * (lane >> 4)) * 2);
  };
  uint32_t ua[S::kRegs ? PARTS : 1][2][S::kRegs ? RP / 16 : 1][4];
  if constexpr (S::kRegs) {
#pragma unroll
    for (int h = 0; h < PARTS; ++h)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int k = 0; k < RP / 16; ++k) u_frag(ua[h][m][k], h, m, 16 * k);
  }
  int slot = 0;
  for (int c0 = first; c0 < last; c0 += kTileCols, slot = slot + 1 == S::kBufs ? 0 : slot + 1) {
    cp_async_wait<S::kBufs - 2>();
    __syncthreads();  // this step's tiles are here, the last step's have been read
    const int ahead = c0 + (S::kBufs - 1) * kTileCols;
    if (ahead < last) load(ahead, slot == 0 ? S::kBufs - 1 : slot - 1);
    cp_async_commit();
    if (!mine) continue;
    const uint32_t sw = sb + PARTS * S::kU + slot * S::kW;
    float acc[2][8][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
#pragma unroll
    for (int k = 0; k < RP / 16; ++k) {
      uint32_t a[S::kRegs ? 1 : PARTS][2][4];
      if constexpr (!S::kRegs) {
#pragma unroll
        for (int h = 0; h < PARTS; ++h)
#pragma unroll
          for (int m = 0; m < 2; ++m) u_frag(a[h][m], h, m, 16 * k);
      }
#pragma unroll
      for (int n = 0; n < 8; n += 2) {
        uint32_t b[4];
        if constexpr (WT)
          ldmatrix_x4(b, sw + ((wn + 8 * n + (lane & 7) + 8 * (lane >> 4)) * S::kWRow + 16 * k + 8 * ((lane >> 3) & 1)) * 2);
        else
          ldmatrix_x4_trans(b, sw + ((16 * k + (lane & 15)) * S::kWRow + wn + 8 * n + 8 * (lane >> 4)) * 2);
#pragma unroll
        for (int h = PARTS - 1; h >= 0; --h)  // the small parts first
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const uint32_t(&f)[4] = S::kRegs ? ua[S::kRegs ? h : 0][m][S::kRegs ? k : 0] : a[S::kRegs ? 0 : h][m];
            mma_bf16(acc[m][n], f, b[0], b[1]);
            mma_bf16(acc[m][n + 1], f, b[2], b[3]);
          }
      }
    }
    // add the base in shared memory (each element by the thread that holds its sum)
    uint8_t* sy = sy0 + slot * 4 * S::kY;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 16 * m + (lane >> 2) + 8 * h;
        if (wm + row < tile.z) {
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            uint8_t* q = sy + row * S::kYRow + (8 * n + 2 * (lane & 3)) * EB;
            const float x = acc[m][n][2 * h], y = acc[m][n][2 * h + 1];
            if constexpr (F32) {
              float2 v = base_in != nullptr ? *reinterpret_cast<float2*>(q) : make_float2(0.f, 0.f);
              *reinterpret_cast<float2*>(q) = make_float2(v.x + x, v.y + y);
            } else {
              const uint32_t v = base_in != nullptr ? *reinterpret_cast<uint32_t*>(q) : 0u;
              *reinterpret_cast<uint32_t*>(q) = pack_bf16x2(bf16_lo(v) + x, bf16_hi(v) + y);
            }
          }
        }
      }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < PIECES; ++k) {
      const int i = lane + 32 * k, row = i / PIECES, c = (i % PIECES) * PER;
      if (wm + row < tile.z && c0 + wn + c < last)
        __stcs(reinterpret_cast<uint4*>(static_cast<uint8_t*>(out) +
                                        (static_cast<size_t>(s_tok[wm + row]) * C + c0 + wn + c) * EB),
               *reinterpret_cast<const uint4*>(sy + row * S::kYRow + c * EB));
    }
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
static int check_adapter(const moe_adapter_config* c) {
  if (c == nullptr) return MOE_ERR_INVALID_ARG;
  if (c->T < 1 || c->K < 1 || c->N < 1 || c->L < 1 || c->r < 1) return MOE_ERR_INVALID_ARG;
  if (c->out_fp32 != 0 && c->out_fp32 != 1) return MOE_ERR_INVALID_ARG;
  if (c->K % 8 != 0 || c->N % 8 != 0 || c->r % 8 != 0) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->r > 128 || c->L > kMaxAdapters || c->T > (1 << 21) || c->K > (1 << 20) || c->N > (1 << 20))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}
static int padded_rank(int r) { return r <= 16 ? 16 : (r <= 32 ? 32 : (r <= 64 ? 64 : 128)); }

// Splits of the long axis of a shrink: three blocks for each SM, and no more than
// the expanding product, whose every block adds them up, reads without loss (rank
// 64, one adapter, 1024 rows: 32 splits 36.9 us, 12 20.0)
static int shrink_splits(const moe_adapter_config& c, int C) {
  const int tiles = c.T / kTileRows + std::min(c.T, c.L);
  const int nkb = (C + kBlockK - 1) / kBlockK;
  return std::max(1, std::min({3 * kAdSMs / tiles, nkb, 12}));
}

// Batches from 2048 rows on take the tensor memory kernels, smaller ones tiles of
// 64 rows on mma.sync. Forward, K = N = 4096, the two forms in us: 64 rows of 48
// adapters, rank 16: tcgen05 17, mma.sync 9; 1024 rows of 8, rank 16: 17, 12; 2048
// rows of 64, rank 64: 37, 43; 4096 rows of one, rank 64: 32, 46.
constexpr int kTcRows = 2048;
static int big_tiles(const moe_adapter_config& c) { return c.T / 128 + std::min(c.T, c.L); }
// two blocks for each SM, at most four splits, or eight up to rank 32 (as above: each
// is read again by every block of the expanding product. Forward with four, eight
// splits in us: 4133 rows, 7168 to 2048, rank 32 47.2, 45.4; 2048 rows, 4096 to 4096,
// rank 16 16.9, 14.9, rank 64 24.8, 26.0; 4096 rows, rank 64 32.4, 36.9)
static int shrink_splits_tc(const moe_adapter_config& c, int C) {
  const int nkb = (C + 63) / 64;
  return std::max(1, std::min({2 * kAdSMs / big_tiles(c), nkb, padded_rank(c.r) <= 32 ? 8 : 4}));
}
// A block for each adapter and column tile instead of runs of rows: small batches
// of many adapters have a run or two, whose one block goes through all their
// adapters; a block of few adapters goes through all of an adapter's rows (backward
// of 4096 to 4096 in us by adapter, by runs: rank 64, 90 rows of 12 adapters 35, 91; 400
// rows of one 33, 31; 1000 of one 47, 38, of two 37, 41; 1500 of two 50, 50, of three 44,
// 50; 2000 of three 56, 56, of four 52, 57; rank 16, 400 of one 18, 18; 1000 of one 30,
// 22, of two 21, 22; 1500 of two 29, 26, of three 25, 27; 2000 of three 31, 30, of six 26, 30).
static bool wgrad_by_adapter(const moe_adapter_config& c) { return c.T < 2048 && c.T <= 512 * c.L; }
// Runs of rows of the weight gradients: together with the column tiles about one
// block for each SM
static RowRuns wgrad_runs(const moe_adapter_config& c, int C, int* col_tiles, size_t* partial_floats) {
  const int rp = padded_rank(c.r), cols = rp <= 64 ? 256 : 128;
  *col_tiles = (C + cols - 1) / cols;
  if (wgrad_by_adapter(c)) {
    *partial_floats = 0;
    return {0, c.L};
  }
  const int want = std::max(1, kAdSMs / *col_tiles);
  RowRuns run;
  run.rows = ((c.T + want - 1) / want + 63) / 64 * 64;
  run.runs = (c.T + run.rows - 1) / run.rows;
  // (a single run holds every adapter whole: nothing is left to add up)
  *partial_floats = run.runs == 1 ? 0 : 2 * static_cast<size_t>(run.runs) * *col_tiles * cols * rp;
  return run;
}

struct AdapterWs {
  size_t parts, du, partial_a, partial_b, total;
};
static AdapterWs adapter_ws(const moe_adapter_config& c, bool training) {
  AdapterWs w{};
  size_t o = 256;
  auto take = [&](size_t b) {
    const size_t at = o;
    o += (b + 255) & ~size_t(255);
    return at;
  };
  const size_t rp = padded_rank(c.r), T = c.T;
  auto splits = [&](int C) { return c.T >= kTcRows ? shrink_splits_tc(c, C) : shrink_splits(c, C); };
  int s = splits(c.K);
  if (training) s = std::max(s, splits(c.N));
  w.parts = take(4 * T * rp * s);
  if (training) {
    w.du = take(6 * T * rp);
    int tiles;
    size_t a, b;
    wgrad_runs(c, c.K, &tiles, &a);
    wgrad_runs(c, c.N, &tiles, &b);
    w.partial_a = take(4 * a);
    w.partial_b = take(4 * b);
  }
  w.total = o;
  return w;
}

// the shared memory of a kernel, allowed once for each device
template <auto Kernel>
static cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || bytes <= 48 * 1024) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
  const cudaError_t a = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (a == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_release);
  return a;
}

// parts of X W: the number of splits it left in *splits
template <int RP, bool WT>
static cudaError_t launch_shrink(const moe_adapter_config& c, int C, const void* X, const void* W, const PlanView& pv,
                                 const PlanLayout& P, float* parts, int* splits, cudaStream_t s) {
  const auto* x = static_cast<const __nv_bfloat16*>(X);
  const auto* w = static_cast<const __nv_bfloat16*>(W);
  if (c.T >= kTcRows) {
    constexpr int sm = TcShrink<RP, WT>::kTotal;
    const cudaError_t e = allow_smem<adapter_shrink_tc<RP, WT>>(sm);
    if (e != cudaSuccess) return e;
    *splits = shrink_splits_tc(c, C);
    return launch_chained(adapter_shrink_tc<RP, WT>, dim3(P.max_big, *splits),
                          TcShrink<RP, WT>::R::kThreads, sm, s, x, w, pv, c.T, C, c.r,
                          *splits, parts, static_cast<uint64_t>(wait_limit_ns()));
  }
  constexpr int sm = ShrinkSmem<RP, WT>::kTotal;
  const cudaError_t e = allow_smem<adapter_shrink_kernel<RP, WT>>(sm);
  if (e != cudaSuccess) return e;
  *splits = shrink_splits(c, C);
  return launch_chained(adapter_shrink_kernel<RP, WT>, dim3(P.max_tiles, *splits), kAdThreads, sm, s, x, w, pv, c.T, C,
                        c.r, *splits, parts);
}

template <int RP, bool WT, bool F32>
static cudaError_t launch_expand(const moe_adapter_config& c, int C, const float* parts, int splits,
                                 const float* scale, const void* W, const PlanView& pv, const PlanLayout& P,
                                 const void* base, void* out, void* keep, cudaStream_t s) {
  const auto* w = static_cast<const __nv_bfloat16*>(W);
  auto* k = static_cast<__nv_bfloat16*>(keep);
  if (c.T >= kTcRows) {
    using S = TcExpand<RP, WT, F32>;
    const cudaError_t e = allow_smem<adapter_expand_tc<RP, WT, F32>>(S::kTotal);
    if (e != cudaSuccess) return e;
    // one wave of blocks where there are no more tiles than that, an adapter's last
    // one counted as three quarters of a tile (rounding to the nearest wave instead:
    // 6900 rows of one adapter, 2048 to 4096, rank 64, forward 53 us for 42; 9500 of 8
    // 70 for 55; an adapter's last tile as a half: 5003 rows of 40, both ways 122 for 108)
    const int cols = (C + S::NC - 1) / S::NC;
    const int ranges = std::max(1, std::min({cols, 16, S::kBlocks * kAdSMs / (c.T / 128 + (3 * std::min(c.T, c.L) + 3) / 4)}));
    const int steps = (cols + ranges - 1) / ranges;
    return launch_chained(adapter_expand_tc<RP, WT, F32>, dim3(P.max_big, (cols + steps - 1) / steps), S::R::kThreads,
                          S::kTotal, s, parts, splits, scale, w, pv, c.T, C, c.r, steps, base, out, k,
                          static_cast<uint64_t>(wait_limit_ns()));
  }
  constexpr int sm = ExpandSmem<RP, WT, F32>::kTotal;
  const cudaError_t e = allow_smem<adapter_expand_kernel<RP, WT, F32>>(sm);
  if (e != cudaSuccess) return e;
  // about three blocks for each SM, as many as run at a time
  const int cols = (C + kTileCols - 1) / kTileCols;
  const int tiles = c.T / kTileRows + std::min(c.T, c.L);
  const int ranges = std::max(1, std::min(cols, (3 * kAdSMs + tiles - 1) / tiles));
  const int steps = (cols + ranges - 1) / ranges;
  return launch_chained(adapter_expand_kernel<RP, WT, F32>, dim3(P.max_tiles, (cols + steps - 1) / steps), kAdThreads,
                        sm, s, parts, splits, scale, w, pv, c.T, C, c.r, steps, base, out, k);
}

template <int RP, bool OUT_T>
static cudaError_t launch_wgrad(const moe_adapter_config& c, const WgradSide& side, const void* X, const void* V,
                                const PlanView& pv, bool v_ready, cudaStream_t s) {
  constexpr int sm = TcWgrad<RP>::kTotal;
  const cudaError_t e = allow_smem<adapter_wgrad_tc<RP, OUT_T>>(sm);
  if (e != cudaSuccess) return e;
  return launch_chained(adapter_wgrad_tc<RP, OUT_T>, dim3(side.col_tiles, side.run.runs), TcWgrad<RP>::R::kThreads, sm, s,
                        static_cast<const __nv_bfloat16*>(X), static_cast<const __nv_bfloat16*>(V), pv, c.T, c.r, side,
                        v_ready, static_cast<uint64_t>(wait_limit_ns()));
}
template <int RP>
static cudaError_t launch_wgrad_join(const moe_adapter_config& c, const WgradSide& dA, const WgradSide& dB,
                                     const PlanView& pv, cudaStream_t s) {
  const int values = std::max(dA.C, dB.C) * c.r, runs = std::max(dA.run.runs, dB.run.runs);
  const int zero_rows = std::min(c.L, 16);
  return launch_chained(adapter_wgrad_join<RP>, dim3((values + kJoinValues - 1) / kJoinValues, runs + zero_rows, 2), 256,
                        0, s, pv, c.r, zero_rows, dA, dB);
}

static bool any_misaligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0) return true;
  return false;
}

#define MOE_RANK(r, ...)                              \
  do {                                                \
    switch (padded_rank(r)) {                         \
      case 16: { constexpr int RP = 16; __VA_ARGS__; break; }   \
      case 32: { constexpr int RP = 32; __VA_ARGS__; break; }   \
      case 64: { constexpr int RP = 64; __VA_ARGS__; break; }   \
      default: { constexpr int RP = 128; __VA_ARGS__; break; }  \
    }                                                 \
  } while (0)

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_adapter_plan_bytes(const moe_adapter_config* cfg) {
  return check_adapter(cfg) != MOE_OK ? 0 : plan_layout(*cfg).total;
}
size_t moe_adapter_workspace_bytes(const moe_adapter_config* cfg, int training) {
  return check_adapter(cfg) != MOE_OK ? 0 : adapter_ws(*cfg, training != 0).total;
}
size_t moe_adapter_saved_bytes(const moe_adapter_config* cfg) {
  return check_adapter(cfg) != MOE_OK ? 0 : 6 * static_cast<size_t>(cfg->T) * padded_rank(cfg->r);
}

int moe_adapter_plan(const moe_adapter_config* cfg, const int32_t* adapter_idx, void* plan, size_t plan_bytes,
                     void* stream) {
  NvtxRange nvtx("moe_adapter_plan");
  const int st = check_adapter(cfg);
  if (st != MOE_OK) return st;
  const moe_adapter_config& c = *cfg;
  if (!adapter_idx || !plan || any_misaligned({adapter_idx, plan})) return MOE_ERR_INVALID_ARG;
  const PlanLayout L = plan_layout(c);
  if (plan_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* b = static_cast<uint8_t*>(plan);
  DevStatus* ds = reinterpret_cast<DevStatus*>(b);
  int32_t* hist = reinterpret_cast<int32_t*>(b + L.hist);
  const bool counted_first = L.chunks > kPlanChunks;
  if (counted_first) {
    const cudaError_t e = launch_chained(plan_hist_kernel, L.chunks, kPlanThreads, 0, s, adapter_idx, c.T, c.L, hist);
    if (e != cudaSuccess) return status_from_cuda(e);
  }
  int4* hdr = reinterpret_cast<int4*>(b + L.hdr);
  int32_t* seg = reinterpret_cast<int32_t*>(b + L.seg);
  int4* tiles = reinterpret_cast<int4*>(b + L.tiles);
  int4* big = reinterpret_cast<int4*>(b + L.big);
  int32_t* order = reinterpret_cast<int32_t*>(b + L.order);
  const int32_t* counted = counted_first ? hist : nullptr;
  const cudaError_t e = launch_chained(plan_place_kernel, L.chunks, kPlanThreads, 0, s, adapter_idx, c.T, c.L, L.chunks,
                                       counted, hdr, seg, tiles, L.max_tiles, big, L.max_big, order, ds);
  const int rc = status_from_cuda(e);
  record_stage(s, 45, counted_first ? 2 : 1);
  return rc;
}

int moe_adapter_fwd(const moe_adapter_config* cfg, const moe_bf16* x, const moe_bf16* A, const moe_bf16* B,
                    const float* scale, const void* plan, const void* base, void* y, void* u_saved, void* ws,
                    size_t ws_bytes, void* stream) {
  NvtxRange nvtx("moe_adapter_fwd");
  const int st = check_adapter(cfg);
  if (st != MOE_OK) return st;
  const moe_adapter_config& c = *cfg;
  if (!x || !A || !B || !scale || !plan || !y || !ws || any_misaligned({x, A, B, scale, plan, base, y, u_saved, ws}))
    return MOE_ERR_INVALID_ARG;
  const size_t yb = static_cast<size_t>(c.T) * c.N * (c.out_fp32 ? 4 : 2);
  if (base != y && overlap(base, yb, y, yb)) return MOE_ERR_INVALID_ARG;
  const AdapterWs L = adapter_ws(c, false);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const PlanLayout P = plan_layout(c);
  const PlanView pv = plan_view(c, plan, P, ws);
  float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + L.parts);
  int splits = 1;
  cudaError_t e = cudaSuccess;
  MOE_RANK(c.r, e = launch_shrink<RP, false>(c, c.K, x, A, pv, P, parts, &splits, s));
  if (e != cudaSuccess) return status_from_cuda(e);
  record_stage(s, 46, 1);
  if (c.out_fp32)
    MOE_RANK(c.r, e = launch_expand<RP, false, true>(c, c.N, parts, splits, scale, B, pv, P, base, y, u_saved, s));
  else
    MOE_RANK(c.r, e = launch_expand<RP, false, false>(c, c.N, parts, splits, scale, B, pv, P, base, y, u_saved, s));
  record_stage(s, 47, 1);
  return status_from_cuda(e);
}

int moe_adapter_bwd(const moe_adapter_config* cfg, const moe_bf16* dy, const moe_bf16* x, const moe_bf16* A,
                    const moe_bf16* B, const float* scale, const void* plan, const void* u_saved, const void* dx_base,
                    void* dx, float* dA, float* dB, void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nvtx("moe_adapter_bwd");
  const int st = check_adapter(cfg);
  if (st != MOE_OK) return st;
  const moe_adapter_config& c = *cfg;
  if (!dy || !x || !A || !B || !scale || !plan || !u_saved || !dx || !dA || !dB || !ws ||
      any_misaligned({dy, x, A, B, scale, plan, u_saved, dx_base, dx, dA, dB, ws}))
    return MOE_ERR_INVALID_ARG;
  // dx is written before x is read for dA
  const size_t xb = static_cast<size_t>(c.T) * c.K * (c.out_fp32 ? 4 : 2);
  if ((dx_base != dx && overlap(dx_base, xb, dx, xb)) || overlap(x, 2 * static_cast<size_t>(c.T) * c.K, dx, xb) ||
      overlap(dy, 2 * static_cast<size_t>(c.T) * c.N, dx, xb))
    return MOE_ERR_INVALID_ARG;
  const AdapterWs L = adapter_ws(c, true);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const PlanLayout P = plan_layout(c);
  const PlanView pv = plan_view(c, plan, P, ws);
  float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + L.parts);
  void* du = static_cast<uint8_t*>(ws) + L.du;
  size_t floats;
  WgradSide side_a{dA, reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + L.partial_a), c.K, 0, {}};
  WgradSide side_b{dB, reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + L.partial_b), c.N, 0, {}};
  side_a.run = wgrad_runs(c, c.K, &side_a.col_tiles, &floats);
  side_b.run = wgrad_runs(c, c.N, &side_b.col_tiles, &floats);
  int splits = 1;
  cudaError_t e = cudaSuccess;
  MOE_RANK(c.r, e = launch_shrink<RP, true>(c, c.N, dy, B, pv, P, parts, &splits, s));
  if (e != cudaSuccess) return status_from_cuda(e);
  record_stage(s, 46, 1);
  // dB reads dy again while much of it is still in L2
  MOE_RANK(c.r, e = launch_wgrad<RP, true>(c, side_b, dy, u_saved, pv, true, s));
  if (e != cudaSuccess) return status_from_cuda(e);
  record_stage(s, 48, 1);
  if (c.out_fp32)
    MOE_RANK(c.r, e = launch_expand<RP, true, true>(c, c.K, parts, splits, scale, A, pv, P, dx_base, dx, du, s));
  else
    MOE_RANK(c.r, e = launch_expand<RP, true, false>(c, c.K, parts, splits, scale, A, pv, P, dx_base, dx, du, s));
  if (e != cudaSuccess) return status_from_cuda(e);
  record_stage(s, 47, 1);
  MOE_RANK(c.r, e = launch_wgrad<RP, false>(c, side_a, x, du, pv, false, s));
  if (e != cudaSuccess) return status_from_cuda(e);
  record_stage(s, 48, 1);
  if (side_a.run.rows == 0) return status_from_cuda(e);
  MOE_RANK(c.r, e = launch_wgrad_join<RP>(c, side_a, side_b, pv, s));
  record_stage(s, 48, 1);
  return status_from_cuda(e);
}

}  // extern "C"
