// The adapters' products on the tensor memory path (tcgen05, one CTA, M = 128):
//   shrink  parts[position][j]  = X[t] W_a          128 rows of one adapter
//   expand  out[t]              = base[t] + u W_a   128 rows of one adapter
//   wgrad   G_a                 = X_a^T V_a         columns of X, rows in equal runs
// The rows of X, base and out are gathered through the plan's order, so the
// tiles come by 16-byte cp.async copies written in the 128-byte swizzle that the
// MMA's descriptors expect, not by TMA boxes.
//
// Warps: first the epilogue's (TMEM lane quarter = warp % 4), then the TMEM owner
// and MMA issuer, then the producers. A stage of operands is full when the copies
// of all producer threads have landed, empty again when the MMAs that read it
// have completed.
//
// fp32 accumulation in tensor memory cuts each addition at the accumulator's last
// bit: measured against fp64 the sum of K products is too small by 1e-9 K of
// itself (K = 512: 5.1e-7, 4096: 4.1e-6). So a sum runs over at most kFlush = 8
// blocks of 64 in tensor memory; the epilogue adds those in registers in ordinary
// fp32 while the MMAs go on with the other accumulator.
#pragma once
#include "host_util.h"
#include "mma.cuh"

namespace moe {

constexpr int kFlush = 8;
// threads of a kernel's roles
template <int EPI_WARPS, int PRODUCER_WARPS>
struct TcRoles {
  static constexpr int kOwner = EPI_WARPS;  // the MMA issuer's warp
  static constexpr int kEpi = EPI_WARPS * 32;
  static constexpr int kProducers = PRODUCER_WARPS * 32;
  static constexpr int kFirstProducer = kEpi + 32;
  static constexpr int kThreads = kFirstProducer + kProducers;
};

struct PlanView {
  const int4* hdr;       // {number of 64-row tiles, T, L, kPlanMagic}, {number of 128-row tiles, 0, 0, 0}
  const int32_t* seg;    // [L + 2]: first position of each adapter, then of the rows without one, then T
  const int4* tiles;     // 64-row tiles {adapter or -1, first position, rows, 0}
  const int4* big;       // the same in 128 rows
  const int32_t* order;  // [T]: token of each position
  int T, L;
  DevStatus* st;
};
constexpr int kPlanMagic = 0x706c616f;
// the number of tiles (of 64 rows, or 128 with `big`); 0, and a device error, for
// a plan of another batch size or number of adapters or a buffer that holds none
__device__ __forceinline__ int plan_tiles(const PlanView& p, bool big = false) {
  const int4 h = __ldcg(p.hdr), h2 = __ldcg(p.hdr + 1);
  if (h.y == p.T && h.z == p.L && h.w == kPlanMagic) return big ? h2.x : h.x;
  set_status(p.st, MOE_ERR_DEVICE_INDEX, 61);
  return 0;
}

// byte offset of 16-byte piece c of row r in a tile of 128-byte rows, swizzled
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
}

// Barriers and roles' common state at the end of dynamic shared memory
template <int NST>
struct TcBars {
  uint64_t full[NST], empty[NST], tfull[2], tempty[2], ready, drain;
  uint32_t tmem;
  int abort;
};
// The block's tensor memory is allocated before the kernel behind may start: that
// kernel's blocks allocate too and may then wait for this one's end, so a block that
// still had to allocate beside them could wait for ever (tcgen05.alloc has no limit).
// As it is, whoever waits with tensor memory in hand waits for blocks that have theirs.
template <class R, int NST>
__device__ __forceinline__ void tc_init(TcBars<NST>* b, int empty_count, uint32_t tmem_cols) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(b->full + s, R::kProducers);
      mbar_init(b->empty + s, empty_count);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(b->tfull + i, 1);
      mbar_init(b->tempty + i, 128);
    }
    mbar_init(&b->ready, R::kThreads);
    mbar_init(&b->drain, 1);
    b->abort = 0;
    fence_barrier_init();
  }
  if (warp_id() == R::kOwner) {
    tmem_alloc(&b->tmem, tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  chain_release();
}
// Every thread ends here. After a wait that ran out the MMAs in flight are given
// their (bounded) time before the tensor memory is freed.
template <class R, int NST>
__device__ __forceinline__ void tc_end(TcBars<NST>* b, uint32_t tmem_cols, uint64_t lim) {
  tc_fence_before();
  __syncthreads();
  if (warp_id() == R::kOwner) {
    tc_fence_after();
    if (*static_cast<volatile int*>(&b->abort)) {
      int zero = 0;
      if (elect_lane0()) umma_commit(&b->drain);
      __syncwarp();
      mbar_wait_bounded(&b->drain, 0, &zero, lim, nullptr, 0);
    }
    tmem_dealloc(b->tmem, tmem_cols);
  }
}

// A producer thread's side of the ring: it waits for a slot, issues its copies and
// goes on; the copies' landing arrives on the stage's barrier by itself.
template <int NST>
struct TcRing {
  TcBars<NST>* b;
  int i = 0;  // stages issued
  __device__ __forceinline__ explicit TcRing(TcBars<NST>* bars) : b(bars) {}
  __device__ __forceinline__ int slot() const { return i % NST; }
  __device__ __forceinline__ bool begin(uint64_t lim, DevStatus* st) {
    return mbar_wait_bounded(b->empty + slot(), ((i / NST) & 1) ^ 1, &b->abort, lim, st, 62);
  }
  __device__ __forceinline__ void commit() {
    cp_async_arrive(b->full + slot());
    ++i;
  }
  // no thread leaves with copies in flight
  __device__ __forceinline__ void end() { cp_async_wait_all(); }
};
// The MMA issuer's wait for a stage. The copies are generic-proxy writes; the
// fence, between the barrier and the MMAs of this thread, orders them before the
// tensor cores' reads.
template <int NST>
__device__ __forceinline__ bool tc_stage_ready(TcBars<NST>* b, int i, uint64_t lim, DevStatus* st, int where) {
  if (!mbar_wait_bounded(b->full + i % NST, (i / NST) & 1, &b->abort, lim, st, where)) return false;
  fence_proxy_async_smem();
  tc_fence_after();
  return true;
}

// ---------------------------------------------------------------------------
// shrink
// ---------------------------------------------------------------------------
template <int RP, bool WT>
struct TcShrink {
  using R = TcRoles<4, 4>;
  static constexpr int kX = 128 * 128;
  static constexpr int kW = WT ? RP * 128 : (RP + 63) / 64 * 8192;
  static constexpr int kStage = kX + kW;
  static constexpr int NST = 4;
  static constexpr int kAcc = RP < 32 ? 32 : RP;  // TMEM columns of an accumulator
  static constexpr uint32_t kTmem = 2 * kAcc;
  static constexpr int kTotal = NST * kStage + sizeof(TcBars<NST>) + 1024;
};

// parts[split][position][j] = sum over the split's part of C of X[t][c] W_a[c][j];
// W_a is [C][r] (WT = false) or [r][C] (WT = true). Bound by the rows of X, read
// once; W_a comes from L2 for every 128 rows (16384 x 4096, rank 64: 138 MB in 33
// us, 4.2 TB/s, the tensor pipe at 13%; a plain gathered read of the same tiles
// takes 30.5 to 35).
template <int RP, bool WT>
__global__ void __launch_bounds__(TcRoles<4, 4>::kThreads, RP <= 64 ? 2 : 1)
    adapter_shrink_tc(const __nv_bfloat16* __restrict__ X, const __nv_bfloat16* __restrict__ W, PlanView plan, int T,
                      int C, int r, int splits, float* __restrict__ parts, uint64_t lim) {
  using S = TcShrink<RP, WT>;
  using R = typename S::R;
  constexpr int NST = S::NST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  auto* bars = reinterpret_cast<TcBars<NST>*>(smem + NST * S::kStage);
  chain_wait();
  const int4 tile = __ldcg(plan.big + blockIdx.x);  // (in bounds for every block, of use to the first ones)
  if (static_cast<int>(blockIdx.x) >= plan_tiles(plan, true)) return;
  if (tile.x < 0) return;
  const int warp = warp_id(), lane = lane_id();
  const int nkb = (C + 63) / 64, per = (nkb + splits - 1) / splits;
  const int kb0 = blockIdx.y * per, kb1 = min(nkb, kb0 + per);
  const uint32_t base = smem_u32(smem);
  tc_init<R>(bars, 1, S::kTmem);
  const uint32_t tmem = bars->tmem;

  if (warp > R::kOwner) {
    const int p = threadIdx.x - R::kFirstProducer;
    const __nv_bfloat16* Wa = W + static_cast<size_t>(tile.x) * C * r;
    const int c8 = p & 7;
    const __nv_bfloat16* row[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int q = (p >> 3) + 16 * i;
      row[i] = q < tile.z ? X + static_cast<size_t>(plan.order[tile.y + q]) * C + c8 * 8 : nullptr;
    }
    TcRing<NST> ring(bars);
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!ring.begin(lim, plan.st)) break;
      const uint32_t sx = base + ring.slot() * S::kStage, sw = sx + S::kX;
      const int c0 = kb * 64;
      const bool in = c0 + c8 * 8 < C;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool ok = in && row[i] != nullptr;
        cp_async16(sx + swz((p >> 3) + 16 * i, c8), ok ? row[i] + c0 : X, ok);
      }
      if constexpr (WT) {
#pragma unroll
        for (int i = p; i < RP * 8; i += R::kProducers) {
          const int j = i >> 3;
          const bool ok = in && j < r;
          cp_async16(sw + swz(j, c8), ok ? Wa + static_cast<size_t>(j) * C + c0 + c8 * 8 : W, ok);
        }
      } else {
#pragma unroll
        for (int i = p; i < 64 * (RP / 8); i += R::kProducers) {
          const int k = i / (RP / 8), j8 = i % (RP / 8);
          const bool ok = c0 + k < C && j8 * 8 < r;
          cp_async16(sw + (j8 >> 3) * 8192 + swz(k, j8 & 7), ok ? Wa + static_cast<size_t>(c0 + k) * r + j8 * 8 : W, ok);
        }
      }
      ring.commit();
    }
    ring.end();
  } else if (warp == R::kOwner) {
    constexpr uint32_t idesc = idesc_bf16_f32(128, RP, false, !WT);
    const uint32_t hi = sdesc_hi_sw128(1024);
    const uint32_t a0 = sdesc_lo(base, 16), b0 = sdesc_lo(base + S::kX, WT ? 16 : 8192);
    for (int kb = kb0; kb < kb1; ++kb) {
      const int i = kb - kb0, s = i % NST, chunk = i / kFlush, buf = chunk & 1;
      if (i % kFlush == 0 && !mbar_wait_bounded(bars->tempty + buf, ((chunk >> 1) & 1) ^ 1, &bars->abort, lim, plan.st, 63))
        break;
      if (!tc_stage_ready(bars, i, lim, plan.st, 64)) break;
      if (lane == 0) {
        const uint32_t so = static_cast<uint32_t>(s * S::kStage) >> 4;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_bf16_w(tmem + buf * S::kAcc, a0 + so + 2 * k, b0 + so + k * (WT ? 2 : 128), hi, idesc,
                      i % kFlush != 0 || k != 0);
        umma_commit(bars->empty + s);
        if (i % kFlush == kFlush - 1 || kb + 1 == kb1) umma_commit(bars->tfull + buf);
      }
      __syncwarp();
    }
  } else {
    float acc[RP];
#pragma unroll
    for (int j = 0; j < RP; ++j) acc[j] = 0.0f;
    const int chunks = (kb1 - kb0 + kFlush - 1) / kFlush;
    bool ok = true;
    for (int c = 0; c < chunks; ++c) {
      const int buf = c & 1;
      if (!mbar_wait_bounded(bars->tfull + buf, (c >> 1) & 1, &bars->abort, lim, plan.st, 65)) {
        ok = false;
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int j = 0; j < RP; j += 32) {
        uint32_t v[32];
        tmem_ld32(tmem + buf * S::kAcc + j + (static_cast<uint32_t>(warp) << 21), v);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 32 && j + q < RP; ++q) acc[j + q] += __uint_as_float(v[q]);
      }
      tc_fence_before();
      mbar_arrive(bars->tempty + buf);
    }
    const int q = warp * 32 + lane;
    if (ok && q < tile.z) {
      float4* out = reinterpret_cast<float4*>(parts + (static_cast<size_t>(blockIdx.y) * T + tile.y + q) * RP);
#pragma unroll
      for (int j = 0; j < RP; j += 4) out[j / 4] = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
    }
  }
  tc_end<R>(bars, S::kTmem, lim);
}

// ---------------------------------------------------------------------------
// expand
// ---------------------------------------------------------------------------
template <int RP, bool WT, bool F32>
struct TcExpand {
  // two sets of epilogue warps take the steps in turn (one set: 57 us for 16384 x
  // 4096, a step's epilogue being longer than its bytes)
  using R = TcRoles<8, 3>;
  static constexpr int kParts = F32 ? 3 : 2;  // of u: 2^-17 of it, or 2^-25 for an fp32 result
  static constexpr int NC = F32 ? 32 : 64;    // columns of a step: 128-byte lines of base and out
  static constexpr int kUChunks = (kParts * RP + 63) / 64;
  static constexpr int kU = kUChunks * 128 * 128;
  static constexpr int kWChunk = WT ? NC * 128 : RP * 128;  // 64 wide
  static constexpr int kW = (WT ? (RP + 63) / 64 : 1) * kWChunk;
  static constexpr int kYRow = NC * (F32 ? 4 : 2) + 16;
  static constexpr int kY = 128 * kYRow;
  static constexpr int kStage = (kW + kY + 1023) / 1024 * 1024;
  static constexpr int NST = RP > 64 || (F32 && RP == 64) ? 2 : 3;
  static constexpr uint32_t kTmem = 2 * NC;
  static constexpr int kBlocks = RP > 64 ? 1 : 2;  // resident on an SM
  static constexpr int kTotal = kU + NST * kStage + sizeof(TcBars<NST>) + 128 * 4 + 1024;
};

// out[t][c] = base[t][c] + sum_j u[position][j] W_a[j][c], u = s_a sum over the
// splits of parts. u's bf16 parts lie side by side along the contraction, each
// against the same tile of W_a, [r][C] (WT = false) or [C][r] (WT = true). Bound by
// base and out (16384 x 4096, rank 64: 268 MB in 54 us, 5.0 TB/s, behind the shrink
// in a graph, 57 to 64 from a cold L2, against 47 to 52 for a tiled copy). The blocks of the first columns keep u's three parts for the
// weight gradients (u_keep: [3][T][RP]). What the caller passes (plan, W_a, base)
// is on its way before the block waits for the kernel ahead, here and in the
// weight gradients (mixed batch of 5003 rows, 40 adapters, rank 24, step 118 -> 109
// us; one row, forward 9.0 -> 7.7).
template <int RP, bool WT, bool F32>
__global__ void __launch_bounds__(TcRoles<8, 3>::kThreads, TcExpand<RP, WT, F32>::kBlocks)
    adapter_expand_tc(const float* __restrict__ parts, int splits, const float* __restrict__ scale,
                      const __nv_bfloat16* __restrict__ W, PlanView plan, int T, int C, int r, int steps,
                      const void* base_in, void* out, __nv_bfloat16* __restrict__ u_keep, uint64_t lim) {
  using S = TcExpand<RP, WT, F32>;
  using R = typename S::R;
  constexpr int NST = S::NST, NC = S::NC, EB = F32 ? 4 : 2, PER = 16 / EB, PIECES = NC / PER;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  auto* bars = reinterpret_cast<TcBars<NST>*>(smem + S::kU + NST * S::kStage);
  int* s_tok = reinterpret_cast<int*>(bars + 1);
  const int4 tile = __ldcg(plan.big + blockIdx.x);  // (in bounds for every block, of use to the first ones)
  const int first = blockIdx.y * steps * NC, last = min(C, first + steps * NC);
  const int warp = warp_id(), lane = lane_id();
  if (static_cast<int>(blockIdx.x) >= plan_tiles(plan, true) || first >= last || (tile.x < 0 && base_in == out))
    return chain_leave();
  if (threadIdx.x < static_cast<unsigned>(tile.z)) s_tok[threadIdx.x] = plan.order[tile.y + threadIdx.x];
  if (tile.x < 0) {
    // rows without an adapter: the base as it is
    chain_wait();
    __syncthreads();
    const int vecs = (last - first) / PER;
    for (int row = warp; row < tile.z; row += R::kThreads / 32) {
      const size_t at = (static_cast<size_t>(s_tok[row]) * C + first) * EB;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base_in) + at);
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(out) + at);
      for (int i = lane; i < vecs; i += 32) dst[i] = base_in != nullptr ? src[i] : make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const uint32_t sb = smem_u32(smem);
  tc_init<R>(bars, 1 + 128, S::kTmem);
  const uint32_t tmem = bars->tmem;
  const int n = (last - first + NC - 1) / NC;
  // u of the tile, by every warp (the producers' first stages are on their way by
  // then): neighbouring lanes along a row, whole lines, the loads of two pieces in
  // flight. (A row a thread, four warps: 11 us of a block's 60.)
  const auto build_u = [&]() {
    const float sc = scale[tile.x];
    chain_wait();
    constexpr int U8 = RP / 8, kItems = 128 * U8;
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < kItems; i0 += 2 * R::kThreads) {
      float f[2][8];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = i0 + k * R::kThreads, row = i / U8, j = i % U8 * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[k][e] = 0.0f;
        if (row < tile.z) {
          const float* up = parts + static_cast<size_t>(tile.y + row) * RP + j;
#pragma unroll 4
          for (int s = 0; s < splits; ++s) {
            const float4* w = reinterpret_cast<const float4*>(up + static_cast<size_t>(s) * T * RP);
            const float4 x = __ldcg(w), y = __ldcg(w + 1);
            f[k][0] += x.x; f[k][1] += x.y; f[k][2] += x.z; f[k][3] += x.w;
            f[k][4] += y.x; f[k][5] += y.y; f[k][6] += y.z; f[k][7] += y.w;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = i0 + k * R::kThreads, row = i / U8, j = i % U8 * 8;
        if (i >= kItems) break;
        __nv_bfloat16 part[3][8];
#pragma unroll
        for (int e = 0; e < 8; ++e) split_bf16(f[k][e] * sc, part[0][e], part[1][e], part[2][e]);
#pragma unroll
        for (int h = 0; h < 3; ++h) {
          const uint4 v = *reinterpret_cast<const uint4*>(part[h]);
          const int ak = h * RP + j;
          if (h < S::kParts) *reinterpret_cast<uint4*>(smem + (ak / 64) * 16384 + swz(row, (ak % 64) / 8)) = v;
          if (u_keep != nullptr && blockIdx.y == 0 && row < tile.z)
            *reinterpret_cast<uint4*>(u_keep + (static_cast<size_t>(h) * T + tile.y + row) * RP + j) = v;
        }
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(&bars->ready);
  };

  if (warp > R::kOwner) {
    const int p = threadIdx.x - R::kFirstProducer;
    const __nv_bfloat16* Wa = W + static_cast<size_t>(tile.x) * C * r;
    // this thread's pieces of the base's rows: piece cp of rows p / PIECES + k kRowStep
    constexpr int kWPieces = WT ? RP / 8 : NC / 8, kWRows = WT ? NC : RP, kWStep = R::kProducers / kWPieces;
    const int wq = p % kWPieces;
    constexpr int kRowStep = R::kProducers / PIECES, kRows = (128 + kRowStep - 1) / kRowStep;
    const int cp = p % PIECES;
    const uint8_t* from[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int row = p / PIECES + k * kRowStep;
      from[k] = base_in != nullptr && row < tile.z
                    ? static_cast<const uint8_t*>(base_in) + (static_cast<size_t>(s_tok[row]) * C + cp * PER) * EB
                    : nullptr;
    }
    TcRing<NST> ring(bars);
    for (int i = 0; i < n; ++i) {
      if (!ring.begin(lim, plan.st)) break;
      const uint32_t sw = sb + S::kU + ring.slot() * S::kStage, sy = sw + S::kW;
      const int c0 = first + i * NC;
      // W: piece wq of rows p / kWPieces + k kWStep (rows: columns of out, or ranks)
#pragma unroll
      for (int k = 0; k < (kWRows + kWStep - 1) / kWStep; ++k) {
        const int row = p / kWPieces + k * kWStep;
        if (row < kWRows) {
          const bool ok = WT ? wq * 8 < r && c0 + row < last : row < r && c0 + wq * 8 < last;
          const __nv_bfloat16* src = WT ? Wa + static_cast<size_t>(c0 + row) * r + wq * 8
                                        : Wa + static_cast<size_t>(row) * C + c0 + wq * 8;
          cp_async16(sw + (wq >> 3) * S::kWChunk + swz(row, wq & 7), ok ? src : W, ok);
        }
      }
      const bool in = c0 + cp * PER < last;
#pragma unroll
      for (int k = 0; k < kRows; ++k)
        if (in && from[k] != nullptr)
          cp_async16(sy + (p / PIECES + k * kRowStep) * S::kYRow + cp * 16, from[k] + static_cast<size_t>(c0) * EB, true);
      ring.commit();
      if (i == min(n, NST) - 1) build_u();
    }
    ring.end();
  } else if (warp == R::kOwner) {
    constexpr uint32_t idesc = idesc_bf16_f32(128, NC, false, !WT);
    const uint32_t hi = sdesc_hi_sw128(1024);
    const uint32_t a0 = sdesc_lo(sb, 16), b0 = sdesc_lo(sb + S::kU, WT ? 16 : S::kWChunk);
    build_u();
    bool ok = mbar_wait_bounded(&bars->ready, 0, &bars->abort, lim, plan.st, 66);
    fence_proxy_async_smem();
    for (int i = 0; i < n && ok; ++i) {
      const int s = i % NST, buf = i & 1;
      if (!mbar_wait_bounded(bars->tempty + buf, ((i >> 1) & 1) ^ 1, &bars->abort, lim, plan.st, 67) ||
          !tc_stage_ready(bars, i, lim, plan.st, 68))
        break;
      if (lane == 0) {
        const uint32_t b = b0 + (static_cast<uint32_t>(s * S::kStage) >> 4);
        // the small parts first
#pragma unroll
        for (int h = S::kParts - 1; h >= 0; --h)
#pragma unroll
          for (int k = 0; k < RP / 16; ++k) {
            const int ak = h * RP + 16 * k;  // column of u's row of parts
            const uint32_t a = a0 + (ak / 64) * (16384 >> 4) + ((ak % 64) * 2 >> 4);
            const uint32_t bk = WT ? (16 * k / 64) * (S::kWChunk >> 4) + ((16 * k % 64) * 2 >> 4) : k * 128;
            umma_bf16_w(tmem + buf * NC, a, b + bk, hi, idesc, h != S::kParts - 1 || k != 0);
          }
        umma_commit(bars->empty + s);
        umma_commit(bars->tfull + buf);
      }
      __syncwarp();
    }
  } else {
    build_u();
    const int quarter = warp & 3;
    const bool live = quarter * 32 + lane < tile.z;
    for (int i = warp >> 2; i < n; i += 2) {
      const int s = i % NST, buf = i & 1, c0 = first + i * NC;
      if (!mbar_wait_bounded(bars->full + s, (i / NST) & 1, &bars->abort, lim, plan.st, 69) ||
          !mbar_wait_bounded(bars->tfull + buf, (i >> 1) & 1, &bars->abort, lim, plan.st, 70))
        break;
      tc_fence_after();
      if (quarter * 32 >= tile.z) {  // no rows for this warp
        mbar_arrive(bars->tempty + buf);
        mbar_arrive(bars->empty + s);
        continue;
      }
      uint8_t* sy = smem + S::kU + s * S::kStage + S::kW + quarter * 32 * S::kYRow;
      uint8_t* mine = sy + lane * S::kYRow;
#pragma unroll
      for (int j = 0; j < NC; j += 32) {
        uint32_t v[32];
        tmem_ld32(tmem + buf * NC + j + (static_cast<uint32_t>(quarter) << 21), v);
        uint4* y = reinterpret_cast<uint4*>(mine + j * EB);
#pragma unroll
        for (int e0 = 0; e0 < 32 / PER; e0 += 4) {
          // the row's pieces of the base, asked for before the first is used
          uint4 w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = base_in != nullptr && live ? y[e0 + e] : make_uint4(0, 0, 0, 0);
          if (e0 == 0) tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t* a = v + (e0 + e) * PER;
            if constexpr (F32) {
              w[e].x = __float_as_uint(__uint_as_float(w[e].x) + __uint_as_float(a[0]));
              w[e].y = __float_as_uint(__uint_as_float(w[e].y) + __uint_as_float(a[1]));
              w[e].z = __float_as_uint(__uint_as_float(w[e].z) + __uint_as_float(a[2]));
              w[e].w = __float_as_uint(__uint_as_float(w[e].w) + __uint_as_float(a[3]));
            } else {
              w[e].x = pack_bf16x2(bf16_lo(w[e].x) + __uint_as_float(a[0]), bf16_hi(w[e].x) + __uint_as_float(a[1]));
              w[e].y = pack_bf16x2(bf16_lo(w[e].y) + __uint_as_float(a[2]), bf16_hi(w[e].y) + __uint_as_float(a[3]));
              w[e].z = pack_bf16x2(bf16_lo(w[e].z) + __uint_as_float(a[4]), bf16_hi(w[e].z) + __uint_as_float(a[5]));
              w[e].w = pack_bf16x2(bf16_lo(w[e].w) + __uint_as_float(a[6]), bf16_hi(w[e].w) + __uint_as_float(a[7]));
            }
          }
          if (live) {
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e0 + e] = w[e];
          }
        }
      }
      tc_fence_before();
      mbar_arrive(bars->tempty + buf);
      __syncwarp();
      // whole lines of the warp's 32 rows
      uint4 o[PIECES];
#pragma unroll
      for (int k = 0; k < PIECES; ++k) {
        const int e = lane + 32 * k, row = e / PIECES, c = (e % PIECES) * PER;
        o[k] = *reinterpret_cast<const uint4*>(sy + row * S::kYRow + c * EB);
      }
      mbar_arrive(bars->empty + s);
#pragma unroll
      for (int k = 0; k < PIECES; ++k) {
        const int e = lane + 32 * k, row = e / PIECES, c = (e % PIECES) * PER;
        if (quarter * 32 + row < tile.z && c0 + c < last)
          __stcs(reinterpret_cast<uint4*>(static_cast<uint8_t*>(out) +
                                          (static_cast<size_t>(s_tok[quarter * 32 + row]) * C + c0 + c) * EB),
                 o[k]);
      }
    }
  }
  tc_end<R>(bars, S::kTmem, lim);
}

// ---------------------------------------------------------------------------
// weight gradients
// ---------------------------------------------------------------------------
template <int RP>
struct TcWgrad {
  using R = TcRoles<4, 7>;  // twelve warps have the registers of nine
  static constexpr int CT = RP <= 64 ? 2 : 1;           // 128-column tiles of X in a block
  static constexpr int kCols = CT * 128;
  static constexpr int kX = CT * 16384;
  static constexpr int kN = 3 * RP;                     // the parts of V side by side
  static constexpr int kV = (kN + 63) / 64 * 8192;
  static constexpr int kStage = kX + kV;
  static constexpr int NST = RP <= 32 ? 4 : 3;
  static constexpr int kSet = (kN + 63) / 64 * 64;      // TMEM columns of a tile's accumulators
  static constexpr int kAcc = CT * kSet;                // of both tiles'
  static constexpr int kBufs = 2 * kAcc <= 512 ? 2 : 1;
  static constexpr uint32_t kTmem = kBufs * kAcc <= 128 ? 128 : (kBufs * kAcc <= 256 ? 256 : 512);
  static constexpr int kTotal = NST * kStage + sizeof(TcBars<NST>) + 1024;
};

// the rows of run y: positions [y rows, (y + 1) rows) of those with an adapter;
// rows = 0: those of adapter y
struct RowRuns {
  int rows, runs;
};
struct WgradSide {
  float* G;
  float* partial;
  int C, col_tiles;
  RowRuns run;
};

// G_a[c][j] = sum over the rows t of adapter a of X[t][c] V[position][j]. A block
// takes kCols columns and one of equal runs of rows, whatever adapters lie in it;
// what it has of an adapter that lies in its run alone is the result, of others a
// partial (at most two a run: at its start and at its end) that
// adapter_wgrad_join adds up. V's three bf16 parts lie side by side as the MMA's N,
// so X is read from shared memory once for the three; their sums are added in the
// epilogue, the small ones first. v_ready: V is the caller's, not the kernel
// ahead's. OUT_T: G_a is stored [r][C] (dB), else [C][r].
// Bound by the rows of X, read once (16384 x 4096, rank 64: 134 MB in 34 us for dB,
// whose dy is in L2 in part, 39 for dA; the tensor pipe at 37%).
template <int RP, bool OUT_T>
__global__ void __launch_bounds__(TcRoles<4, 7>::kThreads, 1)
    adapter_wgrad_tc(const __nv_bfloat16* __restrict__ X, const __nv_bfloat16* __restrict__ V, PlanView plan, int T,
                     int r, WgradSide side, bool v_ready, uint64_t lim) {
  using S = TcWgrad<RP>;
  using R = typename S::R;
  constexpr int NST = S::NST, CT = S::CT;
  const int C = side.C;
  const RowRuns run = side.run;
  float* G = side.G;
  float* partial = side.partial;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  auto* bars = reinterpret_cast<TcBars<NST>*>(smem + NST * S::kStage);
  const bool any = plan_tiles(plan) > 0;
  const int warp = warp_id(), lane = lane_id(), c0 = blockIdx.x * S::kCols;
  int P0, P1, a0 = 0;
  if (run.rows == 0) {
    a0 = blockIdx.y;
    P0 = any ? plan.seg[a0] : 0;
    P1 = any ? plan.seg[a0 + 1] : 0;
    if (P0 >= P1) {  // no rows: zeros
      float* g = G + static_cast<size_t>(a0) * C * r;
      const int cols = min(S::kCols, C - c0);
      for (int i = threadIdx.x; i < cols * r; i += R::kThreads)
        g[OUT_T ? static_cast<size_t>(i / cols) * C + c0 + i % cols : static_cast<size_t>(c0) * r + i] = 0.0f;
      chain_wait();
      return;
    }
  } else {
    P0 = blockIdx.y * run.rows;
    P1 = any ? min(plan.seg[plan.L], P0 + run.rows) : 0;
    if (P0 >= P1) return chain_leave();
    // the first adapter with rows behind P0
    for (int i0 = 0; i0 < plan.L; i0 += R::kThreads) {
      const int i = i0 + static_cast<int>(threadIdx.x);
      a0 += __syncthreads_count(i < plan.L && plan.seg[i + 1] <= P0);
    }
  }
  const uint32_t base = smem_u32(smem);
  tc_init<R>(bars, 1, S::kTmem);
  const uint32_t tmem = bars->tmem;
  // (the copies before their first of V; the others before a wait that has a limit)
  if (!v_ready && warp <= R::kOwner) chain_wait();

  if (warp > R::kOwner) {
    const int p = threadIdx.x - R::kFirstProducer, w = warp - R::kOwner - 1;
    TcRing<NST> ring(bars);
    bool ok = true;
    // tokens of a block's rows, lane l those of rows l and l + 32, asked for one
    // block ahead: positions run on from one block, or adapter, to the next
    int next0 = plan.order[min(P0 + lane, T - 1)], next1 = plan.order[min(P0 + lane + 32, T - 1)];
    for (int a = a0; a < plan.L && ok; ++a) {
      const int lo = max(plan.seg[a], P0), hi = min(plan.seg[a + 1], P1);
      if (plan.seg[a] >= P1) break;
      for (int q0 = lo; q0 < hi; q0 += 64) {
        const int n = min(64, hi - q0);
        const int t0 = next0, t1 = next1;
        next0 = plan.order[min(q0 + n + lane, T - 1)];
        next1 = plan.order[min(q0 + n + lane + 32, T - 1)];
        if (!ring.begin(lim, plan.st)) {
          ok = false;
          break;
        }
        const uint32_t sx = base + ring.slot() * S::kStage, sv = sx + S::kX;
        // X: a warp copies 32 pieces of 16 bytes: 256 columns of a row, or 128 of two
        constexpr int RPI = 32 / (16 * CT), kPW = R::kProducers / 32;
        const int c8 = RPI == 2 ? lane & 15 : lane, c = c0 + c8 * 8;
#pragma unroll
        for (int i = 0; i < (64 / RPI + kPW - 1) / kPW; ++i) {
          const int row = (w + i * kPW) * RPI + (RPI == 2 ? lane >> 4 : 0);
          const int tok = __shfl_sync(0xffffffffu, row < 32 ? t0 : t1, row & 31);
          if (w + i * kPW < 64 / RPI) {
            const bool in = row < n && c < C;
            cp_async16(sx + (c8 >> 3) * 8192 + swz(row, c8 & 7), in ? X + static_cast<size_t>(tok) * C + c : X, in);
          }
        }
        if (ring.i == 0 && !v_ready) chain_wait();
        constexpr int kPieces = 64 * (RP / 8);
#pragma unroll
        for (int k = 0; k < (kPieces + R::kProducers - 1) / R::kProducers; ++k) {
          const int i = p + k * R::kProducers, row = i / (RP / 8), j8 = i % (RP / 8);
          if (i < kPieces) {
            const bool in = row < n;
            const __nv_bfloat16* src = V + (in ? static_cast<size_t>(q0 + row) * RP + j8 * 8 : 0);
#pragma unroll
            for (int h = 0; h < 3; ++h) {
              const int col8 = h * (RP / 8) + j8;
              cp_async16(sv + (col8 >> 3) * 8192 + swz(row, col8 & 7), src + static_cast<size_t>(h) * T * RP, in);
            }
          }
        }
        ring.commit();
      }
    }
    ring.end();
  } else if (warp == R::kOwner) {
    constexpr int NI = S::kN <= 256 ? 1 : 3;  // instructions over N
    constexpr uint32_t idesc = idesc_bf16_f32(128, S::kN / NI, true, true);
    const uint32_t dhi = sdesc_hi_sw128(1024);
    const uint32_t d0 = sdesc_lo(base, 8192), v0 = sdesc_lo(base + S::kX, 8192);
    int i = 0, chunk = 0;
    bool ok = true;
    for (int a = a0; a < plan.L && ok; ++a) {
      const int lo = max(plan.seg[a], P0), hi = min(plan.seg[a + 1], P1);
      if (plan.seg[a] >= P1) break;
      const int blocks = (hi - lo + 63) / 64;
      for (int b = 0; b < blocks; ++b, ++i) {
        const int s = i % NST, buf = S::kBufs == 2 ? chunk & 1 : 0;
        const uint32_t use = S::kBufs == 2 ? chunk >> 1 : chunk;
        if (b % kFlush == 0 && !mbar_wait_bounded(bars->tempty + buf, (use & 1) ^ 1, &bars->abort, lim, plan.st, 71)) {
          ok = false;
          break;
        }
        if (!tc_stage_ready(bars, i, lim, plan.st, 72)) {
          ok = false;
          break;
        }
        const bool done = b % kFlush == kFlush - 1 || b + 1 == blocks;
        if (lane == 0) {
          const uint32_t so = static_cast<uint32_t>(s * S::kStage) >> 4;
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
              for (int h = 0; h < NI; ++h)
                umma_bf16_w(tmem + buf * S::kAcc + ct * S::kSet + h * (S::kN / NI), d0 + so + ct * (16384 >> 4) + k * 128,
                            v0 + so + h * (S::kN / NI / 64) * (8192 >> 4) + k * 128, dhi, idesc,
                            b % kFlush != 0 || k != 0);
          umma_commit(bars->empty + s);
          if (done) umma_commit(bars->tfull + buf);
        }
        __syncwarp();
        if (done) ++chunk;
      }
    }
  } else {
    const uint32_t quarter = static_cast<uint32_t>(warp) << 21;
    int chunk = 0;
    bool ok = true;
    for (int a = a0; a < plan.L && ok; ++a) {
      const int sa = plan.seg[a], se = plan.seg[a + 1];
      if (sa >= P1) break;
      const int lo = max(sa, P0), hi = min(se, P1);
      if (lo >= hi) continue;
      const int chunks = ((hi - lo + 63) / 64 + kFlush - 1) / kFlush;
      float acc[CT][RP];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int j = 0; j < RP; ++j) acc[ct][j] = 0.0f;
      for (int k = 0; k < chunks; ++k, ++chunk) {
        const int buf = S::kBufs == 2 ? chunk & 1 : 0;
        const uint32_t use = S::kBufs == 2 ? chunk >> 1 : chunk;
        if (!mbar_wait_bounded(bars->tfull + buf, use & 1, &bars->abort, lim, plan.st, 73)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          const uint32_t at = tmem + buf * S::kAcc + ct * S::kSet + quarter;
          if constexpr (RP == 16) {
            uint32_t x[32], y[32];  // parts 0 and 1, part 2 (and 16 columns of no use)
            tmem_ld32(at, x);
            tmem_ld32(at + 32, y);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j)
              acc[ct][j] += __uint_as_float(x[j]) + (__uint_as_float(x[16 + j]) + __uint_as_float(y[j]));
          } else {
#pragma unroll
            for (int j = 0; j < RP; j += 32) {
#pragma unroll
              for (int h = 2; h >= 0; --h) {
                uint32_t x[32];
                tmem_ld32(at + h * RP + j, x);
                tmem_ld_wait();
#pragma unroll
                for (int q = 0; q < 32; ++q) acc[ct][j + q] += __uint_as_float(x[q]);
              }
            }
          }
        }
        tc_fence_before();
        mbar_arrive(bars->tempty + buf);
      }
      if (!ok) break;
      const bool whole = lo == sa && hi == se;
      float* slot = partial + (static_cast<size_t>(2 * blockIdx.y + (lo > sa ? 0 : 1)) * gridDim.x + blockIdx.x) *
                                  (S::kCols * RP);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const int row = ct * 128 + warp * 32 + lane, c = c0 + row;
        if (!whole) {
          // as G lies: [j][column] or [column][j]
#pragma unroll
          for (int j = 0; j < RP; j += 4) {
            if constexpr (OUT_T) {
#pragma unroll
              for (int e = 0; e < 4; ++e) slot[static_cast<size_t>(j + e) * S::kCols + row] = acc[ct][j + e];
            } else {
              *reinterpret_cast<float4*>(slot + static_cast<size_t>(row) * RP + j) =
                  make_float4(acc[ct][j], acc[ct][j + 1], acc[ct][j + 2], acc[ct][j + 3]);
            }
          }
        } else if (c < C) {
          float* g = G + static_cast<size_t>(a) * C * r;
          if constexpr (OUT_T) {
#pragma unroll
            for (int j = 0; j < RP; ++j)
              if (j < r) g[static_cast<size_t>(j) * C + c] = acc[ct][j];
          } else {
#pragma unroll
            for (int j = 0; j < RP; j += 4)
              if (j < r)
                *reinterpret_cast<float4*>(g + static_cast<size_t>(c) * r + j) =
                    make_float4(acc[ct][j], acc[ct][j + 1], acc[ct][j + 2], acc[ct][j + 3]);
          }
        }
      }
    }
  }
  chain_wait();
  tc_end<R>(bars, S::kTmem, lim);
}

// What the runs leave of dA (blockIdx.z = 0) and dB (1): for y = blockIdx.y < runs
// the adapter that begins in run y and goes on behind it, the sum of its partials
// run by run; from y = runs on the adapters without rows (every zero_rows-th for
// one y), zeros. A block takes kJoinValues values: blocks of 1024 were twelve
// thousand, most of them with nothing to do, and took 25 us. (Summed by the last
// block of adapter_wgrad_tc to finish an adapter instead: 302 us for a step of 274.) Both
// sides of 16384 x 4096, rank 64, 8 adapters: 12 us, 38 MB of partials.
constexpr int kJoinValues = 4096;
template <int RP, bool OUT_T>
__device__ __forceinline__ void wgrad_join(const PlanView& plan, int r, int zero_rows, const WgradSide& side) {
  constexpr int kCols = TcWgrad<RP>::kCols;
  const bool any = plan_tiles(plan) > 0;
  const RowRuns run = side.run;
  const int C = side.C, col_tiles = side.col_tiles;
  float* G = side.G;
  const float* partial = side.partial;
  const int n = C * r, y = blockIdx.y;  // of the C r values, as G lies
  const int first = blockIdx.x * kJoinValues + static_cast<int>(threadIdx.x) * 4, stop = min(n, first + kJoinValues);
  if (static_cast<int>(blockIdx.x) * kJoinValues >= n) return;
  if (y >= run.runs) {
    if (y >= run.runs + zero_rows) return;
    for (int a = y - run.runs; a < plan.L; a += zero_rows)
      if (!any || plan.seg[a] == plan.seg[a + 1])
        for (int i = first; i < stop; i += 1024)
          *reinterpret_cast<float4*>(G + static_cast<size_t>(a) * n + i) = make_float4(0.f, 0.f, 0.f, 0.f);
    return;
  }
  if (!any) return;
  // the adapter of the run's last position, if it has rows in the next run too
  const int end = (y + 1) * run.rows;
  if (end >= plan.seg[plan.L]) return;
  int a = 0;
  for (int k0 = 0; k0 < plan.L; k0 += 256) {
    const int k = k0 + static_cast<int>(threadIdx.x);
    a += __syncthreads_count(k < plan.L && plan.seg[k + 1] <= end - 1);
  }
  const int lo = plan.seg[a], hi = plan.seg[a + 1];
  if (hi <= end || lo < y * run.rows) return;
  chain_wait();
  const int y1 = (hi - 1) / run.rows;
  constexpr int U = kJoinValues / 1024;
  float4 s[U];
  size_t at[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    // four neighbours of G: columns c .. c + 3 of row j (OUT_T), or rows j .. j + 3 of column c
    const int i = min(first + u * 1024, n - 4);
    const int j = OUT_T ? i / C : i % r, c = OUT_T ? i % C : i / r;
    at[u] = static_cast<size_t>(c / kCols) * (RP * kCols) +
            (OUT_T ? static_cast<size_t>(j) * kCols + c % kCols : static_cast<size_t>(c % kCols) * RP + j);
    s[u] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int k = y; k <= y1; ++k) {
    const float* p = partial + static_cast<size_t>(2 * k + (k == y ? 1 : 0)) * col_tiles * (RP * kCols);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(p + at[u]));
      s[u].x += v.x; s[u].y += v.y; s[u].z += v.z; s[u].w += v.w;
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (first + u * 1024 < n) *reinterpret_cast<float4*>(G + static_cast<size_t>(a) * n + first + u * 1024) = s[u];
}

template <int RP>
__global__ void __launch_bounds__(256) adapter_wgrad_join(PlanView plan, int r, int zero_rows, WgradSide dA,
                                                          WgradSide dB) {
  if (blockIdx.z == 0) wgrad_join<RP, false>(plan, r, zero_rows, dA);
  else wgrad_join<RP, true>(plan, r, zero_rows, dB);
  chain_wait();
}

}  // namespace moe
