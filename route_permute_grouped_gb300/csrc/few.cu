// The whole MoE layer for a few tokens in one kernel (few.cuh: what bounds it, the
// schedule and the operands).
#include <cuda_fp4.h>
#include <string.h>

#include <atomic>
#include <initializer_list>

#include "few.cuh"
#include "router_sel.cuh"

namespace moe {

namespace {

// One thread of a converged warp. The compiler knows that it is one: an MMA then takes
// 79 cycles at 16 columns (the 4 KB of weights it reads from shared memory); behind a
// comparison of the lane it is issued by a loop over the lanes, 153 cycles each.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
// One block's forms of the block-scaled MMA and of the scales' copy (common.cuh has
// the pairs'): E2M1 operands two to a byte, K = 64, two E8M0 scales a row, the bytes 0, 1
// or 2, 3 of a cell by the descriptor's scale ids.
__device__ __forceinline__ void umma_mx_w(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t d_hi, uint32_t idesc,
                                          uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %7, 0;\n\t"
      "mov.b64 da, {%1, %3};\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, %4, [%5], [%6], p;\n\t}" ::"r"(
          d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(d_hi), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_cp_32x128b_x4(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// kind::mxf4: E2M1 A and B (format 1), E8M0 scales (bit 23)
__device__ __forceinline__ uint32_t idesc_mxf4(int N) { return idesc_nvf4_f32(128, N) | (1u << 23); }

__device__ __forceinline__ void bulk_load_hint(void* dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar)), "l"(pol)
      : "memory");
}

__device__ __forceinline__ unsigned ld_acquire(const unsigned* p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void red_release(unsigned* p, unsigned v) {
  asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool ok) {
  const int n = ok ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

// Wait (bounded) until *p has reached n. False when the wait ran out or the block gave up.
__device__ __forceinline__ bool wait_count(const unsigned* p, unsigned n, FewCtl* c, const FewParams& q, int where) {
  const uint64_t t0 = globaltimer();
  for (unsigned it = 1;; ++it) {
    if (ld_acquire(p) >= n) return true;
    if (*static_cast<volatile int*>(&c->abort)) return false;
    if ((it & 63u) == 0 && globaltimer() - t0 > q.lim) {
      *static_cast<volatile int*>(&c->abort) = 1;
      set_status(q.status, MOE_ERR_DEVICE_TIMEOUT, where);
      return false;
    }
  }
}
// the epilogue warps' barrier, alone and with the conjunction of a condition: they
// share barriers, so all of them go on or none does
__device__ __forceinline__ void epi_sync() { named_bar_sync(1, kFewEpi); }
__device__ __forceinline__ bool epi_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u)
      : "memory");
  return r != 0;
}
// a whole warp's bounded wait: all lanes go on or none does
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, FewCtl* c, const FewParams& p, int where) {
  const bool ok = mbar_wait_bounded(bar, parity, &c->abort, p.lim, p.status, where);
  return __all_sync(0xffffffffu, ok) != 0;
}
// All blocks' epilogue warps (thread `et` of a block's 256): what they wrote before is
// visible to all after. False for every thread of a block whose wait ran out.
__device__ __forceinline__ bool grid_sync(unsigned* counter, FewCtl* c, const FewParams& p, int et, int where) {
  epi_sync();
  if (et == 0) {
    __threadfence();
    if (!(p.fault && blockIdx.x == 0)) red_release(counter, 1u);
    wait_count(counter, gridDim.x, c, p, where);
  }
  epi_sync();
  const bool ok = epi_all(*static_cast<volatile int*>(&c->abort) == 0);
  __threadfence();
  return ok;
}

// order-preserving unsigned image of a float that is no NaN (0 is below all of them)
__device__ __forceinline__ uint32_t sort_key(float z) {
  const uint32_t u = __float_as_uint(z + 0.0f);  // -0 and 0 are equal
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// The power of two of a block's first E2M1 part: its unit 2^e has the largest magnitude
// at 6 or below. The second part's unit is 2^-2 of the first's, every further one's 2^-3
// of the one before: a part leaves at most 1 (the step above 4 halved), then at most 1/2
// of its unit, which is 4 of the next. Not below the smallest scale for the last part.
// kFewBad: the block holds an infinity or a NaN.
constexpr int kFewBad = 1 << 20;
__device__ __forceinline__ int part_shift(int part) { return part == 0 ? 0 : 3 * part - 1; }
__device__ __forceinline__ int part_exponent(float amax, int parts) {
  const uint32_t u = __float_as_uint(amax);
  if (u >= 0x7f800000u) return kFewBad;
  const int e = static_cast<int>(u >> 23) - 127 - ((u & 0x7fffffu) > 0x400000u ? 1 : 2);
  const int least = -127 + part_shift(parts - 1);
  return e > least ? e : least;
}
__device__ __forceinline__ uint32_t part_byte(int e, int part) {
  return e >= kFewBad ? 255u : static_cast<uint32_t>(e - part_shift(part) + 127);
}
// 2^-e
__device__ __forceinline__ float part_inverse(int e) {
  return e >= kFewBad ? 0.0f : __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}
// what the part leaves, in the next one's unit
__device__ __forceinline__ float part_rest(float v, float q, int part) { return (v - q) * (part == 0 ? 4.0f : 8.0f); }
__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi) {
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(make_float2(lo, hi), __NV_E2M1, cudaRoundNearest));
}
// value of a code (low four bits): s eem
__device__ __forceinline__ float e2m1_value(uint32_t c) {
  const uint32_t e = (c >> 1) & 3u, m = c & 1u;
  const float v = e == 0 ? 0.5f * static_cast<float>(m) : __uint_as_float(((e + 126u) << 23) | (m << 22));
  return (c & 8u) ? -v : v;
}

// ---------------------------------------------------------------------------
// router
// ---------------------------------------------------------------------------
// logits[t][e], an item of NE experts x 8 tokens a block: its 8 warps share H, 8 products
// to a 16-byte load, fp32 fused multiply-adds; the 32 lanes' sums meet in a halving
// butterfly, the warps' in shared memory
template <int NE>
__device__ __noinline__ void few_logits_of(const FewParams& p, FewCtl* c, int et) {
  const int warp = et >> 5, lane = et & 31;
  const int eg = (p.E + NE - 1) / NE, items = eg * ((p.T + 7) >> 3);
  const int nv = p.H >> 3;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int e0 = item % eg * NE, t0 = item / eg * 8;
    const int ne = min(NE, p.E - e0), nt = min(8, p.T - t0);
    const uint4* w = reinterpret_cast<const uint4*>(p.wr + static_cast<size_t>(e0) * p.H);
    const uint4* x = reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(t0) * p.H);
    float acc[32];  // [expert][token]
#pragma unroll
    for (int j = 0; j < 32; ++j) acc[j] = 0.0f;
#pragma unroll(NE == 1 ? 2 : 1)
    for (int v = et; v < nv; v += kFewEpi) {
      uint4 wv[NE], xv[8];
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (i < ne) wv[i] = __ldg(w + static_cast<size_t>(i) * nv + v);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < nt) xv[j] = __ldg(x + static_cast<size_t>(j) * nv + v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j < nt) {
          const uint32_t xx[4] = {xv[j].x, xv[j].y, xv[j].z, xv[j].w};
#pragma unroll
          for (int i = 0; i < NE; ++i) {
            const uint32_t ww[4] = {wv[i].x, wv[i].y, wv[i].z, wv[i].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              acc[8 * i + j] = fmaf(bf16_lo(xx[q]), bf16_lo(ww[q]), acc[8 * i + j]);
              acc[8 * i + j] = fmaf(bf16_hi(xx[q]), bf16_hi(ww[q]), acc[8 * i + j]);
            }
          }
        }
      }
    }
    c->scratch[warp][lane] = lane_column_sums(acc, lane);
    epi_sync();
    if (et < 32 && (et >> 3) < ne && (et & 7) < nt) {
      float s = 0.0f;
#pragma unroll
      for (int q = 0; q < 8; ++q) s += c->scratch[q][et];
      const int e = e0 + (et >> 3), t = t0 + (et & 7);
      p.logits[static_cast<size_t>(t) * p.E + e] = s + (p.lb != nullptr ? __ldg(p.lb + e) : 0.0f);
    }
    epi_sync();
  }
}
// the more experts an item has the fewer times x is read and unpacked, as long as
// there are items for the blocks (128 experts: 24 tokens two 552 us, one 562, four 559; 64 tokens four
// 716, one 724; 8 tokens one 295.4, four 297.1)
__device__ void few_logits(const FewParams& p, FewCtl* c, int et) {
  const int pairs = p.E * ((p.T + 7) >> 3), G = gridDim.x;
  if (pairs >= 4 * G) few_logits_of<4>(p, c, et);
  else if (pairs >= 2 * G) few_logits_of<2>(p, c, et);
  else few_logits_of<1>(p, c, et);
}

// x in E2M1 parts: four lanes a block of 32 along H, a warp 256 elements. Dealt from the last
// block down: with few tokens those have no logits to compute
__device__ void few_split_x(const FewParams& p, int et) {
  const int nb = p.H >> 5, lane = et & 31, total = p.T * nb;
  for (int u = gridDim.x - 1 - blockIdx.x + gridDim.x * (et >> 5); 8 * u < total; u += 8 * gridDim.x) {
    const int i = min(8 * u + (lane >> 2), total - 1);  // the last warp's spare lanes: its last block once more
    const bool on = 8 * u + (lane >> 2) < total;
    const int t = i / nb, b = i - t * nb, part = lane & 3;
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(t) * p.H + b * 32) + part);
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
    float v[8], amax = 0.0f;
    int bad = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16_lo(ww[j]);
      v[2 * j + 1] = bf16_hi(ww[j]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      amax = fmaxf(amax, fabsf(v[j]));
      bad |= v[j] != v[j];
    }
#pragma unroll
    for (int d = 1; d <= 2; d <<= 1) {
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
      bad |= __shfl_xor_sync(0xffffffffu, bad, d);
    }
    const int e = part_exponent(bad ? INFINITY : amax, p.P1);
    const float inv = part_inverse(e);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = e >= kFewBad ? 0.0f : v[j] * inv;
#pragma unroll 1
    for (int q = 0; q < p.P1; ++q) {
      const size_t row = static_cast<size_t>(t) * p.P1 + q;
      uint32_t codes = 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t c = e2m1_pair(v[2 * j], v[2 * j + 1]);
        codes |= c << (8 * j);
        v[2 * j] = part_rest(v[2 * j], e2m1_value(c), q);
        v[2 * j + 1] = part_rest(v[2 * j + 1], e2m1_value(c >> 4), q);
      }
      if (on) {
        *reinterpret_cast<uint32_t*>(p.xq + row * (p.H >> 1) + b * 16 + part * 4) = codes;
        if (part == 0) p.x_sf[row * nb + b] = static_cast<uint8_t>(part_byte(e, q));
      }
    }
  }
}

// Selection and gates of token t by one warp, as the router's epilogue does it
// (router_sel.cuh): z = logits, probabilities or sigmoids (+ expert bias), NaN as
// -inf, an optional group limit, the k largest with ties to the lower index, gates
// from the unbiased scores. Lane i < k leaves with slot i.
__device__ void few_select(const FewParams& p, float* zs, int t, int lane, int& e_out, float& g_out) {
  const float* L = p.logits + static_cast<size_t>(t) * p.E;
  float l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) l[i] = lane + 32 * i < p.E ? __ldcg(L + lane + 32 * i) : -INFINITY;
  if (p.mode == RSEL_LOGIT && !p.force) {  // where logits are what is selected by, a NaN's gate is 0 too
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (l[i] != l[i]) l[i] = -INFINITY;
  }
  int e_sel = 0;
  if (p.force) {
    e_sel = static_cast<int>((static_cast<long long>(t) * p.k + lane) % p.E);
  } else {
    float z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = l[i];
    if (p.mode == RSEL_SOFTMAX) {
      float m = -INFINITY, s = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, z[i]);
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        z[i] = lane + 32 * i < p.E ? expf(z[i] - m) : 0.0f;
        s += z[i];
      }
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      // (a row with a NaN or no finite maximum: probabilities 0 but for the NaN, the bias selects)
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = s > 0.0f ? z[i] / s : z[i] * 0.0f;
    } else if (p.mode == RSEL_SIGMOID) {
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = 1.0f / (1.0f + expf(-z[i]));
    }
    if (p.mode != RSEL_LOGIT && p.eb != nullptr) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (lane + 32 * i < p.E) z[i] += __ldg(p.eb + lane + 32 * i);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (z[i] != z[i]) z[i] = -INFINITY;
    if (p.groups > 1 && p.topk_groups < p.groups) {
      const int gsz = p.E / p.groups;
#pragma unroll
      for (int i = 0; i < 8; ++i) zs[lane + 32 * i] = z[i];
      __syncwarp();
      uint32_t key = 0;
      if (lane < p.groups) {
        float b1 = -INFINITY, b2 = -INFINITY;
        for (int j = 0; j < gsz; ++j) {
          const float v = zs[lane * gsz + j];
          if (v > b1) {
            b2 = b1;
            b1 = v;
          } else if (v > b2) {
            b2 = v;
          }
        }
        key = sort_key(gsz >= 2 ? b1 + b2 : b1);
      }
      uint32_t kept = 0;
      for (int s = 0; s < p.topk_groups; ++s) {
        const uint32_t best = __reduce_max_sync(0xffffffffu, key);
        const int g = __ffs(__ballot_sync(0xffffffffu, key == best)) - 1;
        kept |= 1u << g;
        if (lane == g) key = 0;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (lane + 32 * i < p.E && !((kept >> ((lane + 32 * i) / gsz)) & 1u)) z[i] = -INFINITY;
      __syncwarp();
    }
    uint32_t key[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) key[i] = lane + 32 * i < p.E ? sort_key(z[i]) : 0u;
    for (int s = 0; s < p.k; ++s) {
      uint32_t mine = 0;
      int at = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (key[i] > mine) {
          mine = key[i];
          at = lane + 32 * i;
        }
      }
      const uint32_t best = __reduce_max_sync(0xffffffffu, mine);
      const int e = static_cast<int>(__reduce_min_sync(0xffffffffu, mine == best ? static_cast<unsigned>(at) : 0xffffffu));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e == lane + 32 * i) key[i] = 0u;
      if (lane == s) e_sel = e;
    }
  }
  const bool on = lane < p.k;
  float ls = -INFINITY;  // the selected expert's logit, from the lane that has it
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = __shfl_sync(0xffffffffu, l[i], e_sel & 31);
    if (on && (e_sel >> 5) == i) ls = v;
  }
  float w;
  if (p.mode == RSEL_SIGMOID) {
    w = on ? 1.0f / (1.0f + expf(-ls)) : 0.0f;
  } else {
    float m = ls;
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    w = on ? expf(ls - m) : 0.0f;
  }
  float sum = w;
#pragma unroll
  for (int d = 8; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  e_out = e_sel;
  g_out = p.gate_scale / sum * w;
}

// The block's plan from the slots' experts and gates: entries of the experts in ascending
// order, their rows in token order (a row's place is the number of its expert's tokens
// before it, from a bit a token)
__device__ void few_plan(const FewParams& p, FewCtl* c, int et) {
  const int R = p.T * p.k, warp = et >> 5, lane = et & 31;
  c->has[et][0] = c->has[et][1] = 0u;
  epi_sync();
  for (int r = et; r < R; r += kFewEpi) {
    const int t = r / p.k;
    atomicOr(&c->has[c->eidx[r]][t >> 5], 1u << (t & 31));
  }
  epi_sync();
  const int m = __popc(c->has[et][0]) + __popc(c->has[et][1]);
  // an expert's rows in as few entries as hold them, of one size
  const int ng = (m + p.mcap - 1) / p.mcap, per = ng > 0 ? (m + ng - 1) / ng : 0;
  int off = m, at = ng, mx = per;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, off, d), b = __shfl_up_sync(0xffffffffu, at, d);
    if (lane >= d) {
      off += a;
      at += b;
    }
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
  if (lane == 31) {
    c->warp_sum[warp] = off;
    c->warp_act[warp] = at;
    c->warp_max[warp] = mx;
  }
  epi_sync();
  int na = 0, most = p.Fs ? min(p.T, p.mcap) : 0;
  off -= m;
  at -= ng;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    if (q < warp) {
      off += c->warp_sum[q];
      at += c->warp_act[q];
    }
    na += c->warp_act[q];
    most = max(most, c->warp_max[q]);
  }
  for (int g = 0; g < ng; ++g) {
    c->act[at + g] = static_cast<uint8_t>(et);
    c->off[at + g] = off + g * per;
  }
  c->eoff[et] = off;
  if (et == 0) {
    c->nact = na;
    c->off[na] = R;
  }
  epi_sync();
  if (et == kFewEpi - 1) c->geo = few_geo(p.P1, p.P2, p.T, most, p.mx);
  for (int r = et; r < R; r += kFewEpi) {
    const int t = r / p.k, e = c->eidx[r];
    const uint32_t below = (1u << (t & 31)) - 1u;
    const int row = c->eoff[e] + (t < 32 ? __popc(c->has[e][0] & below) : __popc(c->has[e][0]) + __popc(c->has[e][1] & below));
    c->tok[row] = static_cast<uint8_t>(t);
    c->gate[row] = c->sgate[r];
  }
  epi_sync();
}

// Router, selection and plan by the epilogue warps; false when a wait ran out
template <bool MX>
__device__ bool few_route(const FewParams& p, FewCtl* c, int et) {
  const int warp = et >> 5, lane = et & 31;
  for (int i = blockIdx.x * kFewEpi + et; i < p.cnt_words; i += gridDim.x * kFewEpi) p.cnt[i] = 0u;
  if constexpr (MX) few_split_x(p, et);
  few_logits(p, c, et);
  if (!grid_sync(p.sync, c, p, et, 81)) return false;
  // a few tokens: every block selects for all of them, which saves the second wait
  const bool all = p.T <= kFewRedundant;
  for (int t = all ? warp : static_cast<int>(blockIdx.x + gridDim.x * warp); t < p.T; t += all ? 8 : 8 * gridDim.x) {
    int e;
    float g;
    few_select(p, c->scratch[warp], t, lane, e, g);
    if (lane < p.k) {
      if (all) {
        c->eidx[t * p.k + lane] = static_cast<uint8_t>(e);
        c->sgate[t * p.k + lane] = g;
      }
      if (!all || blockIdx.x == 0) {
        p.idx[t * p.k + lane] = e;
        p.gate[t * p.k + lane] = g;
      }
    }
  }
  if (!all) {
    if (!grid_sync(p.sync + 1, c, p, et, 82)) return false;
    for (int r = et; r < p.T * p.k; r += kFewEpi) {
      c->eidx[r] = static_cast<uint8_t>(__ldcg(p.idx + r));
      c->sgate[r] = __ldcg(p.gate + r);
    }
  }
  epi_sync();
  few_plan(p, c, et);
  return true;
}

// ---------------------------------------------------------------------------
// ends of a tile
// ---------------------------------------------------------------------------
// The block's share of a tile that is joined elsewhere, to a slot of the workspace
__device__ __forceinline__ void few_leave(const float* acc, int n, float* slot, unsigned* cnt, int et) {
  float4* dst = reinterpret_cast<float4*>(slot);
  const float4* src = reinterpret_cast<const float4*>(acc);
  for (int i = et; i < n / 4; i += kFewEpi) __stcg(dst + i, src[i]);
  epi_sync();
  if (et == 0) red_release(cnt, 1u);
}
// The rest of a tile, `na` shares from slot `a0` of part_a on and then `nb` from b0 of part_b:
// once all are there, added to `acc` in this order. False when the wait ran out.
__device__ __forceinline__ bool few_join(float* acc, int n, size_t stride, const float* part_a, int a0, int na,
                                         const float* part_b, int b0, int nb, const unsigned* cnt, FewCtl* c,
                                         const FewParams& p, int et) {
  bool ok = true;
  if (et == 0) ok = wait_count(cnt, na + nb, c, p, 93);
  if (!epi_all(ok)) return false;
  float4* a = reinterpret_cast<float4*>(acc);
  const int all = na + nb;
  auto piece = [&](int i) {
    return reinterpret_cast<const float4*>(i < na ? part_a + (a0 + i) * stride : part_b + (b0 + i - na) * stride);
  };
  auto add = [](float4& v, const float4& w) {
    v.x += w.x;
    v.y += w.y;
    v.z += w.z;
    v.w += w.w;
  };
  const int n4 = n / 4;
  if (n4 <= kFewEpi) {
    // few floats: four pieces on their way at a time (eight, and four float4 below, spill registers
    // to a stack that the L1 left beside 227 KB does not hold: one MXFP4 token 42.4 us for 41.6,
    // 64 tokens of a layer of 64 x 64 63.6 for 57.9)
    if (et < n4) {
      float4 v = a[et];
      for (int i = 0; i < all; i += 4) {
        float4 w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (i + k < all) w[k] = __ldcg(piece(i + k) + et);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (i + k < all) add(v, w[k]);
      }
      a[et] = v;
    }
  } else {
    // a thread's two float4 of two pieces
    for (int base = et; base < n4; base += 2 * kFewEpi) {
      float4 v[2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (base + k * kFewEpi < n4) v[k] = a[base + k * kFewEpi];
      for (int i = 0; i < all; i += 2) {
        const float4 *s0 = piece(i), *s1 = piece(min(i + 1, all - 1));
        float4 w0[2], w1[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (base + k * kFewEpi < n4) {
            w0[k] = __ldcg(s0 + base + k * kFewEpi);
            w1[k] = __ldcg(s1 + base + k * kFewEpi);
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (base + k * kFewEpi < n4) {
            add(v[k], w0[k]);
            if (i + 1 < all) add(v[k], w1[k]);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (base + k * kFewEpi < n4) a[base + k * kFewEpi] = v[k];
    }
  }
  epi_sync();
  return true;
}

// SwiGLU of an entry's rows x 128 columns from h1, h3 (fp32 sums acc [rows][2][128]), gated, split
// into the parts of the down product's operand
template <bool MX>
__device__ void few_activate(const FewParams& p, const FewCtl* c, const float* acc, const FewRows& rw, int i, int tile,
                             int et) {
  const int f = 128 * tile + (et & 127), lane = et & 31;
  const int Fx = i < 0 ? p.Fs : p.F;
  uint8_t* dst = i < 0 ? p.as : p.a;
  uint8_t* dsf = i < 0 ? p.as_sf : p.a_sf;
  for (int j = et >> 7; j < rw.m; j += 2) {
    const float h1 = acc[j * 256 + (et & 127)], h3 = acc[j * 256 + 128 + (et & 127)];
    float a = h1 / (1.0f + expf(-h1)) * h3;
    if (i >= 0) a *= c->gate[rw.r0 + j];
    const size_t row = static_cast<size_t>(rw.r0 + j) * p.P2;
    if constexpr (MX) {
      // a warp holds a block of 32 along F
      float amax = fabsf(a);
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
      const bool bad = __any_sync(0xffffffffu, a != a);
      const int e = part_exponent(bad ? INFINITY : amax, p.P2);
      float v = e >= kFewBad ? 0.0f : a * part_inverse(e);
      for (int q = 0; q < p.P2; ++q) {
        const uint32_t code = e2m1_pair(v, 0.0f) & 15u;
        const uint32_t next = __shfl_down_sync(0xffffffffu, code, 1);
        if ((lane & 1) == 0) dst[(row + q) * (Fx >> 1) + (f >> 1)] = static_cast<uint8_t>(code | (next << 4));
        if (lane == 0) dsf[(row + q) * (Fx >> 5) + (f >> 5)] = static_cast<uint8_t>(part_byte(e, q));
        v = part_rest(v, e2m1_value(code), q);
      }
    } else if (f < Fx) {
      __nv_bfloat16* d = reinterpret_cast<__nv_bfloat16*>(dst);
      __nv_bfloat16 v[3];
      split_bf16(a, v[0], v[1], v[2]);
#pragma unroll
      for (int q = 0; q < 3; ++q)
        if (q < p.P2) d[(row + q) * Fx + f] = v[q];
    }
  }
}

__device__ __forceinline__ void few_store_y(const FewParams& p, int t, int h, float v) {
  if (h >= p.H) return;
  const size_t o = static_cast<size_t>(t) * p.H + h;
  if (p.out_fp32) static_cast<float*>(p.y)[o] = v;
  else static_cast<__nv_bfloat16*>(p.y)[o] = __float2bfloat16_rn(v);
}

// What a block that gave up has under way ends before it does: copies to shared memory, which
// report to `full`, and MMAs. All threads, behind their roles; n: stages that the thread's warp
// has begun. The threads that fill stages may have left at different ones, and a barrier of
// `full` turns only when all of them have arrived: each arrives for those that another one
// began. (The last stage begun found the one before it in its place taken, so that
// all had arrived there: only the last g.nst barriers are open.)
template <bool MX>
__device__ __noinline__ void few_drain(const FewParams& p, FewCtl* c, int n) {
  const int warp = warp_id();
  int given_up = 0;  // the block's own flag is set
  if (warp != 1 && warp < 4) atomicMax(&c->stages, n);
  __syncthreads();
  const int last = c->stages;
  if (last > 0) {
    // (with a shared expert the stages are the same before and after the plan, without one there are none before)
    const FewGeo g = p.Fs ? few_geo(p.P1, p.P2, p.T, min(p.T, p.mcap), MX) : c->geo;
    const bool weights = warp == 0 && elect_one();
    if (weights || warp == 2 || warp == 3)
      for (int i = n; i < last; ++i) mbar_arrive(c->full + i % g.nst);
    if (weights)
      for (int i = max(0, last - g.nst); i < last; ++i)
        mbar_wait_bounded(c->full + i % g.nst, (i / g.nst) & 1, &given_up, p.lim, nullptr, 0);
  }
  if (warp == 1) {
    if (elect_one()) umma_commit(&c->drain);
    __syncwarp();
    mbar_wait_bounded(&c->drain, 0, &given_up, p.lim, nullptr, 0);
  }
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <bool MX>
__global__ void __launch_bounds__(kFewThreads, 1)
    few_kernel(const __grid_constant__ FewParams p, const __grid_constant__ FewMaps maps) {
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // layout assumption broken: report, touch nothing
    if (threadIdx.x == 0) set_status(p.status, MOE_ERR_CUDA, 99);
    return;
  }
  FewCtl* c = reinterpret_cast<FewCtl*>(smem + kFewCtlOff);
  const int warp = warp_id(), lane = lane_id();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kFewStages; ++s) {
      mbar_init(c->full + s, 1 + kFewCopiers);
      mbar_init(c->empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(c->tfull + b, 1);
      mbar_init(c->tempty + b, kFewEpi / 32);
    }
    mbar_init(&c->plan, 1);
    mbar_init(&c->drain, 1);
    c->abort = 0;
    c->stages = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&c->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c->tmem;
  const int first_phase = p.Fs ? 0 : 1;
  volatile int* abort_flag = &c->abort;
  const int G = gridDim.x;
  constexpr int kSubBytes = 128;
  int n = 0;  // stages so far, of the warps that fill or take them

  if (warp == 0) {
    // ------------------------------------------------------------ weights
    if (elect_one()) {
      if constexpr (!MX)
        for (int i = 0; i < (p.Fs ? 6 : 3); ++i) tma_prefetch_desc(&maps.m[i]);
      const uint64_t pol = l2_policy_evict_first();
      bool ok = true;
      FewGeo g = few_geo(p.P1, p.P2, p.T, min(p.T, p.mcap), MX);
      for (int ph = first_phase; ph < 5 && ok; ++ph) {
        if (ph == 1) {
          if (!mbar_wait_bounded(&c->plan, 0, abort_flag, p.lim, p.status, 83)) break;
          g = c->geo;
        }
        FewWalk w(ph, p, g, ph == 0 ? 0 : c->nact, blockIdx.x, G);
        FewChunk ch;
        while (ok && w.next(ch)) {
          const bool sh = ch.i < 0;
          const int e = sh ? 0 : c->act[ch.i];
          const int nsb = !w.down ? p.nsb1 : sh ? p.nsb2s : p.nsb2;
          for (int kb = ch.kb; kb < ch.kb + ch.nkb; ++kb, ++n) {
            const int s = n % g.nst;
            if (!mbar_wait_bounded(c->empty + s, ((n / g.nst) & 1) ^ 1, abort_flag, p.lim, p.status, 84)) {
              ok = false;
              break;
            }
            uint8_t* sA = smem + s * g.stage;
            uint64_t* bar = c->full + s;
            const int sb0 = !w.down ? kb : kb * kFewSub2, ns = !w.down ? 2 : min(kFewSub2, nsb - sb0);
            if constexpr (MX) {
              // a stage's tiles are one run of bytes
              const uint8_t* src = !w.down ? (sh ? p.w13s : p.w13) : (sh ? p.w2s : p.w2);
              const size_t t = (static_cast<size_t>(e) * (w.down ? p.ns2 : sh ? p.ns1s : p.ns1) + ch.tile) * nsb + sb0;
              mbar_arrive_expect_tx(bar, ns * few_tile(true));
              bulk_load_hint(sA, src + t * (w.down ? 1 : 2) * few_tile(true), ns * few_tile(true), bar, pol);
            } else {
              mbar_arrive_expect_tx(bar, ns * kFewATile);
              for (int q = 0; q < ns; ++q) {
                // W1's and W3's tile of one k sub-block, or W2's of two
                const CUtensorMap* m = &maps.m[(sh ? 3 : 0) + (w.down ? 2 : q)];
                const int row = w.down ? e * (sh ? p.Fs : p.F) + (sb0 + q) * 64 : e * p.H + kb * 64;
                tma_load_2d_hint(sA + q * kFewATile, m, bar, ch.tile * 128, row, pol);
                tma_load_2d_hint(sA + q * kFewATile + 8192, m, bar, ch.tile * 128 + 64, row, pol);
              }
            }
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    int na = 0;  // accumulators so far
    bool ok = true;
    FewGeo g = few_geo(p.P1, p.P2, p.T, min(p.T, p.mcap), MX);
    const uint32_t d_hi = sdesc_hi_sw128(1024);
    const uint64_t sf_hi = static_cast<uint64_t>((128u >> 4) | (1u << 14)) << 32;
    constexpr uint32_t kAStep = MX ? (32u >> 4) : (2048u >> 4);
    int used[2] = {0, 0};  // times that each accumulator has been filled
    auto step = [&](uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, int q, int kk, uint32_t sfb,
                    uint32_t region, bool go) {
      const uint32_t id = 2 * (kk & 1);
      if constexpr (MX)
        umma_mx_w(d, a_lo, b_lo, d_hi, idesc | (id << 29) | (id << 4), region + 8 * q + 4 * (kk >> 1), sfb, go ? 1u : 0u);
      else
        umma_bf16_w(d, a_lo, b_lo, d_hi, idesc, go ? 1u : 0u);
    };
    for (int ph = first_phase; ph < 5 && ok; ++ph) {
      if (ph == 1) {
        if (!warp_wait(&c->plan, 0, c, p, 85)) break;
        g = c->geo;
      }
      FewWalk w(ph, p, g, ph == 0 ? 0 : c->nact, blockIdx.x, G);
      FewChunk ch;
      const int parts = w.down ? p.P2 : p.P1;
      const int nbuf = w.down ? g.nbuf2 : g.nbuf1;
      const int il = w.down ? g.il2 : g.il1, il_cols = w.down ? g.n2 : 2 * g.n1;
      const int acc_cols = il * il_cols;
      na = 0;
      // W2's accumulators are laid out differently: all of the others have been read
      for (int b = 0; b < 2 && ok && ph == 3; ++b)
        if (used[b] > 0) ok = warp_wait(c->tempty + b, (used[b] & 1) ^ 1, c, p, 86);
      while (ok && w.next(ch)) {
        const int N = few_cols(parts, FewRows(p, c, ch.i).m);
        const int buf = na % nbuf;
        ++na;
        // every earlier use of this accumulator has been read
        if (!warp_wait(c->tempty + buf, (used[buf] & 1) ^ 1, c, p, 86)) {
          ok = false;
          break;
        }
        ++used[buf];
        tc_fence_after();
        const uint32_t d0 = tmem + buf * acc_cols;
        for (int kb = ch.kb; kb < ch.kb + ch.nkb; ++kb, ++n) {
          const int s = n % g.nst;
          if (!warp_wait(c->full + s, (n / g.nst) & 1, c, p, 87)) {
            ok = false;
            break;
          }
          // the tokens' copies are generic-proxy writes: ordered before the MMAs' reads
          fence_proxy_async_smem();
          tc_fence_after();
          if (elect_one()) {
            const uint32_t sA = smem_u32(smem) + s * g.stage;
            const uint32_t a0 = sdesc_lo(sA, MX ? 16u : 8192u), b0 = sdesc_lo(sA + 2 * few_tile(MX), 16u);
            int ns = 2;
            if (w.down) ns = min(kFewSub2, (ch.i < 0 ? p.nsb2s : p.nsb2) - kb * kFewSub2);
            const int nblk = w.down ? g.nblk2 : g.nblk1;
            const uint32_t region = tmem + kFewSfCol + (n & 1) * kFewSfRegion;
            if constexpr (MX) {
              // scales to tensor memory, four columns for 128 rows and 128 elements: A's two a
              // tile, behind its codes, then B's two for 128 rows
              const uint32_t sfa = sdesc_lo(sA + kFewATile, 128u), sfb = sdesc_lo(sA + 2 * few_tile(true) + g.b_bytes, 128u);
              const int nb = 2 * (w.down ? ns * nblk : nblk);
              for (int q = 0; q < 2 * ns; ++q)
                tmem_cp_32x128b_x4(region + 4 * q,
                                   sf_hi | (sfa + (((q >> 1) * few_tile(true) + (q & 1) * kFewSf) >> 4)));
              for (int q = 0; q < nb; ++q)
                tmem_cp_32x128b_x4(region + 16 + 4 * q, sf_hi | (sfb + ((kFewSf * q) >> 4)));
            }
            const bool begun = kb > ch.kb;
            for (int n0 = 0; n0 < N; n0 += 256) {
              const int nn = min(256, N - n0);
              const uint32_t idesc = MX ? idesc_mxf4(nn) : idesc_bf16_f32(128, nn, true, false);
              const uint32_t bn = b0 + ((n0 * kSubBytes) >> 4);
              // phases 0 to 2: W1's and W3's tile against the same tokens, accumulators of their
              // own; 3, 4: two sub-blocks of W2, each against its own. Step kk along k of
              // either goes to accumulator kk % il
              if (!w.down) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                  for (int q = 0; q < 2; ++q)
                    step(d0 + (kk & (il - 1)) * il_cols + q * g.n1 + n0, a0 + q * (few_tile(MX) >> 4) + kk * kAStep,
                         bn + kk * (32u >> 4), idesc, q, kk, region + 16 + 4 * nblk * (kk >> 1) + n0 / 32, region,
                         begun || kk >= il);
              } else {
                for (int q = 0; q < ns; ++q)
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk)
                    step(d0 + (kk & (il - 1)) * il_cols + n0, a0 + q * (few_tile(MX) >> 4) + kk * kAStep,
                         bn + q * ((g.n2 * kSubBytes) >> 4) + kk * (32u >> 4), idesc, q, kk,
                         region + 16 + 4 * nblk * (2 * q + (kk >> 1)) + n0 / 32, region, begun || q > 0 || kk >= il);
              }
            }
            umma_commit(c->empty + s);
          }
          __syncwarp();
        }
        if (elect_one()) umma_commit(c->tfull + buf);
        __syncwarp();
      }
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ tokens
    const int ct = threadIdx.x - 64;
    bool ok = true;
    FewGeo g = few_geo(p.P1, p.P2, p.T, min(p.T, p.mcap), MX);
    for (int ph = first_phase; ph < 5 && ok; ++ph) {
      const unsigned* counter = nullptr;
      unsigned want = 0;
      if (ph == 1) {
        if (!warp_wait(&c->plan, 0, c, p, 89)) break;
        g = c->geo;
      }
      FewWalk w(ph, p, g, ph == 0 ? 0 : c->nact, blockIdx.x, G);
      if (ph == 0 && MX) {  // the parts of x come from all blocks
        counter = p.sync;
        want = gridDim.x;
      } else if (ph == 3) {  // the activations of phases 0 and 1
        counter = p.sync + 2;
        want = p.nsh * p.ns1s + few_half(c->nact, MX) * p.ns1;
      } else if (ph == 4) {
        counter = p.sync + 3;
        want = (c->nact - few_half(c->nact, MX)) * p.ns1;
      }
      if (counter != nullptr && w.u < w.u1) {
        if (lane == 0) ok = wait_count(counter, want, c, p, 90);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok) break;
      }
      FewChunk ch;
      const int parts = w.down ? p.P2 : p.P1;
      while (ok && w.next(ch)) {
        const bool sh = ch.i < 0;
        const FewRows rw(p, c, ch.i);
        const int m = rw.m, rows = parts * m;
        // bytes of a row of the operand and of its scales
        const int width = !w.down ? p.H : sh ? p.Fs : p.F, len = MX ? width >> 1 : 2 * width;
        const uint8_t* base = !w.down ? (MX ? p.xq : reinterpret_cast<const uint8_t*>(p.x)) : sh ? p.as : p.a;
        const uint8_t* sf = !w.down ? p.x_sf : sh ? p.as_sf : p.a_sf;
        // column n of the operand is row j's part n / m: the source's row, once a chunk
        // (each of the two warps has a table: no barrier that one of them might not reach)
        uint16_t* table = c->rows[warp - 2];
        __syncwarp();
        for (int r = lane; r < rows; r += 32) {
          const int part = r / m, j = r - part * m;
          table[r] = static_cast<uint16_t>((!w.down && !sh ? c->tok[rw.r0 + j] : rw.r0 + j) * parts + part);
        }
        __syncwarp();
        const int nsb = sh ? p.nsb2s : p.nsb2;
        for (int kb = ch.kb; kb < ch.kb + ch.nkb; ++kb, ++n) {
          const int s = n % g.nst;
          if (!warp_wait(c->empty + s, ((n / g.nst) & 1) ^ 1, c, p, 91)) {
            ok = false;
            break;
          }
          uint32_t sB = smem_u32(smem) + s * g.stage + 2 * few_tile(MX);
          uint32_t sS = sB + g.b_bytes;
          const int sb0 = w.down ? kb * kFewSub2 : kb, ns = w.down ? min(kFewSub2, nsb - sb0) : 1;
          for (int q = 0; q < ns; ++q) {
            // thread: 16-byte chunk ct % 8 of rows ct / 8, + 8, ..; zeros beyond a row's end
            const int at = (sb0 + q) * kSubBytes + (ct & 7) * 16;
            const bool in = at < len;
            const uint8_t* src = base + (in ? at : 0);
            const uint32_t dst = sB + (ct >> 3) * 128 + (((ct & 7) ^ ((ct >> 3) & 7)) << 4);
            for (int r = ct >> 3, i = 0; r < rows; r += 8, ++i)
              cp_async16(dst + i * 1024, src + static_cast<size_t>(table[r]) * len, in);
            if constexpr (MX) {
              const int slen = len >> 4, nblk = w.down ? g.nblk2 : g.nblk1;
              const int half = ct & 1, b = (sb0 + q) * 8 + half * 4;
              const uint8_t* ssrc = sf + (b < slen ? b : 0);
              for (int r = ct >> 1; r < rows; r += kFewCopiers / 2)
                cp_async4(sS + kFewSf * (nblk * half + (r >> 7)) + 16 * (r & 31) + 4 * ((r >> 5) & 3),
                          ssrc + static_cast<size_t>(table[r]) * slen, b < slen);
              sS += 2 * kFewSf * nblk;
            }
            sB += g.n2 * kSubBytes;
          }
          cp_async_arrive(c->full + s);
        }
      }
    }
    cp_async_wait_all();
  } else {
    // ------------------------------------------------------------ router, epilogue
    const int et = threadIdx.x - 128, q4 = warp & 3, half = (warp - 4) >> 2;
    const int row = 32 * q4 + lane;  // the thread's column of the weight tile (TMEM lane)
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * q4) << 16);
    bool ok = few_route<MX>(p, c, et);
    if (ok && et == 0) mbar_arrive(&c->plan);
    int used[2] = {0, 0};
    const FewGeo g = c->geo;
    float* acc = reinterpret_cast<float*>(smem + g.acc_off);
    unsigned* cnt = p.cnt;
    const bool halved = ok && few_half(c->nact, MX) < c->nact;
    for (int ph = first_phase; ph < 5 && ok; ++ph) {
      FewWalk w(ph, p, g, ph == 0 ? 0 : c->nact, blockIdx.x, G);
      FewChunk ch;
      const int nbuf = w.down ? g.nbuf2 : g.nbuf1;
      const int il = w.down ? g.il2 : g.il1, il_cols = w.down ? g.n2 : 2 * g.n1;
      const int acc_cols = il * il_cols;
      const int parts = w.down ? p.P2 : p.P1;
      int na = 0;
      while (ok && w.next(ch)) {
        const FewRows rw(p, c, ch.i);
        const int m = rw.m;
        const int buf = na % nbuf;
        ++na;
        if (w.down && ch.first) {
          for (int i = et; i < p.T * 32; i += kFewEpi) reinterpret_cast<float4*>(acc)[i] = make_float4(0, 0, 0, 0);
          epi_sync();
        }
        ok = epi_all(mbar_wait_bounded(c->tfull + buf, used[buf] & 1, abort_flag, p.lim, p.status, 92));
        if (!ok) break;
        ++used[buf];
        tc_fence_after();
        const uint32_t d0 = tl + buf * acc_cols + (w.down ? 0 : half * g.n1);
        for (int j0 = w.down ? 8 * half : 0; j0 < m; j0 += w.down ? 16 : 8) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = 0.0f;
          // every part's columns in every accumulator, four reads on their way at a time
          for (int q = 0; q < parts; ++q) {
            uint32_t r[4][8];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < il) tmem_ld8(d0 + k * il_cols + q * m + j0, r[k]);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < il)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += __uint_as_float(r[k][j]);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (j0 + j < m) {
              if (!w.down) {
                float* a = acc + (j0 + j) * 256 + half * 128 + row;
                *a = ch.first ? v[j] : *a + v[j];
              } else {
                acc[(ch.i < 0 ? rw.r0 + j0 + j : c->tok[rw.r0 + j0 + j]) * 128 + row] += v[j];
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(c->tempty + buf);
        epi_sync();
        if (!ch.last) continue;
        const int ti = w.tile_index(), n = w.down ? p.T * 128 : m * 256, me = blockIdx.x;
        const FewPieces pc = w.pieces(ti);
        const size_t stride = static_cast<size_t>(p.T) * (w.down ? 128 : 256);
        const bool early = ph == 3 && halved;  // joined in the next phase
        if (early || me != pc.c0) {
          few_leave(acc, n, p.part[ph] + (early ? me + ti : me) * stride, cnt + ti, et);
        } else {
          FewPieces pa{0, -1};
          if (ph == 4) pa = FewWalk(3, p, g, c->nact, 0, G).pieces(ti);
          const int na = pa.c1 - pa.c0 + 1, nb = pc.c1 - pc.c0;
          if (na + nb > 0) ok = few_join(acc, n, stride, p.part[3], pa.c0 + ti, na, p.part[ph], me + 1, nb, cnt + ti, c, p, et);
          if (!ok) break;
          if (!w.down) {
            few_activate<MX>(p, c, acc, rw, ch.i, ch.tile, et);
          } else {
            for (int i = et; i < n; i += kFewEpi) few_store_y(p, i >> 7, 128 * ch.tile + (i & 127), acc[i]);
          }
        }
        epi_sync();
        if (!w.down && me == pc.c0 && et == 0) red_release(p.sync + (ph == 2 ? 3 : 2), 1u);
      }
      // the counters of the next phase's tiles; both phases of W2 share theirs
      const int half = few_half(c->nact, MX);
      cnt += ph == 0 ? p.nsh * p.ns1s : ph == 1 ? half * p.ns1 : ph == 2 ? (c->nact - half) * p.ns1 : 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) few_drain<MX>(p, c, n);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0) {
    // the last block to end leaves the counters at 0, as it found them
    __threadfence();
    if (atomicAdd(p.sync + 4, 1u) == gridDim.x - 1) {
      for (int i = 0; i < 5; ++i) p.sync[i] = 0u;
    }
  }
}

}  // namespace

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
static size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

// Where things lie in the workspace
struct FewLayout {
  size_t logits, cnt, part[5], a, as, a_sf, as_sf, xq, x_sf, total;
  int cnt_words;
};
static FewLayout few_layout(const moe_config& c, bool mx, int G) {
  FewLayout L{};
  const size_t T = c.T, R = T * c.k, F = c.F, Fs = c.F_shared, H = c.H, P2 = few_parts2(mx, c.out_fp32);
  const size_t P1 = few_parts1(mx, c.out_fp32);
  size_t o = sizeof(DevStatus);
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += up256(bytes);
    return at;
  };
  // (the shared expert has at most as many entries as tokens)
  L.cnt_words = c.T * ((c.F_shared + 127) / 128) + kFewMaxEnt * ((c.F + 127) / 128) + (c.H + 127) / 128;
  L.logits = take(4 * T * c.E);
  L.cnt = take(4 * static_cast<size_t>(L.cnt_words));
  // a phase's partial sums: a slot a block, in phase 3 another for each of its tiles
  const bool halves = c.T * c.k >= kFewHalve;
  for (int ph = 0; ph < 5; ++ph) {
    const bool used = ph == 0 ? Fs > 0 : (ph & 1) || halves;
    const size_t slots = static_cast<size_t>(G) + (ph == 3 ? (c.H + 127) / 128 : 0);
    L.part[ph] = take(used ? slots * T * (ph < 3 ? 256 : 128) * 4 : 0);
  }
  L.a = take(mx ? R * P2 * F / 2 : R * P2 * F * 2);
  L.as = take(mx ? T * P2 * Fs / 2 : T * P2 * Fs * 2);
  if (mx) {
    L.a_sf = take(R * P2 * F / 32);
    L.as_sf = take(T * P2 * Fs / 32);
    L.xq = take(T * P1 * H / 2);
    L.x_sf = take(T * P1 * H / 32);
  }
  L.total = o;
  return L;
}

size_t few_workspace_bytes(const moe_config& c, bool mx) { return few_layout(c, mx, num_sms()).total; }

template <bool MX>
static cudaError_t few_start(const FewParams& p, const FewMaps& maps, cudaStream_t st) {
  static std::atomic<unsigned long long> set{0};  // devices whose kernel has its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(set.load() & bit)) {
    e = cudaFuncSetAttribute(few_kernel<MX>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem);
    if (e != cudaSuccess) return e;
    set.fetch_or(bit);
  }
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeCooperative;  // the blocks wait for one another
  attr.val.cooperative = 1;
  cfg.gridDim = dim3(num_sms());
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = kFewSmem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few_kernel<MX>, p, maps);
}

int run_few(const moe_config& c, const FewArgs& q, bool mx, void* ws, cudaStream_t st) {
  const int G = num_sms();
  const FewLayout L = few_layout(c, mx, G);
  uint8_t* base = static_cast<uint8_t*>(ws);
  FewParams p{};
  p.T = c.T; p.H = c.H; p.E = c.E; p.k = c.k; p.F = c.F; p.Fs = c.F_shared;
  const bool grouped = !c.force_balanced && c.n_groups > 1 && c.topk_groups < c.n_groups;
  const bool softmax = c.score == MOE_SCORE_SOFTMAX;
  p.mode = !softmax ? RSEL_SIGMOID : ((q.expert_bias == nullptr && !grouped) ? RSEL_LOGIT : RSEL_SOFTMAX);
  p.groups = grouped ? c.n_groups : 1;
  p.topk_groups = c.topk_groups;
  p.force = c.force_balanced;
  p.gate_scale = c.gate_scale;
  p.P1 = few_parts1(mx, c.out_fp32);
  p.P2 = few_parts2(mx, c.out_fp32);
  p.mx = mx ? 1 : 0;
  p.mcap = few_mcap(p.P1, mx);
  p.nsh = c.F_shared ? (c.T + p.mcap - 1) / p.mcap : 0;
  p.msh = p.nsh ? (c.T + p.nsh - 1) / p.nsh : 0;
  const int ks = mx ? 256 : 64;
  // the tensor cores' sums round towards zero: fp32 results take them in chains of 128
  // products (512 under block scales, which lose less), joined in fp32: 4e-7 of the
  // result, 1.4e-6 with chains of 512
  p.chain = c.out_fp32 ? (mx ? 512 : 128) : 1 << 24;
  p.ks = ks;
  p.out_fp32 = c.out_fp32;
  p.ns1 = (c.F + 127) / 128;
  p.ns1s = (c.F_shared + 127) / 128;
  p.ns2 = (c.H + 127) / 128;
  p.nsb1 = (c.H + ks - 1) / ks;
  p.nsb2 = (c.F + ks - 1) / ks;
  p.nsb2s = (c.F_shared + ks - 1) / ks;
  p.x = q.x; p.wr = q.router_w; p.eb = q.expert_bias; p.lb = q.logit_bias;
  p.idx = q.topk_idx; p.gate = q.topk_gate; p.y = q.y;
  p.status = reinterpret_cast<DevStatus*>(base);
  p.sync = reinterpret_cast<unsigned*>(base + 64);
  p.logits = reinterpret_cast<float*>(base + L.logits);
  p.cnt = reinterpret_cast<unsigned*>(base + L.cnt);
  p.cnt_words = L.cnt_words;
  for (int ph = 0; ph < 5; ++ph) p.part[ph] = reinterpret_cast<float*>(base + L.part[ph]);
  p.a = base + L.a; p.as = base + L.as; p.a_sf = base + L.a_sf; p.as_sf = base + L.as_sf;
  p.xq = base + L.xq; p.x_sf = base + L.x_sf;
  p.lim = wait_limit_ns();
  p.fault = debug_fault();
  FewMaps maps;
  memset(&maps, 0, sizeof(maps));
  bool ok = true;
  if (mx) {
    const moe_mx4_weights& w = *q.mx4;
    p.w13 = w.w13; p.w2 = w.w2; p.w13s = w.w13s; p.w2s = w.w2s;
  } else {
    const uint64_t E = c.E, H = c.H, F = c.F, Fs = c.F_shared;
    ok = make_map_bf16(&maps.m[0], q.W1, F, E * H, 2 * F, 64, 64) && make_map_bf16(&maps.m[1], q.W3, F, E * H, 2 * F, 64, 64) &&
         make_map_bf16(&maps.m[2], q.W2, H, E * F, 2 * H, 64, 64);
    if (Fs)
      ok = ok && make_map_bf16(&maps.m[3], q.Ws1, Fs, H, 2 * Fs, 64, 64) &&
           make_map_bf16(&maps.m[4], q.Ws3, Fs, H, 2 * Fs, 64, 64) && make_map_bf16(&maps.m[5], q.Ws2, H, Fs, 2 * H, 64, 64);
  }
  if (!ok) return MOE_ERR_CUDA;
  return status_from_cuda(mx ? few_start<true>(p, maps, st) : few_start<false>(p, maps, st));
}

}  // namespace moe

using namespace moe;

static int check_few(const moe_config* cfg, bool mx) {
  const int s = validate_config(cfg);
  if (s != MOE_OK) return s;
  const int unit = mx ? 128 : 64;
  if (cfg->T > MOE_FEW_MAX_T || cfg->H % unit || cfg->F % unit || cfg->F_shared % unit) return MOE_ERR_UNSUPPORTED_SHAPE;
  // tile and unit counts stay within 32 bits
  if (cfg->H > (1 << 17) || cfg->F > (1 << 17) || cfg->F_shared > (1 << 17)) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}
static bool few_aligned(std::initializer_list<const void*> ps, uintptr_t to) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) & (to - 1)) return false;
  return true;
}
// bytes of what a call reads and writes: outputs may overlap nothing else, but y may be x
struct FewArray {
  const void* p;
  size_t bytes;
};
static int few_call(const moe_config* cfg, const FewArgs& q, bool mx, void* ws, size_t ws_bytes, void* stream) {
  const moe_config& c = *cfg;
  if (!q.x || !q.router_w || !q.topk_idx || !q.topk_gate || !q.y || !ws) return MOE_ERR_INVALID_ARG;
  if (!few_aligned({q.x, q.router_w, q.expert_bias, q.logit_bias, q.topk_idx, q.topk_gate, q.y, ws}, 16))
    return MOE_ERR_INVALID_ARG;
  const size_t need = few_workspace_bytes(c, mx);
  const size_t TH = static_cast<size_t>(c.T) * c.H, Tk = 4 * static_cast<size_t>(c.T) * c.k, HF = static_cast<size_t>(c.H) * c.F;
  const size_t HFs = static_cast<size_t>(c.H) * c.F_shared;
  const FewArray out[4] = {{q.y, TH * (c.out_fp32 ? 4 : 2)}, {q.topk_idx, Tk}, {q.topk_gate, Tk}, {ws, need}};
  FewArray in[10] = {{q.x, 2 * TH}, {q.router_w, 2 * static_cast<size_t>(c.E) * c.H}, {q.expert_bias, 4ull * c.E},
                     {q.logit_bias, 4ull * c.E}, {q.W1, 2 * c.E * HF}, {q.W3, 2 * c.E * HF}, {q.W2, 2 * c.E * HF},
                     {c.F_shared ? q.Ws1 : nullptr, 2 * HFs}, {c.F_shared ? q.Ws3 : nullptr, 2 * HFs},
                     {c.F_shared ? q.Ws2 : nullptr, 2 * HFs}};
  if (mx) {
    const uint8_t* w[4] = {q.mx4->w13, q.mx4->w2, c.F_shared ? q.mx4->w13s : nullptr, c.F_shared ? q.mx4->w2s : nullptr};
    for (int i = 0; i < 4; ++i) in[4 + i] = FewArray{w[i], moe_mx4_weight_bytes(cfg, i)};
  }
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return MOE_ERR_INVALID_ARG;
    for (int j = 0; j < 10; ++j)
      if (overlap(out[i].p, out[i].bytes, in[j].p, in[j].bytes) && !(i == 0 && j == 0 && q.y == q.x && !c.out_fp32))
        return MOE_ERR_INVALID_ARG;
  }
  if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int r = run_few(c, q, mx, ws, s);
  if (r == MOE_OK) record_stage(s, 50, 1);
  return r;
}

extern "C" {

size_t moe_few_workspace_bytes(const moe_config* cfg, int mxfp4) {
  return check_few(cfg, mxfp4 != 0) != MOE_OK ? 0 : few_workspace_bytes(*cfg, mxfp4 != 0);
}

int moe_layer_few_fwd(const moe_config* cfg, const moe_bf16* x, const moe_bf16* router_w, const float* expert_bias,
                      const float* logit_bias, const moe_bf16* W1, const moe_bf16* W3, const moe_bf16* W2,
                      const moe_bf16* Ws1, const moe_bf16* Ws3, const moe_bf16* Ws2, int32_t* topk_idx,
                      float* topk_gate, void* y, void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nvtx("moe_layer_few_fwd");
  const int s = check_few(cfg, false);
  if (s != MOE_OK) return s;
  if (!W1 || !W3 || !W2 || (cfg->F_shared && (!Ws1 || !Ws3 || !Ws2))) return MOE_ERR_INVALID_ARG;
  if (!few_aligned({W1, W3, W2, Ws1, Ws3, Ws2}, 16)) return MOE_ERR_INVALID_ARG;
  auto b = [](const moe_bf16* v) { return reinterpret_cast<const __nv_bfloat16*>(v); };
  const FewArgs q{b(x), b(router_w), expert_bias, logit_bias, b(W1), b(W3), b(W2), b(Ws1), b(Ws3), b(Ws2), nullptr,
                  topk_idx, topk_gate, y};
  return few_call(cfg, q, false, ws, ws_bytes, stream);
}

int moe_layer_few_fwd_mxfp4(const moe_config* cfg, const moe_bf16* x, const moe_bf16* router_w,
                            const float* expert_bias, const float* logit_bias, const moe_mx4_weights* w,
                            int32_t* topk_idx, float* topk_gate, void* y, void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nvtx("moe_layer_few_fwd_mxfp4");
  const int s = check_few(cfg, true);
  if (s != MOE_OK) return s;
  if (!w || !w->w13 || !w->w2 || (cfg->F_shared && (!w->w13s || !w->w2s))) return MOE_ERR_INVALID_ARG;
  if (!few_aligned({w->w13, w->w2, w->w13s, w->w2s}, 16)) return MOE_ERR_INVALID_ARG;
  auto b = [](const moe_bf16* v) { return reinterpret_cast<const __nv_bfloat16*>(v); };
  const FewArgs q{b(x), b(router_w), expert_bias, logit_bias, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, w,
                  topk_idx, topk_gate, y};
  return few_call(cfg, q, true, ws, ws_bytes, stream);
}

}  // extern "C"
