// The whole MoE layer for a few tokens (T <= 64) in one cooperative kernel:
// types and schedule shared by the kernel (few.cu) and its host side.
//
//   y[t] = sum_{e in topk(t)} g[t,e] (SiLU(x[t] W1_e) * (x[t] W3_e)) W2_e (+ shared expert)
//
// What bounds it is the weights of the selected experts, read once each: at one
// token of a 128-expert layer 302 MB of bf16, 80 MB of MXFP4. So the weights are
// the M operand of the tensor cores (128 output columns a tile), the few tokens
// the N operand, and everything is arranged so that the stream of weight tiles
// never stops:
//  - the units of a phase (one weight tile of 32 KB each in shared memory) are
//    dealt to the blocks in equal contiguous runs, whatever the experts' number;
//    a tile cut by a run's border is joined from fp32 partials by whichever of
//    its blocks comes last, always in the blocks' order;
//  - one thread copies weights (TMA) as far ahead as the ring of stages allows,
//    over the borders of tiles and phases: while the blocks wait for one another
//    between the phases, the next phase's weights are already on their way;
//  - the tokens' operand follows by 16-byte copies of two other warps as soon as
//    it exists.
//
// Phases: 0 the shared expert's gate and up products (needs no routing: its
// weights stream while the router works), 1 the routed experts', 2 all down
// products. A stage of phases 0 and 1 holds one k sub-block (128 bytes: 64 bf16,
// 128 MXFP4 elements) of 128 columns of W1 and of W3, a stage of phase 2 up to two
// sub-blocks of 128 columns of W2.
//
// Operands: bf16 weights multiply bf16 parts of the tokens (x itself; the
// activation a in two parts, three for fp32 results: 2^-17 and 2^-25 of a).
// MXFP4 weights (E2M1 with a power of two for 32 elements along k) multiply E4M3
// parts of the tokens, each with its own power of two for 32 elements: x in two
// parts, which hold a bf16 exactly unless it lies 2^-15 below its block's maximum
// (2^-22 of that maximum then); a in three (2^-12), five for fp32 results (2^-20).
// The parts are further columns of the N operand, of which the tensor cores have
// plenty to spare.
#pragma once
#include "host_util.h"
#include "mma.cuh"

namespace moe {

constexpr int kFewMaxT = 64;
constexpr int kFewThreads = 384;   // warp 0 weights, 1 MMA, 2-3 tokens, 4-11 router and epilogue
constexpr int kFewEpi = 256;
constexpr int kFewCopiers = 64;
constexpr int kFewStages = 8;      // at most
constexpr int kFewMaxR = kFewMaxT * 16;
constexpr int kFewATile = 16384;   // 128 columns x 128 bytes
constexpr int kFewABytes = 2 * kFewATile;
constexpr int kFewSmem = 232448;   // 227 KB
constexpr int kFewRedundant = 16;  // tokens up to which every block selects for itself

// A block's own plan of the batch (shared memory)
struct FewCtl {
  uint64_t full[kFewStages], empty[kFewStages], tfull[2], tempty[2], plan, drain;
  uint32_t tmem;
  int abort;
  int nact, mmax;            // experts with rows, most rows of one (shared expert: T)
  int flag;
  int warp_sum[8], warp_act[8], warp_max[8];
  int off[257];              // first row of active expert i
  uint8_t act[256];          // expert of active expert i
  uint8_t tok[kFewMaxR];     // row -> token
  float gate[kFewMaxR];      // row -> gate
  uint8_t eidx[kFewMaxR];    // slot (token-major) -> expert
  float sgate[kFewMaxR];     // slot -> gate
  float scratch[8][256];     // a warp's selection values; the router's partial sums
};
constexpr int kFewCtl = (sizeof(FewCtl) + 1023) / 1024 * 1024;
constexpr int kFewCtlOff = kFewSmem - kFewCtl;

struct FewParams {
  int T, H, E, k, F, Fs;
  int mode, groups, topk_groups, force;  // router (RouterSelMode)
  float gate_scale;
  int P1, P2;                // parts of x and of a
  int flush;                 // most products accumulated in tensor memory, in k sub-blocks
  int out_fp32;
  int ns1, ns1s, ns2;        // tiles of 128 columns: F, Fs, H
  int nsb1, nsb2, nsb2s;     // k sub-blocks: H, F, Fs
  const __nv_bfloat16 *x, *wr;
  const float *eb, *lb;
  int32_t* idx;
  float* gate;
  void* y;
  float* logits;             // [T, E]
  unsigned* sync;            // barrier 1, barrier 2, finished tiles, ended blocks
  unsigned* cnt;             // arrivals of a cut tile: phase 0, 1, 2
  int cnt_words;
  float *part0, *part1, *part2;
  uint8_t *a, *as;           // parts of the activations: rows x parts x (F or Fs)
  uint8_t *a_sf, *as_sf;     // MXFP4: their scale bytes
  uint8_t *xq, *x_sf;        // MXFP4: parts of x and their scale bytes
  const uint8_t *sf13, *sf2, *sf13s, *sf2s;
  DevStatus* status;
  unsigned long long lim;
};
struct FewMaps {
  CUtensorMap m[6];          // W1, W3, W2, Ws1, Ws3, Ws2; MXFP4: w13, -, w2, ws13, -, ws2
};

// What a stage holds and how many there are, from the largest number of rows
struct FewGeo {
  int n1, n2;                // columns of an expert's N operand, at most
  int sub2;                  // sub-blocks of a phase 2 stage
  int b_bytes, nblk1, nblk2, stage, nst;
  int acc_off;               // fp32 sums in shared memory
  int nbuf1, nbuf2;          // accumulators in tensor memory
};
__host__ __device__ __forceinline__ int few_cols(int parts, int m) { return (parts * ((m + 7) & ~7) + 15) & ~15; }
__host__ __device__ __forceinline__ FewGeo few_geo(int P1, int P2, int T, int mmax, bool mx) {
  FewGeo g;
  g.n1 = few_cols(P1, mmax);
  g.n2 = few_cols(P2, mmax);
  // two sub-blocks of W2 a stage unless the tokens' side outgrows the weights'
  g.sub2 = 2 * g.n2 * 128 <= kFewATile ? 2 : 1;
  g.b_bytes = 128 * (g.n1 > g.sub2 * g.n2 ? g.n1 : g.sub2 * g.n2);
  g.nblk1 = (g.n1 + 127) >> 7;
  g.nblk2 = (g.n2 + 127) >> 7;
  const int sfb = 512 * (g.nblk1 > g.sub2 * g.nblk2 ? g.nblk1 : g.sub2 * g.nblk2);
  g.stage = kFewABytes + g.b_bytes + (mx ? (1024 + sfb + 1023) / 1024 * 1024 : 0);
  const int acc = mmax * 1024 > T * 512 ? mmax * 1024 : T * 512;
  g.acc_off = kFewCtlOff - (acc + 1023) / 1024 * 1024;
  g.nst = g.acc_off / g.stage;
  if (g.nst > kFewStages) g.nst = kFewStages;
  const int cols = mx ? 448 : 512;  // the rest holds scales
  g.nbuf1 = 4 * g.n1 <= cols ? 2 : 1;
  g.nbuf2 = 2 * g.n2 <= cols ? 2 : 1;
  return g;
}

// Equal contiguous runs of U units over G blocks
struct FewSplit {
  int U, G;
  __host__ __device__ __forceinline__ int start(int c) const {
    return static_cast<int>(static_cast<long long>(U) * c / G);
  }
  // the block that has unit u
  __host__ __device__ __forceinline__ int owner(int u) const {
    return static_cast<int>(((static_cast<long long>(u) + 1) * G - 1) / U);
  }
  // blocks that share units [u0, u1): all blocks owner(u0) .. owner(u1 - 1) with a unit
  __host__ __device__ __forceinline__ int pieces(int u0, int u1) const {
    const int a = owner(u0), b = owner(u1 - 1);
    int n = 0;
    for (int c = a; c <= b; ++c) n += start(c + 1) > start(c) ? 1 : 0;
    return n;
  }
};

// A run of k blocks of one tile and one expert, accumulated at once
struct FewChunk {
  int i;       // active expert; -1: the shared one
  int tile;    // 128-column tile: of F (phases 0 and 1), of H (phase 2)
  int kb, nkb; // first stage of the expert's k, stages
  bool first, last;  // of this block's segment of the tile
};

// A block's share of a phase, chunk by chunk; every role walks it by itself.
struct FewWalk {
  FewSplit s;
  int phase, u, u0, u1;
  int kbs, kbr, per;   // stages of the shared expert's and a routed expert's k, of a tile
  int ns, flush;
  __host__ __device__ __forceinline__ FewWalk(int ph, const FewParams& p, const FewGeo& g, int nact, int c, int G) {
    phase = ph;
    if (ph < 2) {
      ns = ph == 0 ? p.ns1s : p.ns1;
      per = p.nsb1;
      s.U = (ph == 0 ? 1 : nact) * ns * per;
      kbs = kbr = per;
      flush = p.flush;
    } else {
      ns = p.ns2;
      kbr = (p.nsb2 + g.sub2 - 1) / g.sub2;
      kbs = p.Fs ? (p.nsb2s + g.sub2 - 1) / g.sub2 : 0;
      per = kbs + nact * kbr;
      s.U = ns * per;
      flush = p.flush / g.sub2;
    }
    s.G = G;
    u = u0 = s.start(c);
    u1 = s.start(c + 1);
  }
  __host__ __device__ __forceinline__ bool next(FewChunk& c) {
    if (u >= u1) return false;
    const int t = u / per, r = u - t * per;
    int lim;
    if (phase < 2) {
      c.i = phase == 0 ? -1 : t / ns;
      c.tile = phase == 0 ? t : t - c.i * ns;
      c.kb = r;
      lim = per - r;
    } else {
      c.tile = t;
      if (r < kbs) {
        c.i = -1;
        c.kb = r;
        lim = kbs - r;
      } else {
        c.i = (r - kbs) / kbr;
        c.kb = r - kbs - c.i * kbr;
        lim = kbr - c.kb;
      }
    }
    if (lim > u1 - u) lim = u1 - u;
    if (lim > flush) lim = flush;
    c.nkb = lim;
    c.first = u == u0 || r == 0;
    u += lim;
    c.last = u == u1 || r + lim == per;
    return true;
  }
  // the tile that the chunk just walked belongs to: index in the phase, first unit
  __host__ __device__ __forceinline__ int tile_index() const { return (u - 1) / per; }
};

}  // namespace moe
