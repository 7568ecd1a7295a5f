// The whole MoE layer for a few tokens (T <= 64) in one cooperative kernel:
// types and schedule shared by the kernel (few.cu) and its host side.
//
//   y[t] = sum_{e in topk(t)} g[t,e] (SiLU(x[t] W1_e) * (x[t] W3_e)) W2_e (+ shared expert)
//
// What bounds it is the weights of the selected experts, read once each: at one
// token of a 128-expert layer 302 MB of bf16, 80 MB of MXFP4. So the weights are
// the M operand of the tensor cores (128 output columns a tile), the few tokens
// the N operand, and everything is arranged so that the stream of weight tiles
// goes on from the first to the last, as far as the ring of stages holds them:
//  - the units of a phase (one weight tile of 32 KB each in shared memory) are
//    dealt to the blocks in equal contiguous runs, whatever the experts' number;
//    a tile cut by a run's border is joined from fp32 partials by the block that has its
//    beginning, in the blocks' order. The others have theirs at the start of their
//    runs, so that the partials are mostly there when they are wanted: the end of a
//    phase is then four trips to L2 (a partial, the activations there and back, a
//    count), 9 us of 71 less for one token than with the last block to arrive joining;
//  - one thread copies weights (TMA) as far ahead as the ring of stages allows,
//    over the borders of tiles and phases: while the blocks wait for one another
//    between the phases, the next phase's weights are already on their way;
//  - the tokens' operand follows by 16-byte copies of two other warps as soon as
//    it exists.
// A stage holds both, and is as large as the entry with most rows wants, in every phase
// (few_geo); with a shared expert that is min(T, mcap) rows whatever the routing, more than its
// entries have where there are several. Four stages become two from 41 rows on (fp32 results 33;
// MXFP4 weights 20, with fp32 results 13) and one from 54 rows with fp32 results, under MXFP4
// from 36 (25): then no weights are on their way during a stage's MMAs. 32 experts of 4096 x 1536 with a
// shared expert of that size, and without: 64 tokens 245 and 220 us, fp32 results 459 and 271; MXFP4
// weights, 40 tokens 167 and 119, 64 tokens 195 and 158, fp32 results 313 and 273 (the shared
// expert's weights themselves are 6 us, 1.5 in MXFP4).
//
// Phases: 0 the shared expert's gate and up products (needs no routing: its weights
// stream while the router works); 1 and 2 those of the first and second half of the
// routed entries; 3 the down products of the shared expert and the first half, 4 those of
// the second. So a half's activations are joined and finished while the other half's
// weights stream. Few entries (one token: eight) are not halved (few_half): phases 2 and 4 are
// empty then, since a half would end before the other's activations are there. A stage of
// phases 0 to 2 holds one k sub-block (128 bytes: 64 bf16, 256 MXFP4 elements) of 128
// columns of W1 and of W3, a stage of phases 3 and 4 up to two sub-blocks of 128 columns of W2.
//
// Measured, 128 experts of 4096 x 1536, eight a token: one token 68 us (302 MB: 4.4 TB/s; the
// router and the plan take 10, the ends of the two phases 6 and 3, during which little is
// read), 8 tokens 295, 61 tokens 699 (4.74 GB: 6.8 TB/s, as fast as memory is read);
// with MXFP4 weights one token 40 (80 MB: 2.0 TB/s), 33 tokens 207 (1.1 GB: 5.4 TB/s, a unit's
// eight small MMAs and their scales take 0.4 of its 0.7 us).
//
// Operands: bf16 weights multiply bf16 parts of the tokens (x itself; the activation
// a in two parts, three for fp32 results: 2^-17 and 2^-25 of a). MXFP4 weights stay
// packed, two to a byte, in shared memory: the block-scaled MMA takes them with E2M1
// tokens, a power of two for 32 elements on either side. So x and a enter as sums of E2M1
// parts, every part with its own powers of two: a part leaves at most half the largest
// step of the one before, 3 bits a part, 2^-12 of a block's unit after five (2^-21 after
// eight, for fp32 results), 2^-13 of its largest element: elements below a sixteenth of that
// keep fewer bits than bf16 has (after eight, below 2^-13 of it). The parts are further columns of the N operand, of which the
// tensor cores have plenty to spare. (Unpacked 4-bit weights with E4M3 tokens need fewer
// parts, but the copies that unpack move 8 bytes a cycle: 2.5 TB/s over all SMs.)
#pragma once
#include "host_util.h"
#include "mma.cuh"

namespace moe {

constexpr int kFewMaxT = 64;
constexpr int kFewThreads = 384;   // warp 0 weights, 1 MMA, 2-3 tokens, 4-11 router and epilogue
constexpr int kFewEpi = 256;
constexpr int kFewCopiers = 64;
constexpr int kFewStages = 4;      // at most (8 tokens: three 301, four 295.7, five 295.6 us; one token 69.1, 68.1, 68.2)
constexpr int kFewMaxR = kFewMaxT * 16;
constexpr int kFewMaxEnt = 320;    // runs of rows of one expert
constexpr int kFewSub2 = 2;        // k sub-blocks of a stage of W2, as many tiles as one of W1 and W3 (one: 8 tokens 319 us
                                   // for 295, 33 with MXFP4 weights 227 for 209)
constexpr int kFewATile = 16384;   // 128 columns x 128 bytes
constexpr int kFewSf = 512;        // scales of 128 columns (rows) x 128 MXFP4 elements
constexpr int kFewSmem = 232448;   // 227 KB
// tokens up to which every block selects for itself, without a second wait of all blocks for one
// another (128 experts, one token 68.2 us for 70.4, 8 295.6 for 296.1; 12 tokens 388.3 for 387.9, 24 556 for 553)
constexpr int kFewRedundant = 8;

// What a stage holds and how many there are, from the largest number of rows
struct FewGeo {
  int n1, n2;                // columns of an expert's N operand, at most
  int b_bytes, nblk1, nblk2, stage, nst;
  int acc_off;               // fp32 sums in shared memory
  int il1, il2;              // accumulators that the steps along k take in turn
  int nbuf1, nbuf2;          // chunks in tensor memory at a time
};
// A block's own plan of the batch (shared memory)
struct FewCtl {
  uint64_t full[kFewStages], empty[kFewStages], tfull[2], tempty[2], plan, drain;
  uint32_t tmem;
  int abort;
  int nact;                  // entries: runs of rows of one expert
  int stages;                // that a block has begun which gave up
  int warp_sum[8], warp_act[8], warp_max[8];
  uint32_t has[256][2];      // expert -> its tokens
  int eoff[256];             // expert -> its first row
  int off[kFewMaxEnt + 1];   // first row of entry i
  uint8_t act[kFewMaxEnt];   // its expert
  uint8_t tok[kFewMaxR];     // row -> token
  float gate[kFewMaxR];      // row -> gate
  uint8_t eidx[kFewMaxR];    // slot (token-major) -> expert
  float sgate[kFewMaxR];     // slot -> gate
  uint16_t rows[2][448];     // a copying warp's chunk: column of the N operand -> row of its source
  float scratch[8][256];     // a warp's selection values; the router's partial sums
  FewGeo geo;
};
constexpr int kFewCtl = (sizeof(FewCtl) + 1023) / 1024 * 1024;
constexpr int kFewCtlOff = kFewSmem - kFewCtl;

struct FewParams {
  int T, H, E, k, F, Fs;
  int mode, groups, topk_groups, force;  // router (RouterSelMode)
  float gate_scale;
  int P1, P2;                // parts of x and of a
  int mx;                    // MXFP4 weights
  int mcap;                  // rows of an entry, at most
  int nsh, msh;              // entries of the shared expert, rows of one
  int chain;                 // products summed by one accumulator in tensor memory, at most
  int out_fp32;
  int ns1, ns1s, ns2;        // tiles of 128 columns: F, Fs, H
  int ks;                    // elements of a k sub-block
  int nsb1, nsb2, nsb2s;     // k sub-blocks: H, F, Fs
  const __nv_bfloat16 *x, *wr;
  const float *eb, *lb;
  int32_t* idx;
  float* gate;
  void* y;
  float* logits;             // [T, E]
  unsigned* sync;            // barrier 1, barrier 2, finished tiles of phases 0 and 1 and of 2, ended blocks
  unsigned* cnt;             // partials of a cut tile that are there: phases 0, 1, 2, both of W2
  int cnt_words;
  float* part[5];            // a phase's partial sums
  uint8_t *a, *as;           // parts of the activations: rows x parts x (F or Fs)
  uint8_t *a_sf, *as_sf;     // MXFP4: their scale bytes
  uint8_t *xq, *x_sf;        // MXFP4: parts of x and their scale bytes
  const uint8_t *w13, *w2, *w13s, *w2s;  // MXFP4 tiles, codes and scales
  DevStatus* status;
  unsigned long long lim;
  int fault;                 // test hook: block 0 does not arrive at the blocks' barriers
};
struct FewMaps {
  CUtensorMap m[6];          // W1, W3, W2, Ws1, Ws3, Ws2 (bf16)
};

__host__ __device__ constexpr int few_tile(bool mx) { return kFewATile + (mx ? 2 * kFewSf : 0); }
// parts of x and of a
__host__ __device__ constexpr int few_parts1(bool mx, bool fp32) { return mx ? (fp32 ? 8 : 5) : 1; }
__host__ __device__ constexpr int few_parts2(bool mx, bool fp32) { return mx ? (fp32 ? 8 : 5) : fp32 ? 3 : 2; }
// columns of the N operand: part q of row j is column q m + j
__host__ __device__ __forceinline__ int few_cols(int parts, int m) { return (parts * m + 15) & ~15; }
// accumulator columns of tensor memory: the rest holds scales, or is left to reads of
// eight columns that begin below
__host__ __device__ constexpr int few_acc_cols(bool mx) { return mx ? 416 : 496; }
constexpr int kFewSfCol = 416, kFewSfRegion = 48;  // two regions, in turn: 16 columns of A's, 32 of B's
__host__ __device__ __forceinline__ int few_mcap(int P1, bool mx) {
  return mx ? few_acc_cols(true) / 2 / 16 * 16 / P1 : kFewMaxT;
}
__host__ __device__ __forceinline__ FewGeo few_geo(int P1, int P2, int T, int mmax, bool mx) {
  FewGeo g;
  g.n1 = few_cols(P1, mmax);
  g.n2 = few_cols(P2, mmax);
  g.nblk1 = (g.n1 + 127) >> 7;
  g.nblk2 = (g.n2 + 127) >> 7;
  const int acc = mmax * 1024 > T * 512 ? mmax * 1024 : T * 512;
  g.acc_off = kFewCtlOff - (acc + 1023) / 1024 * 1024;
  g.b_bytes = 128 * (g.n1 > kFewSub2 * g.n2 ? g.n1 : kFewSub2 * g.n2);
  const int nblk = g.nblk1 > kFewSub2 * g.nblk2 ? g.nblk1 : kFewSub2 * g.nblk2;
  g.stage = 2 * few_tile(mx) + g.b_bytes + (mx ? 2 * kFewSf * nblk : 0);
  g.nst = g.acc_off / g.stage;  // (one at least: 64 rows of an expert, three parts)
  if (g.nst > kFewStages) g.nst = kFewStages;
  const int cols = few_acc_cols(mx);
  // the steps along k of fp32 results take several accumulators in turn: each adds a part of the
  // products, so that their chains end once a stage or two (one accumulator: 16 tokens of 8
  // experts of 4096 x 14336 571 us for 437). bf16 results are as near with one, which is read
  // sooner (one MXFP4 token 40.7 us with four, 40.2; 33 tokens 208, 207)
  const bool fp32 = P2 != few_parts2(mx, false);
  g.il1 = !fp32 ? 1 : 8 * g.n1 * 2 <= cols ? 4 : 4 * g.n1 * 2 <= cols ? 2 : 1;
  g.il2 = !fp32 ? 1 : 4 * g.n2 * 2 <= cols ? 4 : 2 * g.n2 * 2 <= cols ? 2 : 1;
  // two sets of them, where they fit, while the epilogue reads one (one set: 8 tokens 297.7 us for
  // 294.1, 33 with MXFP4 weights 212 for 208)
  g.nbuf1 = 4 * g.n1 * g.il1 <= cols ? 2 : 1;
  g.nbuf2 = 2 * g.n2 * g.il2 <= cols ? 2 : 1;
  return g;
}

// Routed entries of phases 1 and 3: half of them where there are enough that a half outlasts the
// join of the other (128 experts of 4096 x 1536, bf16: 8 tokens 295 us for 301, 33 613 for 621, 61 699 for
// 702; one token 68 either way, with MXFP4 weights 48 for 42), under MXFP4 while the halves' further
// partial sums weigh less than that (4 tokens, some 28 entries, 71 us for 73; 8, some 51, 113 for 111, 24 196 for 191)
constexpr int kFewHalve = 16, kFewHalveMx = 48;
__host__ __device__ __forceinline__ int few_half(int nact, bool mx) {
  return nact < kFewHalve || (mx && nact >= kFewHalveMx) ? nact : (nact + 1) >> 1;
}

// Equal contiguous runs of U units over the first G blocks of the grid (runs of at least four
// units instead: one MXFP4 token of 512 x 256 30.3 us for 23.6, one of 4096 x 1536 41.7 for 41.3)
struct FewSplit {
  int U, G, q, r;  // units, blocks; the first r blocks have q + 1 units, the others q
  __host__ __device__ __forceinline__ void set(int units, int blocks) {
    U = units;
    G = blocks < U ? blocks : U;
    q = G > 0 ? U / G : 0;
    r = U - q * G;
  }
  __host__ __device__ __forceinline__ int start(int c) const { return c >= G ? U : c * q + (c < r ? c : r); }
  // the block that has unit u
  __host__ __device__ __forceinline__ int owner(int u) const {
    const int big = r * (q + 1);
    return u < big ? u / (q + 1) : r + (u - big) / q;
  }
};
// Blocks c0 .. c1 share a tile of a phase. c0 has its beginning and joins it; the others
// leave their sums in their slot of the workspace (a block has at most one share that
// begins inside a tile: its first). W2's tiles are joined in their last phase: the shares
// of the phase before lie in slots of their own, block + tile.
struct FewPieces {
  int c0, c1;
};

// Consecutive stages of one tile and one expert, summed in tensor memory, that the
// epilogue takes at once
struct FewChunk {
  int i;       // entry; -1 - g: the shared expert's entry g
  int tile;    // 128-column tile: of F (phases 0 to 2), of H
  int kb, nkb; // first stage of the expert's k, stages
  bool first, last;  // of this block's segment of the tile
};

// A block's share of a phase, chunk by chunk; every role walks it by itself.
struct FewWalk {
  FewSplit s;
  int phase, u, u0, u1;
  bool down;
  int i0;                     // first routed entry of the phase
  int kbs, kbr, shared, per;  // stages of the shared expert's and a routed expert's k, of all shared entries, of a tile
  int ns, flush;
  __host__ __device__ __forceinline__ FewWalk(int ph, const FewParams& p, const FewGeo& g, int nact, int c, int G) {
    phase = ph;
    down = ph >= 3;
    const int half = few_half(nact, p.mx), n = ph == 0 ? 0 : (ph & 1) ? half : nact - half;
    i0 = ph == 0 || (ph & 1) ? 0 : half;
    if (!down) {
      ns = ph == 0 ? p.ns1s : p.ns1;
      per = p.nsb1;
      s.set((ph == 0 ? p.nsh : n) * ns * per, G);
      kbs = kbr = shared = per;
      flush = p.chain * g.il1 / p.ks;
    } else {
      ns = p.ns2;
      kbr = (p.nsb2 + kFewSub2 - 1) / kFewSub2;
      kbs = (p.nsb2s + kFewSub2 - 1) / kFewSub2;
      shared = ph == 3 ? p.nsh * kbs : 0;
      per = shared + n * kbr;
      s.set(ns * per, G);
      flush = p.chain * g.il2 / (p.ks * kFewSub2);
    }
    if (flush < 1) flush = 1;
    u = u0 = s.start(c);
    u1 = s.start(c + 1);
  }
  // the blocks that share tile t of the phase (which has work)
  __host__ __device__ __forceinline__ FewPieces pieces(int t) const {
    return FewPieces{s.owner(t * per), s.owner((t + 1) * per - 1)};
  }
  __host__ __device__ __forceinline__ bool next(FewChunk& c) {
    if (u >= u1) return false;
    const int t = u / per, r = u - t * per;
    int lim;
    if (!down) {
      const int e = t / ns;
      c.i = phase == 0 ? -1 - e : i0 + e;
      c.tile = t - e * ns;
      c.kb = r;
      lim = per - r;
    } else {
      c.tile = t;
      if (r < shared) {
        const int e = r / kbs;
        c.i = -1 - e;
        c.kb = r - e * kbs;
        lim = kbs - c.kb;
      } else {
        const int e = (r - shared) / kbr;
        c.i = i0 + e;
        c.kb = r - shared - e * kbr;
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

// An entry's rows: the first (of the routed rows; the shared expert's: token) and how many
struct FewRows {
  int r0, m;
  __device__ __forceinline__ FewRows(const FewParams& p, const FewCtl* c, int i) {
    if (i < 0) {
      r0 = (-1 - i) * p.msh;
      m = p.T - r0 < p.msh ? p.T - r0 : p.msh;
    } else {
      r0 = c->off[i];
      m = c->off[i + 1] - r0;
    }
  }
};

}  // namespace moe
