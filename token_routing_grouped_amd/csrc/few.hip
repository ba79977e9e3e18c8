// The expert layer for a few tokens (at most 64: a decode step, a short
// draft), forward only, and one dense product with 4-bit weights.
//
//   p[t,:] = softmax(x[t] wr^T);  the k largest, ties to the lower expert
//   h[t,e] = p[t,e] * silu(W1[e] x[t]) * (W3[e] x[t])    for the chosen e
//   y[t]   = sum_e W2[e] h[t,e]
//
// With few tokens the layer is a stream of weights: each chosen expert's three
// matrices are read once (2, 4 or 17/32 bytes a weight) for a handful of
// multiplications each, so HBM bounds it and everything else has to hide
// behind the loads.  The products still go through the matrix cores, weights
// as the A operand (16 output rows), tokens as the B operand (up to 16
// columns): that costs the vector units nothing, needs no cross-lane sums, and
// reads each weight once for all the tokens of its expert.
//
// Operand loads go straight from memory to registers.  In one step a wave
// reads a 128-byte line of each of 16 weight rows: lane (row l % 16, quarter
// l / 16) takes 32 consecutive bytes of its row as two 16-byte loads.  The
// order of a product's k is free, so the quarters' places in the line are the
// matrix instruction's k groups, and the tokens' operand is read with the same
// places.  A probe of this pattern read 4 GiB at 6.1-6.7 TB/s, the same as
// whole-wave contiguous loads.
//
// fp32 accumulation throughout.  The hidden vector h (gate included) is kept
// for the second product as two bf16 halves, hi = bf16(h) and lo = bf16(h -
// hi): 16 mantissa bits, so its rounding is far below y's own; a second matrix
// instruction is free next to the weight stream.  Measured, 24 tokens, 384
// experts: 0.3 % of the bf16 outputs round to the neighbour of what an fp32 h
// gives, and the error against 64 bits is the same, 1.6615e-3 of y's norm with
// either.  fp32 weights use the fp32 matrix instruction and h stays fp32.
//
// Launches (in_prologue has the rule):
//   a token or a few, few experts  router logits; up projection, which routes in
//                                  its prologue; down projection, summing over
//                                  the experts in its accumulators (a column is
//                                  a token, whichever experts it chose).  With
//                                  at most 16 experts the up projection computes
//                                  the logits as well: two launches.
//   more                           logits; routing; up; down, a row an entry (a
//                                  token's place among its k); join, which adds a
//                                  token's rows
// Every sum has a fixed order.
#include "common.h"
#include "kernels.h"

namespace trg {

namespace {

enum { kF32 = 0, kBF16 = 1, kE2M1 = 2 };  // weight storage

constexpr int kWaves = 8;          // waves of the product kernels' workgroups
constexpr int kThreads = kWaves * 64;

typedef unsigned long long mask_t;  // tokens, a bit each

// One chosen expert (few_down_kernel's): its index, its first hidden row, and
// which tokens chose it.
struct FewSlot {
  int e, off;
  mask_t mask;
};
// What token t's choice of expert e says, at [t E + e] (nothing where t did not
// choose e): its weight, and its entry t k + j.
struct FewEntry {
  float w;
  int row;
};

// The most experts that T tokens can choose.
int slots_of(int T, int E, int k) { return T * k < E ? T * k : E; }

constexpr int kProTokens = kWaves;  // tokens that the up projection routes itself: a wave each
constexpr int kProEntries = 64;     // and their entries: a lane each
// Routing in the up projection's prologue, and few_down_kernel: the launches of
// the routing and the join are saved (3 to 6 us), but every workgroup routes, so
// only where the chip takes all of them at once (256 CUs, two of 8 waves each).
// Measured, prologue / own launch, us, d = 2048, bf16 and 4 bits, with 512
// workgroups: one token, 128 experts, h = 2048, k = 4 30.1 / 34.2, 18.2 / 21.3; 2
// tokens, 384 experts, h = 512, k = 8 31.8 / 36.9, 22.6 / 24.1; 8 tokens, 8
// experts, h = 1024, k = 4 32.1 / 33.3, 20.5 / 21.6.  With 1024: one token, 384
// experts, h = 2048, k = 8 57.5 / 54.0, 32.3 / 29.2; 8 tokens, 8 experts, h = 2048,
// k = 2 57.2 / 55.2, 30.6 / 25.4.
bool in_prologue(int T, int E, int k, int h) {
  return T <= kProTokens && T * k <= kProEntries && slots_of(T, E, k) * ((h + 15) / 16) <= 512;
}
// Rows of the hidden buffer: an entry's own, or (few_down_kernel) T for every
// slot.
int hid_rows(int T, int E, int k, int h) { return in_prologue(T, E, k, h) ? slots_of(T, E, k) * T : T * k; }
// Partial sums that the router's logits come in (its E / 16 row tiles alone would
// leave most of the chip idle): as many as leave each of a workgroup's 8 waves a
// line.  Whoever adds them reads them all, so no more than that.  One part of 16
// waves with two lines each measured 12.8 us instead of 5.0 (61 tokens, 128
// experts, d = 2048).
constexpr int kLogitParts = 8;
int logit_parts(int row_bytes) {
  const int p = ((row_bytes + 127) / 128 + 7) / 8;
  return p < 1 ? 1 : (p > kLogitParts ? kLogitParts : p);
}

struct FewLayout {
  size_t n_active, slots, masks, entries, logits, hid, yp, bytes;
};

FewLayout few_layout(int T, int d, int E, int k, int h) {
  const size_t R = (size_t)T * k, S = slots_of(T, E, k);
  const bool rows = !in_prologue(T, E, k, h);
  FewLayout l;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t p = at;
    at += (n + 255) / 256 * 256;
    return p;
  };
  l.n_active = take(rows ? 0 : sizeof(int));
  l.slots = take(rows ? 0 : S * sizeof(FewSlot));
  l.masks = take(rows ? E * sizeof(mask_t) : 0);
  l.entries = take(rows ? (size_t)T * E * sizeof(FewEntry) : 0);
  l.logits = take((size_t)logit_parts(d * 4) * T * E * sizeof(float));  // fp32 rows have the most lines
  l.hid = take((size_t)hid_rows(T, E, k, h) * h * sizeof(float));         // fp32, or the hi and lo bf16 halves
  l.yp = take(rows ? R * d * sizeof(float) : 0);
  l.bytes = at;
  return l;
}

// The wave's number in its workgroup, known to the compiler as uniform.
TRG_DEV int wave_id() { return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)); }

TRG_DEV bf16x8_t as_bf16x8(uint4 v) { return __builtin_bit_cast(bf16x8_t, v); }

// Scale operand of an E8M0 byte (255 stands for NaN).
TRG_DEV float e8m0(uint32_t b) {
  return b == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(b ? b << 23 : 0x00400000u);
}

// Eight E2M1 codes (one dword) times their block's scale, as bf16 (exact:
// two significant bits).
TRG_DEV bf16x8_t e2m1x8(uint32_t c, float sc) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 0);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 1);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 2);
  const bf16x2_t e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 3);
  return bf16x8_t{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}

// k values of one 16-byte piece of a weight row.
template <int WT>
struct Piece {
  static constexpr int kK = WT == kF32 ? 4 : (WT == kBF16 ? 8 : 32);
  static constexpr int kX = WT == kE2M1 ? 4 : 1;  // 16-byte pieces of the tokens' operand it meets
  static constexpr int kXE = WT == kF32 ? 4 : 2;  // bytes of an element of that operand
};

// acc += piece of 16 rows x piece of 16 columns.
template <int WT>
TRG_DEV f32x4_t mma_piece(uint4 w, float sc, const uint4* x, f32x4_t acc) {
  if constexpr (WT == kBF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(w), as_bf16x8(x[0]), acc, 0, 0, 0);
  } else if constexpr (WT == kF32) {
    const f32x4_t a = __builtin_bit_cast(f32x4_t, w), b = __builtin_bit_cast(f32x4_t, x[0]);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], acc, 0, 0, 0);
    return acc;
  } else {
    const uint32_t c[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(e2m1x8(c[i], sc), as_bf16x8(x[i]), acc, 0, 0, 0);
    return acc;
  }
}

// The same with an operand in P parts (2: x and y are its halves): a 4-bit
// piece is decoded once for both.
template <int WT, int P>
TRG_DEV f32x4_t mma_parts(uint4 w, float sc, const uint4* x, const uint4* y, f32x4_t acc) {
  if constexpr (WT == kE2M1) {
    const uint32_t c[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bf16x8_t a = e2m1x8(c[i], sc);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, as_bf16x8(x[i]), acc, 0, 0, 0);
      if constexpr (P == 2) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, as_bf16x8(y[i]), acc, 0, 0, 0);
    }
    return acc;
  } else {
    acc = mma_piece<WT>(w, sc, x, acc);
    return P == 2 ? mma_piece<WT>(w, sc, y, acc) : acc;
  }
}

// A lane's place in a weight matrix: uniform bases (of an expert's matrix, and of
// the whole matrix's scales) and 32-bit offsets (the caller's sizes keep an
// expert's matrix and all scales of one under 2 GiB), so that a row costs two
// registers.
struct WBase {
  const char* p;
  const uint8_t* s;   // E2M1: scales
  uint32_t first;     // E2M1: this matrix's first row among the n rows of the scales
  uint32_t sstride;   // E2M1: bytes from a 128-value chunk's scales to the next one's, n * 4
};
struct WRow {
  uint32_t off, soff;
};
// Matrix e of E matrices of `rows` rows of rb bytes.
template <int WT>
TRG_DEV WBase w_base(const void* w, const uint8_t* ws, int e, int E, int rows, int rb) {
  return {(const char*)w + (long)e * rows * rb, ws, (uint32_t)e * (uint32_t)rows, (uint32_t)E * (uint32_t)rows * 4u};
}
template <int WT>
TRG_DEV WRow w_row(const WBase& b, int row, int rb) {
  return {(uint32_t)row * (uint32_t)rb, WT == kE2M1 ? (b.first + (uint32_t)row) * 4u : 0u};
}

// Row tile of the t-th of `tiles` workgroups (a permutation).  A cache line of
// 4-bit rows' scales is 32 rows' of one chunk, G tiles'; workgroups go round the
// 8 dies, so with tiles in order G of them would each fetch it.  So G
// neighbouring tiles go to one die.  61 tokens, 128 experts, up projection: 50.2
// -> 47.0 us.
template <int WT, int G>
TRG_DEV int near_tile(int t, int tiles) {
  if constexpr (WT != kE2M1 || G <= 1) return t;
  const int o = t % (8 * G), b = t - o;
  return b + 8 * G <= tiles ? b + o % 8 * G + o / 8 : t;
}

// One step's share of a weight row: two 16-byte pieces and their scale bytes.
struct WStep {
  uint4 v[2];
  uint32_t sb;
};
// c: 128-byte line of the row; q: the lane's quarter of it.  A piece past the
// row's end (rb is a multiple of 16, so it is in or out whole) becomes zeros,
// loaded from the row's last piece: every load is unconditional, so that the
// compiler can count which of them it has to wait for.
template <int WT>
TRG_DEV WStep w_load(const WBase& b, const WRow& r, int c, int q, int rb) {
  WStep o;
  const int off = c * 128 + q * 32, last = rb - 16;
  o.v[0] = *(const uint4*)(b.p + (r.off + (uint32_t)min(off, last)));
  o.v[1] = *(const uint4*)(b.p + (r.off + (uint32_t)min(off + 16, last)));
  o.sb = 0;
  if constexpr (WT == kE2M1) {
    // block b = off / 16, its byte in chunk b / 4; b is even, so both bytes of
    // the step are in one chunk (the second may be a place past the last block)
    const int bk = min(off, last) / 16 & ~1;
    o.sb = *(const uint16_t*)(b.s + (r.soff + (uint32_t)(bk >> 2) * b.sstride + (uint32_t)(bk & 3)));
  }
  return o;
}
template <int WT>
TRG_DEV void w_mask(WStep& o, int c, int q, int rb) {
  const int off = c * 128 + q * 32;
  const bool in0 = off < rb, in1 = off + 16 < rb;
  o.v[0].x = in0 ? o.v[0].x : 0; o.v[0].y = in0 ? o.v[0].y : 0;
  o.v[0].z = in0 ? o.v[0].z : 0; o.v[0].w = in0 ? o.v[0].w : 0;
  o.v[1].x = in1 ? o.v[1].x : 0; o.v[1].y = in1 ? o.v[1].y : 0;
  o.v[1].z = in1 ? o.v[1].z : 0; o.v[1].w = in1 ? o.v[1].w : 0;
  if (WT == kE2M1) o.sb = in1 ? o.sb : (in0 ? o.sb & 0xFFu : 0u);
}

// The tokens' operand of one step for a lane's column: both pieces, KX 16-byte
// parts each.  Past the row's end it is the row's last piece again, until
// x_mask puts zeros there: the weights are zeros too, but 0 * inf is not.
template <int WT>
struct XStep {
  uint4 v[2][Piece<WT>::kX];
};
// Piece i of the operand; xb: a uniform base, xo: the lane's column's row.
template <int WT>
TRG_DEV void x_piece(const char* xb, uint32_t xo, int c, int q, int i, int rb, uint4* x) {
  const int at = min(c * 128 + q * 32 + 16 * i, rb - 16) / 16 * (Piece<WT>::kK * Piece<WT>::kXE);
  const char* p = xb + (xo + (uint32_t)at);
#pragma unroll
  for (int j = 0; j < Piece<WT>::kX; ++j) x[j] = *(const uint4*)(p + j * 16);
}
template <int WT>
TRG_DEV void x_load(const char* xb, uint32_t xo, int c, int q, int rb, XStep<WT>& o) {
  x_piece<WT>(xb, xo, c, q, 0, rb, o.v[0]);
  x_piece<WT>(xb, xo, c, q, 1, rb, o.v[1]);
}
template <int WT>
TRG_DEV void x_mask(uint4* x, int c, int q, int i, int rb) {
  const bool in = c * 128 + q * 32 + 16 * i < rb;
#pragma unroll
  for (int j = 0; j < Piece<WT>::kX; ++j)
    x[j] = make_uint4(in ? x[j].x : 0, in ? x[j].y : 0, in ? x[j].z : 0, in ? x[j].w : 0);
}
template <int WT>
TRG_DEV f32x4_t mma_step(const WStep& w, const XStep<WT>& x, f32x4_t acc) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    acc = mma_piece<WT>(w.v[i], WT == kE2M1 ? e8m0((w.sb >> (8 * i)) & 255u) : 0.f, x.v[i], acc);
  return acc;
}

// ---- the tokens' operand of 4-bit lines, through LDS ---------------------------
// A line of 4-bit weights meets 512 bytes of every token, and a lane needs 16 of
// each 128: loaded directly, 64 lanes touch up to 64 cache lines an instruction,
// eight times the same ones, and the address unit, not HBM, sets the pace (13
// tokens, 24576 x 6144: 24.3 us, of which 15.6 are left without these loads;
// staged 16.4).  So a wave copies them to its own kStage bytes of LDS, whole
// cache lines an instruction, and its lanes read their pieces there: XB = 2
// pieces at a time (a line: 512 bytes of a token), or, where registers are short,
// one (256 bytes a token, and room for both parts of the hidden vector).  A dense
// product with one piece at a time: 19.0 instead of 16.7 us.  Place s of token n
// is stored at s ^ n, so that the 16 tokens' reads of one place fall into
// different banks.  No workgroup barrier: the buffer is one wave's, and its LDS
// instructions run in order (wave_order keeps the compiler to it).
constexpr int kStage = 8192;
TRG_DEV void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// In two steps, so that the weights' loads can go out in between.  xo: lane r's
// row offset of column r, which repeats the last column where there is none;
// the first XN * (tokens an instruction) columns are copied.
template <int P, int XN, int XB>
struct Stage {
  static constexpr int LT = 16 * XB;           // lanes (16-byte places) a token
  static constexpr int TI = 64 / LT;           // tokens an instruction
  uint4 g[XN][P];
};
// Where in a token's row place s of a copy is.
template <int XB>
TRG_DEV int stage_at(int s, int line, int piece) {
  return line * 512 + (XB == 2 ? s * 16 : (s >> 2) * 128 + piece * 64 + (s & 3) * 16);
}
template <int P, int XN, int XB>
TRG_DEV void stage_load(Stage<P, XN, XB>& o, const char* xb, long xpart, uint32_t xo, int line, int piece,
                        int row_bytes) {
  constexpr int LT = Stage<P, XN, XB>::LT, TI = Stage<P, XN, XB>::TI;
  const int lane = threadIdx.x & 63, s = lane % LT;
  const uint32_t off = (uint32_t)min(stage_at<XB>(s, line, piece), row_bytes - 16);
#pragma unroll
  for (int t = 0; t < XN; ++t) {
    const uint32_t at = (uint32_t)__builtin_amdgcn_ds_bpermute((t * TI + lane / LT) * 4, (int)xo) + off;
#pragma unroll
    for (int p = 0; p < P; ++p) o.g[t][p] = *(const uint4*)(xb + p * xpart + at);
  }
}
// Zeros past the row's end, where the row's last place was loaded again.
template <int P, int XN, int XB>
TRG_DEV void stage_mask(Stage<P, XN, XB>& o, int line, int piece, int row_bytes) {
  const bool in = stage_at<XB>((threadIdx.x & 63) % Stage<P, XN, XB>::LT, line, piece) < row_bytes;
#pragma unroll
  for (int t = 0; t < XN; ++t)
#pragma unroll
    for (int p = 0; p < P; ++p) {
      uint4& g = o.g[t][p];
      g = make_uint4(in ? g.x : 0, in ? g.y : 0, in ? g.z : 0, in ? g.w : 0);
    }
}
template <int P, int XN, int XB>
TRG_DEV void stage_store(const Stage<P, XN, XB>& o, char* xl) {
  constexpr int LT = Stage<P, XN, XB>::LT, TI = Stage<P, XN, XB>::TI;
  const int lane = threadIdx.x & 63, s = lane % LT;
#pragma unroll
  for (int t = 0; t < XN; ++t) {
    const int tok = t * TI + lane / LT;
#pragma unroll
    for (int p = 0; p < P; ++p) *(uint4*)(xl + p * (kStage / 2) + tok * (LT * 16) + (s ^ tok) * 16) = o.g[t][p];
  }
}
// Lane's four 16-byte parts of piece `piece` of part p.
template <int XB>
TRG_DEV void staged_x(const char* xl, int r, int q, int piece, int p, uint4* x) {
  constexpr int LT = 16 * XB;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int s = XB == 2 ? q * 8 + piece * 4 + j : q * 4 + j;
    x[j] = *(const uint4*)(xl + p * (kStage / 2) + r * (LT * 16) + (s ^ r) * 16);
  }
}

// ---- products of NM 16-row tiles with NT * 16 columns --------------------------
// acc[m][n] over lines c0, c0 + step, ... < c1 of the rows, U lines at a time:
// all their weights are loaded (from HBM), then the tokens' operand (P parts,
// xpart bytes apart; from the caches).  The waves of a CU hide each other's
// loads: NM * U * 2 KB a wave in flight is several times what HBM's latency
// needs.  Tile m is rows wr[m] of matrix wb[m % NB], NB bases; cols: columns
// that are there.
// Only the lanes of those columns load the operand (a few tokens are a few
// lanes); the others' registers hold anything: columns do not mix, and theirs
// are not stored.  xl: the wave's staging buffer, XN the copying instructions
// (4-bit weights; cols and more columns fit).  PEEL: a body without masks for the
// lines before a row's end (4-bit weights).  A dense product gains by it (24576 x
// 6144, one / 13 / 64 tokens 16.4 / 17.4 / 39.9 -> 14.9 / 16.7 / 38.4 us); the
// experts' short rows lose (61 tokens, 128 experts 95.6 -> 101.8).
// One line of 4-bit rows; MASK: the row may end inside it.
template <bool MASK, int NB, int NM, int NT, int P, int XN, int XB>
TRG_DEV void line_e2m1(const WBase* wb, const WRow* wr, const char* xb, const uint32_t* xo, long xpart, int rb, int c,
                       int r, int q, f32x4_t (*acc)[NT], char* xl) {
  const bool tail = MASK && (c + 1) * 128 > rb;
  WStep w[NM];
  // the first copy's loads go out before the weights', so that it is in LDS when
  // they arrive
  Stage<P, XN, XB> st;
  stage_load(st, xb, xpart, xo[0], c, 0, rb * 4);
#pragma unroll
  for (int m = 0; m < NM; ++m) w[m] = w_load<kE2M1>(wb[m % NB], wr[m], c, q, rb);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int b = 0; b < 2; b += XB) {
      uint4 x[XB][P][4];
      if (n + b > 0) stage_load(st, xb, xpart, xo[n], c, b, rb * 4);
      if (tail) stage_mask(st, c, b, rb * 4);
      stage_store(st, xl);
      wave_order();
#pragma unroll
      for (int i = 0; i < XB; ++i)
#pragma unroll
        for (int p = 0; p < P; ++p) staged_x<XB>(xl, r, q, b + i, p, x[i][p]);
      wave_order();
      // the codes are waited for only here, after the copy: one token 15.8 -> 14.9
      // us, 32 tokens 26.4 -> 25.1 (24576 x 6144)
      __builtin_amdgcn_sched_barrier(0);
      if (tail && n + b == 0) {
#pragma unroll
        for (int m = 0; m < NM; ++m) w_mask<kE2M1>(w[m], c, q, rb);
      }
#pragma unroll
      for (int i = 0; i < XB; ++i) {
#pragma unroll
        for (int m = 0; m < NM; ++m)
          acc[m][n] = mma_parts<kE2M1, P>(w[m].v[b + i], e8m0((w[m].sb >> (8 * (b + i))) & 255u), x[i][0], x[i][P - 1],
                                          acc[m][n]);
        __builtin_amdgcn_sched_barrier(0);  // a piece's codes are decoded when it is used, not ahead
      }
    }
}

template <int WT, int NB, int NM, int NT, int U, int P, int XN, int XB = 2, bool PEEL = false>
TRG_DEV void stream_tile(const WBase* wb, const WRow* wr, const char* xb, const uint32_t* xo, long xpart, int cols,
                         int rb, int c0, int c1, int step, int r, int q, f32x4_t (*acc)[NT], char* xl) {
  if constexpr (WT == kE2M1) {
    static_assert(U == 1, "a staging buffer holds one line");
    if constexpr (PEEL)
      for (; c0 < min(c1, rb >> 7); c0 += step)
        line_e2m1<false, NB, NM, NT, P, XN, XB>(wb, wr, xb, xo, xpart, rb, c0, r, q, acc, xl);
    for (; c0 < c1; c0 += step)
      line_e2m1<true, NB, NM, NT, P, XN, XB>(wb, wr, xb, xo, xpart, rb, c0, r, q, acc, xl);
  } else {
    const int past = (rb + 127) >> 7;  // a line that is past every row's end
    for (; c0 < c1; c0 += step * U) {
      WStep w[U][NM];
      int line[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        line[u] = c0 + u * step < c1 ? c0 + u * step : past;
#pragma unroll
        for (int m = 0; m < NM; ++m) w[u][m] = w_load<WT>(wb[m % NB], wr[m], line[u], q, rb);
      }
      const bool whole = (line[U - 1] + 1) * 128 <= rb;  // lines rise, so all of them are
      // the operand of all columns at once: one trip to the caches a batch
      constexpr int NB_X = NT * 2 * U * P <= 16 ? NT : 1;  // column tiles in registers: at most 64 of them
#pragma unroll
      for (int n0 = 0; n0 < NT; n0 += NB_X) {
        uint4 x[NB_X][2 * U][P];
        if (NT > 1 || r < cols) {
#pragma unroll
          for (int n = 0; n < NB_X; ++n)
#pragma unroll
            for (int i = 0; i < 2 * U; ++i)
#pragma unroll
              for (int p = 0; p < P; ++p)
                x_piece<WT>(xb + p * xpart, xo[n0 + n], line[i / 2], q, i & 1, rb, &x[n][i][p]);
        }
        if (!whole) {
          if (n0 == 0) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int m = 0; m < NM; ++m) w_mask<WT>(w[u][m], line[u], q, rb);
          }
#pragma unroll
          for (int n = 0; n < NB_X; ++n)
#pragma unroll
            for (int i = 0; i < 2 * U; ++i)
#pragma unroll
              for (int p = 0; p < P; ++p) x_mask<WT>(&x[n][i][p], line[i / 2], q, i & 1, rb);
        }
#pragma unroll
        for (int n = 0; n < NB_X; ++n)
#pragma unroll
          for (int i = 0; i < 2 * U; ++i)
#pragma unroll
            for (int m = 0; m < NM; ++m)
              acc[m][n0 + n] =
                  mma_parts<WT, P>(w[i / 2][m].v[i & 1], 0.f, &x[n][i][0], &x[n][i][P - 1], acc[m][n0 + n]);
        if (NB_X < NT) __builtin_amdgcn_sched_barrier(0);  // or all tiles' operands are loaded at once, into scratch
      }
    }
  }
}

// Sum of `waves` accumulators of one 16 x 16 tile, in wave order.  red: 256
// floats a wave; entry (lane, r) of the matrix layout: column lane % 16, row
// lane / 16 * 4 + r.
TRG_DEV void put_tile(float* red, int lane, f32x4_t a) { *(f32x4_t*)(red + lane * 4) = a; }
TRG_DEV float sum_tile(const float* red, int waves, int row, int col) {
  const float* p = red + ((row >> 2) * 16 + col) * 4 + (row & 3);
  float t = p[0];
  for (int w = 1; w < waves; ++w) t += p[w * 256];
  return t;
}

// Live tokens: all T, or what the device count says.
TRG_DEV int live_tokens(const int* n_live, int T) { return n_live != nullptr ? min(max(*n_live, 0), T) : T; }

// ---- a dense product, and the router's logits -----------------------------------
// out[t, row] = <x[t], w[row]> for T <= NT * 16 columns.  A workgroup takes NM
// tiles of 16 rows, its waves share the lines; blockIdx.y takes the part_lines
// lines from blockIdx.y * part_lines and writes its own [T, n] of out.  The first
// one also clears the nz masks that the next launch sets.
// 4 bits, 24576 x 6144 (80 MB, HBM-bound; decoding and the operand's way through
// LDS take their share of the issue slots): one token 14.5 us, 5.5 TB/s, 13
// tokens 17 to 19 (by the card), 4.3 to 4.8 TB/s.  Above 16 tokens each of the 8
// waves stages its own line for every column tile, and a staged byte serves only
// that wave's rows: 32 tokens 27.5 us, 64 tokens 44, for 13 of bytes.  Logits of 61
// tokens, 128 experts, d = 2048: 5.2 us, latency.
template <int WT, int NM, int NT, int U, int XN, int WAVES, class OUT>
__global__ __launch_bounds__(WAVES * 64, NT > 1 && NM* NT > 3 ? 2 : 4) void few_linear_kernel(
    const char* __restrict__ x, const void* __restrict__ w, const uint8_t* __restrict__ ws, int T, int n, int rb,
    int xb, int part_lines, const int* __restrict__ n_live, OUT* __restrict__ out, mask_t* __restrict__ masks,
    int nz) {
  // the waves' staging buffers, then (1 KB a wave) their accumulators
  __shared__ __attribute__((aligned(16))) char lds[WAVES * (WT == kE2M1 ? kStage : 1024)];
  float* red = (float*)lds;
  const int lane = threadIdx.x & 63, wv = wave_id(), r = lane & 15, q = lane >> 4;
  const int live = live_tokens(n_live, T);
  if (blockIdx.x + blockIdx.y == 0)
    for (int i = threadIdx.x; i < nz; i += WAVES * 64) masks[i] = 0;
  const int row0 = blockIdx.x * (16 * NM);
  const int c0 = blockIdx.y * part_lines, c1 = min((rb + 127) >> 7, c0 + part_lines);
  const WBase wb[1] = {w_base<WT>(w, ws, 0, 1, n, rb)};
  WRow wr[NM];
#pragma unroll
  for (int m = 0; m < NM; ++m) wr[m] = w_row<WT>(wb[0], min(row0 + m * 16 + r, n - 1), rb);
  uint32_t xo[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) xo[i] = (uint32_t)min(i * 16 + r, T - 1) * (uint32_t)xb;
  f32x4_t acc[NM][NT];
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[m][i] = f32x4_t{0, 0, 0, 0};
  stream_tile<WT, 1, NM, NT, U, 1, XN, 2, true>(wb, wr, x, xo, 0, live, rb, c0 + wv, c1, WAVES, r, q, acc,
                                                lds + wv * kStage);
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if (WT == kE2M1 || m + i > 0) __syncthreads();
      put_tile(red + wv * 256, lane, acc[m][i]);
      __syncthreads();
      const int row = row0 + m * 16 + (threadIdx.x & 15), t = i * 16 + ((threadIdx.x >> 4) & 15);
      if (threadIdx.x < 256 && t < live && row < n)
        Elt<OUT>::st(out + ((long)blockIdx.y * T + t) * n + row,
                     sum_tile(red, WAVES, threadIdx.x & 15, (threadIdx.x >> 4) & 15));
    }
}

// ---- routing ---------------------------------------------------------------------
// Reductions over the wave inside the vector registers: within rows of 16 lanes,
// then over the rows' last lanes; lane 63 has the result.  Lanes without a
// partner combine with 0, the identity of both.
template <int CTRL>
TRG_DEV uint32_t max_dpp(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false));
}
template <int CTRL>
TRG_DEV float sum_dpp(float v) {
  return v + __uint_as_float(__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, false));
}
// row_shr 1, 2, 4, 8, row_bcast 15, 31
TRG_DEV uint32_t wave_max_u32(uint32_t v) {
  v = max_dpp<0x118>(max_dpp<0x114>(max_dpp<0x112>(max_dpp<0x111>(v))));
  return (uint32_t)__builtin_amdgcn_readlane((int)max_dpp<0x143>(max_dpp<0x142>(v)), 63);
}
TRG_DEV float wave_sum_dpp(float v) {
  v = sum_dpp<0x118>(sum_dpp<0x114>(sum_dpp<0x112>(sum_dpp<0x111>(v))));
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(sum_dpp<0x143>(sum_dpp<0x142>(v))), 63));
}

// One wave routes a token from its logits (v[i] of lane l: expert l + 64 i): the
// k largest, ties to the lower expert, a NaN never before a number (moe_route's
// rules), and their softmax values.  A logit becomes a 32-bit key that orders
// like it (0 is below every key), so a round is one wave maximum and the first
// lane of the first register that holds it.
template <int EPL>
struct Routed {
  int mine;               // lane j: the j-th choice
  int place[EPL];         // places of this lane's experts, -1: not chosen
  float p[EPL], s;        // softmax p / s
};
template <int EPL>
TRG_DEV void route_token(float* v, int E, int k, int lane, Routed<EPL>& o) {
  uint32_t key[EPL], top = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const bool in = lane + 64 * i < E;
    v[i] = (v[i] != v[i] || !in) ? -INFINITY : v[i] + 0.0f;  // -0 and 0 are equal
    const uint32_t b = __float_as_uint(v[i]);
    key[i] = in ? ((b & 0x80000000u) ? ~b : b | 0x80000000u) : 0u;
    top = max(top, key[i]);
  }
  top = wave_max_u32(top);
  const float m = __uint_as_float((top & 0x80000000u) ? top & 0x7FFFFFFFu : ~top);  // the largest logit
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    o.p[i] = lane + 64 * i < E ? expf(v[i] - m) : 0.f;
    s += o.p[i];
  }
  o.s = wave_sum_dpp(s);
  o.mine = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) o.place[i] = -1;
  for (int j = 0; j < k; ++j) {
    // no branches: a round is a chain of dependent instructions as it is
    int e = 0;
#pragma unroll
    for (int i = EPL - 1; i >= 0; --i) {
      const unsigned long long at = __ballot(key[i] == top);
      e = at != 0 ? 64 * i + __ffsll(at) - 1 : e;
    }
    o.mine = lane == j ? e : o.mine;
    uint32_t next = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const bool hit = lane + 64 * i == e;
      key[i] = hit ? 0u : key[i];
      o.place[i] = hit ? j : o.place[i];
      next = max(next, key[i]);
    }
    top = wave_max_u32(next);
  }
}

// out[j] = the router's partial logits at at[j] (of plane = T E values), added in
// order; G parts of all N are in flight at once (other XCDs wrote them: every
// trip goes past L2), past the last one it is loaded again and not added.
template <int N>
TRG_DEV void add_logits(const float* __restrict__ logits, int parts, uint32_t plane, const uint32_t* at, float* out) {
  constexpr int G = N <= 8 ? 4 : 2;
#pragma unroll
  for (int j = 0; j < N; ++j) out[j] = 0.f;
  for (int a0 = 0; a0 < parts; a0 += G) {
    float raw[G][N];
#pragma unroll
    for (int a = 0; a < G; ++a) {
      const float* L = logits + (long)min(a0 + a, parts - 1) * plane;
#pragma unroll
      for (int j = 0; j < N; ++j) raw[a][j] = L[at[j]];
    }
#pragma unroll
    for (int a = 0; a < G; ++a)
#pragma unroll
      for (int j = 0; j < N; ++j) out[j] = a0 + a < parts ? out[j] + raw[a][j] : out[j];
  }
}

// Routing in a launch of its own: a wave, and a workgroup, a token.  An expert's mask collects its tokens
// by an integer OR, which has one result in any order; the products find the
// chosen experts in the masks themselves (nth_expert), so that nothing has to wait
// for all tokens.  One workgroup routing all of them and listing the experts took
// 10.0 us with 61 tokens and 128 experts, 18.2 with 24 and 384; this takes 4.9 and
// 5.8, latency of the logits' loads and of the rounds.
template <int EPL>
__global__ __launch_bounds__(64) void few_route_kernel(const float* __restrict__ logits, int parts, int T, int E, int k,
                                                       const int* __restrict__ n_live, int* __restrict__ idx_out,
                                                       float* __restrict__ w_out, mask_t* __restrict__ masks,
                                                       FewEntry* __restrict__ entries) {
  const int lane = threadIdx.x, t = blockIdx.x;
  uint32_t at[EPL];
  float v[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) at[i] = (uint32_t)(t * E + min(lane + 64 * i, E - 1));
  if (t >= live_tokens(n_live, T)) return;
  add_logits<EPL>(logits, parts, (uint32_t)T * (uint32_t)E, at, v);
  Routed<EPL> o;
  route_token<EPL>(v, E, k, lane, o);
  if (lane < k) {
    atomicOr(&masks[o.mine], 1ull << t);
    if (idx_out != nullptr) idx_out[t * k + lane] = o.mine;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    if (o.place[i] >= 0) {
      const int row = t * k + o.place[i];
      entries[at[i]] = FewEntry{o.p[i] / o.s, row};
      if (w_out != nullptr) w_out[row] = o.p[i] / o.s;
    }
}

// The n-th expert, from 0, that has tokens, and its tokens' mask; -1: there are
// no more.  The same in every lane.
TRG_DEV int nth_expert(const mask_t* __restrict__ masks, int E, int n, int lane, mask_t* mask) {
  constexpr int B = 4;  // loads in flight
  for (int e0 = 0; e0 < E; e0 += 64 * B) {
    mask_t m[B];
#pragma unroll
    for (int i = 0; i < B; ++i) m[i] = masks[min(e0 + 64 * i + lane, E - 1)];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const mask_t on = __ballot(m[i] != 0 && e0 + 64 * i + lane < E);
      const int c = __popcll(on);
      if (n < c) {
        const mask_t at = __ballot((on >> lane & 1) && (int)__popcll(on & ((1ull << lane) - 1)) == n);
        const int l = __ffsll(at) - 1;
        *mask = (mask_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(m[i] >> 32), l) << 32 |
                (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)m[i], l);
        return e0 + 64 * i + l;
      }
      n -= c;
    }
  }
  return -1;
}

// ---- up projection ------------------------------------------------------------------
// Token of column c of a slot: the c-th set bit of its mask.  Lane l's token is
// pushed to the lane of its rank among the set bits (lanes without one behind
// them, so every lane receives one value), and read from there.
TRG_DEV int nth_token(unsigned long long mask, int lane, int c) {
  const unsigned long long below = (1ull << lane) - 1;
  const bool set = (mask >> lane) & 1;
  const int to = set ? __popcll(mask & below) : __popcll(mask) + __popcll(~mask & below);
  const int list = __builtin_amdgcn_ds_permute(to * 4, lane);
  return __builtin_amdgcn_ds_bpermute(c * 4, list);
}

// Lane c: column c's choice, for the tokens of expert e's mask (not empty); lanes
// without a column have the last one's.
TRG_DEV FewEntry column_entry(const FewEntry* __restrict__ entries, int E, int e, mask_t mask, int lane) {
  const int cnt = __popcll(mask), t = nth_token(mask, lane, min(lane, cnt - 1));  // every lane takes part
  return entries[t * E + e];
}

// RM * 16 rows of h for an expert's columns: both matrices' rows, shared by the
// workgroup's wk waves along k (this one is kw), then h = gate * silu(g) * u.
// ent: lane c has column c's.  lds: 2 KB a wave (kStage with 4-bit weights).
template <int WT, int RM, int NT, int U, int XN>
TRG_DEV void up_tile(const char* __restrict__ x, int xb, const WBase* wb, int rb, mask_t mask,
                     FewEntry ent, int cnt, int col0, int row0, int h, char* hid, long hid_n, int wk, int kw,
                     char* lds) {
  float* red = (float*)lds;
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  WRow wr[2 * RM];
#pragma unroll
  for (int m = 0; m < RM; ++m) {
    const int row = min(row0 + m * 16 + r, h - 1);
    wr[2 * m] = w_row<WT>(wb[0], row, rb);
    wr[2 * m + 1] = w_row<WT>(wb[1], row, rb);
  }
  uint32_t xo[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) xo[i] = (uint32_t)nth_token(mask, lane, min(col0 + i * 16 + r, cnt - 1)) * (uint32_t)xb;
  f32x4_t acc[2 * RM][NT];
#pragma unroll
  for (int m = 0; m < 2 * RM; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[m][i] = f32x4_t{0, 0, 0, 0};
  stream_tile<WT, 2, 2 * RM, NT, U, 1, XN>(wb, wr, x, xo, 0, cnt - col0, rb, kw, (rb + 127) >> 7, wk, r, q, acc,
                                       lds + kw * kStage);
#pragma unroll
  for (int m = 0; m < RM; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if (WT == kE2M1 || m + i > 0) __syncthreads();
      put_tile(red + kw * 256, lane, acc[2 * m][i]);
      put_tile(red + (wk + kw) * 256, lane, acc[2 * m + 1][i]);
      __syncthreads();
      for (int o = threadIdx.x; o < 256; o += wk * 64) {
        const int lr = o & 15, col = o >> 4, c = col0 + i * 16 + col, row = row0 + m * 16 + lr;
        const float gate = __int_as_float(__builtin_amdgcn_ds_bpermute(c * 4, __float_as_int(ent.w)));
        const int hrow = __builtin_amdgcn_ds_bpermute(c * 4, ent.row);
        if (c < cnt && row < h) {
          const float g = sum_tile(red, wk, lr, col), u = sum_tile(red + wk * 256, wk, lr, col);
          const float v = gate * (g / (1.0f + expf(-g)) * u);
          const long at = (long)hrow * h + row;
          if constexpr (WT == kF32) {
            ((float*)hid)[at] = v;
          } else {
            const uint16_t hi = f2bf(v);
            ((uint16_t*)hid)[at] = hi;
            const float lo = v - bf2f(hi);  // not a number where v is infinite: then hi says it all
            ((uint16_t*)hid)[hid_n + at] = fabsf(bf2f(hi)) < INFINITY ? f2bf(lo) : (uint16_t)0;
          }
        }
      }
    }
}

constexpr int kProRouter = 65536;  // bytes of router weights that a prologue reads

// PRO: every workgroup routes the (few) tokens in its prologue, a wave a token,
// instead of waiting for a launch that does it once.  Each slot's first workgroup
// leaves it for the down projection; slots are in the order of their first (token,
// place), and slot s has hid rows s * T.  ROUTER: it computes the logits too (at
// most 16 experts and kProRouter bytes of router weights, which every workgroup
// reads).
// Measured: bf16, 24 tokens, d = 6144, 384 experts, h = 2048 1228 us, 6.2 TB/s,
// HBM's read rate; 4 bits, 61 tokens, d = 2048, 128 experts, h = 1024 47.7 us, 5.1
// TB/s: rows of 1 KB are four loads a wave.  One token, 4 experts of 8, bf16 12.7
// to 13.4 us for 5.3 us of bytes: the router and the choice come before the first
// load.  64 tokens, 8 experts (32 an expert): bf16 24.7 us, 2.8 TB/s, the tokens'
// operand as many bytes through the caches as the weights; 4 bits 16.6 us for 2.9
// of bytes, the codes read and decoded again for every 16 tokens.
template <int WT, int RM, int U, int EPL, bool PRO, bool ROUTER>
__global__ __launch_bounds__(kThreads, 4) void few_up_kernel(
    const char* __restrict__ x, int xb, const void* __restrict__ w1, const uint8_t* __restrict__ w1s,
    const void* __restrict__ w3, const uint8_t* __restrict__ w3s, const void* __restrict__ wr, int T, int E, int k,
    int h, int rb, const float* __restrict__ logits, int parts, const int* __restrict__ n_live,
    int* __restrict__ idx_out, float* __restrict__ w_out, int* __restrict__ n_active, FewSlot* __restrict__ slots,
    const mask_t* __restrict__ masks, const FewEntry* __restrict__ entries, char* __restrict__ hid, long hid_n) {
  const int wk = blockDim.x >> 6;  // all its waves share a row tile
  extern __shared__ __attribute__((aligned(16))) char lds[];  // lds_bytes<WT>(waves, 2)
  const int lane = threadIdx.x & 63, wv = wave_id();
  const int tiles = (h + 16 * RM - 1) / (16 * RM);
  const int slot = blockIdx.x / tiles, tile = near_tile<WT, 2 / RM>(blockIdx.x - slot * tiles, tiles);
  const int row0 = tile * 16 * RM;
  int ex;          // the expert
  mask_t toks;     // its tokens
  FewEntry ent;    // lane c: column c's
  if constexpr (PRO) {
    __shared__ mask_t mask[EPL * 64];
    __shared__ uint16_t sel[kProEntries];
    __shared__ float selw[kProEntries];
    const int live = live_tokens(n_live, T), ne = live * k;
    for (int e = threadIdx.x; e < EPL * 64; e += kThreads) mask[e] = 0;  // launched with kThreads
    float* red = (float*)lds;
    if constexpr (ROUTER) {
      // at most 16 experts: one row tile, its lines shared by the waves
      constexpr int RT = WT == kF32 ? kF32 : kBF16;  // the router's weights are in x's type
      const int r = lane & 15, q = lane >> 4;
      const WBase wb[1] = {w_base<RT>(wr, nullptr, 0, 1, E, xb)};
      const WRow row[1] = {w_row<RT>(wb[0], min(r, E - 1), xb)};
      const uint32_t xo[1] = {(uint32_t)min(r, T - 1) * (uint32_t)xb};
      f32x4_t acc[1][1] = {{{0, 0, 0, 0}}};
      stream_tile<RT, 1, 1, 1, 4, 1, 1>(wb, row, x, xo, 0, live, xb, wv, (xb + 127) >> 7, kWaves, r, q, acc, nullptr);
      put_tile(red + wv * 256, lane, acc[0][0]);
    }
    __syncthreads();
    if (wv < live) {
      float v[EPL];
      if constexpr (ROUTER) {
        v[0] = sum_tile(red, kWaves, lane & 15, wv);
      } else {
        uint32_t at[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) at[i] = (uint32_t)(wv * E + min(lane + 64 * i, E - 1));
        add_logits<EPL>(logits, parts, (uint32_t)T * (uint32_t)E, at, v);
      }
      Routed<EPL> o;
      route_token<EPL>(v, E, k, lane, o);
      if (lane < k) {
        sel[wv * k + lane] = (uint16_t)o.mine;
        atomicOr(&mask[o.mine], 1ull << wv);  // integer: the order does not matter
      }
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (o.place[i] >= 0) selw[wv * k + o.place[i]] = o.p[i] / o.s;
    }
    __syncthreads();
    // every wave: lane = entry (token lane / k, place lane % k)
    const int e = lane < ne ? sel[lane] : 0, t = lane / k;
    const mask_t mk = lane < ne ? mask[e] : 0;
    const mask_t lead = __ballot(lane < ne && (mk & ((1ull << t) - 1)) == 0);
    const int na = __popcll(lead);
    if (blockIdx.x == 0 && wv == 0) {
      if (lane == 0) *n_active = na;
      if (lane < ne && idx_out != nullptr) idx_out[lane] = e;
      if (lane < ne && w_out != nullptr) w_out[lane] = selw[lane];
    }
    if (slot >= na) return;  // the whole workgroup
    const int at = nth_token(lead, lane, slot);  // the entry that leads this slot
    ex = __builtin_amdgcn_readfirstlane(__shfl(e, at, 64));
    toks = mask[ex];
    // its entries are in its tokens' order
    ent = FewEntry{selw[nth_token(__ballot(lane < ne && e == ex), lane, lane)], slot * T + lane};
    if (tile == 0 && threadIdx.x == 0) slots[slot] = FewSlot{ex, slot * T, toks};
  } else {
    ex = nth_expert(masks, E, slot, lane, &toks);
    if (ex < 0) return;  // the whole workgroup
    ent = column_entry(entries, E, ex, toks, lane);
  }
  const int cnt = __popcll(toks);
  const WBase wb[2] = {w_base<WT>(w1, w1s, ex, E, h, rb), w_base<WT>(w3, w3s, ex, E, h, rb)};
#define TRG_TILE(RM, NT, U, XN, ROW0) \
  up_tile<WT, RM, NT, U, XN>(x, xb, wb, rb, toks, ent, cnt, c0, ROW0, h, hid, hid_n, wk, wv, lds)
  int c0 = 0;
  if constexpr (PRO) {
    if (WT == kE2M1 && cnt > 2) TRG_TILE(RM, 1, U, 4, row0);
    else TRG_TILE(RM, 1, U, 1, row0);
  } else if constexpr (WT == kE2M1) {
    // 4-bit rows are read again for every 16 tokens (from L2): the accumulators
    // of more columns and the staging do not fit into the registers together
    if (cnt <= 4) TRG_TILE(RM, 1, U, 2, row0);
    else
      for (; c0 < cnt; c0 += 16) {
        if (c0 > 0) __syncthreads();
        TRG_TILE(RM, 1, U, 8, row0);
      }
  } else if (cnt <= 16) {
    TRG_TILE(RM, 1, U, 1, row0);
  } else {
    // more columns: their accumulators take the registers of the second line, or of
    // the second row tile.  64 tokens, 32 experts, k = 8, bf16: 122.9 us with the row
    // tiles in turn (17 to 32 columns), 116.2 together.
    if (cnt <= 32) TRG_TILE(RM, 2, (RM == 1 ? U : 1), 1, row0);
    else
      for (int m = 0; m < RM; ++m) {
        if (m > 0) __syncthreads();
        // 33 to 48 columns are three tiles: 62 tokens, 8 experts, k = 4, fp32, both
        // projections 88.1 -> 81.7 us
        if (cnt <= 48) TRG_TILE(1, 3, 1, 1, row0 + 16 * m);
        else TRG_TILE(1, 4, 1, 1, row0 + 16 * m);
      }
  }
#undef TRG_TILE
}

// ---- down projection after a prologue's routing: at most 8 tokens ----------------------
// A workgroup takes 16 / KS rows of d and all chosen experts: item f is KS
// lines of a row, from line f % nit * KS of slot f / nit.  A column is a token;
// an expert's item meets only the columns of its own tokens.  T <= 16 / KS: the
// 16 rows and columns of the matrix instruction are KS groups; group g of rows
// holds the same weight rows at the item's line g, group g of columns the
// tokens at that line, and the blocks where the groups agree are summed at the
// end: more, smaller row tiles, at the same loads.  One token, 4 experts, d =
// 2048, h = 1024: bf16 5.7 us (2.7 of bytes), 4 bits 5.1; latency.
template <int WT, int U, int KS>
__global__ __launch_bounds__(kThreads, 4) void few_down_kernel(const char* __restrict__ hid, long hid_n,
                                                               const void* __restrict__ w2,
                                                               const uint8_t* __restrict__ w2s, int E, int d, int h,
                                                               int rb, const int* __restrict__ n_active,
                                                               const FewSlot* __restrict__ slots, int slots_max,
                                                               int T, const int* __restrict__ n_live,
                                                               void* __restrict__ y) {
  constexpr int P = WT == kF32 ? 1 : 2;  // parts of h
  constexpr int XE = Piece<WT>::kXE;
  constexpr int RT = 16 / KS, CT = 16 / KS;
  __shared__ __attribute__((aligned(16))) float red[kWaves * 256];
  const int lane = threadIdx.x & 63, wv = wave_id(), r = lane & 15, q = lane >> 4;
  const int live = live_tokens(n_live, T);
  const int na = *n_active;
  const int row0 = near_tile<WT, 32 / RT>(blockIdx.x, gridDim.x) * RT;
  const int row = min(row0 + r % RT, d - 1), kr = r / RT;  // this lane's weight row and line group
  const int ct = r % CT, kc = r / CT;                      // this lane's column: token and line group
  const int nall = (rb + 127) >> 7, nit = (nall + KS - 1) / KS;
  const int F = na * nit;
  f32x4_t acc = {0, 0, 0, 0};
  struct Items {
    WStep w[U];
    unsigned long long mask[U];
    int off[U], c[U];
  };
  int s = wv / nit, c = wv - s * nit;  // the next item to load
  // items f, f + kWaves, ...: one past the end reads expert 0 (so its loads are
  // in bounds) for no token
  auto load = [&](Items& o, int f) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = f + u * kWaves < F;
      // read without waiting for n_active; from there on slots hold anything
      const FewSlot sl = slots[min(s, slots_max - 1)];
      o.mask[u] = in ? sl.mask : 0;
      o.off[u] = in ? sl.off : 0;
      o.c[u] = in ? c * KS : 0;
      const WBase wb = w_base<WT>(w2, w2s, in ? sl.e : 0, E, d, rb);
      o.w[u] = w_load<WT>(wb, w_row<WT>(wb, row, rb), o.c[u] + kr, q, rb);
      c += kWaves;
      while (c >= nit) {
        c -= nit;
        ++s;
      }
    }
  };
  auto multiply = [&](Items& o) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool on = (o.mask[u] >> ct) & 1;
      const uint32_t xo = (uint32_t)(o.off[u] + __popcll(o.mask[u] & ((1ull << ct) - 1))) * (uint32_t)(h * XE);
      XStep<WT> x[P];
      if (on) {
#pragma unroll
        for (int p = 0; p < P; ++p) x_load<WT>(hid + p * hid_n * XE, xo, o.c[u] + kc, q, rb, x[p]);
      }
      if ((o.c[u] + KS) * 128 > rb) {  // the same for the whole wave
        w_mask<WT>(o.w[u], o.c[u] + kr, q, rb);
#pragma unroll
        for (int p = 0; p < P; ++p) {
          x_mask<WT>(x[p].v[0], o.c[u] + kc, q, 0, rb);
          x_mask<WT>(x[p].v[1], o.c[u] + kc, q, 1, rb);
        }
      }
      f32x4_t t = {0, 0, 0, 0};
#pragma unroll
      for (int p = 0; p < P; ++p) t = mma_step<WT>(o.w[u], x[p], t);
      // columns of tokens that did not choose this expert are left alone, not
      // given 0 * w: an infinite or NaN weight is its own tokens' matter
#pragma unroll
      for (int z = 0; z < 4; ++z) acc[z] = on ? acc[z] + t[z] : acc[z];
    }
  };
  Items a, b;
  load(a, wv);
  if (wv < F) {
    for (int f = wv + kWaves * U; f < F; f += kWaves * U) {
      load(b, f);
      multiply(a);
      a = b;
    }
    multiply(a);
  }
  put_tile(red + wv * 256, lane, acc);
  __syncthreads();
  const int orow = threadIdx.x % RT, t = threadIdx.x / RT;
  if (threadIdx.x < RT * CT && t < live && row0 + orow < d) {
    float v = 0.f;
#pragma unroll
    for (int g = 0; g < KS; ++g) v += sum_tile(red, kWaves, g * RT + orow, g * CT + t);
    const long at = (long)t * d + row0 + orow;
    if constexpr (WT == kF32) ((float*)y)[at] = v;
    else ((uint16_t*)y)[at] = f2bf(v);
  }
}

// ---- down projection, a row an entry --------------------------------------------------
// As the up projection: workgroup (expert, row tiles of d), columns the expert's own
// tokens, lines shared by wk waves; ent: lane c has column c's entry, the hidden
// row it reads and the row it writes; every entry's row goes out in fp32 and the
// join adds each token's k rows in order.  Those rows are R d floats, out and
// in: 3 % of the weights' bytes with two tokens an expert at h = 1024 and 4
// bits, 0.25 % in bf16 at h = 2048.
// H > 0 (at most H <= 8 tokens, h in halves): columns 0..H-1 are the tokens' hi
// halves and H..2H-1 their lo halves, added at the end: half the matrix
// instructions and operand reads of two passes over the columns.  4-bit weights,
// 61 tokens, 128 experts: 32.0 -> 29.9 us; bf16, whose reads set the pace, no
// different, so it keeps the one form.
// Measured: bf16, 24 tokens, 384 experts, d = 6144, h = 2048 621 us, 6.2 TB/s; 4
// bits, 61 tokens, 128 experts, d = 2048, h = 1024 29.4 us, 4.1 TB/s (4.5 with the
// hidden vector): a row is 512 bytes, so a workgroup's life is one trip to memory.
// 64 tokens, 8 experts: bf16 18.3 us, 4 bits 14.4, for the up projection's reasons.
template <int WT, int RM, int NT, int U, int XN, int H>
TRG_DEV void down_tile(const char* __restrict__ hid, long hid_n, const WBase* wb, int rb, int ent, int cnt, int col0,
                       int row0, int d, int h, int wk, int kw, char* lds, float* __restrict__ yp) {
  float* red = (float*)lds;
  constexpr int P = WT == kF32 || H > 0 ? 1 : 2, XE = Piece<WT>::kXE;
  constexpr int CT = H > 0 ? H : 16;  // tokens a column tile
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  WRow wr[RM];
#pragma unroll
  for (int m = 0; m < RM; ++m) wr[m] = w_row<WT>(wb[0], min(row0 + m * 16 + r, d - 1), rb);
  uint32_t xo[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int c = col0 + i * CT + r % CT;
    xo[i] = (uint32_t)__builtin_amdgcn_ds_bpermute(min(c, cnt - 1) * 4, ent) * (uint32_t)(h * XE);
    if (r >= CT) xo[i] += (uint32_t)hid_n * XE;
  }
  f32x4_t acc[RM][NT];
#pragma unroll
  for (int m = 0; m < RM; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[m][i] = f32x4_t{0, 0, 0, 0};
  stream_tile<WT, 1, RM, NT, U, P, XN, 1>(wb, wr, hid, xo, hid_n * XE, H > 0 ? 2 * H : cnt - col0, rb, kw,
                                       (rb + 127) >> 7, wk, r, q, acc, lds + kw * kStage);
#pragma unroll
  for (int m = 0; m < RM; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if (WT == kE2M1 || m + i > 0) __syncthreads();
      put_tile(red + kw * 256, lane, acc[m][i]);
      __syncthreads();
      for (int o = threadIdx.x; o < 256; o += wk * 64) {
        const int lr = o & 15, col = o >> 4, c = col0 + i * CT + col, row = row0 + m * 16 + lr;
        const int yrow = __builtin_amdgcn_ds_bpermute(c * 4, ent);
        if (col < CT && c < cnt && row < d) {
          float v = sum_tile(red, wk, lr, col);
          if constexpr (H > 0) v += sum_tile(red, wk, lr, col + H);
          yp[(long)yrow * d + row] = v;
        }
      }
    }
}

template <int WT, int RM, int U>
__global__ __launch_bounds__(kThreads, 4) void few_down_rows_kernel(const char* __restrict__ hid, long hid_n,
                                                                    const void* __restrict__ w2,
                                                                    const uint8_t* __restrict__ w2s, int E, int d,
                                                                    int h, int rb, const mask_t* __restrict__ masks,
                                                                    const FewEntry* __restrict__ entries,
                                                                    float* __restrict__ yp) {
  extern __shared__ __attribute__((aligned(16))) char lds[];  // lds_bytes<WT>(waves, 1)
  const int wv = wave_id(), wk = blockDim.x >> 6, lane = threadIdx.x & 63;
  const int tiles = (d + 16 * RM - 1) / (16 * RM);
  const int slot = blockIdx.x / tiles, tile = blockIdx.x - slot * tiles;
  const int row0 = tile * 16 * RM;
  mask_t toks;
  const int ex = nth_expert(masks, E, slot, lane, &toks);
  if (ex < 0) return;
  const int cnt = __popcll(toks), ent = column_entry(entries, E, ex, toks, lane).row;
  const WBase wb[1] = {w_base<WT>(w2, w2s, ex, E, d, rb)};
#define TRG_TILE(RM, NT, U, XN, H, ROW0) \
  down_tile<WT, RM, NT, U, XN, H>(hid, hid_n, wb, rb, ent, cnt, c0, ROW0, d, h, wk, wv, lds, yp)
  int c0 = 0;
  if constexpr (WT == kE2M1) {
    if (cnt <= 2) TRG_TILE(RM, 1, U, 1, 2, row0);
    else if (cnt <= 8) TRG_TILE(RM, 1, U, 4, 8, row0);
    else
      for (; c0 < cnt; c0 += 16) {
        if (c0 > 0) __syncthreads();
        TRG_TILE(RM, 1, U, 4, 0, row0);
      }
  } else if (cnt <= 16) {
    TRG_TILE(RM, 1, U, 1, 0, row0);
  } else if (cnt <= 32) {
    // all row tiles at once: 64 tokens, 32 experts, k = 8, bf16 117.3 -> 110.7 us
    TRG_TILE(RM, 2, 1, 1, 0, row0);
  } else {
    // two at a time: with four the accumulators spill (k = 16: 156.9 -> 174.1)
    constexpr int RN = RM > 2 ? 2 : RM;
    for (int m = 0; m < RM; m += RN) {
      if (m > 0) __syncthreads();
      if (cnt <= 48) TRG_TILE(RN, 3, 1, 1, 0, row0 + 16 * m);
      else TRG_TILE(RN, 4, 1, 1, 0, row0 + 16 * m);
    }
  }
#undef TRG_TILE
}

// y[t] = sum over its k entries' rows, in the order of its choices.  61 tokens, 4
// entries, d = 2048: 4.8 us, latency of the launch and one trip.
template <class OUT>
__global__ __launch_bounds__(256) void few_join_kernel(const float* __restrict__ yp, int T, int d, int k,
                                                       const int* __restrict__ n_live, OUT* __restrict__ y) {
  const int i = (blockIdx.x * 256 + threadIdx.x) * 4;  // d is a multiple of 4
  const int t = blockIdx.y;
  if (i >= d || t >= live_tokens(n_live, T)) return;
  float4 a = make_float4(0, 0, 0, 0);
  constexpr int B = 8;  // rows in flight; past the last one it is loaded again and not added
  for (int j0 = 0; j0 < k; j0 += B) {
    float4 b[B];
#pragma unroll
    for (int j = 0; j < B; ++j) b[j] = *(const float4*)(yp + (long)(t * k + min(j0 + j, k - 1)) * d + i);
#pragma unroll
    for (int j = 0; j < B; ++j)
      if (j0 + j < k) {
        a.x += b[j].x;
        a.y += b[j].y;
        a.z += b[j].z;
        a.w += b[j].w;
      }
  }
  OUT* o = y + (long)t * d + i;
  Elt<OUT>::st(o, a.x);
  Elt<OUT>::st(o + 1, a.y);
  Elt<OUT>::st(o + 2, a.z);
  Elt<OUT>::st(o + 3, a.w);
}

template <int WT, int NM, int NT, int U, int XN, int WAVES, class OUT>
hipError_t linear_nt(const void* x, const void* w, const uint8_t* ws, int T, int n, int rb, int xb, int parts,
                     const int* n_live, OUT* out, hipStream_t st, mask_t* masks = nullptr, int nz = 0) {
  const int lines = (rb + 127) / 128, pl = (lines + parts - 1) / parts;
  few_linear_kernel<WT, NM, NT, U, XN, WAVES, OUT>
      <<<dim3((n + 16 * NM - 1) / (16 * NM), parts), WAVES * 64, 0, st>>>((const char*)x, w, ws, T, n, rb, xb, pl,
                                                                          n_live, out, masks, nz);
  return hipGetLastError();
}

// Waves that share a row tile along k, from a weight row's bytes and the row
// tiles there may be: long rows need the waves (a wave by itself has too few
// loads in flight), short ones leave a wave too little to do, and with many
// tiles the chip is full without them.  Measured, us a pass with 8 / 4 / 2 / 1
// waves: 24 tokens, 384 experts, rows of 12 and 4 KB 1843 / 1926 / 2018 / 2029; 61
// tokens, 128 experts, rows of 4 and 2 KB 260 / 268 / 276 / 270.  4 bits, waves of
// the up and of the down projection: 61 tokens, 128 experts, rows of 1 KB and 512
// bytes 4, 4: 99.3; 2, 4: 94.5; 2, 2: 90.5; 2, 1: 88.6; 1, 2: 93.0; 64 tokens, 8
// experts 4, 4: 39.5; 4, 2: 40.5; 2, 2: 42.0.
int row_waves(int rb, long tiles) { return rb >= 4096 ? 8 : rb > 1024 || tiles < 4096 ? 4 : rb > 512 ? 2 : 1; }

// LDS of a product's workgroup: the waves' accumulators of `tiles` matrices, or
// their staging buffers.
template <int WT>
size_t lds_bytes(int waves, int tiles) {
  return (size_t)waves * (WT == kE2M1 ? kStage : tiles * 1024);
}

// Which of its launches' variants a call takes.
FewPlan few_plan_of(int T, int d, int E, int k, int h, int wt) {
  const int xe = wt == kF32 ? 4 : 2, xb = d * xe;
  // bytes of a weight row
  const int rb1 = wt == kE2M1 ? d / 2 : xb, rb2 = wt == kE2M1 ? h / 2 : h * xe;
  const long slots = slots_of(T, E, k), up_tiles = slots * ((h + 15) / 16), down_tiles = slots * ((d + 15) / 16);
  FewPlan p;
  p.pro = in_prologue(T, E, k, h);
  p.router = p.pro && E <= 16 && E * xb <= kProRouter;
  p.logit_tiles = T <= 16 ? 1 : T <= 32 ? 2 : 4;
  // 129 to 256 experts take the next width's 8 a lane: 4 would save 0.2 to 1.3 us of 18 to 81 (256 experts, 1 to
  // 40 tokens)
  p.epl = p.router ? 1 : E <= 64 && !p.pro ? 1 : E <= 128 ? 2 : E <= 512 ? 8 : 16;
  // two row tiles a wave would leave CUs idle where there are few; 4-bit rows' staging and accumulators leave
  // no registers for a second one
  p.up_rows = p.pro || wt == kE2M1 || up_tiles < 1024 ? 1 : 2;
  p.up_waves = p.pro ? kWaves : row_waves(rb1, up_tiles);
  // Four row tiles a wave read the operand once for 64 rows; with few tiles that
  // leaves CUs idle.  Measured, us a call with 1 / 2 / 4 a wave, 8 experts (2 taken):
  // 64 tokens 58.4 / 51.3 / 54.5 in bf16 and 41.0 / 39.1 / 40.5 in 4 bits, 16 tokens
  // 37.1 / 36.2 / 36.6 and 21.5 / 22.8 / 23.6; 128 experts, 61 tokens (4 taken) 287 /
  // 260 / 262 and 98.9 / 92.5 / 88.4.
  p.down_rows = down_tiles < 4096 ? 2 : 4;
  p.down_waves = row_waves(rb2, down_tiles);
  return p;
}

template <int WT>
hipError_t few_any(const moe_few_args& a, hipStream_t st) {
  constexpr int XE = WT == kF32 ? 4 : 2;
  const FewLayout l = few_layout(a.T, a.d, a.E, a.k, a.h);
  const FewPlan p = few_plan_of(a.T, a.d, a.E, a.k, a.h, WT);
  char* ws = (char*)a.ws;
  int* n_active = (int*)(ws + l.n_active);
  FewSlot* slots = (FewSlot*)(ws + l.slots);
  mask_t* masks = (mask_t*)(ws + l.masks);
  FewEntry* entries = (FewEntry*)(ws + l.entries);
  float* logits = (float*)(ws + l.logits);
  char* hid = ws + l.hid;
  float* yp = (float*)(ws + l.yp);
  const int slots_max = slots_of(a.T, a.E, a.k);
  const long hid_n = (long)hid_rows(a.T, a.E, a.k, a.h) * a.h;
  const int xb = a.d * XE;
  const int parts = logit_parts(xb);
  hipError_t e = hipSuccess;
  if (!p.router) {
    constexpr int RT = WT == kF32 ? kF32 : kBF16;
#define TRG_LOGITS(NT) \
  linear_nt<RT, 1, NT, 1, 1, kWaves, float>(a.x, a.wr, nullptr, a.T, a.E, xb, xb, parts, a.n_live, logits, st, \
                                                masks, p.pro ? 0 : a.E)
    e = p.logit_tiles == 1 ? TRG_LOGITS(1) : p.logit_tiles == 2 ? TRG_LOGITS(2) : TRG_LOGITS(4);
#undef TRG_LOGITS
    if (e != hipSuccess) return e;
  }
  if (!p.pro) {
#define TRG_ROUTE(N)                                                                                                  \
  few_route_kernel<N><<<a.T, 64, 0, st>>>(logits, parts, a.T, a.E, a.k, a.n_live, a.topk_idx, a.topk_w, masks, entries)
    if (p.epl == 1) TRG_ROUTE(1);
    else if (p.epl == 2) TRG_ROUTE(2);
    else if (p.epl == 8) TRG_ROUTE(8);
    else TRG_ROUTE(16);
#undef TRG_ROUTE
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  // bytes of a weight row
  const int rb1 = WT == kE2M1 ? a.d / 2 : a.d * XE, rb2 = WT == kE2M1 ? a.h / 2 : a.h * XE;
  constexpr int U = WT == kE2M1 ? 1 : 2, UP = WT == kE2M1 ? 1 : 4;  // lines at a time
  constexpr int UR = WT == kE2M1 ? 1 : 2;                             // row tiles a wave, at most
  const int uw = p.up_waves, dw = p.down_waves;
#define TRG_UP(RM, U, EPL, PRO, ROUTER)                                                                             \
  few_up_kernel<WT, RM, U, EPL, PRO, ROUTER>                                                                       \
      <<<(unsigned)slots_max * ((a.h + 16 * RM - 1) / (16 * RM)), uw * 64, lds_bytes<WT>(uw, 2), st>>>(            \
          (const char*)a.x, xb, a.w1, a.w1s, a.w3, a.w3s, a.wr, a.T, a.E, a.k, a.h, rb1, logits, parts, a.n_live,  \
          a.topk_idx, a.topk_w, n_active, slots, masks, entries, hid, hid_n)
  if (!p.pro && p.up_rows == 1) TRG_UP(1, U, 1, false, false);
  else if (!p.pro) TRG_UP(UR, U, 1, false, false);
  else if (p.router) TRG_UP(1, UP, 1, true, true);
  else if (p.epl == 2) TRG_UP(1, UP, 2, true, false);
  else if (p.epl == 8) TRG_UP(1, UP, 8, true, false);
  else TRG_UP(1, UP, 16, true, false);
#undef TRG_UP
  e = hipGetLastError();
  if (e != hipSuccess) return e;
#define TRG_DOWN(KS)                                                                                                \
  few_down_kernel<WT, U, KS><<<(a.d + 16 / KS - 1) / (16 / KS), kThreads, 0, st>>>(hid, hid_n, a.w2, a.w2s, a.E, a.d, \
                                                                                   a.h, rb2, n_active, slots,       \
                                                                                   slots_max, a.T, a.n_live, a.y)
  if (p.pro) {
    if (a.T <= 4) TRG_DOWN(4);
    else TRG_DOWN(2);
    return hipGetLastError();
  }
#undef TRG_DOWN
#define TRG_ROWS(RM, U)                                                                                             \
  few_down_rows_kernel<WT, RM, U><<<(unsigned)slots_max * ((a.d + 16 * RM - 1) / (16 * RM)), 64 * dw,               \
                                    lds_bytes<WT>(dw, 1), st>>>(hid, hid_n, a.w2, a.w2s, a.E, a.d, a.h, rb2, masks, \
                                                                entries, yp)
  if (p.down_rows == 2) TRG_ROWS(2, 1);
  else TRG_ROWS(4, 1);
#undef TRG_ROWS
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 jg((a.d / 4 + 255) / 256, a.T);
  if constexpr (WT == kF32)
    few_join_kernel<float><<<jg, 256, 0, st>>>(yp, a.T, a.d, a.k, a.n_live, (float*)a.y);
  else
    few_join_kernel<uint16_t><<<jg, 256, 0, st>>>(yp, a.T, a.d, a.k, a.n_live, (uint16_t*)a.y);
  return hipGetLastError();
}

}  // namespace

size_t few_ws_bytes(int T, int d, int E, int k, int h) { return few_layout(T, d, E, k, h).bytes; }
size_t few_ws_bytes_up_to(int T, int d, int E, int k, int h) {
  size_t most = 0;  // not always the largest batch's: smaller ones may take another path
  for (int t = 1; t <= T; ++t) {
    const size_t b = few_layout(t, d, E, k, h).bytes;
    most = b > most ? b : most;
  }
  return most;
}

hipError_t launch_few_fwd(const moe_few_args& a, hipStream_t st) {
  if (a.wt == MOE_E2M1) return few_any<kE2M1>(a, st);
  if (a.wt == MOE_BF16) return few_any<kBF16>(a, st);
  return few_any<kF32>(a, st);
}

FewPlan few_plan(int T, int d, int E, int k, int h, int wt) {
  return few_plan_of(T, d, E, k, h, wt == MOE_E2M1 ? kE2M1 : wt == MOE_BF16 ? kBF16 : kF32);
}

// Row tiles a wave: more read the tokens' operand fewer times, fewer leave less
// of the chip idle at the end.  The model: a workgroup costs its row tiles plus
// the staging of its column tiles, a CU does ceil(workgroups / 256) of them.  It
// orders the counts by their rounds and is no estimate of the times.  Four row
// tiles are left out above 32 tokens: with four column tiles their accumulators
// spill 42 registers.  Measured in us, K = 6144, with 1 / 2 / 3 / 4 row tiles:
//   n       13 tokens                 32                        64
//   24576   22.3 / 18.7 / 17.4 / 25.7 37.1 / 35.6 / 27.5 / 32.6 75.8 / 51.4 / 44.3 / 79.3
//   28672   31.4 / 26.4 / 25.8 / 27.5 50.6 / 45.4 / 42.3 / 34.6 96.6 / 69.8 / 61.5 / 84.3
//   32768   37.3 / 31.0 / 29.9 / 31.6 59.7 / 49.5 / 45.3 / 38.2 111 / 73.6 / 64.9 / 87.4
//   40960   47.0 / 39.1 / 37.0 / 47.5 75.5 / 61.5 / 59.4 / 53.9 140 / 90.8 / 85.6 / 129
// and 6144 x 2048, 64 tokens 11.8 / 8.6 / 10.0 / 15.9.  The rule takes the fastest
// of them but for 13 tokens with n = 28672 and 32768 (four, 7 % slower than three).
int linear_row_tiles(int T, int n) {
  const long tiles = (n + 15) / 16;
  const int nt = T <= 16 ? 1 : T <= 32 ? 2 : 4;
  int nm = 1;
  long best = 0;
  for (int m = 1; m <= (nt == 4 ? 3 : 4); ++m) {
    const long cost = ((tiles + m - 1) / m + 255) / 256 * (m + nt);
    if (m == 1 || cost < best) {
      best = cost;
      nm = m;
    }
  }
  return nm;
}

hipError_t launch_linear_e2m1(const void* x, const uint8_t* q, const uint8_t* s, int T, int n, int K, void* y,
                              hipStream_t st) {
  const int nt = T <= 16 ? 1 : T <= 32 ? 2 : 4, nm = linear_row_tiles(T, n);
#define TRG_LINEAR(NM, NT, XN) \
  linear_nt<kE2M1, NM, NT, 1, XN, kWaves, uint16_t>(x, q, s, T, n, K / 2, K * 2, 1, nullptr, (uint16_t*)y, st)
#define TRG_NT(NM) \
  if (nm == NM) return T <= 4 ? TRG_LINEAR(NM, 1, 2) : nt == 1 ? TRG_LINEAR(NM, 1, 8) : TRG_LINEAR(NM, 2, 8)
  if (nt == 4) return nm == 1 ? TRG_LINEAR(1, 4, 8) : nm == 2 ? TRG_LINEAR(2, 4, 8) : TRG_LINEAR(3, 4, 8);
  TRG_NT(1);
  TRG_NT(2);
  TRG_NT(3);
  return T <= 4 ? TRG_LINEAR(4, 1, 2) : nt == 1 ? TRG_LINEAR(4, 1, 8) : TRG_LINEAR(4, 2, 8);
#undef TRG_LINEAR
#undef TRG_NT
}

}  // namespace trg
