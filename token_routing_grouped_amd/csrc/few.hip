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
// instruction is free next to the weight stream.  fp32 weights use the fp32
// matrix instruction and h stays fp32.
//
// Launches: router logits; routing (one workgroup); up projection with the
// SwiGLU and gate epilogue; down projection, summing over the experts in its
// accumulators (a column is a token, whichever experts it chose), so there is
// no combine step and no partial result.  Every sum has a fixed order.
#include "common.h"
#include "kernels.h"

namespace trg {

namespace {

enum { kF32 = 0, kBF16 = 1, kE2M1 = 2 };  // weight storage

constexpr int kWaves = 8;          // waves of the product kernels' workgroups
constexpr int kThreads = kWaves * 64;

// One chosen expert: its index, the place of its first entry in the
// expert-ordered entry list, and which tokens chose it.
struct FewSlot {
  int e, off;
  unsigned long long mask;
};

// Rows of the hidden buffer: an entry's own, or (routing in the up
// projection's prologue) T for every slot.
bool in_prologue(int T, int k);
int hid_rows(int T, int E, int k) {
  const int R = T * k, S = R < E ? R : E;
  return in_prologue(T, k) ? S * T : R;
}
int logit_parts(int d, int es);
int down_parts(int T, int d);

struct FewLayout {
  size_t n_active, slots, gate, logits, hid, part, bytes;
};

FewLayout few_layout(int T, int d, int E, int k, int h) {
  const size_t R = (size_t)T * k, S = R < (size_t)E ? R : (size_t)E;
  FewLayout l;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t p = at;
    at += (n + 255) / 256 * 256;
    return p;
  };
  l.n_active = take(sizeof(int));
  l.slots = take(S * sizeof(FewSlot));
  l.gate = take(R * sizeof(float));
  l.logits = take((size_t)logit_parts(d, 4) * T * E * sizeof(float));  // fp32 rows have the most lines
  l.hid = take((size_t)hid_rows(T, E, k) * h * sizeof(float));         // fp32, or the hi and lo bf16 halves
  const int dp = down_parts(T, d);
  l.part = take(dp > 1 ? (size_t)dp * T * d * sizeof(float) : 0);
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

TRG_DEV uint4 zero16() { return make_uint4(0, 0, 0, 0); }

// A lane's place in a weight matrix of n rows with rb bytes a row.
struct WRow {
  const char* p;        // its row
  const uint8_t* s;     // E2M1: its row's scales in chunk 0
  long sstride;         // E2M1: bytes from a 128-value chunk's scales to the next one's
};
template <int WT>
TRG_DEV WRow w_row(const void* w, const uint8_t* ws, long n, long row, int rb) {
  WRow r;
  r.p = (const char*)w + row * rb;
  r.s = WT == kE2M1 ? ws + row * 4 : nullptr;
  r.sstride = n * 4;
  return r;
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
TRG_DEV WStep w_load(const WRow& r, int c, int q, int rb) {
  WStep o;
  const int off = c * 128 + q * 32, last = rb - 16;
  o.v[0] = *(const uint4*)(r.p + min(off, last));
  o.v[1] = *(const uint4*)(r.p + min(off + 16, last));
  o.sb = 0;
  if constexpr (WT == kE2M1) {
    // block b = off / 16, its byte in chunk b / 4; b is even, so both bytes of
    // the step are in one chunk (the second may be a place past the last block)
    const int bk = min(off, last) / 16 & ~1;
    o.sb = *(const uint16_t*)(r.s + (long)(bk >> 2) * r.sstride + (bk & 3));
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
// parts each.  Where the weights are past the row's end this is the row's last
// piece again, which meets zeros.
template <int WT>
struct XStep {
  uint4 v[2][Piece<WT>::kX];
};
template <int WT>
TRG_DEV void x_load(const char* xr, int c, int q, int rb, XStep<WT>& o) {
  const int off = c * 128 + q * 32;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const char* p = xr + min(off + 16 * i, rb - 16) / 16 * (Piece<WT>::kK * Piece<WT>::kXE);
#pragma unroll
    for (int j = 0; j < Piece<WT>::kX; ++j) o.v[i][j] = *(const uint4*)(p + j * 16);
  }
}
template <int WT>
TRG_DEV f32x4_t mma_step(const WStep& w, const XStep<WT>& x, f32x4_t acc) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    acc = mma_piece<WT>(w.v[i], WT == kE2M1 ? e8m0((w.sb >> (8 * i)) & 255u) : 0.f, x.v[i], acc);
  return acc;
}

// ---- products of NM 16-row tiles with NT * 16 columns --------------------------
// acc[m][n] over lines c0, c0 + step, ... < c1 of the rows, U lines a batch.  A
// batch's weights are loaded while the one before is multiplied; the tokens'
// operand comes from the caches and is loaded where it is used.  With one tile
// of columns only the lanes of columns that are `on` load it (a few tokens are
// a few lanes); the others' registers hold anything: columns do not mix, and
// theirs are not stored.
template <int WT, int NM, int NT, int U>
TRG_DEV void stream_tile(const WRow* wr, const char* const* xr, bool on, int rb, int c0, int c1, int step, int q,
                         f32x4_t (*acc)[NT]) {
  if (c0 >= c1) return;
  const int past = (rb + 127) >> 7;  // a line that is past every row's end
  WStep w[U][NM];
  auto line = [&](int c) { return c < c1 ? c : past; };
  auto load_w = [&](int c, WStep (*o)[NM]) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < NM; ++m) o[u][m] = w_load<WT>(wr[m], line(c + u * step), q, rb);
  };
  auto load_x = [&](int c, int n, XStep<WT>* x) {
#pragma unroll
    for (int u = 0; u < U; ++u) x_load<WT>(xr[n], line(c + u * step), q, rb, x[u]);
  };
  auto multiply = [&](int c, int n, XStep<WT>* x) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < NM; ++m) acc[m][n] = mma_step<WT>(w[u][m], x[u], acc[m][n]);
  };
  auto mask_w = [&](int c) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < NM; ++m) w_mask<WT>(w[u][m], line(c + u * step), q, rb);
  };
  load_w(c0, w);
  for (; c0 + step * U < c1; c0 += step * U) {
    WStep wn[U][NM];
    XStep<WT> x[U];
    if (NT > 1 || on) load_x(c0, 0, x);
    load_w(c0 + step * U, wn);
    multiply(c0, 0, x);  // not the last batch: every line of it is inside
#pragma unroll
    for (int n = 1; n < NT; ++n) {
      load_x(c0, n, x);
      multiply(c0, n, x);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < NM; ++m) w[u][m] = wn[u][m];
  }
  XStep<WT> x[U];
  if (NT > 1 || on) load_x(c0, 0, x);
  mask_w(c0);
  multiply(c0, 0, x);
#pragma unroll
  for (int n = 1; n < NT; ++n) {
    load_x(c0, n, x);
    multiply(c0, n, x);
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
// lines from blockIdx.y * part_lines and writes its own [T, n] of out.
template <int WT, int NM, int NT, int U, class OUT>
__global__ __launch_bounds__(kThreads, NM* NT > 4 ? 2 : 4) void few_linear_kernel(const char* __restrict__ x,
                                                                 const void* __restrict__ w,
                                                                 const uint8_t* __restrict__ ws, int T, int n, int rb,
                                                                 int xb, int part_lines,
                                                                 const int* __restrict__ n_live,
                                                                 OUT* __restrict__ out) {
  __shared__ __attribute__((aligned(16))) float red[kWaves * 256];
  const int lane = threadIdx.x & 63, wv = wave_id(), r = lane & 15, q = lane >> 4;
  const int live = live_tokens(n_live, T);
  const int row0 = blockIdx.x * (16 * NM);
  const int c0 = blockIdx.y * part_lines, c1 = min((rb + 127) >> 7, c0 + part_lines);
  WRow wr[NM];
#pragma unroll
  for (int m = 0; m < NM; ++m) wr[m] = w_row<WT>(w, ws, n, min(row0 + m * 16 + r, n - 1), rb);
  const char* xr[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) xr[i] = x + (long)min(i * 16 + r, T - 1) * xb;
  f32x4_t acc[NM][NT];
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[m][i] = f32x4_t{0, 0, 0, 0};
  stream_tile<WT, NM, NT, U>(wr, xr, r < live, rb, c0 + wv, c1, kWaves, q, acc);
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if (m + i > 0) __syncthreads();
      put_tile(red + wv * 256, lane, acc[m][i]);
      __syncthreads();
      const int row = row0 + m * 16 + (threadIdx.x & 15), t = i * 16 + ((threadIdx.x >> 4) & 15);
      if (threadIdx.x < 256 && t < live && row < n)
        Elt<OUT>::st(out + ((long)blockIdx.y * T + t) * n + row,
                     sum_tile(red, kWaves, threadIdx.x & 15, (threadIdx.x >> 4) & 15));
    }
}

// ---- routing ---------------------------------------------------------------------
// Largest of v over the wave (0 is the identity), known to every lane: five
// steps inside the vector registers (rows of 16, then the rows' ends).
template <int CTRL>
TRG_DEV uint32_t max_dpp(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false));
}
TRG_DEV uint32_t wave_max_u32(uint32_t v) {
  v = max_dpp<0x111>(v);  // row_shr:1
  v = max_dpp<0x112>(v);  // row_shr:2
  v = max_dpp<0x114>(v);  // row_shr:4
  v = max_dpp<0x118>(v);  // row_shr:8
  v = max_dpp<0x142>(v);  // row_bcast:15
  v = max_dpp<0x143>(v);  // row_bcast:31
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// One wave routes token t: the k largest logits, ties to the lower expert, a
// NaN never before a number (moe_route's rules), and their softmax values.
// Logits come as `parts` partial sums [parts][T][E], added in order.  A logit
// becomes a 32-bit key that orders like it (0 is below every key), so a round
// is one wave maximum and the first lane of the first register that holds it:
// expert e is lane e % 64, register e / 64.  sel, selw: this token's k places.
template <int EPL>
TRG_DEV void route_token(const float* __restrict__ logits, int parts, int T, int E, int k, int t, int lane, int* sel,
                         float* selw, unsigned long long* mask) {
  float v[EPL], p[EPL];
  uint32_t key[EPL];
  float m = -INFINITY, s = 0.f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    float x = -INFINITY;
    if (e < E) {
      const float* L = logits + (long)t * E + e;
      x = L[0];
      for (int a = 1; a < parts; ++a) x += L[(long)a * T * E];
    }
    v[i] = (x != x) ? -INFINITY : x;
    m = fmaxf(m, v[i]);
    const uint32_t b = __float_as_uint(v[i] + 0.0f);  // -0 and 0 are equal
    key[i] = e < E ? ((b & 0x80000000u) ? ~b : b | 0x80000000u) : 0u;
  }
  m = wave_max(m);
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    p[i] = lane + 64 * i < E ? expf(v[i] - m) : 0.f;
    s += p[i];
  }
  s = wave_sum(s);
  for (int j = 0; j < k; ++j) {
    uint32_t b = key[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) b = max(b, key[i]);
    b = wave_max_u32(b);
    bool found = false;  // the same for the whole wave
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const unsigned long long at = __ballot(key[i] == b);
      if (!found && at != 0) {
        found = true;
        const int l = __ffsll((unsigned long long)at) - 1;
        if (lane == l) {
          const int e = l + 64 * i;
          key[i] = 0;
          sel[j] = e;
          selw[j] = p[i] / s;
          atomicOr(&mask[e], 1ull << t);  // integer: the order does not matter
        }
      }
    }
  }
}

// Routing in a launch of its own (more than kProTokens tokens or kProEntries
// entries): one workgroup, a wave a token at a time; then the chosen experts'
// token masks are compacted, in expert order, into slots.
template <int EPL>
__global__ __launch_bounds__(1024) void few_route_kernel(const float* __restrict__ logits, int parts, int T, int E,
                                                         int k, const int* __restrict__ n_live,
                                                         int* __restrict__ idx_out, float* __restrict__ w_out,
                                                         int* __restrict__ n_active, FewSlot* __restrict__ slots,
                                                         float* __restrict__ gate) {
  __shared__ unsigned long long mask[1024];
  __shared__ int first[1024];
  __shared__ int tmp[32];
  __shared__ int sel[64 * 32];
  __shared__ float selw[64 * 32];
  const int lane = threadIdx.x & 63, wv = wave_id();
  mask[threadIdx.x] = 0;
  __syncthreads();
  const int live = live_tokens(n_live, T);
  for (int t = wv; t < live; t += 16)
    route_token<EPL>(logits, parts, T, E, k, t, lane, sel + t * 32, selw + t * 32, mask);
  __syncthreads();
  // experts with tokens, in order: (slots, entries) before each, in one scan
  const unsigned long long mk = mask[threadIdx.x];
  const int cnt = __popcll(mk);
  int total;
  const int before = block_excl_scan_1024((cnt > 0 ? 1 << 16 : 0) | cnt, tmp, &total);  // at most 2048 entries
  first[threadIdx.x] = before & 0xFFFF;
  if (cnt > 0) slots[before >> 16] = FewSlot{(int)threadIdx.x, before & 0xFFFF, mk};
  if (threadIdx.x == 0) *n_active = total >> 16;
  __syncthreads();
  for (int i = threadIdx.x; i < live * k; i += 1024) {
    const int t = i / k, j = i - t * k, e = sel[t * 32 + j];
    gate[first[e] + __popcll(mask[e] & ((1ull << t) - 1))] = selw[t * 32 + j];
    if (idx_out != nullptr) idx_out[i] = e;
    if (w_out != nullptr) w_out[i] = selw[t * 32 + j];
  }
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

// 16 rows of h for a slot's columns: both matrices' rows, shared by wk waves
// along k, then h = gate * silu(g) * u.  red: this group's 2 * wk * 256 floats;
// tid: thread within the group.
template <int WT, int NT, int U>
TRG_DEV void up_tile(const char* __restrict__ x, int xb, const WRow* wr, int rb, unsigned long long mask,
                     const float* gate, int cnt, int row0, int h, char* hid, long hid_n, long pos0, int wk, int kw,
                     int tid, float* red) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const char* xr[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) xr[i] = x + (long)nth_token(mask, lane, min(i * 16 + r, cnt - 1)) * xb;
  f32x4_t acc[2][NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[0][i] = acc[1][i] = f32x4_t{0, 0, 0, 0};
  stream_tile<WT, 2, NT, U>(wr, xr, r < cnt, rb, kw, (rb + 127) >> 7, wk, q, acc);
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    if (i > 0) __syncthreads();
    put_tile(red + kw * 256, lane, acc[0][i]);
    put_tile(red + (wk + kw) * 256, lane, acc[1][i]);
    __syncthreads();
    for (int o = tid; o < 256; o += wk * 64) {
      const int row = o & 15, col = o >> 4, c = i * 16 + col;
      if (c < cnt && row0 + row < h) {
        const float g = sum_tile(red, wk, row, col), u = sum_tile(red + wk * 256, wk, row, col);
        const float v = gate[c] * (g / (1.0f + expf(-g)) * u);
        const long at = (pos0 + c) * h + row0 + row;
        if constexpr (WT == kF32) {
          ((float*)hid)[at] = v;
        } else {
          const uint16_t hi = f2bf(v);
          ((uint16_t*)hid)[at] = hi;
          ((uint16_t*)hid)[hid_n + at] = f2bf(v - bf2f(hi));
        }
      }
    }
  }
}

constexpr int kProTokens = kWaves;  // tokens and entries that the up projection routes itself
constexpr int kProEntries = 64;

// PRO: every workgroup routes the (few) tokens in its prologue, a wave a token,
// instead of waiting for a launch that does it once; the slots' first
// workgroups leave them for the down projection.  Slots are then in the order
// of their first (token, place), a lane an entry, and slot s has hid rows s * T.
template <int WT, int NT, int U, int EPL, bool PRO>
__global__ __launch_bounds__(kThreads, 4) void few_up_kernel(
    const char* __restrict__ x, int xb, const void* __restrict__ w1, const uint8_t* __restrict__ w1s,
    const void* __restrict__ w3, const uint8_t* __restrict__ w3s, int T, int E, int k, int h, int rb, int wk,
    const float* __restrict__ logits, int parts, const int* __restrict__ n_live, int* __restrict__ idx_out,
    float* __restrict__ w_out, int* __restrict__ n_active, FewSlot* __restrict__ slots, float* __restrict__ gate,
    char* __restrict__ hid, long hid_n) {
  const int G = kWaves / wk;  // row tiles of a workgroup
  __shared__ __attribute__((aligned(16))) float red[2 * kWaves * 256];
  const int lane = threadIdx.x & 63, wv = wave_id(), r = lane & 15;
  const int tiles = (h + 16 * G - 1) / (16 * G);
  const int slot = blockIdx.x / tiles, tile = blockIdx.x - slot * tiles;
  const int grp = wv / wk, kw = wv % wk, tid = threadIdx.x - grp * wk * 64;
  const int row0 = (tile * G + grp) * 16;
  FewSlot sl;
  const float* gt;
  if constexpr (PRO) {
    __shared__ unsigned long long mask[EPL * 64];
    __shared__ int sel[kProEntries];
    __shared__ float selw[kProEntries];
    __shared__ float mygate[kProTokens];
    const int live = live_tokens(n_live, T), entries = live * k;
    for (int e = threadIdx.x; e < EPL * 64; e += kThreads) mask[e] = 0;
    __syncthreads();
    if (wv < live) route_token<EPL>(logits, parts, T, E, k, wv, lane, sel + wv * k, selw + wv * k, mask);
    __syncthreads();
    // every wave: lane = entry (token lane / k, place lane % k)
    const int e = lane < entries ? sel[lane] : 0, t = lane / k;
    const unsigned long long mk = lane < entries ? mask[e] : 0;
    const unsigned long long lead = __ballot(lane < entries && (mk & ((1ull << t) - 1)) == 0);
    const int na = __popcll(lead);
    if (blockIdx.x == 0 && wv == 0) {
      if (lane == 0) *n_active = na;
      if (lane < entries && idx_out != nullptr) idx_out[lane] = e;
      if (lane < entries && w_out != nullptr) w_out[lane] = selw[lane];
    }
    if (slot >= na) return;  // the whole workgroup
    const int at = nth_token(lead, lane, slot);  // the entry that leads this slot
    sl.e = __builtin_amdgcn_readfirstlane(__shfl(e, at, 64));
    sl.mask = mask[sl.e];
    sl.off = slot * T;
    if (wv == 0 && lane < entries && e == sl.e) mygate[__popcll(sl.mask & ((1ull << t) - 1))] = selw[lane];
    if (tile == 0 && threadIdx.x == 0) slots[slot] = sl;
    gt = mygate;  // read after the products' barrier
  } else {
    const int na = *n_active;
    sl = slots[slot];  // in bounds; meaningful if slot < na
    if (slot >= na) return;
    gt = gate + sl.off;
  }
  const int cnt = __popcll(sl.mask);
  const long n = (long)E * h, row = (long)sl.e * h + min(row0 + r, h - 1);
  const WRow wr[2] = {w_row<WT>(w1, w1s, n, row, rb), w_row<WT>(w3, w3s, n, row, rb)};
  float* rd = red + grp * 2 * wk * 256;
  // a tile past the last row (row0 >= h) still takes part in the barriers
#define TRG_TILE(N) \
  up_tile<WT, N, (N == 1 ? U : 1)>(x, xb, wr, rb, sl.mask, gt, cnt, row0, h, hid, hid_n, sl.off, wk, kw, tid, rd)
  if (NT == 1 || cnt <= 16) TRG_TILE(1);
  else if (cnt <= 32) TRG_TILE((NT > 1 ? NT / 2 : 1));
  else TRG_TILE(NT);
#undef TRG_TILE
}

// ---- down projection ----------------------------------------------------------------
// A workgroup takes 16 / KS rows of d and one part (blockIdx.y of gridDim.y) of
// the items of all chosen experts: item f is KS lines of a row from line
// f % nit * KS of slot f / nit.  A column is a token; an expert's item meets
// only the columns of its own tokens.  With few tokens (T <= 16 / KS) the 16
// rows and columns of the matrix instruction are KS groups: group g of rows
// holds the same weight rows at the item's line g, group g of columns the
// tokens at that line, and the blocks where the groups agree are summed at the
// end: more, smaller row tiles, at the same loads.
// PART: the sum goes to part[blockIdx.y] in fp32, else to y.
template <int WT, int NT, int U, int KS, bool PART>
__global__ __launch_bounds__(kThreads, 4) void few_down_kernel(const char* __restrict__ hid, long hid_n,
                                                               const void* __restrict__ w2,
                                                               const uint8_t* __restrict__ w2s, int E, int d, int h,
                                                               int rb, const int* __restrict__ n_active,
                                                               const FewSlot* __restrict__ slots, int T,
                                                               const int* __restrict__ n_live, void* __restrict__ y,
                                                               float* __restrict__ part) {
  static_assert(KS == 1 || NT == 1, "line groups share one tile of columns");
  constexpr int P = WT == kF32 ? 1 : 2;  // parts of h
  constexpr int XE = Piece<WT>::kXE;
  constexpr int RT = 16 / KS, CT = 16 / KS;
  __shared__ __attribute__((aligned(16))) float red[kWaves * 256];
  const int lane = threadIdx.x & 63, wv = wave_id(), r = lane & 15, q = lane >> 4;
  const int live = live_tokens(n_live, T);
  const int na = *n_active;
  const int row0 = blockIdx.x * RT;
  const int row = min(row0 + r % RT, d - 1), kr = r / RT;  // this lane's weight row and line group
  const int ct = r % CT, kc = r / CT;                      // this lane's column: token and line group
  const int nall = (rb + 127) >> 7, nit = (nall + KS - 1) / KS;
  const int F = na * nit;
  const int f1 = (int)((long)F * (blockIdx.y + 1) / gridDim.y);
  const int f0 = (int)((long)F * blockIdx.y / gridDim.y) + wv;
  f32x4_t acc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i] = f32x4_t{0, 0, 0, 0};
  struct Items {
    WStep w[U];
    unsigned long long mask[U];
    int off[U], c[U];
  };
  int s = f0 / nit, c = f0 - s * nit;  // the next item to load
  // items f, f + kWaves, ...: one past the share's end repeats the share's last
  // slot (so its loads are in bounds) for no token
  auto load = [&](Items& o, int f) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = f + u * kWaves < f1;
      const FewSlot sl = slots[in ? s : na - 1];
      o.mask[u] = in ? sl.mask : 0;
      o.off[u] = sl.off;
      o.c[u] = in ? c * KS : 0;
      const WRow wr = w_row<WT>(w2, w2s, (long)E * d, (long)sl.e * d + row, rb);
      o.w[u] = w_load<WT>(wr, o.c[u] + kr, q, rb);
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
      w_mask<WT>(o.w[u], o.c[u] + kr, q, rb);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (NT > 1 && ((unsigned)(o.mask[u] >> (16 * n)) & 0xFFFFu) == 0) continue;  // the same for the whole wave
        const int t = 16 * n + ct;
        const bool on = (o.mask[u] >> t) & 1;
        const long pos = o.off[u] + __popcll(o.mask[u] & ((1ull << t) - 1));
        const char* hr = hid + pos * h * XE;
        f32x4_t t4 = {0, 0, 0, 0};
        // both parts' operands at once, or with several tiles of columns (whose
        // accumulators need the registers) one after the other
        constexpr int AT = NT > 1 ? 1 : P;
#pragma unroll
        for (int p0 = 0; p0 < P; p0 += AT) {
          XStep<WT> x[AT];
          if (on) {
#pragma unroll
            for (int p = 0; p < AT; ++p) x_load<WT>(hr + (p0 + p) * hid_n * XE, o.c[u] + kc, q, rb, x[p]);
          }
#pragma unroll
          for (int p = 0; p < AT; ++p) t4 = mma_step<WT>(o.w[u], x[p], t4);
        }
        // columns of tokens that did not choose this expert are left alone, not
        // given 0 * w: an infinite or NaN weight is its own tokens' matter
#pragma unroll
        for (int z = 0; z < 4; ++z) acc[n][z] = on ? acc[n][z] + t4[z] : acc[n][z];
      }
    }
  };
  if (f0 < f1) {
    Items a, b;
    load(a, f0);
    int f = f0;
    for (; f + kWaves * U < f1; f += kWaves * U) {
      load(b, f + kWaves * U);
      multiply(a);
      a = b;
    }
    multiply(a);
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    if (i > 0) __syncthreads();
    put_tile(red + wv * 256, lane, acc[i]);
    __syncthreads();
    const int orow = threadIdx.x % RT, col = threadIdx.x / RT, t = i * 16 + col;
    if (threadIdx.x < RT * CT && t < live && row0 + orow < d) {
      float v = 0.f;
#pragma unroll
      for (int g = 0; g < KS; ++g) v += sum_tile(red, kWaves, g * RT + orow, g * CT + col);
      const long at = (long)t * d + row0 + orow;
      if constexpr (PART) part[(long)blockIdx.y * T * d + at] = v;
      else if constexpr (WT == kF32) ((float*)y)[at] = v;
      else ((uint16_t*)y)[at] = f2bf(v);
    }
  }
}

// y = the parts' sum, in order.
template <class OUT>
__global__ __launch_bounds__(256) void few_join_kernel(const float* __restrict__ part, int parts, int T, int d,
                                                       const int* __restrict__ n_live, OUT* __restrict__ y) {
  const long i = ((long)blockIdx.x * 256 + threadIdx.x) * 4;  // d is a multiple of 4
  if (i >= (long)live_tokens(n_live, T) * d) return;
  float4 a = *(const float4*)(part + i);
  for (int p = 1; p < parts; ++p) {
    const float4 b = *(const float4*)(part + (long)p * T * d + i);
    a.x += b.x;
    a.y += b.y;
    a.z += b.z;
    a.w += b.w;
  }
  Elt<OUT>::st(y + i, a.x);
  Elt<OUT>::st(y + i + 1, a.y);
  Elt<OUT>::st(y + i + 2, a.z);
  Elt<OUT>::st(y + i + 3, a.w);
}

template <int WT, int NM, int NT, int U, class OUT>
hipError_t linear_nt(const void* x, const void* w, const uint8_t* ws, int T, int n, int rb, int xb, int parts,
                     const int* n_live, OUT* out, hipStream_t st) {
  const int lines = (rb + 127) / 128, pl = (lines + parts - 1) / parts;
  few_linear_kernel<WT, NM, NT, U, OUT><<<dim3((n + 16 * NM - 1) / (16 * NM), parts), kThreads, 0, st>>>(
      (const char*)x, w, ws, T, n, rb, xb, pl, n_live, out);
  return hipGetLastError();
}

// Partial sums of the router's logits: enough workgroups that a wave has about
// one line (E / 16 tiles alone leave most of the chip idle).
int logit_parts(int d, int es) {
  const int lines = (d * es + 127) / 128;
  const int p = (lines + kWaves - 1) / kWaves;
  return p < 1 ? 1 : (p > 8 ? 8 : p);
}

// Parts of the down projection (1: straight to y).
int down_parts(int T, int d) {
  if (T <= 8) return 1;
  const int tiles = (d + 15) / 16;
  const int p = 1024 / tiles;
  return p < 2 ? 2 : (p > 8 ? 8 : p);
}

// Waves that share a row tile of the up projection: as many as leave each wave
// about 16 KB of weights.
int up_waves(int T, int E, int k, int h, int rb) {
  (void)T; (void)E; (void)k; (void)h;
  const int bytes = 32 * rb;  // a tile's: 16 rows of both matrices
  return bytes >= 8 * 12288 ? 8 : (bytes >= 4 * 8192 ? 4 : 2);
}

bool in_prologue(int T, int k) { return T <= kProTokens && T * k <= kProEntries; }

template <int WT, int NT, int U>
hipError_t up_any(const moe_few_args& a, int rb, int xb, int slots_max, const float* logits, int parts, int* n_active,
                  FewSlot* slots, float* gate, char* hid, long hid_n, hipStream_t st) {
  const int wk = up_waves(a.T, a.E, a.k, a.h, rb), G = kWaves / wk;
  const unsigned grid = (unsigned)slots_max * ((a.h + 16 * G - 1) / (16 * G));
#define TRG_UP(EPL, PRO)                                                                                             \
  few_up_kernel<WT, NT, U, EPL, PRO><<<grid, kThreads, 0, st>>>((const char*)a.x, xb, a.w1, a.w1s, a.w3, a.w3s, a.T, \
                                                                a.E, a.k, a.h, rb, wk, logits, parts, a.n_live,     \
                                                                a.topk_idx, a.topk_w, n_active, slots, gate, hid,   \
                                                                hid_n)
  if constexpr (NT == 1) {
    if (in_prologue(a.T, a.k)) {
      if (a.E <= 128) TRG_UP(2, true);
      else if (a.E <= 512) TRG_UP(8, true);
      else TRG_UP(16, true);
      return hipGetLastError();
    }
  }
  TRG_UP(1, false);
#undef TRG_UP
  return hipGetLastError();
}

template <int WT>
hipError_t few_any(const moe_few_args& a, hipStream_t st) {
  constexpr int XE = WT == kF32 ? 4 : 2;
  const FewLayout l = few_layout(a.T, a.d, a.E, a.k, a.h);
  char* ws = (char*)a.ws;
  int* n_active = (int*)(ws + l.n_active);
  FewSlot* slots = (FewSlot*)(ws + l.slots);
  float* gate = (float*)(ws + l.gate);
  float* logits = (float*)(ws + l.logits);
  char* hid = ws + l.hid;
  float* part = (float*)(ws + l.part);
  const int R = a.T * a.k, slots_max = R < a.E ? R : a.E;
  const long hid_n = (long)hid_rows(a.T, a.E, a.k) * a.h;
  const int lp = logit_parts(a.d, XE);
  constexpr int RT = WT == kF32 ? kF32 : kBF16;  // the router's weights are in x's type
  const int xb = a.d * XE;
  hipError_t e = a.T <= 16   ? linear_nt<RT, 1, 1, 1, float>(a.x, a.wr, nullptr, a.T, a.E, xb, xb, lp, a.n_live, logits, st)
                 : a.T <= 32 ? linear_nt<RT, 1, 2, 1, float>(a.x, a.wr, nullptr, a.T, a.E, xb, xb, lp, a.n_live, logits, st)
                             : linear_nt<RT, 1, 4, 1, float>(a.x, a.wr, nullptr, a.T, a.E, xb, xb, lp, a.n_live, logits, st);
  if (e != hipSuccess) return e;
  if (!in_prologue(a.T, a.k)) {
#define TRG_ROUTE(N)                                                                                                  \
  few_route_kernel<N><<<1, 1024, 0, st>>>(logits, lp, a.T, a.E, a.k, a.n_live, a.topk_idx, a.topk_w, n_active, slots, \
                                          gate)
    if (a.E <= 64) TRG_ROUTE(1);
    else if (a.E <= 128) TRG_ROUTE(2);
    else if (a.E <= 512) TRG_ROUTE(8);
    else TRG_ROUTE(16);
#undef TRG_ROUTE
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  // bytes of a weight row
  const int rb1 = WT == kE2M1 ? a.d / 2 : a.d * XE, rb2 = WT == kE2M1 ? a.h / 2 : a.h * XE;
  constexpr int U = WT == kE2M1 ? 1 : 2;
  e = a.T <= 16 ? up_any<WT, 1, U>(a, rb1, xb, slots_max, logits, lp, n_active, slots, gate, hid, hid_n, st)
                : up_any<WT, 4, U>(a, rb1, xb, slots_max, logits, lp, n_active, slots, gate, hid, hid_n, st);
  if (e != hipSuccess) return e;
  const int dp = down_parts(a.T, a.d);
#define TRG_DOWN(NT, U, KS, PART)                                                                                     \
  few_down_kernel<WT, NT, U, KS, PART><<<dim3((a.d + 16 / KS - 1) / (16 / KS), dp), kThreads, 0, st>>>(               \
      hid, hid_n, a.w2, a.w2s, a.E, a.d, a.h, rb2, n_active, slots, a.T, a.n_live, a.y, part)
  if (a.T <= 4) TRG_DOWN(1, U, 4, false);
  else if (a.T <= 8) TRG_DOWN(1, U, 2, false);
  else if (a.T <= 16) TRG_DOWN(1, U, 1, true);
  else TRG_DOWN(4, U, 1, true);
#undef TRG_DOWN
  e = hipGetLastError();
  if (e != hipSuccess || dp == 1) return e;
  const unsigned jg = (unsigned)(((long)a.T * a.d / 4 + 255) / 256);
  if constexpr (WT == kF32)
    few_join_kernel<float><<<jg, 256, 0, st>>>(part, dp, a.T, a.d, a.n_live, (float*)a.y);
  else
    few_join_kernel<uint16_t><<<jg, 256, 0, st>>>(part, dp, a.T, a.d, a.n_live, (uint16_t*)a.y);
  return hipGetLastError();
}

}  // namespace

size_t few_ws_bytes(int T, int d, int E, int k, int h) { return few_layout(T, d, E, k, h).bytes; }

hipError_t launch_few_fwd(const moe_few_args& a, hipStream_t st) {
  if (a.wt == MOE_E2M1) return few_any<kE2M1>(a, st);
  if (a.wt == MOE_BF16) return few_any<kBF16>(a, st);
  return few_any<kF32>(a, st);
}

hipError_t launch_linear_e2m1(const void* x, const uint8_t* q, const uint8_t* s, int T, int n, int K, void* y,
                              hipStream_t st) {
  // four row tiles a wave once there are rows enough for two workgroups a CU:
  // the tokens' operand, four times the weights' bytes, is then read once for
  // 64 rows
#define TRG_LINEAR(NM, NT) \
  linear_nt<kE2M1, NM, NT, 1, uint16_t>(x, q, s, T, n, K / 2, K * 2, 1, nullptr, (uint16_t*)y, st)
  if (n >= 64 * 384) return T <= 16 ? TRG_LINEAR(4, 1) : T <= 32 ? TRG_LINEAR(4, 2) : TRG_LINEAR(4, 4);
  return T <= 16 ? TRG_LINEAR(1, 1) : T <= 32 ? TRG_LINEAR(1, 2) : TRG_LINEAR(1, 4);
#undef TRG_LINEAR
}

}  // namespace trg
