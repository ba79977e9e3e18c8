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

struct FewLayout {
  size_t n_active, slots, tok, gate, logits, hid, bytes;
};

FewLayout few_layout(int T, int E, int k, int h) {
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
  l.tok = take(R * sizeof(int));
  l.gate = take(R * sizeof(float));
  l.logits = take((size_t)T * E * sizeof(float));
  l.hid = take(R * h * sizeof(float));  // fp32, or the hi and lo bf16 halves
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
// c: 128-byte line of the row; q: the lane's quarter of it.  Pieces past the
// row's end are zero (rb is a multiple of 16, so a piece is in or out whole).
template <int WT>
TRG_DEV WStep w_load(const WRow& r, int c, int q, int rb, bool whole) {
  WStep o;
  const int off = c * 128 + q * 32;
  o.sb = 0;
  if (whole) {
    o.v[0] = *(const uint4*)(r.p + off);
    o.v[1] = *(const uint4*)(r.p + off + 16);
    if (WT == kE2M1) o.sb = *(const uint16_t*)(r.s + (long)(2 * c + (q >> 1)) * r.sstride + (q & 1) * 2);
  } else {
    o.v[0] = o.v[1] = zero16();
    if (off < rb) {
      o.v[0] = *(const uint4*)(r.p + off);
      // the second byte is a place past the row's last block (0) if only the
      // first piece is inside
      if (WT == kE2M1) o.sb = *(const uint16_t*)(r.s + (long)(2 * c + (q >> 1)) * r.sstride + (q & 1) * 2);
    }
    if (off + 16 < rb) o.v[1] = *(const uint4*)(r.p + off + 16);
  }
  return o;
}
// The tokens' operand for piece i of the same step: kX 16-byte pieces.
template <int WT>
TRG_DEV void x_load(const char* xr, int c, int q, int i, int rb, bool whole, uint4* x) {
  const int off = c * 128 + q * 32 + i * 16;
  const long k = (long)off / 16 * Piece<WT>::kK;
  const char* p = xr + k * Piece<WT>::kXE;
  if (whole || off < rb) {
#pragma unroll
    for (int j = 0; j < Piece<WT>::kX; ++j) x[j] = *(const uint4*)(p + j * 16);
  } else {
#pragma unroll
    for (int j = 0; j < Piece<WT>::kX; ++j) x[j] = zero16();
  }
}

// ---- products of NM matrices' 16-row tiles with up to NT * 16 columns -------
// acc[m][n] over this wave's lines wv, wv + kWaves, ... of the rows.
template <int WT, int NM, int NT, int U>
TRG_DEV void stream_tile(const WRow* wr, const char* const* xr, int rb, int wv, int q, f32x4_t (*acc)[NT]) {
  const int nfull = rb >> 7, nall = (rb + 127) >> 7;
  for (int c0 = wv; c0 < nall; c0 += kWaves * U) {
    WStep w[U][NM];
    const bool whole = c0 + kWaves * (U - 1) < nfull;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < NM; ++m) w[u][m] = w_load<WT>(wr[m], c0 + u * kWaves, q, rb, whole);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!whole && c0 + u * kWaves >= nall) break;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float sc[NM];
#pragma unroll
        for (int m = 0; m < NM; ++m) sc[m] = WT == kE2M1 ? e8m0((w[u][m].sb >> (8 * i)) & 255u) : 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint4 x[Piece<WT>::kX];
          x_load<WT>(xr[n], c0 + u * kWaves, q, i, rb, whole, x);
#pragma unroll
          for (int m = 0; m < NM; ++m) acc[m][n] = mma_piece<WT>(w[u][m].v[i], sc[m], x, acc[m][n]);
        }
      }
    }
  }
}

// Sum of the waves' accumulators of one 16 x 16 tile, in wave order.  red:
// kWaves * 256 floats; entry (lane, r) of the matrix layout: column lane % 16,
// row lane / 16 * 4 + r.
TRG_DEV void put_tile(float* red, int wv, int lane, f32x4_t a) { *(f32x4_t*)(red + wv * 256 + lane * 4) = a; }
TRG_DEV float sum_tile(const float* red, int row, int col) {
  const float* p = red + ((row >> 2) * 16 + col) * 4 + (row & 3);
  float t = 0.f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) t += p[w * 256];
  return t;
}

// ---- router logits, and a dense product ---------------------------------------
// out[t, row] = <x[t], w[row]> for T <= NT * 16 columns; F32OUT: fp32 results
// (the router), else bf16.  A workgroup takes 16 rows, its waves share k.
template <int WT, int NT, int U, class OUT>
__global__ __launch_bounds__(kThreads) void few_linear_kernel(const char* __restrict__ x, const void* __restrict__ w,
                                                              const uint8_t* __restrict__ ws, int T, int n, int rb,
                                                              int xb, const int* __restrict__ n_live,
                                                              OUT* __restrict__ out) {
  __shared__ __attribute__((aligned(16))) float red[kWaves * 256];
  const int lane = threadIdx.x & 63, wv = wave_id(), r = lane & 15, q = lane >> 4;
  const int live = n_live != nullptr ? min(max(*n_live, 0), T) : T;
  const int row0 = blockIdx.x * 16;
  const WRow wr[1] = {w_row<WT>(w, ws, n, min(row0 + r, n - 1), rb)};
  const char* xr[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) xr[i] = x + (long)min(i * 16 + r, T - 1) * xb;  // columns past T repeat the last token
  f32x4_t acc[1][NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[0][i] = f32x4_t{0, 0, 0, 0};
  stream_tile<WT, 1, NT, U>(wr, xr, rb, wv, q, acc);
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    if (i > 0) __syncthreads();
    put_tile(red, wv, lane, acc[0][i]);
    __syncthreads();
    const int row = threadIdx.x & 15, col = (threadIdx.x >> 4) & 15, t = i * 16 + col;
    if (threadIdx.x < 256 && t < live && row0 + row < n) Elt<OUT>::st(out + (long)t * n + row0 + row, sum_tile(red, row, col));
  }
}

// ---- routing ---------------------------------------------------------------------
// One workgroup.  Each wave takes tokens wv, wv + 16, ...: softmax and k rounds
// of arg-max as moe_route does them (a NaN logit never wins a slot), then the
// chosen experts' token masks are compacted, in expert order, into slots and an
// entry list.  EPL: experts a lane.
TRG_DEV bool wins(float v, int e, float bv, int be) { return v > bv || (v == bv && e < be); }

template <int EPL>
__global__ __launch_bounds__(1024) void few_route_kernel(const float* __restrict__ logits, int T, int E, int k,
                                                         const int* __restrict__ n_live, int* __restrict__ idx_out,
                                                         float* __restrict__ w_out, int* __restrict__ n_active,
                                                         FewSlot* __restrict__ slots, int* __restrict__ tok,
                                                         float* __restrict__ gate) {
  __shared__ unsigned long long mask[1024];
  __shared__ int first[1024];
  __shared__ int tmp[32];
  __shared__ int sel[64 * 32];
  __shared__ float selw[64 * 32];
  const int lane = threadIdx.x & 63, wv = wave_id();
  mask[threadIdx.x] = 0;
  __syncthreads();
  const int live = n_live != nullptr ? min(max(*n_live, 0), T) : T;
  for (int t = wv; t < live; t += 16) {
    const float* L = logits + (long)t * E;
    float v[EPL], p[EPL];
    float m = -INFINITY, s = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 64 * i;
      const float x = e < E ? L[e] : -INFINITY;
      v[i] = (x != x) ? -INFINITY : x;
      m = fmaxf(m, v[i]);
    }
    m = wave_max(m);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      p[i] = lane + 64 * i < E ? expf(v[i] - m) : 0.f;
      s += p[i];
    }
    s = wave_sum(s);
    unsigned chosen = 0;
    for (int j = 0; j < k; ++j) {
      float bv = -INFINITY;
      int be = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane + 64 * i;
        if (e < E && !((chosen >> i) & 1u) && wins(v[i], e, bv, be)) {
          bv = v[i];
          be = e;
        }
      }
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) {
        const float ov = __shfl_xor(bv, o, 64);
        const int oe = __shfl_xor(be, o, 64);
        if (wins(ov, oe, bv, be)) {
          bv = ov;
          be = oe;
        }
      }
      // the lane that holds expert be (< E: k <= E leaves one unchosen)
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        if (lane + 64 * i == be) {
          chosen |= 1u << i;
          const float g = p[i] / s;
          sel[t * 32 + j] = be;
          selw[t * 32 + j] = g;
          if (idx_out != nullptr) idx_out[t * k + j] = be;
          if (w_out != nullptr) w_out[t * k + j] = g;
          atomicOr(&mask[be], 1ull << t);  // integer: the order does not matter
        }
      }
    }
  }
  __syncthreads();
  // experts with tokens, in order: (slots, entries) before each, in one scan
  const unsigned long long mk = mask[threadIdx.x];
  const int cnt = __popcll(mk);
  int total;
  const int before = block_excl_scan_1024((cnt > 0 ? 1 << 16 : 0) | cnt, tmp, &total);  // at most 2048 entries
  first[threadIdx.x] = before & 0xFFFF;
  if (cnt > 0) {
    FewSlot sl;
    sl.e = threadIdx.x;
    sl.off = before & 0xFFFF;
    sl.mask = mk;
    slots[before >> 16] = sl;
  }
  if (threadIdx.x == 0) *n_active = total >> 16;
  __syncthreads();
  for (int i = threadIdx.x; i < live * k; i += 1024) {
    const int t = i / k, j = i - t * k, e = sel[t * 32 + j];
    const int pos = first[e] + __popcll(mask[e] & ((1ull << t) - 1));
    tok[pos] = t;
    gate[pos] = selw[t * 32 + j];
  }
}

// ---- up projection ------------------------------------------------------------------
// Workgroup (slot, 16 rows of h): both matrices' rows against the slot's
// tokens, then h = gate * silu(g) * u.
template <int WT, int NT, int U>
TRG_DEV void up_tile(const char* __restrict__ x, int xb, const WRow* wr, int rb, const int* tok, const float* gate,
                     int cnt, int col_base, int row0, int h, char* hid, long hid_n, long pos0, float* red) {
  const int lane = threadIdx.x & 63, wv = wave_id(), r = lane & 15, q = lane >> 4;
  const char* xr[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) xr[i] = x + (long)tok[min(col_base + i * 16 + r, cnt - 1)] * xb;
  f32x4_t acc[2][NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[0][i] = acc[1][i] = f32x4_t{0, 0, 0, 0};
  stream_tile<WT, 2, NT, U>(wr, xr, rb, wv, q, acc);
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    if (i > 0) __syncthreads();
    put_tile(red, wv, lane, acc[0][i]);
    put_tile(red + kWaves * 256, wv, lane, acc[1][i]);
    __syncthreads();
    const int row = threadIdx.x & 15, col = (threadIdx.x >> 4) & 15, c = col_base + i * 16 + col;
    if (threadIdx.x < 256 && c < cnt && row0 + row < h) {
      const float g = sum_tile(red, row, col), u = sum_tile(red + kWaves * 256, row, col);
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

template <int WT, int NT>
__global__ __launch_bounds__(kThreads) void few_up_kernel(const char* __restrict__ x, int xb,
                                                          const void* __restrict__ w1, const uint8_t* __restrict__ w1s,
                                                          const void* __restrict__ w3, const uint8_t* __restrict__ w3s,
                                                          int E, int h, int rb, const int* __restrict__ n_active,
                                                          const FewSlot* __restrict__ slots,
                                                          const int* __restrict__ tok, const float* __restrict__ gate,
                                                          char* __restrict__ hid, long hid_n) {
  __shared__ __attribute__((aligned(16))) float red[2 * kWaves * 256];
  const int tiles = (h + 15) / 16;
  const int slot = blockIdx.x / tiles, row0 = (blockIdx.x - slot * tiles) * 16;
  if (slot >= *n_active) return;
  const FewSlot sl = slots[slot];
  const int cnt = __popcll(sl.mask);
  const int r = threadIdx.x & 15;
  const long n = (long)E * h, row = (long)sl.e * h + min(row0 + r, h - 1);
  const WRow wr[2] = {w_row<WT>(w1, w1s, n, row, rb), w_row<WT>(w3, w3s, n, row, rb)};
  const int* tk = tok + sl.off;
  const float* gt = gate + sl.off;
  if (NT == 1 || cnt <= 16) {
    up_tile<WT, 1, 4>(x, xb, wr, rb, tk, gt, cnt, 0, row0, h, hid, hid_n, sl.off, red);
  } else {
    up_tile<WT, NT, 2>(x, xb, wr, rb, tk, gt, cnt, 0, row0, h, hid, hid_n, sl.off, red);
  }
}

// ---- down projection ----------------------------------------------------------------
// Workgroup: RT rows of d, all chosen experts.  Its waves share the lines of
// the row over all slots: item f is line f % nall of slot f / nall.  A column
// is a token; an expert's item meets only the columns of its own tokens.
template <int WT, int NT, int U>
__global__ __launch_bounds__(kThreads) void few_down_kernel(const char* __restrict__ hid, long hid_n,
                                                            const void* __restrict__ w2,
                                                            const uint8_t* __restrict__ w2s, int E, int d, int h,
                                                            int rb, int rt, const int* __restrict__ n_active,
                                                            const FewSlot* __restrict__ slots, int T,
                                                            const int* __restrict__ n_live, void* __restrict__ y) {
  constexpr int P = WT == kF32 ? 1 : 2;  // parts of h
  constexpr int XE = Piece<WT>::kXE, KX = Piece<WT>::kX;
  __shared__ __attribute__((aligned(16))) float red[kWaves * 256];
  const int lane = threadIdx.x & 63, wv = wave_id(), r = lane & 15, q = lane >> 4;
  const int live = n_live != nullptr ? min(max(*n_live, 0), T) : T;
  const int na = *n_active;
  const int row0 = blockIdx.x * rt;
  const bool row_in = r < rt && row0 + r < d;
  const int row = min(row0 + r, d - 1);
  const int nall = (rb + 127) >> 7, F = na * nall;
  f32x4_t acc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i] = f32x4_t{0, 0, 0, 0};
  int s = wv / nall, c = wv - s * nall;
  for (int f0 = wv; f0 < F; f0 += kWaves * U) {
    WStep w[U];
    FewSlot sl[U];
    int cc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      cc[u] = c;
      if (f0 + u * kWaves < F) {
        sl[u] = slots[s];
        const WRow wr = w_row<WT>(w2, w2s, (long)E * d, (long)sl[u].e * d + row, rb);
        if (row_in) {
          w[u] = w_load<WT>(wr, c, q, rb, (c + 1) * 128 <= rb);
        } else {
          w[u].v[0] = w[u].v[1] = zero16();
          w[u].sb = 0;
        }
      }
      c += kWaves;
      while (c >= nall) {
        c -= nall;
        ++s;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (f0 + u * kWaves >= F) break;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const unsigned m16 = (unsigned)(sl[u].mask >> (16 * n)) & 0xFFFFu;
        if (NT > 1 && m16 == 0) continue;  // the same for the whole wave
        const bool on = (m16 >> r) & 1u;
        f32x4_t t = {0, 0, 0, 0};
        const long pos = sl[u].off + __popcll(sl[u].mask & ((1ull << (16 * n + r)) - 1));
        const char* hr = hid + (on ? pos : (long)sl[u].off) * h * XE;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int off = cc[u] * 128 + q * 32 + i * 16;
          const bool in = on && off < rb;
          const float sc = WT == kE2M1 ? e8m0((w[u].sb >> (8 * i)) & 255u) : 0.f;
          uint4 xv[P][KX];
#pragma unroll
          for (int p = 0; p < P; ++p)
#pragma unroll
            for (int j = 0; j < KX; ++j) xv[p][j] = zero16();
          if (in) {
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
              for (int j = 0; j < KX; ++j)
                xv[p][j] = *(const uint4*)(hr + (p ? hid_n * 2 : 0) + (long)off / 16 * Piece<WT>::kK * XE + j * 16);
          }
#pragma unroll
          for (int p = 0; p < P; ++p) t = mma_piece<WT>(w[u].v[i], sc, xv[p], t);
        }
        // columns of tokens that did not choose this expert are left alone, not
        // given 0 * w: an infinite or NaN weight is its own tokens' matter
#pragma unroll
        for (int z = 0; z < 4; ++z) acc[n][z] = on ? acc[n][z] + t[z] : acc[n][z];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    if (i > 0) __syncthreads();
    put_tile(red, wv, lane, acc[i]);
    __syncthreads();
    const int orow = threadIdx.x & 15, col = (threadIdx.x >> 4) & 15, t = i * 16 + col;
    if (threadIdx.x < 256 && t < live && orow < rt && row0 + orow < d) {
      const float v = sum_tile(red, orow, col);
      const long at = (long)t * d + row0 + orow;
      if constexpr (WT == kF32) ((float*)y)[at] = v;
      else ((uint16_t*)y)[at] = f2bf(v);
    }
  }
}

template <int WT, class OUT>
hipError_t linear_any(const void* x, const void* w, const uint8_t* ws, int T, int n, int rb, int xb, const int* n_live,
                      OUT* out, hipStream_t st) {
  const dim3 grid((n + 15) / 16);
  if (T <= 16)
    few_linear_kernel<WT, 1, 4, OUT><<<grid, kThreads, 0, st>>>((const char*)x, w, ws, T, n, rb, xb, n_live, out);
  else if (T <= 32)
    few_linear_kernel<WT, 2, 2, OUT><<<grid, kThreads, 0, st>>>((const char*)x, w, ws, T, n, rb, xb, n_live, out);
  else
    few_linear_kernel<WT, 4, 2, OUT><<<grid, kThreads, 0, st>>>((const char*)x, w, ws, T, n, rb, xb, n_live, out);
  return hipGetLastError();
}

template <int WT>
hipError_t few_any(const moe_few_args& a, hipStream_t st) {
  constexpr int XE = WT == kF32 ? 4 : 2;
  const FewLayout l = few_layout(a.T, a.E, a.k, a.h);
  char* ws = (char*)a.ws;
  int* n_active = (int*)(ws + l.n_active);
  FewSlot* slots = (FewSlot*)(ws + l.slots);
  int* tok = (int*)(ws + l.tok);
  float* gate = (float*)(ws + l.gate);
  float* logits = (float*)(ws + l.logits);
  char* hid = ws + l.hid;
  const long R = (long)a.T * a.k, hid_n = R * a.h;
  const int slots_max = R < a.E ? (int)R : a.E;
  hipError_t e = linear_any<WT == kF32 ? kF32 : kBF16, float>(a.x, a.wr, nullptr, a.T, a.E, a.d * XE, a.d * XE,
                                                              a.n_live, logits, st);
  if (e != hipSuccess) return e;
#define TRG_ROUTE(N)                                                                                             \
  few_route_kernel<N><<<1, 1024, 0, st>>>(logits, a.T, a.E, a.k, a.n_live, a.topk_idx, a.topk_w, n_active, slots, \
                                          tok, gate)
  if (a.E <= 64) TRG_ROUTE(1);
  else if (a.E <= 128) TRG_ROUTE(2);
  else if (a.E <= 256) TRG_ROUTE(4);
  else if (a.E <= 512) TRG_ROUTE(8);
  else TRG_ROUTE(16);
#undef TRG_ROUTE
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  // bytes of a weight row
  const int rb1 = WT == kE2M1 ? a.d / 2 : a.d * XE, rb2 = WT == kE2M1 ? a.h / 2 : a.h * XE;
  const unsigned up_grid = (unsigned)slots_max * ((a.h + 15) / 16);
  const int rt = 16;
  const unsigned down_grid = (a.d + rt - 1) / rt;
#define TRG_FEW(NT, U)                                                                                               \
  few_up_kernel<WT, NT><<<up_grid, kThreads, 0, st>>>((const char*)a.x, a.d * XE, a.w1, a.w1s, a.w3, a.w3s, a.E, a.h, \
                                                      rb1, n_active, slots, tok, gate, hid, hid_n);                  \
  e = hipGetLastError();                                                                                             \
  if (e != hipSuccess) return e;                                                                                     \
  few_down_kernel<WT, NT, U><<<down_grid, kThreads, 0, st>>>(hid, hid_n, a.w2, a.w2s, a.E, a.d, a.h, rb2, rt,        \
                                                             n_active, slots, a.T, a.n_live, a.y)
  if (a.T <= 16) { TRG_FEW(1, 4); }
  else if (a.T <= 32) { TRG_FEW(2, 4); }
  else { TRG_FEW(4, 4); }
#undef TRG_FEW
  return hipGetLastError();
}

}  // namespace

size_t few_ws_bytes(int T, int E, int k, int h) { return few_layout(T, E, k, h).bytes; }

hipError_t launch_few_fwd(const moe_few_args& a, hipStream_t st) {
  if (a.wt == MOE_E2M1) return few_any<kE2M1>(a, st);
  if (a.wt == MOE_BF16) return few_any<kBF16>(a, st);
  return few_any<kF32>(a, st);
}

hipError_t launch_linear_e2m1(const void* x, const uint8_t* q, const uint8_t* s, int T, int n, int K, void* y,
                              hipStream_t st) {
  return linear_any<kE2M1, uint16_t>(x, q, s, T, n, K / 2, K * 2, nullptr, (uint16_t*)y, st);
}

}  // namespace trg
