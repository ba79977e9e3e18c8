// The dense products beside the experts: a matrix product with bias, activation
// and residual in its epilogue, and its gradients.
//   forward   z = x W^T + b,  y = act(z) + res         x [T,K], W [n,K]
//   backward  dz = dy act'(z), db = sum_t dz,  dx = dz W,  dW = dz^T x
// The products are dense_impl.h's tiles; dz is made by one pass over dy and z
// that also sums the bias gradient's partials in fp32 (HBM bound; formed inside the
// products instead, every tile of a row would evaluate the slope again).  A training
// step's gradients, 16384 x 6144 x 2048 gelu, 812 us: the pass 116, the bias 5, dx 332, dW
// 375.
#include <math.h>

#include "dense_impl.h"

namespace trg {
namespace dn {

// act and its slope in fp32.  Phi is the normal distribution function, Phi(z) =
// erfc(-z / sqrt 2) / 2, whose left tail keeps its relative exactness (1 + erf(z / sqrt 2)
// cancels there: 4 % of Phi(-5) was wrong, all of it below -5.7).  For values stored in bf16 it comes from
//   erfc(x) = exp(-x^2) t P(t),  t = 1 / (1 + p x),  x = |z| / sqrt 2,
// P of degree 6 and p fitted over x in [0, 9.5] (all that fp32 holds) for the least largest
// relative error, 5.3e-7; the exponential and the reciprocal are the hardware's (1 ulp):
// with erff and expf an epilogue of 256 x 256 values took a sixth of its tile's products
// (16384 x 6144 x 2048, gelu and z kept: 412 us, 1001 TFLOP/s).
// The exponential is that of the density, too.
template <class T>
TRG_DEV float phi_f(float z, float& density) {
  if constexpr (sizeof(T) == 4) {
    density = 0.39894228040143268f * expf(-0.5f * z * z);
    return 0.5f * erfcf(z * -0.70710678118654752f);
  } else {
    const float e = __builtin_amdgcn_exp2f(z * z * -0.72134752044448170f);
    const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(z), 0.37314241f * 0.70710678118654752f, 1.0f));
    const float q =
        t * (0.21022014557f + t * (0.21564321789f + t * (0.16017091088f + t * (0.29918176371f + t * (-0.15544663812f +
             t * (0.40920448903f + t * -0.13897441406f))))));
    const float h = 0.5f * q * e;  // Phi(-|z|)
    density = 0.39894228040143268f * e;
    return z > 0.f ? 1.0f - h : h;
  }
}
template <class T>
TRG_DEV float sigmoid_of(float z) {
  if constexpr (sizeof(T) == 4) return 1.0f / (1.0f + expf(-z));
  else return sigmoid_f(z);
}
template <class T, int ACT>
TRG_DEV float act_f(float z) {
  float d;
  if constexpr (ACT == MOE_ACT_RELU) return z > 0.f ? z : (z == z ? 0.f : z);
  else if constexpr (ACT == MOE_ACT_GELU) return z * phi_f<T>(z, d);
  else if constexpr (ACT == MOE_ACT_SILU) return z * sigmoid_of<T>(z);
  else return z;
}
template <class T, int ACT>
TRG_DEV float act_slope(float z) {
  if constexpr (ACT == MOE_ACT_RELU) {
    return z > 0.f ? 1.f : (z == z ? 0.f : z);
  } else if constexpr (ACT == MOE_ACT_GELU) {
    float d;
    const float p = phi_f<T>(z, d);
    return fmaf(z, d, p);
  } else if constexpr (ACT == MOE_ACT_SILU) {
    const float s = sigmoid_of<T>(z);
    return s + z * s * (1.0f - s);
  } else {
    return 1.f;
  }
}

// y = act(v + bias) + res, z = v + bias; everything but y may be absent.
template <class T, int ACT>
struct EpiLinear {
  static constexpr bool kMirror = false;
  T* y;
  T* z;
  const T* bias;
  const T* res;
  int N;
  struct Tile {
    TileMat<T> y, z, bias, res;
    bool has_z, has_bias, has_res;
    TRG_DEV void fetch(const At& a, Held& h) const {
      if (has_res) res.fetch(a, h);
    }
    TRG_DEV void apply(const At& a, float (&v)[8], const Held& h) const {
      float f[8];
      if (has_bias) {
        bias.load(a, f);  // (rows 0 bytes apart)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += f[i];
      }
      if (has_z) z.store(a, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = act_f<T, ACT>(v[i]);
      if (has_res) {
        TileMat<T>::unpack(h, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += f[i];
      }
      y.store(a, v);
    }
  };
  TRG_DEV int cols() const { return N; }
  TRG_DEV Tile tile(int, int, int m0, int n0) const {
    const long at = (long)m0 * N + n0;
    return {TileMat<T>(y, at, N), TileMat<T>(z, at, N), TileMat<T>(bias, n0, 0), TileMat<T>(res, at, N),
            z != nullptr, bias != nullptr, res != nullptr};
  }
};

// 8 values of a row from column n on; `both`: the last four exist too (fp32).
TRG_DEV void ld8(const uint16_t* p, bool, float (&f)[8]) { unpack16<uint16_t>(*(const uint4*)p, f); }
TRG_DEV void ld8(const float* p, bool both, float (&f)[8]) {
  unpack16<float>(*(const uint4*)p, f);
  if (both) unpack16<float>(*(const uint4*)(p + 4), f + 4);
  else f[4] = f[5] = f[6] = f[7] = 0.f;
}
TRG_DEV void st8(uint16_t* p, bool, const float (&f)[8]) { *(uint4*)p = pack16<uint16_t>(f); }
TRG_DEV void st8(float* p, bool both, const float (&f)[8]) {
  *(uint4*)p = pack16<float>(f);
  if (both) *(uint4*)(p + 4) = pack16<float>(f + 4);
}

// dz = dy act'(z) and the bias gradient's partial sums: a thread takes 8
// columns of every 8th row of its block's rows (wave w of 8: rows w, w + 8, ...),
// adds them in fp32, and the waves' sums are added in order.  dz or part may be
// absent; z too where the activation has none.
// dz is rounded to its type here, once, for the two products (the bias sums what is not
// rounded): bf16 gradients are 2.3e-3 off the exact ones in the norm, where rounding the
// results alone leaves 1.7e-3.  Two bf16 planes of dz would keep those at twice both
// products' time (16384 x 6144 x 2048: 707 of 812 us).
constexpr int kDzWaves = 8;
template <class T, int ACT>
__global__ __launch_bounds__(64 * kDzWaves) void dz_kernel(const T* __restrict__ dy, const T* __restrict__ z,
                                                           int rows, int n, int block_rows, T* __restrict__ dz,
                                                           float* __restrict__ part) {
  __shared__ float red[kDzWaves][64][9];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int col = (blockIdx.x * 64 + lane) * 8;
  const int r0 = blockIdx.y * block_rows, r1 = min(rows, r0 + block_rows);
  float sum[8] = {};
  if (col < n) {
    const bool both = col + 8 <= n;
    for (int r = r0 + wv; r < r1; r += kDzWaves) {
      const long at = (long)r * n + col;
      float g[8];
      ld8(dy + at, both, g);
      if constexpr (ACT != MOE_ACT_NONE) {
        float zz[8];
        ld8(z + at, both, zz);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] *= act_slope<T, ACT>(zz[i]);
      }
      if (dz) st8(dz + at, both, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += g[i];
    }
  }
  if (part == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) red[wv][lane][i] = sum[i];
  __syncthreads();
  const int l = threadIdx.x >> 3, i = threadIdx.x & 7, c = (blockIdx.x * 64 + l) * 8 + i;
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kDzWaves; ++w) s += red[w][l][i];
  if (c < n) part[(long)blockIdx.y * n + c] = s;
}

// The same for at most kDzShort rows, in one launch with the bias gradient: a
// workgroup has 64 columns and every row, eight lanes a row and 64 rows at a time;
// its lanes' sums are added in order.  The border depends on the rows alone: of the two
// launches' time this takes, over 64, 256, ... 16384 columns with gelu, bf16 0.42-0.79 at
// 64 rows, 0.62-0.89 at 320, 0.67-0.97 at 384, 0.78-1.11 at 512; fp32 0.44-0.82, 0.79-1.02,
// 0.89-1.12, 1.03-1.33 (without activation 0.57-0.67 at 320, 0.72-0.84 at 512).
constexpr int kDzShort = 320;
template <class T, int ACT>
__global__ __launch_bounds__(512) void dz_short_kernel(const T* __restrict__ dy, const T* __restrict__ z, int rows,
                                                       int n, T* __restrict__ dz, T* __restrict__ db) {
  __shared__ float red[64][68], half[8][64];
  const int row = threadIdx.x >> 3, c8 = (threadIdx.x & 7) * 8, col = blockIdx.x * 64 + c8;
  float sum[8] = {};
  if (col < n) {
    const bool both = col + 8 <= n;
#pragma unroll
    for (int i = 0; i < kDzShort / 64; ++i) {
      const int r = i * 64 + row;
      if (r >= rows) continue;
      const long at = (long)r * n + col;
      float g[8];
      ld8(dy + at, both, g);
      if constexpr (ACT != MOE_ACT_NONE) {
        float zz[8];
        ld8(z + at, both, zz);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] *= act_slope<T, ACT>(zz[e]);
      }
      if (dz) st8(dz + at, both, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += g[e];
    }
  }
  *(f32x4_t*)&red[row][c8] = f32x4_t{sum[0], sum[1], sum[2], sum[3]};
  *(f32x4_t*)&red[row][c8 + 4] = f32x4_t{sum[4], sum[5], sum[6], sum[7]};
  __syncthreads();
  const int l = threadIdx.x & 63, q = threadIdx.x >> 6, c = blockIdx.x * 64 + l;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += red[q * 8 + i][l];
  half[q][l] = s;
  __syncthreads();
  if (q > 0 || c >= n) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) s += half[i][l];
  Elt<T>::st(db + c, s);
}

// db[c] = sum of the blocks' partials: four threads a column take every fourth
// block in order, and their sums are added in order.
template <class T>
__global__ __launch_bounds__(256) void dbias_kernel(const float* __restrict__ part, int blocks, int n,
                                                    T* __restrict__ db) {
  __shared__ float red[4][64];
  const int l = threadIdx.x & 63, q = threadIdx.x >> 6, c = blockIdx.x * 64 + l;
  float s = 0.f;
  if (c < n)
#pragma unroll 4
    for (int b = q; b < blocks; b += 4) s += part[(long)b * n + c];
  red[q][l] = s;
  __syncthreads();
  if (q == 0 && c < n) Elt<T>::st(db + c, (red[0][l] + red[1][l]) + (red[2][l] + red[3][l]));
}

// Row blocks of dz_kernel: at least 32 rows each, at most 64 blocks.
static int dz_block_rows(int T) {
  const int r = gg::cdiv(T, 64);
  return r < 32 ? 32 : r;
}

static size_t up256(size_t b) { return (b + 255) / 256 * 256; }
static int es_of(int dt) { return dt == MOE_F32 ? 4 : 2; }
static Plan plan_of(int M, int N, int K, int dt) {
  const int es = es_of(dt);
  return plan(1, M, N, gg::cdiv((long)K * es, 128), es, false);
}

// ---- a few tokens -------------------------------------------------------------
// A few tokens are a stream of weights.  Those go straight from memory to
// registers as the matrix instruction's A operand (16 rows), tokens as its B
// operand (16 columns): in one step a wave reads a 128-byte line of each of 16
// rows, lane l 32 bytes (quarter l / 16) of row l % 16, and the tokens' operand
// with the same places, so the order of k is the same for both.  A workgroup has
// 16 rows, its waves take the row's lines in turn and their sums are added in
// order through LDS, so one launch does it all.
constexpr int kFewWaves = 8;
constexpr int few_lines(int row_tiles, int tokens) { return row_tiles == 2 && tokens > 16 ? 2 : 4; }
struct FewBf16 {
  using Acc = f32x4_t;
  static TRG_DEV Acc mma(u32x4v a, u32x4v b, Acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
  }
};
struct FewF32 {  // (instruction r takes value r of both pieces)
  using Acc = f32x4_t;
  static TRG_DEV Acc mma(u32x4v a, u32x4v b, Acc c) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[r]), __uint_as_float(b[r]), c, 0, 0, 0);
    return c;
  }
};

// NM: tiles of 16 rows; NT: of 16 tokens; U: lines of a row in one round of a wave's
// loop, whose loads the compiler spreads over the products: two to eight 16-byte pieces
// are under way at a time.  (y may be res.)
template <class Few, class T, int ACT, int NM, int NT, int U, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void linear_few_kernel(const T* __restrict__ x, const T* __restrict__ w,
                                                                const T* __restrict__ bias, const T* res, int tokens,
                                                                int n, int K, T* __restrict__ z, T* y) {
  __shared__ __attribute__((aligned(16))) float red[WAVES][NM][NT][256];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = (lane >> 4) * 16, row0 = blockIdx.x * (16 * NM);
  const int rb = K * (int)sizeof(T), lines = (rb + 127) >> 7;
  const auto rw = tile_rsrc((const char*)(w + (long)row0 * K), min(16 * NM, n - row0) * rb);
  const auto rx = tile_rsrc((const char*)x, tokens * rb);
  int wo[NM], xo[NT];
#pragma unroll
  for (int m = 0; m < NM; ++m) wo[m] = min(m * 16 + r, n - 1 - row0) * rb;
#pragma unroll
  for (int i = 0; i < NT; ++i) xo[i] = min(i * 16 + r, tokens - 1) * rb;
  f32x4_t acc[NM][NT] = {};
  for (int l0 = wv; l0 < lines; l0 += WAVES * U) {
    u32x4v a[U][2][NM], b[U][2][NT];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int at = (l0 + u * WAVES) * 128 + p * 64 + q;  // zeros past the row's end
#pragma unroll
        for (int m = 0; m < NM; ++m)
          a[u][p][m] = __builtin_bit_cast(u32x4v, __builtin_amdgcn_raw_buffer_load_b128(rw, at < rb ? wo[m] + at : kPast, 0, 0));
#pragma unroll
        for (int i = 0; i < NT; ++i)
          b[u][p][i] = __builtin_bit_cast(u32x4v, __builtin_amdgcn_raw_buffer_load_b128(rx, at < rb ? xo[i] + at : kPast, 0, 0));
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
          for (int i = 0; i < NT; ++i) acc[m][i] = Few::mma(a[u][p][m], b[u][p][i], acc[m][i]);
  }
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i) *(f32x4_t*)&red[wv][m][i][lane * 4] = acc[m][i];
  __syncthreads();
  for (int o = threadIdx.x; o < 16 * NM * tokens; o += 64 * WAVES) {
    const int ro = o % (16 * NM), t = o / (16 * NM), row = row0 + ro;
    if (row >= n) continue;
    // (lane 16 (row / 4) + column of a tile holds four rows)
    const int at = (((ro & 15) >> 2) * 16 + (t & 15)) * 4 + (ro & 3);
    float v = red[0][ro >> 4][t >> 4][at];
#pragma unroll
    for (int s = 1; s < WAVES; ++s) v += red[s][ro >> 4][t >> 4][at];
    if (bias) v += Elt<T>::ld(bias + row);
    const long yo = (long)t * n + row;
    if (z) Elt<T>::st(z + yo, v);
    v = act_f<T, ACT>(v);
    if (res) v += Elt<T>::ld(res + yo);
    Elt<T>::st(y + yo, v);
  }
}

// Row tiles a workgroup has, 1 or 2, or 0 where the other kernels' tiles take a
// product.  By estimates in us, fitted to 5134 times (1 to 32 tokens, 64 to 65536 rows
// of 64 to 17000 values, bf16 and fp32, weights that come from memory): a launch, the
// rounds of loads that a wave waits for, all weights, and the fullest CU's weights and
// tokens (every token's whole row for each workgroup, which two row tiles halve).  What
// is picked takes 0.7 % longer than the best of the three on average, 26 % at most.  Both
// sides of some borders, us with one row tile / two / the other tiles:
//   16 tokens, rows of 2048 bf16: 4096 rows 6.9 / 9.0 / 10.4, 5120 10.1 / 8.8 / 9.7, 8192
//   11.3 / 11.9 / 11.4, 12288 14.9 / 17.1 / 11.9
//   32 tokens, rows of 1024 fp32: 4096 rows 9.5 / 11.9 / 12.5, 8192 16.1 / 14.4 / 16.6,
//   16384 27.5 / 24.2 / 24.3; 8 tokens 5120 rows 8.9 / 8.5 / 13.6, 12288 13.5 / 16.0 / 23.1
static int few_row_tiles(int tokens, int n, int K, int dt) {
  if (tokens > 32 || tokens < 1) return 0;
  const double row = (double)K * es_of(dt), lines = row / 128, all = 1e-6 * row * n;
  auto us = [&](int tiles, double launch, double wait, double mb, double w_kb, double x_kb) {
    const int rounds = gg::cdiv(gg::cdiv(n, 16 * tiles), 256);  // workgroups of the fullest CU
    const double waits = lines / (kFewWaves * few_lines(tiles, tokens));
    return launch + mb * all + rounds * (wait * (waits > 1 ? waits : 1) + 1e-3 * row * (16 * tiles * w_kb + tokens * x_kb));
  };
  const double one = us(1, 2.2, 0.4, 0.1, 0.016, 0.028), two = us(2, 2.45, 0.55, 0.129, 0.0203, 0.0212);
  const int tiles = two < one ? 2 : 1;
  // the other tiles: 4.5 TB/s, or their plan, which has a least that saves asking it
  const double best = two < one ? two : one, least = 1.05 * (3.45 + (lines < 30 ? lines * 0.175 : 5.25));
  if (best <= all / 4.5 || best <= least) return tiles;
  return best <= 1.05 * plan_of(tokens, n, K, dt).us ? tiles : 0;
}

template <class Few, class T, int ACT>
static hipError_t few(int row_tiles, const T* x, const T* w, const T* bias, const T* res, int tokens, int n, int K, T* z,
                      T* y, hipStream_t s) {
  auto go = [&](auto NM, auto NT) {
    constexpr int nm = decltype(NM)::value, nt = decltype(NT)::value;
    linear_few_kernel<Few, T, ACT, nm, nt, few_lines(nm, nt * 16), kFewWaves>
        <<<gg::cdiv(n, 16 * nm), 64 * kFewWaves, 0, s>>>(x, w, bias, res, tokens, n, K, z, y);
  };
  const std::integral_constant<int, 1> c1{};
  const std::integral_constant<int, 2> c2{};
  if (tokens <= 16) row_tiles == 1 ? go(c1, c1) : go(c2, c1);
  else row_tiles == 1 ? go(c1, c2) : go(c2, c2);
  return hipGetLastError();
}

// f(std::integral_constant<int, act>{})
template <class F>
static auto with_act(int act, F&& f) {
  switch (act) {
    case MOE_ACT_RELU: return f(std::integral_constant<int, MOE_ACT_RELU>{});
    case MOE_ACT_GELU: return f(std::integral_constant<int, MOE_ACT_GELU>{});
    case MOE_ACT_SILU: return f(std::integral_constant<int, MOE_ACT_SILU>{});
    default: return f(std::integral_constant<int, MOE_ACT_NONE>{});
  }
}

static Args product(const void* A, long lda, const void* B, long ldb, int M, int N, int K) {
  Args a{};
  a.A = A;
  a.lda = lda;
  a.B = B;
  a.ldb = ldb;
  a.M = M;
  a.N = a.b_rows = N;
  a.K = K;
  a.batch = a.nseg = 1;
  return a;
}

template <class El, class T>
static hipError_t fwd(const void* x, const void* w, const void* bias, const void* res, int rows, int n, int K, int act,
                      int dt, void* z, void* y, void* ws, hipStream_t s) {
  const Args a = product(x, K, w, K, rows, n, K);
  return with_act(act, [&](auto ACT) {
    if (const int row_tiles = few_row_tiles(rows, n, K, dt))
      return few<std::conditional_t<sizeof(T) == 4, FewF32, FewBf16>, T, decltype(ACT)::value>(
          row_tiles, (const T*)x, (const T*)w, (const T*)bias, (const T*)res, rows, n, K, (T*)z, (T*)y, s);
    const EpiLinear<T, decltype(ACT)::value> e{(T*)y, (T*)z, (const T*)bias, (const T*)res, n};
    return run<El, true, true>(plan_of(rows, n, K, dt), a, e, (float*)ws, s);
  });
}

template <class El, class T>
static hipError_t bwd(const void* dy, const void* x, const void* w, const void* z, int rows, int n, int K, int act,
                      int dt, void* dx, void* dw, void* db, char* ws, hipStream_t s) {
  T* dz = act == MOE_ACT_NONE ? nullptr : (T*)ws;
  if (dz) ws += up256((size_t)rows * n * sizeof(T));
  const int br = dz_block_rows(rows), blocks = gg::cdiv(rows, br);
  float* part = (float*)ws;
  const bool need_dz = dz && (dx || dw);
  const bool brief = db && rows > 0 && rows <= kDzShort;
  if (brief)
    with_act(act, [&](auto ACT) {
      dz_short_kernel<T, decltype(ACT)::value><<<gg::cdiv(n, 64), 512, 0, s>>>((const T*)dy, (const T*)z, rows, n,
                                                                               need_dz ? dz : nullptr, (T*)db);
    });
  else if (rows > 0 && (need_dz || db))
    with_act(act, [&](auto ACT) {
      dz_kernel<T, decltype(ACT)::value><<<dim3(gg::cdiv(n, 512), blocks), 64 * kDzWaves, 0, s>>>(
          (const T*)dy, (const T*)z, rows, n, br, need_dz ? dz : nullptr, db ? part : nullptr);
    });
  if (db && !brief) dbias_kernel<T><<<gg::cdiv(n, 64), 256, 0, s>>>(part, rows > 0 ? blocks : 0, n, (T*)db);
  hipError_t err = hipGetLastError();
  const void* g = dz ? (const void*)dz : dy;
  if (dx && err == hipSuccess) {  // dx = dz W
    const EpiLinear<T, MOE_ACT_NONE> e{(T*)dx, nullptr, nullptr, nullptr, K};
    err = run<El, true, false>(plan_of(rows, K, n, dt), product(g, n, w, K, rows, K, n), e, (float*)ws, s);
  }
  if (dw && err == hipSuccess) {  // dW = dz^T x
    const EpiLinear<T, MOE_ACT_NONE> e{(T*)dw, nullptr, nullptr, nullptr, K};
    err = run<El, false, false>(plan_of(n, K, rows, dt), product(g, n, x, K, n, K, rows), e, (float*)ws, s);
  }
  return err;
}

}  // namespace dn

using namespace dn;

static DensePlan chosen(int M, int N, int K, int dt, int row_tiles) {
  const Plan p = plan_of(M, N, K, dt);
  return {row_tiles, p.tile, p.stages(p.nsplit * tiles_of(M, N, p.tile, false)), p.nsplit};
}

DensePlan linear_plan(int T, int n, int K, int dt) { return chosen(T, n, K, dt, few_row_tiles(T, n, K, dt)); }

DensePlan linear_bwd_plan(int T, int n, int K, int dt, bool dw) {
  return dw ? chosen(n, K, T, dt, 0) : chosen(T, K, n, dt, 0);
}

size_t linear_ws_bytes(int T, int n, int K, int dt) {
  return few_row_tiles(T, n, K, dt) ? 0 : plan_of(T, n, K, dt).part_bytes(1, T, n);
}

size_t linear_bwd_ws_bytes(int T, int n, int K, int dt) {
  size_t need = (size_t)gg::cdiv(T, dz_block_rows(T)) * n * 4;
  const size_t px = plan_of(T, K, n, dt).part_bytes(1, T, K), pw = plan_of(n, K, T, dt).part_bytes(1, n, K);
  need = need > px ? need : px;
  need = need > pw ? need : pw;
  return up256((size_t)T * n * es_of(dt)) + need;
}

hipError_t launch_linear_fwd(const void* x, const void* w, const void* bias, const void* res, int T, int n, int K,
                             int act, int dt, void* z, void* y, void* ws, hipStream_t s) {
  return dt == MOE_F32 ? fwd<ElF32, float>(x, w, bias, res, T, n, K, act, dt, z, y, ws, s)
                       : fwd<ElBf16, uint16_t>(x, w, bias, res, T, n, K, act, dt, z, y, ws, s);
}

hipError_t launch_linear_bwd(const void* dy, const void* x, const void* w, const void* z, int T, int n, int K, int act,
                             int dt, void* dx, void* dw, void* db, void* ws, hipStream_t s) {
  return dt == MOE_F32 ? bwd<ElF32, float>(dy, x, w, z, T, n, K, act, dt, dx, dw, db, (char*)ws, s)
                       : bwd<ElBf16, uint16_t>(dy, x, w, z, T, n, K, act, dt, dx, dw, db, (char*)ws, s);
}

}  // namespace trg
