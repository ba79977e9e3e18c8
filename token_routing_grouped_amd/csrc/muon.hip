// Orthogonalised updates (Newton-Schulz products, as the Muon optimiser uses
// them) for batches of matrices: the experts' weight gradients.
//   X_0 = G / (|G|_F + eps);  A = X X^T (X^T X for tall ones: the smaller side)
//   X <- B X,  B = a + b A + c A^2,  (a, b, c) = (3.4445, -4.7750, 2.0315)
// The odd quintic takes singular values in (0, 1] towards 1 (it stays under
// 1.21 on [0, 1.21]), so every iterate is bounded and fits fp16: fp16 has the
// matrix rate of bf16 and three more mantissa bits, which the quintic's slope at 0
// (3.4 a step, 485 over five) makes worth having.  fp32 matrices are kept as two
// fp16 planes (22 bits) and multiplied as split sums (takes_planes: which others are).
//
// A step is three products of dense_impl.h: A (symmetric: tiles on and above
// the diagonal), B (symmetric, with a and b A in the epilogue) and B X.  With a in
// B's diagonal the last one, half of a step's operations, has nothing to read in
// its epilogue, and B's diagonal is stored as what is left of the sum: near the
// end 0.70, not -2.74 to be added to 3.44, so fp16 rounds it to a quarter of
// that (the result's error is a tenth smaller).  A wide matrix reads X as rows in the first and as columns (the
// transpose read) in the last, a tall one the other way round, so no
// transposed copy is made.  Before them one pass forms the momentum and the
// sum of squares (in 64 bits: the square of any fp32 value fits) and one
// scales into fp16; the last product's epilogue writes the result, or moves
// the weights.
#include "dense_impl.h"

namespace trg {
namespace dn {

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
// Scale of the stored X, A and B: |X| <= 1.21, |A| <= 1.47 and |B| <= 3.45 (as
// norms, so as entries) stay under fp16's 65504, and what is small, entries of
// large matrices and low planes, keeps as many bits above fp16's smallest.
constexpr float kS = 8192.0f;
constexpr int kSumBlocks = 256;  // partial sums of squares a matrix, at most

// Stored = hi + lo where there are two planes.
TRG_DEV void split_planes(const float (&v)[8], f16x8_t& hi, f16x8_t& lo) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    hi[i] = (_Float16)v[i];
    lo[i] = (_Float16)(v[i] - (float)hi[i]);
  }
}

// A tile of a matrix in one plane, or two `plane` values apart.
template <bool TWO>
struct TilePlanes {
  TileMat<uint16_t> hi, lo;
  TRG_DEV TilePlanes(const _Float16* p, long at, long ld, long plane)
      : hi((const uint16_t*)p, at, ld), lo((const uint16_t*)p, at + (TWO ? plane : 0), ld) {}
  TRG_DEV void store(const At& a, const float (&v)[8]) const {
    const int o = a.ok ? hi.off(a) : kPast;
    f16x8_t h, l;
    split_planes(v, h, l);
    hi.raw_st(o, __builtin_bit_cast(uint4, h));
    if (TWO) lo.raw_st(o, __builtin_bit_cast(uint4, l));
  }
  TRG_DEV void fetch(const At& a, Held& h) const {
    const int o = a.ok ? hi.off(a) : kPast;
    h.v[0] = hi.raw(o);
    if (TWO) h.v[1] = lo.raw(o);
  }
  // v = alpha v + beta stored
  static TRG_DEV void mix(const Held& held, float alpha, float beta, float (&v)[8]) {
    const f16x8_t h = __builtin_bit_cast(f16x8_t, held.v[0]);
    f16x8_t l = {};
    if (TWO) l = __builtin_bit_cast(f16x8_t, held.v[1]);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = alpha * v[i] + beta * (TWO ? (float)h[i] + (float)l[i] : (float)h[i]);
  }
};

// out = alpha v + beta in + gamma I (IN), or alpha v, in planes.
template <bool TWO, bool IN>
struct EpiIter {
  static constexpr bool kMirror = true;
  _Float16* out;
  const _Float16* in;
  long ld, bs, plane;
  float alpha, beta, gamma;
  struct Tile {
    TilePlanes<TWO> out, in;
    float alpha, beta, gamma;
    int diag;  // the tile's row less its column
    TRG_DEV void fetch(const At& a, Held& h) const {
      if (IN) in.fetch(a, h);
    }
    TRG_DEV void apply(const At& a, float (&v)[8], const Held& h) const {
      if (IN) {
        TilePlanes<TWO>::mix(h, alpha, beta, v);
        const int d = diag + a.row - a.col;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += d == i ? gamma : 0.f;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= alpha;
      }
      out.store(a, v);
    }
  };
  TRG_DEV int cols() const { return (int)ld; }
  TRG_DEV Tile tile(int b, int, int m0, int n0) const {
    const long at = b * bs + m0 * ld + n0;
    return {TilePlanes<TWO>(out, at, ld, plane), TilePlanes<TWO>(in, at, ld, plane), alpha, beta, gamma, m0 - n0};
  }
};

// The last product: o = alpha v, written as it is or as a step of
// the weights, w <- w (1 - decay) - step o, in fp32 and rounded once.
struct Update {
  const void* w;  // null: write o
  const float* master;
  float* master_out;
  void* out;
  float step, decay;
  const float* lr_scale;
};
template <class T>
struct EpiUpdate {
  static constexpr bool kMirror = false;
  float alpha;
  int rows, ncols;
  Update u;
  struct Tile {
    TileMat<T> out, w;
    TileMat<float> master, master_out, base;  // base: where master or w starts
    float alpha, keep, step;
    bool has_w, has_master;
    TRG_DEV void fetch(const At& a, Held& h) const {  // the base: master, w, or nothing
      const int o = has_master ? master.off(a) : w.off(a);
      h.v[0] = base.raw(has_w && a.ok ? o : kPast);
      h.v[1] = base.raw(has_w && a.ok2 && (has_master || sizeof(T) == 4) ? o + 16 : kPast);
    }
    TRG_DEV void apply(const At& a, float (&v)[8], const Held& h) const {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= alpha;
      if (has_w) {
        float f[8];
        if (has_master) TileMat<float>::unpack(h, f);
        else TileMat<T>::unpack(h, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = f[i] * keep - step * v[i];
        if (has_master) master_out.store(a, v);
      }
      out.store(a, v);
    }
  };
  TRG_DEV int cols() const { return ncols; }
  TRG_DEV Tile tile(int b, int, int m0, int n0) const {
    const long at = ((long)b * rows + m0) * ncols + n0;
    const float s = u.w && u.lr_scale ? *u.lr_scale : 1.0f;
    return {TileMat<T>((const T*)u.out, at, ncols),
            TileMat<T>((const T*)u.w, at, ncols),
            TileMat<float>(u.master, at, ncols),
            TileMat<float>(u.master_out, at, ncols),
            u.master ? TileMat<float>(u.master, at, ncols)
                     : TileMat<float>((const float*)((const T*)u.w + at), 0, ncols),
            alpha, 1.0f - u.decay * s, u.step * s, u.w != nullptr, u.master != nullptr};
  }
};

// What is orthogonalised: g, or (buf given) the momentum's step.
struct Momentum {
  const float* buf;
  float* buf_out;
  float mu;
  int nesterov;
};

// One pass over a batch's gradients: buf_out = mu buf + g and the partial sums
// of u^2, u = g, g + mu buf_out, or buf_out.  blockIdx.y: the matrix.
template <class T>
__global__ __launch_bounds__(256) void sumsq_kernel(const T* __restrict__ g, Momentum mo, long count, int blocks,
                                                    double* __restrict__ part) {
  constexpr int V = Elt<T>::kVec;
  __shared__ double red[4];
  const long first = (long)blockIdx.y * count;
  double sum = 0.0;
  for (long c = (long)blockIdx.x * 256 + threadIdx.x; c < count / V; c += (long)blocks * 256) {
    const long at = first + c * V;
    float u[V];
    unpack16<T>(*(const uint4*)(g + at), u);
    if (mo.buf) {
      float bn[V];
#pragma unroll
      for (int h = 0; h < V; h += 4) unpack16<float>(*(const uint4*)(mo.buf + at + h), bn + h);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        bn[i] = mo.mu * bn[i] + u[i];
        u[i] = mo.nesterov ? u[i] + mo.mu * bn[i] : bn[i];
      }
#pragma unroll
      for (int h = 0; h < V; h += 4) *(uint4*)(mo.buf_out + at + h) = pack16<float>(bn + h);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) sum += (double)u[i] * (double)u[i];
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, kWave);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) part[(long)blockIdx.y * blocks + blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

// X = u 2^13 / (|u| + eps) in planes of rows of ldx values (zeros behind cols).
// A zero matrix stays zero; one that holds an infinity or NaN becomes NaN.  A
// thread's NC pieces of 8 values are loaded before the norm is put together from
// its partial sums.
template <class T, bool MOM, int NC>
__global__ __launch_bounds__(256) void scale_kernel(const T* __restrict__ g, Momentum mo, int rows, int cols, int ldx,
                                                    float eps, const double* __restrict__ part, int blocks, int two,
                                                    long plane, _Float16* __restrict__ x) {
  constexpr int V = Elt<T>::kVec;
  __shared__ double s_inv;
  const int b = blockIdx.y, chunks = ldx / 8;
  const long total = (long)rows * chunks, i0 = (long)blockIdx.x * (256 * NC) + threadIdx.x;
  const bool use_g = !MOM || mo.nesterov;
  float u[NC][8];
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const long i = i0 + k * 256;
    const int r = ldx == cols ? 0 : (int)(i / chunks);  // (rows without padding are one long row)
    const long c = (i - (long)r * chunks) * 8;
#pragma unroll
    for (int h = 0; h < 8; h += V) {
#pragma unroll
      for (int e = 0; e < V; ++e) u[k][h + e] = 0.f;
      if (i >= total || (ldx != cols && c + h >= cols)) continue;
      const long at = ((long)b * rows + r) * cols + c + h;
      if (use_g) unpack16<T>(*(const uint4*)(g + at), u[k] + h);
      if (MOM) {
        float bn[V];
#pragma unroll
        for (int q = 0; q < V; q += 4) unpack16<float>(*(const uint4*)(mo.buf_out + at + q), bn + q);
#pragma unroll
        for (int e = 0; e < V; ++e) u[k][h + e] = mo.nesterov ? u[k][h + e] + mo.mu * bn[e] : bn[e];
      }
    }
  }
  if (threadIdx.x < 64) {
    double s = 0.0;
    for (int i = threadIdx.x; i < blocks; i += 64) s += part[(long)b * blocks + i];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, kWave);
    if (threadIdx.x == 0) s_inv = s == 0.0 ? 0.0 : (s < INFINITY ? (double)kS / (sqrt(s) + (double)eps) : (double)NAN);
  }
  __syncthreads();
  const double inv = s_inv;
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const long i = i0 + k * 256;
    if (i >= total) return;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)((double)u[k][e] * inv);
    f16x8_t hi, lo;
    split_planes(v, hi, lo);
    _Float16* o = x + (long)b * rows * ldx + i * 8;
    *(f16x8_t*)o = hi;
    if (two) *(f16x8_t*)(o + plane) = lo;
  }
}

// Sizes, plans and places of a chunk of the batch.
struct Layout {
  int rows, cols, m, ldx, lda, planes;
  int chunk;            // matrices at a time
  long xs, as;          // values of one X, of one A
  Plan gram, sq, upd;
  int sum_blocks;
  size_t x_b, a_b, sum_b, part_b, total;
};
// Matrices go through in chunks whose X and A (two of each) take at most 2 GiB:
// far more than fills the chip (the smallest chunk that does takes some tens of
// MiB; 8 to 128 matrices of [2048, 1024] at a time take 132 to 145 us each), and what
// a training step can spare of 288 GB.
constexpr size_t kChunkBytes = (size_t)2 << 30;

// One plane leaves 1e-3 to 2e-3 of the result as error, about what rounding it to
// bf16 does.  fp32 results have two (with master weights 2e-3 of a step is some 1e-5
// of a small matrix's weights, hundreds of their roundings).  So have matrices with a
// side of at most 32, where few roundings add up and one plane's error reaches twice
// the result's own rounding.  In time: 128 x [2048, 1024] with master weights 17.7 ms
// against one plane's 6.9; 8 x [16, 1000] 90 us / 70, 128 x [32, 4096] 432 / 257.
static bool takes_planes(int rows, int cols, int dt, bool master) {
  return dt == MOE_F32 || master || rows <= 32 || cols <= 32;
}

static Layout layout(int B, int rows, int cols, bool planes) {
  Layout l{};
  l.rows = rows;
  l.cols = cols;
  l.m = rows < cols ? rows : cols;
  l.ldx = (cols + 7) / 8 * 8;
  l.lda = (l.m + 7) / 8 * 8;
  l.planes = planes ? 2 : 1;
  l.xs = (long)rows * l.ldx;
  l.as = (long)l.m * l.lda;
  const size_t per = 4UL * l.planes * (l.xs + l.as);
  size_t most = kChunkBytes / per;
  most = most < 1 ? 1 : most > 32768 ? 32768 : most;  // a launch's blockIdx.y counts matrices
  l.chunk = (size_t)B <= most ? B : (int)most;
  const int runs = l.planes == 2 ? 3 : 1, n = rows < cols ? cols : rows;
  l.gram = plan(l.chunk, l.m, l.lda, (long)runs * gg::cdiv(n, 64), 2, true);
  l.sq = plan(l.chunk, l.m, l.lda, (long)runs * gg::cdiv(l.m, 64), 2, true);
  l.upd = plan(l.chunk, rows, l.ldx, (long)runs * gg::cdiv(l.m, 64), 2, false);
  // 16384 values a workgroup; 4096 where that gives a matrix at most 64 of them (8 x
  // [128, 256]: 6.1 -> 3.3 us; more partial sums cost the scaling pass that reads them,
  // 128 x [2048, 1024] 345 -> 369 us with 256 instead of 128)
  const long v = (long)rows * cols, many = gg::cdiv(v, 16384), few = gg::cdiv(v, 4096);
  l.sum_blocks = (int)(many > kSumBlocks ? kSumBlocks : few <= 64 ? few : many > 64 ? many : 64);
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  l.x_b = up(2UL * l.planes * l.chunk * l.xs);
  l.a_b = up(2UL * l.planes * l.chunk * l.as);
  l.sum_b = up(8UL * l.chunk * l.sum_blocks);
  size_t p = l.gram.part_bytes(l.chunk, l.m, l.lda);
  const size_t p2 = l.sq.part_bytes(l.chunk, l.m, l.lda), p3 = l.upd.part_bytes(l.chunk, rows, l.ldx);
  p = p > p2 ? p : p2;
  l.part_b = up(p > p3 ? p : p3);
  l.total = 2 * l.x_b + 2 * l.a_b + l.sum_b + l.part_b;
  return l;
}

template <class T, bool TWO>
static hipError_t orthogonalize(const void* g, int B, int rows, int cols, int steps, float eps, Momentum mo,
                                Update u, char* ws, hipStream_t s) {
  const Layout l = layout(B, rows, cols, TWO);
  const bool tall = rows > cols;
  _Float16* x0 = (_Float16*)ws;
  _Float16* x1 = (_Float16*)(ws + l.x_b);
  _Float16* A = (_Float16*)(ws + 2 * l.x_b);
  _Float16* Bm = (_Float16*)(ws + 2 * l.x_b + l.a_b);
  double* sums = (double*)(ws + 2 * l.x_b + 2 * l.a_b);
  float* parts = (float*)(ws + 2 * l.x_b + 2 * l.a_b + l.sum_b);
  const long mat = (long)rows * cols;
  for (int b0 = 0; b0 < B; b0 += l.chunk) {
    const int nb = B - b0 < l.chunk ? B - b0 : l.chunk;
    const T* gc = (const T*)g + b0 * mat;
    Momentum mc = mo;
    if (mo.buf) {
      mc.buf += b0 * mat;
      mc.buf_out += b0 * mat;
    }
    Update uc = u;
    uc.out = (T*)u.out + b0 * mat;
    if (u.w) uc.w = (const T*)u.w + b0 * mat;
    if (u.master) {
      uc.master += b0 * mat;
      uc.master_out += b0 * mat;
    }
    const long xplane = nb * l.xs, aplane = nb * l.as;
    sumsq_kernel<T><<<dim3(l.sum_blocks, nb), 256, 0, s>>>(gc, mc, mat, l.sum_blocks, sums);
    // four pieces a thread; one where that leaves CUs without a workgroup (8 x [128,
    // 256] with momentum 7.4 -> 3.9 us)
    const long pieces = l.xs / 8;
    auto scale = [&](auto kernel, int nc) {
      kernel<<<dim3(gg::cdiv(pieces, 256L * nc), nb), 256, 0, s>>>(gc, mc, rows, cols, l.ldx, eps, sums, l.sum_blocks, TWO,
                                                                   xplane, x0);
    };
    const bool few = gg::cdiv(pieces, 1024L) * nb < 256;
    if (mo.buf) few ? scale(scale_kernel<T, true, 1>, 1) : scale(scale_kernel<T, true, 4>, 4);
    else few ? scale(scale_kernel<T, false, 1>, 1) : scale(scale_kernel<T, false, 4>, 4);
    hipError_t err = hipGetLastError();
    _Float16 *x = x0, *y = x1;
    for (int it = 0; it < steps && err == hipSuccess; ++it) {
      Args a{};
      a.batch = nb;
      a.nseg = TWO ? 3 : 1;
      // A = X X^T, or X^T X
      a.A = a.B = x;
      a.lda = a.ldb = l.ldx;
      a.a_bs = a.b_bs = l.xs;
      a.a_plane = a.b_plane = xplane;
      a.M = a.b_rows = l.m;
      a.N = l.lda;
      a.K = tall ? rows : cols;
      a.sym = 1;
      const EpiIter<TWO, false> ea{A, nullptr, l.lda, l.as, aplane, 1.0f / kS, 0.f, 0.f};
      err = tall ? run<ElF16, false, false>(l.gram, a, ea, parts, s) : run<ElF16, true, true>(l.gram, a, ea, parts, s);
      if (err != hipSuccess) break;
      // B = a + b A + c A^2
      a.A = a.B = A;
      a.lda = a.ldb = l.lda;
      a.a_bs = a.b_bs = l.as;
      a.a_plane = a.b_plane = aplane;
      a.K = l.m;
      const EpiIter<TWO, true> eb{Bm, A, l.lda, l.as, aplane, kC / kS, kB, kA * kS};
      err = run<ElF16, true, true>(l.sq, a, eb, parts, s);
      if (err != hipSuccess) break;
      // X' = B X, or X B
      a.sym = 0;
      a.M = rows;
      a.N = l.ldx;
      if (tall) {
        a.A = x;
        a.lda = l.ldx;
        a.a_bs = l.xs;
        a.a_plane = xplane;
        a.B = Bm;
      } else {
        a.A = Bm;
        a.B = x;
        a.ldb = l.ldx;
        a.b_bs = l.xs;
        a.b_plane = xplane;
      }
      if (it + 1 < steps) {
        const EpiIter<TWO, false> ex{y, nullptr, l.ldx, l.xs, xplane, 1.0f / kS, 0.f, 0.f};
        err = tall ? run<ElF16, true, true>(l.upd, a, ex, parts, s) : run<ElF16, true, false>(l.upd, a, ex, parts, s);
        _Float16* t = x;
        x = y;
        y = t;
      } else {
        const EpiUpdate<T> eu{1.0f / (kS * kS), rows, cols, uc};
        err = tall ? run<ElF16, true, true>(l.upd, a, eu, parts, s) : run<ElF16, true, false>(l.upd, a, eu, parts, s);
      }
    }
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace dn

using namespace dn;

static hipError_t by_type(const void* g, int B, int rows, int cols, int dt, int steps, float eps, Momentum mo, Update u,
                          void* ws, hipStream_t s) {
  if (dt == MOE_F32) return orthogonalize<float, true>(g, B, rows, cols, steps, eps, mo, u, (char*)ws, s);
  if (takes_planes(rows, cols, dt, u.master != nullptr))
    return orthogonalize<uint16_t, true>(g, B, rows, cols, steps, eps, mo, u, (char*)ws, s);
  return orthogonalize<uint16_t, false>(g, B, rows, cols, steps, eps, mo, u, (char*)ws, s);
}

size_t orthogonalize_ws_bytes(int B, int rows, int cols, int dt) {
  const size_t two = layout(B, rows, cols, true).total;  // (with master weights, any may take two planes)
  const size_t one = takes_planes(rows, cols, dt, false) ? 0 : layout(B, rows, cols, false).total;
  return two > one ? two : one;
}

OrthoPlan ortho_plan(int B, int rows, int cols, int dt, bool master) {
  const Layout l = layout(B, rows, cols, takes_planes(rows, cols, dt, master));
  auto of = [&](const Plan& p, int M, int N, bool sym) {
    return DensePlan{0, p.tile, p.stages((long)l.chunk * p.nsplit * tiles_of(M, N, p.tile, sym)), p.nsplit};
  };
  return {l.planes, l.chunk, of(l.gram, l.m, l.lda, true), of(l.sq, l.m, l.lda, true), of(l.upd, rows, l.ldx, false)};
}

hipError_t launch_orthogonalize(const void* g, int B, int rows, int cols, int dt, int steps, float eps, void* out,
                                void* ws, hipStream_t s) {
  Update u{};
  u.out = out;
  return by_type(g, B, rows, cols, dt, steps, eps, Momentum{}, u, ws, s);
}

hipError_t launch_muon_step(const moe_muon_args& a, hipStream_t s) {
  const Momentum mo{a.buf, a.buf_out, a.momentum, a.nesterov};
  const Update u{a.w, a.master, a.master_out, a.w_out, a.step, a.decay, a.lr_scale};
  return by_type(a.g, a.B, a.rows, a.cols, a.dt, a.steps, a.eps, mo, u, a.ws, s);
}

}  // namespace trg
