// The dense products beside the experts: a matrix product with bias, activation
// and residual in its epilogue, and its gradients.
//   forward   z = x W^T + b,  y = act(z) + res         x [T,K], W [n,K]
//   backward  dz = dy act'(z), db = sum_t dz,  dx = dz W,  dW = dz^T x
// The products are dense_impl.h's tiles; dz is made by one pass over dy and z
// that also sums the bias gradient's partials in fp32.
#include <math.h>

#include "dense_impl.h"

namespace trg {
namespace dn {

// act and its slope in fp32.  gelu is z Phi(z) with the error function.
TRG_DEV float act_f(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.f ? z : (z == z ? 0.f : z);
    case MOE_ACT_GELU: return z * (0.5f + 0.5f * erff(z * 0.70710678118654752f));
    case MOE_ACT_SILU: return z / (1.0f + expf(-z));
    default: return z;
  }
}
TRG_DEV float act_slope(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.f ? 1.f : (z == z ? 0.f : z);
    case MOE_ACT_GELU:
      return 0.5f + 0.5f * erff(z * 0.70710678118654752f) + z * 0.39894228040143268f * expf(-0.5f * z * z);
    case MOE_ACT_SILU: {
      const float s = 1.0f / (1.0f + expf(-z));
      return s + z * s * (1.0f - s);
    }
    default: return 1.f;
  }
}

// y = act(v + bias) + res, z = v + bias; everything but y may be absent.
template <class T>
struct EpiLinear {
  T* y;
  T* z;
  const T* bias;
  const T* res;
  long ld;
  int N, act;
  TRG_DEV void apply(int, int, int m, int n, float (&v)[8]) const {
    const bool both = n + 8 <= N;
    const long at = m * ld + n;
    float f[8];
    if (bias) {
      ld8(bias + n, both, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += f[i];
    }
    if (z) st8(z + at, both, v);
    if (act != MOE_ACT_NONE)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = act_f(v[i], act);
    if (res) {
      ld8(res + at, both, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += f[i];
    }
    st8(y + at, both, v);
  }
};

// dz = dy act'(z) and the bias gradient's partial sums: a thread takes 8
// columns of every 8th row of its block's rows (wave w of 8: rows w, w + 8, ...),
// adds them in fp32, and the waves' sums are added in order.  dz or part may be
// absent; z too where the activation has none.
constexpr int kDzWaves = 8;
template <class T>
__global__ __launch_bounds__(64 * kDzWaves) void dz_kernel(const T* __restrict__ dy, const T* __restrict__ z, int act,
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
      if (act != MOE_ACT_NONE) {
        float zz[8];
        ld8(z + at, both, zz);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] *= act_slope(zz[i], act);
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

// db[c] = sum of the blocks' partials, in order.
template <class T>
__global__ __launch_bounds__(256) void dbias_kernel(const float* __restrict__ part, int blocks, int n,
                                                    T* __restrict__ db) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= n) return;
  float s = 0.f;
  for (int b = 0; b < blocks; ++b) s += part[(long)b * n + c];
  Elt<T>::st(db + c, s);
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

template <class El, class T>
static hipError_t fwd(const void* x, const void* w, const void* bias, const void* res, int rows, int n, int K, int act,
                      int dt, void* z, void* y, void* ws, hipStream_t s) {
  Args a{};
  a.A = x;
  a.lda = K;
  a.B = w;
  a.ldb = K;
  a.M = rows;
  a.N = a.b_rows = n;
  a.K = K;
  a.batch = a.nseg = 1;
  const EpiLinear<T> e{(T*)y, (T*)z, (const T*)bias, (const T*)res, n, n, act};
  return run<El, true, true>(plan_of(rows, n, K, dt), a, e, (float*)ws, s);
}

template <class El, class T>
static hipError_t bwd(const void* dy, const void* x, const void* w, const void* z, int rows, int n, int K, int act,
                      int dt, void* dx, void* dw, void* db, char* ws, hipStream_t s) {
  T* dz = act == MOE_ACT_NONE ? nullptr : (T*)ws;
  if (dz) ws += up256((size_t)rows * n * sizeof(T));
  const int br = dz_block_rows(rows), blocks = gg::cdiv(rows, br);
  float* part = (float*)ws;
  const bool need_dz = dz && (dx || dw);
  if (rows > 0 && (need_dz || db))
    dz_kernel<T><<<dim3(gg::cdiv(n, 512), blocks), 64 * kDzWaves, 0, s>>>((const T*)dy, (const T*)z, act, rows, n, br,
                                                                         need_dz ? dz : nullptr, db ? part : nullptr);
  if (db) dbias_kernel<T><<<gg::cdiv(n, 256), 256, 0, s>>>(part, rows > 0 ? blocks : 0, n, (T*)db);
  hipError_t err = hipGetLastError();
  const void* g = dz ? (const void*)dz : dy;
  if (dx && err == hipSuccess) {  // dx = dz W
    Args a{};
    a.A = g;
    a.lda = n;
    a.B = w;
    a.ldb = K;
    a.M = rows;
    a.N = K;
    a.K = n;
    a.batch = a.nseg = 1;
    const EpiLinear<T> e{(T*)dx, nullptr, nullptr, nullptr, K, K, MOE_ACT_NONE};
    err = run<El, true, false>(plan_of(rows, K, n, dt), a, e, (float*)ws, s);
  }
  if (dw && err == hipSuccess) {  // dW = dz^T x
    Args a{};
    a.A = g;
    a.lda = n;
    a.B = x;
    a.ldb = K;
    a.M = n;
    a.N = K;
    a.K = rows;
    a.batch = a.nseg = 1;
    const EpiLinear<T> e{(T*)dw, nullptr, nullptr, nullptr, K, K, MOE_ACT_NONE};
    err = run<El, false, false>(plan_of(n, K, rows, dt), a, e, (float*)ws, s);
  }
  return err;
}

}  // namespace dn

using namespace dn;

size_t linear_ws_bytes(int T, int n, int K, int dt) { return plan_of(T, n, K, dt).part_bytes(1, T, n); }

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
