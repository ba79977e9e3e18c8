// Root-mean-square norm in front of the expert layer, with the residual's
// addition and an MXFP8 copy of the output, and its gradients.
//
//   v = x + res            (fp32; res optional)         s = v rounded to dt
//   rstd = 1 / sqrt(mean_c v^2 + eps)
//   y = v * rstd * w                                    rounded to dt
//   q, qs: E4M3 elements and E8M0 scales of y, taken from the fp32 values (one
//          rounding), rowwise with the scales K-chunk major
//   dx = rstd * (g - xh * mean_c(g xh)) + ds,  g = dy w,  xh = s rstd
//   dw = sum_t dy xh
//
// All sums are fp32.  Both directions are bound by HBM: one read of each
// input, one write of each output, nothing kept between the passes but the
// row in registers.  A row is held by WPR waves (1, 4 or 16), NP 16-byte
// pieces a lane, so the row's sum is a wave sum (plus, for WPR > 1, one
// barrier per row over WPR partial sums).
//
// Measured, 16384 x 2048 bf16 (a large copy reads and writes 4.74 TB/s): forward
// with residual and MXFP8 copy 60.4 us, 5.0 TB/s; backward with ds 54.9 us, 4.9
// TB/s, of which the second launch 4; 1021 x 6144 fp32 without ds 18.1 us, 4.2
// TB/s.  One row of 2048: 3.0 us.
#include "common.h"
#include "kernels.h"

namespace trg {

namespace {

// Sum of v over the WPR waves that hold one row, known to all of them.  red:
// WPR floats of this row and parity; two parities let the next row's sums go
// out while a slow wave still reads this one's, so one barrier a row is enough.
template <int WPR>
TRG_DEV float row_sum(float v, float* red, int wave_in_row) {
  v = wave_sum(v);
  if constexpr (WPR == 1) {
    return v;
  } else {
    if ((threadIdx.x & 63) == 0) red[wave_in_row] = v;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < WPR; ++i) t += red[i];
    return t;
  }
}

// E8M0 exponent and E4M3 codes: s = clamp(floor(log2 amax) - 8, -127, 127)
// from the exponent bits; elements are divided by 2^s (an exact multiplication
// by 2^-s; s is at most 120, so 2^-s is normal or, at s = -127, 2^127),
// clamped to +-448 and rounded to nearest even.  NaN keeps the NaN code: the
// clamp alone would turn it into a number.
TRG_DEV int norm_scale_exp(float amax) {
  const int ex = (int)((__float_as_uint(amax) >> 23) & 0xFF);
  return ex == 0 ? -127 : max(ex - 135, -127);
}
TRG_DEV float pow2f(int n) { return __uint_as_float((uint32_t)(n + 127) << 23); }  // n in [-126, 127]
TRG_DEV float clamp448(float x) { return x != x ? x : __builtin_amdgcn_fmed3f(x, -448.f, 448.f); }
TRG_DEV uint32_t e4m3x4(const float* f, float inv) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(f[0] * inv), clamp448(f[1] * inv), 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(f[2] * inv), clamp448(f[3] * inv), w, true);
  return (uint32_t)w;
}

// Forward.  One row per WPR waves; 256 threads (four rows a workgroup) for WPR = 1,
// WPR * 64 threads otherwise.
template <class T, int WPR, int NP>
__global__ __launch_bounds__(WPR == 16 ? 1024 : 256) void rmsnorm_fwd_kernel(
    const T* x, const T* res, const T* __restrict__ w, int rows, int d, float eps, T* s, T* y,
    uint8_t* __restrict__ q, uint8_t* __restrict__ qs, float* __restrict__ rstd_out) {
  constexpr int V = 16 / (int)sizeof(T);
  constexpr int RPB = WPR == 1 ? 4 : 1;
  __shared__ float red[WPR];
  const int wv = threadIdx.x >> 6;
  const int row = blockIdx.x * RPB + (WPR == 1 ? wv : 0);
  if (WPR == 1 && row >= rows) return;  // the whole wave leaves; no barrier follows when WPR == 1
  const int lane = WPR == 1 ? (int)(threadIdx.x & 63) : (int)threadIdx.x;  // lane within the row
  const int np = d / V;                                                    // pieces in a row
  const long base = (long)row * d;
  float v[NP][V];
  float ss = 0.f;
  uint4 a[NP], b[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int i = p * WPR * 64 + lane;
    if (i < np) {
      a[p] = *(const uint4*)(x + base + (long)i * V);
      if (res != nullptr) b[p] = *(const uint4*)(res + base + (long)i * V);
    }
  }
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int i = p * WPR * 64 + lane;
    if (i < np) {
      unpack16<T>(a[p], v[p]);
      if (res != nullptr) {
        float r[V];
        unpack16<T>(b[p], r);
#pragma unroll
        for (int c = 0; c < V; ++c) v[p][c] += r[c];
      }
    } else {
#pragma unroll
      for (int c = 0; c < V; ++c) v[p][c] = 0.f;
    }
#pragma unroll
    for (int c = 0; c < V; ++c) ss = fmaf(v[p][c], v[p][c], ss);
  }
  ss = row_sum<WPR>(ss, red, wv);
  const float rstd = 1.0f / sqrtf(ss / (float)d + eps);
  if (lane == 0 && rstd_out != nullptr) rstd_out[row] = rstd;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int i = p * WPR * 64 + lane;
    const bool in = i < np;
    if (in && s != nullptr) *(uint4*)(s + base + (long)i * V) = pack16<T>(v[p]);
    float f[V];
    if (in) {
      float wf[V];
      unpack16<T>(*(const uint4*)(w + (long)i * V), wf);
#pragma unroll
      for (int c = 0; c < V; ++c) f[c] = v[p][c] * rstd * wf[c];
      if (y != nullptr) *(uint4*)(y + base + (long)i * V) = pack16<T>(f);
    } else {
#pragma unroll
      for (int c = 0; c < V; ++c) f[c] = 0.f;
    }
    if (q != nullptr) {
      // a block of 32 values is LB neighbouring lanes; d is a multiple of 32,
      // so a block is inside the row or wholly past its end
      constexpr int LB = 32 / V;
      float am = 0.f;
#pragma unroll
      for (int c = 0; c < V; ++c) am = fmaxf(am, fabsf(f[c]));
#pragma unroll
      for (int o = 1; o < LB; o <<= 1) am = fmaxf(am, __shfl_xor(am, o, 64));
      const int se = norm_scale_exp(am);
      const float inv = pow2f(-se);
      if (in) {
        if constexpr (V == 8) {
          *(uint2*)(q + base + (long)i * V) = make_uint2(e4m3x4(f, inv), e4m3x4(f + 4, inv));
        } else {
          *(uint32_t*)(q + base + (long)i * V) = e4m3x4(f, inv);
        }
      }
      // the four scale bytes of a 128-value chunk are one dword, gathered from
      // the blocks' first lanes (a chunk is 4 * LB lanes of one wave); places
      // past the row's end hold 0
      uint32_t sb = in ? (uint32_t)(se + 127) << (8 * ((lane / LB) & 3)) : 0u;
#pragma unroll
      for (int o = LB; o < 4 * LB; o <<= 1) sb |= __shfl_xor(sb, o, 64);
      if (in && lane % (4 * LB) == 0) *(uint32_t*)(qs + ((long)(i / (4 * LB)) * rows + row) * 4) = sb;
    }
  }
}

// Backward.  Rows r0, r0 + RPB, ... of one workgroup's share; each lane keeps the weight
// gradient of its columns in registers over all its rows.  part: [grid, d].
template <class T, int WPR, int NP>
__global__ __launch_bounds__(WPR == 16 ? 1024 : 256) void rmsnorm_bwd_kernel(
    const T* dy, const T* ds, const T* s, const T* __restrict__ w, const float* __restrict__ rstd_in, int rows, int d,
    T* dx, float* __restrict__ part) {
  constexpr int V = 16 / (int)sizeof(T);
  constexpr int RPB = WPR == 1 ? 4 : 1;
  __shared__ float red[2][WPR];
  __shared__ float fold[WPR == 1 ? 3 * 64 * V : 1];
  const int wv = threadIdx.x >> 6;
  const int lane = WPR == 1 ? (int)(threadIdx.x & 63) : (int)threadIdx.x;
  const int np = d / V;
  float acc[NP][V];
#pragma unroll
  for (int p = 0; p < NP; ++p)
#pragma unroll
    for (int c = 0; c < V; ++c) acc[p][c] = 0.f;
  uint4 wp[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int i = p * WPR * 64 + lane;
    wp[p] = i < np ? *(const uint4*)(w + (long)i * V) : make_uint4(0, 0, 0, 0);
  }
  const float inv_d = 1.0f / (float)d;
  int par = 0;
  for (int row = blockIdx.x * RPB + (WPR == 1 ? wv : 0); row < rows; row += gridDim.x * RPB, par ^= 1) {
    const long base = (long)row * d;
    uint4 a[NP], b[NP], e[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int i = p * WPR * 64 + lane;
      const bool in = i < np;
      a[p] = in ? *(const uint4*)(dy + base + (long)i * V) : make_uint4(0, 0, 0, 0);
      b[p] = in ? *(const uint4*)(s + base + (long)i * V) : make_uint4(0, 0, 0, 0);
      if (ds != nullptr && in) e[p] = *(const uint4*)(ds + base + (long)i * V);
    }
    const float rstd = rstd_in[row];
    float sum = 0.f;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      float gy[V], xs[V], wf[V];
      unpack16<T>(a[p], gy);
      unpack16<T>(b[p], xs);
      unpack16<T>(wp[p], wf);
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float xh = xs[c] * rstd;
        acc[p][c] = fmaf(gy[c], xh, acc[p][c]);
        sum = fmaf(gy[c] * wf[c], xh, sum);
      }
    }
    const float m = row_sum<WPR>(sum, red[par], wv) * inv_d;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int i = p * WPR * 64 + lane;
      if (i >= np) continue;
      float gy[V], xs[V], wf[V], o[V];
      unpack16<T>(a[p], gy);
      unpack16<T>(b[p], xs);
      unpack16<T>(wp[p], wf);
#pragma unroll
      for (int c = 0; c < V; ++c) o[c] = rstd * (gy[c] * wf[c] - xs[c] * rstd * m);
      if (ds != nullptr) {
        float g[V];
        unpack16<T>(e[p], g);
#pragma unroll
        for (int c = 0; c < V; ++c) o[c] += g[c];
      }
      *(uint4*)(dx + base + (long)i * V) = pack16<T>(o);
    }
  }
  // the workgroup's partial weight gradient: with one wave a row, waves 1..3
  // hand theirs to wave 0, one piece at a time
  float* P = part + (long)blockIdx.x * d;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int i = p * WPR * 64 + lane;
    if constexpr (WPR == 1) {
      __syncthreads();
      if (wv > 0) {
#pragma unroll
        for (int c = 0; c < V; ++c) fold[((wv - 1) * V + c) * 64 + lane] = acc[p][c];
      }
      __syncthreads();
      if (wv == 0) {
#pragma unroll
        for (int c = 0; c < V; ++c)
          acc[p][c] += fold[c * 64 + lane] + fold[(V + c) * 64 + lane] + fold[(2 * V + c) * 64 + lane];
      }
      if (wv != 0) continue;
    }
    if (i < np) {
#pragma unroll
      for (int c = 0; c < V; c += 4)
        *(float4*)(P + (long)i * V + c) = make_float4(acc[p][c], acc[p][c + 1], acc[p][c + 2], acc[p][c + 3]);
    }
  }
}

// dw[c] = sum over the workgroups' partials, in a fixed order: 64 groups of rows,
// then the 64 group sums.  16 columns (a 64-byte line each) x 64 groups a
// workgroup, so that 2048 columns are 128 workgroups with 8 loads in flight a
// thread: 4 us instead of 11 with 64 columns x 16 groups (512 partials).
template <class T>
__global__ __launch_bounds__(1024) void rmsnorm_dw_kernel(const float* __restrict__ part, int np, int d,
                                                          T* __restrict__ dw) {
  __shared__ float red[64][17];
  const int col = threadIdx.x & 15, g = threadIdx.x >> 4;
  const int c = min(blockIdx.x * 16 + col, d - 1);  // d is a multiple of 4: the last workgroup may be short
  float a = 0.f;
  for (int p0 = g; p0 < np; p0 += 64 * 8) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = part[(long)min(p0 + 64 * i, np - 1) * d + c];
#pragma unroll
    for (int i = 0; i < 8; ++i) a += p0 + 64 * i < np ? v[i] : 0.f;
  }
  red[g][col] = a;
  __syncthreads();
  if (threadIdx.x < 64) {  // lane: column lane % 16, a quarter of the groups each
    const int q = threadIdx.x >> 4;
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += red[q * 16 + i][col];
    t += __shfl_xor(t, 16, 64);
    t += __shfl_xor(t, 32, 64);
    if (q == 0 && blockIdx.x * 16 + col < d) Elt<T>::st(dw + c, t);
  }
}

// Rows' shape: waves a row and pieces a lane that hold d elements.  The backward
// keeps three inputs, the weight and the gradient's sums of a lane's columns,
// so more waves beat more pieces.  With 16 waves a lane has 128 registers, and the
// backward's rows over 32 KiB in bf16 do not fit: 4 pieces spill 97, 8 spill 398
// (fp32: 4 and 186).  Measured, backward with ds, 64 MiB a matrix: bf16 d = 16384 63
// us, 4.2 TB/s; 16392 (16 x 4) 220, 1.2; 65536 (16 x 8) 440, 0.6; fp32 16384 67, 4.0;
// 32768 165, 1.6.  The forward has no such step: 4.2 to 5.1 TB/s at all of them.
struct RowShape {
  int wpr, np;
};
RowShape row_shape(int d, int esize) {
  const int pieces = d * esize / 16;  // at most 16 * 64 * 8 (checked by the caller)
  const int wpr = pieces <= 64 * 4 ? 1 : (pieces <= 256 * 4 ? 4 : 16);
  const int per = (pieces + wpr * 64 - 1) / (wpr * 64);
  return {wpr, per <= 1 ? 1 : per <= 2 ? 2 : per <= 4 ? 4 : 8};
}

// Workgroups of the backward's row pass: two a CU when there are rows enough that
// their partial weight gradients (d floats each, out and in) are little next to
// the rows, else one.
int bwd_groups(int rows, int rpb) {
  const int full = (rows + rpb - 1) / rpb, most = rows >= 4096 ? 512 : 256;
  return full < most ? (full < 1 ? 1 : full) : most;
}

// The shapes that row_shape gives.
template <class F>
hipError_t with_shape(RowShape r, F&& f) {
#define TRG_SHAPE(W, N) \
  if (r.wpr == W && r.np == N) return f(std::integral_constant<int, W>{}, std::integral_constant<int, N>{})
  TRG_SHAPE(1, 1);
  TRG_SHAPE(1, 2);
  TRG_SHAPE(1, 4);
  TRG_SHAPE(4, 2);
  TRG_SHAPE(4, 4);
  TRG_SHAPE(16, 2);
  TRG_SHAPE(16, 4);
  TRG_SHAPE(16, 8);
#undef TRG_SHAPE
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_rmsnorm_fwd(const void* x, const void* res, const void* w, int rows, int d, float eps, bool bf16,
                              void* s, void* y, uint8_t* q, uint8_t* qs, float* rstd, hipStream_t st) {
  const RowShape r = row_shape(d, bf16 ? 2 : 4);
  return with_shape(r, [&](auto W, auto N) {
    const int rpb = W == 1 ? 4 : 1, threads = W == 1 ? 256 : W * 64;
    const dim3 grid((rows + rpb - 1) / rpb);
    if (bf16)
      rmsnorm_fwd_kernel<uint16_t, W, N><<<grid, threads, 0, st>>>((const uint16_t*)x, (const uint16_t*)res,
                                                                   (const uint16_t*)w, rows, d, eps, (uint16_t*)s,
                                                                   (uint16_t*)y, q, qs, rstd);
    else
      rmsnorm_fwd_kernel<float, W, N><<<grid, threads, 0, st>>>((const float*)x, (const float*)res, (const float*)w,
                                                                rows, d, eps, (float*)s, (float*)y, q, qs, rstd);
    return hipGetLastError();
  });
}

size_t rmsnorm_bwd_ws_bytes(int rows, int d) {
  // partial weight gradients of every workgroup; one row a workgroup is the
  // most that either storage type uses
  return (size_t)bwd_groups(rows, 1) * d * sizeof(float);
}

hipError_t launch_rmsnorm_bwd(const void* dy, const void* ds, const void* s, const void* w, const float* rstd, int rows,
                              int d, bool bf16, void* dx, void* dw, void* ws, hipStream_t st) {
  const RowShape r = row_shape(d, bf16 ? 2 : 4);
  const int np = bwd_groups(rows, r.wpr == 1 ? 4 : 1);
  const hipError_t e = with_shape(r, [&](auto W, auto N) {
    const int threads = W == 1 ? 256 : W * 64;
    if (bf16)
      rmsnorm_bwd_kernel<uint16_t, W, N><<<np, threads, 0, st>>>((const uint16_t*)dy, (const uint16_t*)ds,
                                                                 (const uint16_t*)s, (const uint16_t*)w, rstd, rows, d,
                                                                 (uint16_t*)dx, (float*)ws);
    else
      rmsnorm_bwd_kernel<float, W, N><<<np, threads, 0, st>>>((const float*)dy, (const float*)ds, (const float*)s,
                                                              (const float*)w, rstd, rows, d, (float*)dx, (float*)ws);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  if (bf16)
    rmsnorm_dw_kernel<uint16_t><<<(d + 15) / 16, 1024, 0, st>>>((const float*)ws, np, d, (uint16_t*)dw);
  else
    rmsnorm_dw_kernel<float><<<(d + 15) / 16, 1024, 0, st>>>((const float*)ws, np, d, (float*)dw);
  return hipGetLastError();
}

}  // namespace trg
