// 4-bit weights: E2M1 elements (0, 1/2, 1, 3/2, 2, 3, 4, 6 and their
// negatives) with one E8M0 scale per 32 consecutive values of a row, the OCP
// microscaling format of the same family as the MXFP8 copies:
//   s = clamp(floor(log2(amax)) - 2, -127, 127) from the exponent bits of the
//       block's largest magnitude (s = -127 for an all-zero block); byte s + 127;
//   element = v * 2^-s rounded to nearest even, saturating to +-6, the sign of
//       zero kept.
// A block that holds an infinity or NaN gets the scale byte 255, which stands
// for NaN in all of its 32 values, and zero codes: E2M1 itself has no NaN, and
// a number in its place would hide the fault.
// Codes are packed two to a byte, the even value in the low half; scales are
// K-chunk major as for MXFP8: block b of row r of n at byte (b/4 * n + r)*4 +
// b%4, so a row's four scales of a 128-value chunk are one dword.  Places past
// the row's last block hold 0.
//
// Both directions are one streaming pass bound by HBM: a lane takes one
// 16-byte piece of the values, 4 (bf16) or 8 (fp32) lanes a block.
#include "common.h"
#include "kernels.h"

namespace trg {

namespace {

// Code of x (already divided by the block's scale), ties to the even code:
// steps of 1/2 below 2, of 1 below 4, of 2 above.  Saturates at 6.
TRG_DEV uint32_t e2m1_code(float x) {
  const float a = fminf(fabsf(x), 6.0f);
  const float lo = rintf(a * 2.0f), mid = rintf(a) + 2.0f, hi = rintf(a * 0.5f) + 4.0f;
  const float m = a < 2.0f ? lo : (a < 4.0f ? mid : hi);
  return (uint32_t)m | (__float_as_uint(x) >> 31 << 3);
}

// Value of a code without its scale.
TRG_DEV float e2m1_value(uint32_t c) {
  const uint32_t ex = (c >> 1) & 3, m = c & 1;
  // ex > 0: (1 + m/2) 2^(ex-1); ex = 0: m/2
  const uint32_t bits = ex != 0 ? ((ex + 126) << 23 | m << 22) : (m != 0 ? 0x3F000000u : 0u);
  return __uint_as_float(bits | (c >> 3) << 31);
}

// 2^n for n in [-126, 127].  The block exponents lie in [-127, 125], so 2^-s is
// a normal float and the division by 2^s an exact multiplication.
TRG_DEV float pow2n(int n) { return __uint_as_float((uint32_t)(n + 127) << 23); }

// One thread per 16-byte piece; pieces of a row are padded to whole 128-value
// chunks so that a chunk is a run of lanes of one wave.
template <class T>
__global__ __launch_bounds__(256) void quantize_e2m1_kernel(const T* __restrict__ in, int rows, int cols,
                                                            uint8_t* __restrict__ q, uint8_t* __restrict__ s) {
  constexpr int V = 16 / (int)sizeof(T);
  constexpr int LB = 32 / V;   // lanes a block
  constexpr int LC = 128 / V;  // lanes a chunk
  const int nch = (cols + 127) / 128;
  const long g = (long)blockIdx.x * 256 + threadIdx.x;
  const long ch = g / LC;  // chunk: row-major over (row, chunk of the row)
  const int l = (int)(g % LC);
  const long row = ch / nch;
  const int c0 = (int)(ch % nch) * 128 + l * V;
  const bool in_row = row < rows && c0 < cols;  // cols is a multiple of 32: a whole block is in or out
  float f[V];
  if (in_row) {
    unpack16<T>(*(const uint4*)(in + row * cols + c0), f);
  } else {
#pragma unroll
    for (int c = 0; c < V; ++c) f[c] = 0.f;
  }
  uint32_t am = 0;  // magnitudes order like their bit patterns, infinity and NaN on top
#pragma unroll
  for (int c = 0; c < V; ++c) am = max(am, __float_as_uint(f[c]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 1; o < LB; o <<= 1) am = max(am, (uint32_t)__shfl_xor((int)am, o, 64));
  const int ex = (int)(am >> 23);
  const bool bad = ex == 255;
  const int se = ex == 0 ? -127 : max(ex - 129, -127);
  uint32_t code = 0;
  if (!bad) {
    const float inv = pow2n(-se);
#pragma unroll
    for (int c = 0; c < V; ++c) code |= e2m1_code(f[c] * inv) << (4 * c);
  }
  if (in_row) {
    uint8_t* o = q + (row * cols + c0) / 2;
    if constexpr (V == 8) *(uint32_t*)o = code;
    else *(uint16_t*)o = (uint16_t)code;
  }
  uint32_t sb = in_row ? (uint32_t)(bad ? 255 : se + 127) << (8 * ((l / LB) & 3)) : 0u;
#pragma unroll
  for (int o = LB; o < LC; o <<= 1) sb |= (uint32_t)__shfl_xor((int)sb, o, 64);
  if (l == 0 && row < rows) *(uint32_t*)(s + ((ch % nch) * rows + row) * 4) = sb;
}

template <class T>
__global__ __launch_bounds__(256) void dequantize_e2m1_kernel(const uint8_t* __restrict__ q,
                                                              const uint8_t* __restrict__ s, int rows, int cols,
                                                              T* __restrict__ out) {
  constexpr int V = 16 / (int)sizeof(T);
  const long g = (long)blockIdx.x * 256 + threadIdx.x;  // 16-byte piece of the output
  const int ppr = cols / V;
  const long row = g / ppr;
  if (row >= rows) return;
  const int c0 = (int)(g % ppr) * V;
  const uint8_t* p = q + (row * cols + c0) / 2;
  const uint32_t code = V == 8 ? *(const uint32_t*)p : *(const uint16_t*)p;
  const int b = c0 / 32;
  const int sb = s[((long)(b / 4) * rows + row) * 4 + b % 4];
  const float sc = sb == 255 ? __uint_as_float(0x7FC00000u)
                             : (sb == 0 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)sb << 23));
  float f[V];
#pragma unroll
  for (int c = 0; c < V; ++c) f[c] = e2m1_value((code >> (4 * c)) & 15u) * sc;
  *(uint4*)(out + row * cols + c0) = pack16<T>(f);
}

}  // namespace

hipError_t launch_quantize_e2m1(const void* in, bool bf16, int rows, int cols, uint8_t* q, uint8_t* s, hipStream_t st) {
  const long chunks = (long)rows * ((cols + 127) / 128);
  if (bf16)
    quantize_e2m1_kernel<uint16_t><<<(unsigned)((chunks * 16 + 255) / 256), 256, 0, st>>>((const uint16_t*)in, rows,
                                                                                         cols, q, s);
  else
    quantize_e2m1_kernel<float><<<(unsigned)((chunks * 32 + 255) / 256), 256, 0, st>>>((const float*)in, rows, cols, q,
                                                                                      s);
  return hipGetLastError();
}

hipError_t launch_dequantize_e2m1(const uint8_t* q, const uint8_t* s, bool bf16, int rows, int cols, void* out,
                                  hipStream_t st) {
  const long pieces = (long)rows * cols / (bf16 ? 8 : 4);
  if (bf16)
    dequantize_e2m1_kernel<uint16_t><<<(unsigned)((pieces + 255) / 256), 256, 0, st>>>(q, s, rows, cols,
                                                                                      (uint16_t*)out);
  else
    dequantize_e2m1_kernel<float><<<(unsigned)((pieces + 255) / 256), 256, 0, st>>>(q, s, rows, cols, (float*)out);
  return hipGetLastError();
}

}  // namespace trg
