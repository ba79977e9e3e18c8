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
// Both directions are one streaming pass bound by HBM: a lane takes 16-byte
// pieces of the values, 4 (bf16) or 8 (fp32) lanes a block.  Measured, 8192 x 2048
// bf16: quantise 9.4 us, 4.5 TB/s; dequantise 8.5, 5.0; both in turn 16.5 a pass.
#include "common.h"
#include "kernels.h"

namespace trg {

namespace {

// Eight (or four) codes of values divided by the block's scale: gfx950's scaled
// conversion divides by the scale operand (2^s; a float subnormal for s = -127),
// rounds to nearest even and saturates at +-6, the format's rule.  The tests put
// every bf16 pattern and the fp32 values beside every border through it.
TRG_DEV uint32_t e2m1_codes4(const float* f, float scale, uint32_t old) {
  uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, f[0], f[1], scale, 0);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[2], f[3], scale, 1);
}

// Two values of byte SEL of eight codes, times the scale (gfx950's scaled
// conversion: exact, fp32 subnormals included).
typedef float f32x2_t __attribute__((ext_vector_type(2)));
template <int SEL>
TRG_DEV void e2m1_values(uint32_t codes, float scale, float* f) {
  const f32x2_t v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, SEL);
  f[0] = v.x;
  f[1] = v.y;
}

// Value of a lane's neighbours inside a row of 16 lanes, in the vector registers.
template <int CTRL>
TRG_DEV uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E;         // within four lanes
constexpr int kHalfMirror = 0x141;                // lane i of eight <-> 7 - i
constexpr int kRor4 = 0x124, kRor8 = 0x128;       // rotations of the row

// N 16-byte pieces a thread, a workgroup's pieces apart, all loaded before the
// first is used; pieces of a row are padded to whole 128-value chunks so that a
// chunk is a run of lanes of one wave.
template <class T, int N>
__global__ __launch_bounds__(256) void quantize_e2m1_kernel(const T* __restrict__ in, int rows, int cols,
                                                            uint8_t* __restrict__ q, uint8_t* __restrict__ s) {
  constexpr int V = 16 / (int)sizeof(T);
  constexpr int LB = 32 / V;   // lanes a block
  constexpr int LC = 128 / V;  // lanes a chunk
  const uint32_t nch = (uint32_t)(cols + 127) / 128;
  const int l = (int)(threadIdx.x % LC);
  uint4 raw[N];
  uint32_t row[N], chunk[N];
  bool in_row[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    // chunks are numbered row-major over (row, chunk of the row); fewer than 2^27
    const uint32_t ch = (uint32_t)(blockIdx.x * N + n) * (256 / LC) + threadIdx.x / LC;
    row[n] = ch / nch;
    chunk[n] = ch - row[n] * nch;
    const int c0 = (int)chunk[n] * 128 + l * V;
    in_row[n] = row[n] < (uint32_t)rows && c0 < cols;  // cols is a multiple of 32: a whole block is in or out
    raw[n] = in_row[n] ? *(const uint4*)(in + (long)row[n] * cols + c0) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float f[V];
    unpack16<T>(raw[n], f);
    uint32_t am = 0;  // magnitudes order like their bit patterns, infinity and NaN on top
#pragma unroll
    for (int c = 0; c < V; ++c) am = max(am, __float_as_uint(f[c]) & 0x7FFFFFFFu);
    am = max(am, dpp<kXor1>(am));
    am = max(am, dpp<kXor2>(am));
    if constexpr (LB == 8) am = max(am, dpp<kHalfMirror>(am));
    const int ex = (int)(am >> 23);
    const bool bad = ex == 255;
    const int sb = max(ex - 2, 0);  // s + 127; a zero or subnormal block gets 0
    const float scale = __uint_as_float(sb != 0 ? (uint32_t)sb << 23 : 0x00400000u);
    uint32_t code = e2m1_codes4(f, scale, 0);
    if constexpr (V == 8) code = (code & 0xFFFFu) | e2m1_codes4(f + 4, scale, 0) << 16;
    if (bad) code = 0;
    const int c0 = (int)chunk[n] * 128 + l * V;
    if (in_row[n]) {
      uint8_t* o = q + ((long)row[n] * cols + c0) / 2;
      if constexpr (V == 8) *(uint32_t*)o = code;
      else *(uint16_t*)o = (uint16_t)code;
    }
    // the chunk's four scale bytes as one dword
    uint32_t sw = in_row[n] ? (uint32_t)(bad ? 255 : sb) << (8 * ((l / LB) & 3)) : 0u;
    if constexpr (LC == 16) {
      sw |= dpp<kRor4>(sw);
      sw |= dpp<kRor8>(sw);
    } else {
      sw |= dpp<kRor8>(sw);
      sw |= (uint32_t)__shfl_xor((int)sw, 16, 64);
    }
    if (l == 0 && row[n] < (uint32_t)rows) *(uint32_t*)(s + ((long)chunk[n] * rows + row[n]) * 4) = sw;
  }
}

// A workgroup takes 256 / LC rows of N neighbouring 128-value chunks: a chunk's
// scale dwords of consecutive rows are contiguous, so they are read in pieces of
// that many dwords (with whole rows a workgroup, one dword of a line each, 8192 x
// 2048 took 12.6 us).
template <class T, int N>
__global__ __launch_bounds__(256) void dequantize_e2m1_kernel(const uint8_t* __restrict__ q,
                                                              const uint8_t* __restrict__ s, int rows, int cols,
                                                              T* __restrict__ out) {
  constexpr int V = 16 / (int)sizeof(T);
  constexpr int LC = 128 / V;  // lanes a chunk
  const uint32_t nch = (uint32_t)(cols + 127) / 128, ncb = (nch + N - 1) / N;
  const uint32_t rb = blockIdx.x / ncb, cb = blockIdx.x - rb * ncb;
  const uint32_t row = rb * (256 / LC) + threadIdx.x / LC;
  const int l = threadIdx.x % LC;
  if (row >= (uint32_t)rows) return;
  uint32_t code[N], sb[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int c0 = (int)(cb * N + n) * 128 + l * V;
    code[n] = sb[n] = 0;
    if (c0 < cols) {
      const uint8_t* p = q + ((long)row * cols + c0) / 2;
      code[n] = V == 8 ? *(const uint32_t*)p : *(const uint16_t*)p;
      sb[n] = s[((long)(cb * N + n) * rows + row) * 4 + (l * V) / 32];
    }
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int c0 = (int)(cb * N + n) * 128 + l * V;
    if (c0 >= cols) continue;
    const float sc = sb[n] == 255 ? __uint_as_float(0x7FC00000u)
                                  : (sb[n] == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(sb[n] << 23));
    float f[V];
    e2m1_values<0>(code[n], sc, f);
    e2m1_values<1>(code[n], sc, f + 2);
    if constexpr (V == 8) {
      e2m1_values<2>(code[n], sc, f + 4);
      e2m1_values<3>(code[n], sc, f + 6);
    }
    *(uint4*)(out + (long)row * cols + c0) = pack16<T>(f);
  }
}

// Pieces a thread: four once that still leaves two workgroups a CU.
template <class F>
hipError_t with_pieces(long pieces, F&& f) {
  if (pieces >= 4L * 256 * 512) return f(std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, 1>{});
}

}  // namespace

hipError_t launch_quantize_e2m1(const void* in, bool bf16, int rows, int cols, uint8_t* q, uint8_t* s, hipStream_t st) {
  const long pieces = (long)rows * ((cols + 127) / 128) * (bf16 ? 16 : 32);
  return with_pieces(pieces, [&](auto N) {
    const unsigned grid = (unsigned)((pieces + 256 * N - 1) / (256 * N));
    if (bf16) quantize_e2m1_kernel<uint16_t, N><<<grid, 256, 0, st>>>((const uint16_t*)in, rows, cols, q, s);
    else quantize_e2m1_kernel<float, N><<<grid, 256, 0, st>>>((const float*)in, rows, cols, q, s);
    return hipGetLastError();
  });
}

hipError_t launch_dequantize_e2m1(const uint8_t* q, const uint8_t* s, bool bf16, int rows, int cols, void* out,
                                  hipStream_t st) {
  const long nch = (cols + 127) / 128, per = bf16 ? 16 : 8;  // rows a workgroup
  return with_pieces((long)rows * nch * (256 / per), [&](auto N) {
    const unsigned grid = (unsigned)((rows + per - 1) / per * ((nch + N - 1) / N));
    if (bf16) dequantize_e2m1_kernel<uint16_t, N><<<grid, 256, 0, st>>>(q, s, rows, cols, (uint16_t*)out);
    else dequantize_e2m1_kernel<float, N><<<grid, 256, 0, st>>>(q, s, rows, cols, (float*)out);
    return hipGetLastError();
  });
}

}  // namespace trg
