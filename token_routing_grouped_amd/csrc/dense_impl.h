// Dense (batched) matrix products with an epilogue, for the projections beside
// the experts (dense.hip) and the orthogonalised weight update (muon.hip):
//   C[b] = epilogue(A[b] B[b]^T),  A [M,K], B [N,K], fp32 accumulation,
// each operand stored K-contiguous (KC) or MN-contiguous (X[k][mn]), in bf16,
// fp16 or fp32.  The tile pipeline is the grouped GEMMs' (ggemm.hip): operands
// move from memory to LDS without registers, two stages of 128 bytes of K, the
// next 16-byte slice's fragments are read while the current one's matrix
// instructions run.  What differs:
//  * Any K, M, N: a buffer resource bounds each operand's rows, and the lanes
//    past a K-contiguous row's end load from past the resource, so both
//    operands are zero there.
//  * Three types in one kernel: a stage holds 128 bytes of K of every row, so
//    bf16 and fp16 take 64 values a step and fp32 32; a 16-byte fragment is one
//    32x32x16 instruction or four 32x32x2.
//  * Split sums: an operand in two fp16 planes, hi and 2^11 lo, is multiplied in
//    three runs over K (lo hi, hi lo, then hi hi after scaling by 2^-11), which
//    keeps 22 mantissa bits at a third of the fp16 rate (the fp32 instruction
//    has a sixteenth of it).
//  * Symmetric products compute the tiles on and above the diagonal and store
//    each twice.
//  * K may be cut into parts (few output tiles): each part's sums go to memory
//    and join_kernel adds them in order and runs the epilogue.
#pragma once

#include "common.h"
#include "ggemm_impl.h"

namespace trg {
namespace dn {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));

constexpr int kPast = 0x7ffffff0;  // a byte offset past every operand tile's resource (under 2^31 bytes each)

struct ElBf16 {
  static constexpr int ES = 2;
  static TRG_DEV f32x16_t mma(u32x4v b, u32x4v a, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, b), __builtin_bit_cast(bf16x8_t, a), c,
                                                   0, 0, 0);
  }
};
struct ElF16 {
  static constexpr int ES = 2;
  static TRG_DEV f32x16_t mma(u32x4v b, u32x4v a, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, b), __builtin_bit_cast(f16x8_t, a), c, 0,
                                                  0, 0);
  }
};
// fp32: instruction r takes value r of both operands' 16 bytes, so its two k
// are 4 apart: any order of K will do as long as both operands have the same.
struct ElF32 {
  static constexpr int ES = 4;
  static TRG_DEV f32x16_t mma(u32x4v b, u32x4v a, f32x16_t c) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(b[r]), __uint_as_float(a[r]), c, 0, 0, 0);
    return c;
  }
};

struct Args {
  const void* A;
  const void* B;
  long lda, ldb;          // elements between rows
  long a_bs, b_bs;        // between matrices of the batch
  long a_plane, b_plane;  // between the hi and lo planes (nseg = 3)
  int M, N, K;            // K * ES a multiple of 16 where an operand is K-contiguous
  int b_rows;             // rows of a K-contiguous B (C's columns from there to N are 0)
  int batch, nsplit, split_steps;  // K parts, and K steps in each
  int nseg;                        // 1, or 3: split sums
  int sym;                         // C symmetric: tiles with m <= n, stored twice
  int tiles_m, tiles_n, tiles;     // tiles of one part of one matrix
};

// 8 values of a row, from column n (a multiple of 8) on; fp32 rows may end
// after four of them.
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

// ---- operand tiles: memory -> LDS ------------------------------------------
// K-contiguous: as gg::load_kc, with the lanes at or past the row's end (kend
// bytes) sent past the resource.
template <int BMN, int NW>
TRG_DEV void load_kc(char* dst, int wave, int lane, __amdgpu_buffer_rsrc_t rs, int kbyte, int kend, int ld_bytes) {
  constexpr int PER = BMN / 8 / NW;
  static_assert(PER >= 1 && BMN / 8 % NW == 0, "blocks per wave");
  const int l8 = lane >> 3;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int blk = wave * PER + i;
    const int c = ((lane & 7) ^ (((blk & 1) << 2) | (l8 >> 1))) << 4;
    const int off = (blk * 8 + l8) * ld_bytes + kbyte + c;
    gg::lds_load16(rs, dst + blk * 1024, kbyte + c < kend ? off : kPast);
  }
}

// MN-contiguous: 128 / ES rows of BMN values; the resource starts at the step's
// first row and the tile's first column and ends with the last row.
template <int ES, int BMN>
TRG_DEV int mn_swizzle(int kr) {  // XOR of a 16-byte chunk's place in row kr
  return ES == 2 ? (kr & 3) << 2 : ((kr >> 2) & 1) << 3;
}
template <int ES, int BMN, int NW>
TRG_DEV void load_mn(char* dst, int wave, int lane, __amdgpu_buffer_rsrc_t rs, int ld_bytes) {
  constexpr int ROWB = BMN * ES, NBLK = BMN / 8, PER = NBLK / NW;
  static_assert(PER >= 1 && NBLK % NW == 0, "blocks per wave");
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int blk = wave * PER + i;
    const int at = blk * 1024 + lane * 16;
    const int kr = at / ROWB;
    const int c = ((at % ROWB) >> 4) ^ mn_swizzle<ES, BMN>(kr);
    gg::lds_load16(rs, dst + blk * 1024, kr * ld_bytes + c * 16);
  }
}

// ---- fragments: LDS -> registers --------------------------------------------
// 16 bytes of K (slice kk of 4, half lane / 32) of row base + lane % 32.
template <class El, int BMN, bool KC>
TRG_DEV u32x4v frag(const char* s, int base, int kk, int lane) {
  if constexpr (KC) {
    return __builtin_bit_cast(u32x4v, gg::frag_kc(s, base, kk, lane));
  } else if constexpr (El::ES == 2) {
    return __builtin_bit_cast(u32x4v, gg::frag_mnc<BMN>(s, base, kk, lane));
  } else {
    const int h = lane >> 5, col = base + (lane & 31);
    const char* p = s + (kk * 2 + h) * 4 * (BMN * 4) + (((col >> 2) ^ (h << 3)) << 4) + (col & 3) * 4;
    u32x4v v;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = *(const uint32_t*)(p + r * (BMN * 4));
    return v;
  }
}

struct TileAt {
  int b, part, mt, nt;
};
// Tile t: matrix, K part, row and column tile.  Inside a part, eight row tiles
// at a time run down the columns (an XCD's workgroups then share 8 tiles of A
// and a few of B in its L2); symmetric: column by column of the upper triangle.
TRG_DEV TileAt tile_at(const Args& g, int t) {
  TileAt r;
  const int bp = t / g.tiles;
  int i = t - bp * g.tiles;
  r.b = bp / g.nsplit;
  r.part = bp - r.b * g.nsplit;
  if (g.sym) {
    int nt = 0;
    while (i > nt) i -= ++nt;
    r.nt = nt;
    r.mt = i;
  } else {
    const int per = 8 * g.tiles_n;
    const int grp = i / per, in = i - grp * per;
    const int gm = min(8, g.tiles_m - grp * 8);
    r.nt = in / gm;
    r.mt = grp * 8 + in - r.nt * gm;
  }
  return r;
}

// Epi::apply(b, part, row, col, v): the epilogue of 8 consecutive columns of a
// row, col a multiple of 8 under N.
template <class El, int BM, int BN, int WM, int WN, int OCC, bool AKC, bool BKC, class Epi>
__global__ __launch_bounds__(64 * WM * WN, OCC) void dense_kernel(Args g, Epi epi) {
  constexpr int NW = WM * WN, ES = El::ES, KSTEP = 128 / ES;
  constexpr int WTM = BM / WM, WTN = BN / WN, TM = WTM / 32, TN = WTN / 32;
  constexpr int SA = BM * 128, SB = BN * 128, STAGE = SA + SB;
  __shared__ __attribute__((aligned(1024))) char smem[2 * STAGE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;

  const int total = g.batch * g.nsplit * g.tiles;
  const int xcd = blockIdx.x & 7, lb = blockIdx.x >> 3, nbx = gridDim.x >> 3;
  const int per = (total + 7) >> 3;
  const int t_end = min(total, (xcd + 1) * per);
  const int lda_b = (int)g.lda * ES, ldb_b = (int)g.ldb * ES;

  struct Cur {
    TileAt at;
    int m0, n0, k0, nk;  // nk: K steps of one run over the part
  };
  auto decode = [&](int t) {
    Cur c;
    c.at = tile_at(g, t);
    c.m0 = c.at.mt * BM;
    c.n0 = c.at.nt * BN;
    c.k0 = c.at.part * g.split_steps * KSTEP;
    const int left = (g.K - c.k0 + KSTEP - 1) / KSTEP;
    c.nk = max(0, min(left, g.split_steps));
    return c;
  };
  // step it of nseg * nk: operand bytes of one K step into a stage
  auto issue = [&](const Cur& c, int it, int stage) {
    int seg = 0, ks = it;
    if (g.nseg > 1) {
      seg = it >= 2 * c.nk ? 2 : it >= c.nk ? 1 : 0;
      ks = it - seg * c.nk;
    }
    const int k = c.k0 + ks * KSTEP;
    const char* A = (const char*)g.A + (c.at.b * g.a_bs + (g.nseg > 1 && seg == 0 ? g.a_plane : 0)) * ES;
    const char* B = (const char*)g.B + (c.at.b * g.b_bs + (seg == 1 ? g.b_plane : 0)) * ES;
    char* sA = smem + stage * STAGE;
    char* sB = sA + SA;
    if constexpr (AKC) {
      const auto rs = gg::make_rsrc(A + (long)c.m0 * lda_b, (long)min(BM, g.M - c.m0) * lda_b);
      load_kc<BM, NW>(sA, wave, lane, rs, k * ES, g.K * ES, lda_b);
    } else {
      const auto rs = gg::make_rsrc(A + (long)k * lda_b + c.m0 * ES, (long)min(KSTEP, g.K - k) * lda_b - c.m0 * ES);
      load_mn<ES, BM, NW>(sA, wave, lane, rs, lda_b);
    }
    if constexpr (BKC) {
      const auto rs = gg::make_rsrc(B + (long)c.n0 * ldb_b, (long)min(BN, g.b_rows - c.n0) * ldb_b);
      load_kc<BN, NW>(sB, wave, lane, rs, k * ES, g.K * ES, ldb_b);
    } else {
      const auto rs = gg::make_rsrc(B + (long)k * ldb_b + c.n0 * ES, (long)min(KSTEP, g.K - k) * ldb_b - c.n0 * ES);
      load_mn<ES, BN, NW>(sB, wave, lane, rs, ldb_b);
    }
  };

  // As in the grouped GEMMs: a tile's first step is loaded into stage 0 before
  // the previous tile's epilogue, which stages through stage 1.
  int t = xcd * per + lb;
  Cur cur;
  if (t < t_end) {
    cur = decode(t);
    if (cur.nk > 0) issue(cur, 0, 0);
  }
  for (; t < t_end; t += nbx) {
    const Cur c = cur;
    f32x16_t acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    const int steps = c.nk * g.nseg;
    for (int it = 0; it < steps; ++it) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();  // this step's stage is complete; the other one is free
      if (it + 1 < steps) issue(c, it + 1, (it + 1) & 1);
      if (g.nseg > 1 && it == 2 * c.nk) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] *= 1.0f / 2048.0f;
      }
      const char* sA = smem + (it & 1) * STAGE;
      const char* sB = sA + SA;
      u32x4v af[2][TM], bf[2][TN];
#pragma unroll
      for (int i = 0; i < TM; ++i) af[0][i] = frag<El, BM, AKC>(sA, wm * WTM + i * 32, 0, lane);
#pragma unroll
      for (int j = 0; j < TN; ++j) bf[0][j] = frag<El, BN, BKC>(sB, wn * WTN + j * 32, 0, lane);
      __builtin_amdgcn_sched_barrier(0);  // the next slice's reads stay ahead of this one's products
      static_for<4>([&](auto KK) {
        constexpr int kk = decltype(KK)::value, fb = kk & 1;
        if constexpr (kk < 3) {
#pragma unroll
          for (int i = 0; i < TM; ++i) af[fb ^ 1][i] = frag<El, BM, AKC>(sA, wm * WTM + i * 32, kk + 1, lane);
#pragma unroll
          for (int j = 0; j < TN; ++j) bf[fb ^ 1][j] = frag<El, BN, BKC>(sB, wn * WTN + j * 32, kk + 1, lane);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) acc[i][j] = El::mma(bf[fb][j], af[fb][i], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
      });
    }
    __syncthreads();  // every wave is done with the last stage
    if (t + nbx < t_end) {
      cur = decode(t + nbx);
      if (cur.nk > 0) issue(cur, 0, 0);
    }

    // Epilogue.  Each wave stages 16 rows of its tile in fp32 in its part of
    // stage 1, then a lane takes 8 consecutive columns of a row (and, for the
    // mirrored tile, 8 rows of a column).
    constexpr int WLDS = STAGE / NW, P = WTN * 4 + 16, SR = 16;
    static_assert(SR * P <= WLDS, "epilogue staging");
    char* wl = smem + STAGE + wave * WLDS;
    const int lrow = lane & 31, lgrp = (lane >> 5) * 4;
    const bool mirror = g.sym && c.at.mt != c.at.nt;
    static_for<TM * 2>([&](auto IH) {
      constexpr int i = decltype(IH)::value / 2, part = decltype(IH)::value % 2;
      const int ms = c.m0 + wm * WTM + i * 32 + part * SR, ns = c.n0 + wn * WTN;
      if (ms < g.M && ns < g.N) {
        if (lrow / SR == part) {
          static_for<TN>([&](auto J) {
            constexpr int j = decltype(J)::value;
            static_for<4>([&](auto Q) {
              constexpr int q = decltype(Q)::value;
              const f32x4_t v = {acc[i][j][q * 4], acc[i][j][q * 4 + 1], acc[i][j][q * 4 + 2], acc[i][j][q * 4 + 3]};
              *(f32x4_t*)(wl + (lrow & (SR - 1)) * P + (j * 32 + q * 8 + lgrp) * 4) = v;
            });
          });
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int s = 0; s < SR * (WTN / 8) / 64; ++s) {
          const int ch = lane + s * 64, row = ch / (WTN / 8), col = ch % (WTN / 8) * 8;
          float v[8];
          *(f32x4_t*)v = *(const f32x4_t*)(wl + row * P + col * 4);
          *(f32x4_t*)(v + 4) = *(const f32x4_t*)(wl + row * P + col * 4 + 16);
          if (ms + row < g.M && ns + col < g.N) epi.apply(c.at.b, c.at.part, ms + row, ns + col, v);
        }
        if (mirror) {
#pragma unroll
          for (int s = 0; s < SR / 8 * WTN / 64; ++s) {
            const int ch = lane + s * 64, col = ch / (SR / 8), r8 = ch % (SR / 8) * 8;
            float v[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) v[r] = *(const float*)(wl + (r8 + r) * P + col * 4);
            if (ns + col < g.M && ms + r8 < g.N) epi.apply(c.at.b, c.at.part, ns + col, ms + r8, v);
          }
        }
      }
      __builtin_amdgcn_wave_barrier();  // the staging area is rewritten next
    });
  }
}

// One K part's sums: [part][batch][M][ld] fp32.
struct EpiPart {
  float* p;
  long ld, mat, all;  // row; one matrix; one part of all matrices
  TRG_DEV void apply(int b, int part, int m, int n, const float (&v)[8]) const {
    float* o = p + part * all + b * mat + m * ld + n;
    *(f32x4_t*)o = *(const f32x4_t*)v;
    *(f32x4_t*)(o + 4) = *(const f32x4_t*)(v + 4);
  }
};

template <class Epi>
__global__ __launch_bounds__(256) void join_kernel(EpiPart in, int nsplit, int batch, int M, Epi epi) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x, chunks = in.ld / 8;
  if (i >= batch * (long)M * chunks) return;
  const long row = i / chunks;
  const int n = (int)(i - row * chunks) * 8, b = (int)(row / M), m = (int)(row - (long)b * M);
  const float* p = in.p + b * in.mat + m * in.ld + n;
  float v[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) v[c] = p[c];
  for (int s = 1; s < nsplit; ++s) {
    p += in.all;
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] += p[c];
  }
  epi.apply(b, 0, m, n, v);
}

// ---- host: which tiles, how many parts ----------------------------------------
struct Plan {
  int tile;    // 256 or 128
  int nsplit;  // parts of K
  size_t part_bytes(int batch, int M, int N) const {
    return nsplit > 1 ? (size_t)nsplit * batch * M * ((N + 7) / 8 * 8) * 4 : 0;
  }
};

inline long tiles_of(int M, int N, int tile, bool sym) {
  const long tm = gg::cdiv(M, tile), tn = gg::cdiv(N, tile);
  return sym ? tm * (tm + 1) / 2 : tm * tn;
}

// es: bytes an element; ksteps: 128-byte steps of K, over all runs.
inline Plan plan(int batch, int M, int N, long ksteps, int es, bool sym) {
  Plan best{128, 1};
  double t_best = 1e300;
  for (int tile = 256; tile >= 128; tile /= 2) {
    if (tile == 256 && es == 4) continue;
    const int slots = tile == 256 ? 256 : 512;
    for (int split = 1; split <= 16; split *= 2) {
      if (split > 1 && ksteps < 4L * split) break;
      const long tiles = batch * tiles_of(M, N, tile, sym && split == 1);
      const long steps = gg::cdiv(ksteps, split);
      const double step = tile == 256 ? 1.6 : (es == 4 ? 4.0 : 1.1);
      const double rounds = (double)gg::cdiv(tiles * split, slots);
      double t = rounds * (steps * step + (tile == 256 ? 8.0 : 4.0));
      if (split > 1) t += 5.0 + 8.0 * split * batch * (double)M * N / 3e6;
      if (t < t_best) {
        t_best = t;
        best = Plan{tile, split};
      }
    }
  }
  return best;
}

template <class El, bool AKC, bool BKC, class Epi>
hipError_t run(const Plan& p, Args a, const Epi& epi, float* parts, hipStream_t s) {
  if (a.M <= 0 || a.N <= 0 || a.batch <= 0) return hipSuccess;
  constexpr int KSTEP = 128 / El::ES;
  a.tiles_m = gg::cdiv(a.M, p.tile);
  a.tiles_n = gg::cdiv(a.N, p.tile);
  a.sym = a.sym && p.nsplit == 1;
  a.tiles = (int)tiles_of(a.M, a.N, p.tile, a.sym);
  a.nsplit = p.nsplit;
  const int ksteps = gg::cdiv(a.K, KSTEP);
  a.split_steps = gg::cdiv(ksteps, p.nsplit);
  const long total = (long)a.tiles * a.nsplit * a.batch;
  const int need = (int)((total + 7) / 8 * 8);
  auto go = [&](const auto& e) {
    if (p.tile == 256) {
      if constexpr (El::ES == 2)
        dense_kernel<El, 256, 256, 2, 4, 2, AKC, BKC><<<need < 256 ? need : 256, 512, 0, s>>>(a, e);
    } else {
      dense_kernel<El, 128, 128, 2, 2, 2, AKC, BKC><<<need < 512 ? need : 512, 256, 0, s>>>(a, e);
    }
  };
  if (p.nsplit == 1) {
    go(epi);
  } else {
    const long ld = (a.N + 7) / 8 * 8;
    const EpiPart part{parts, ld, a.M * ld, a.batch * (long)a.M * ld};
    go(part);
    const long n = (long)a.batch * a.M * (ld / 8);
    join_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(part, p.nsplit, a.batch, a.M, epi);
  }
  return hipGetLastError();
}

}  // namespace dn
}  // namespace trg
