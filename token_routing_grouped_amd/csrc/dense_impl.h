// Dense (batched) matrix products with an epilogue, for the projections beside
// the experts (dense.hip) and the orthogonalised weight update (muon.hip):
//   C[b] = epilogue(A[b] B[b]^T),  A [M,K], B [N,K], fp32 accumulation,
// each operand stored K-contiguous (KC) or MN-contiguous (X[k][mn]), in bf16,
// fp16 or fp32.  The tile pipeline is the grouped GEMMs' (ggemm.hip): operands
// move from memory to LDS without registers, two or four stages of 128 bytes of K, the
// next 16-byte slice's fragments are read while the current one's matrix
// instructions run.  What differs:
//  * Any K, M, N: a buffer resource bounds each operand's rows, and the lanes
//    past a K-contiguous row's end load from past the resource, so both
//    operands are zero there.
//  * Three types in one kernel: a stage holds 128 bytes of K of every row, so
//    bf16 and fp16 take 64 values a step and fp32 32; a 16-byte fragment is one
//    32x32x16 instruction or four 32x32x2.
//  * Split sums: operands in two fp16 planes, hi + lo, are multiplied in three
//    runs over K (lo hi, hi lo, hi hi), which keeps 22 mantissa bits at a third
//    of the fp16 rate (the fp32 instruction has a sixteenth of it).
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
  static constexpr bool kRuns = false;  // nseg may be 3
  static TRG_DEV f32x16_t mma(u32x4v b, u32x4v a, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, b), __builtin_bit_cast(bf16x8_t, a), c,
                                                   0, 0, 0);
  }
};
struct ElF16 {
  static constexpr int ES = 2;
  static constexpr bool kRuns = true;
  static TRG_DEV f32x16_t mma(u32x4v b, u32x4v a, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, b), __builtin_bit_cast(f16x8_t, a), c, 0,
                                                  0, 0);
  }
};
// fp32: instruction r takes value r of both operands' 16 bytes, so its two k
// are 4 apart: any order of K will do as long as both operands have the same.
struct ElF32 {
  static constexpr int ES = 4;
  static constexpr bool kRuns = false;
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

// The part of a matrix that an epilogue's tile covers, through a buffer resource
// with 32-bit offsets from the tile's corner: 8 values from (row, col) on, or
// nothing where the offset is kPast (a load gives zeros, a store is dropped), so
// that a tile's edge costs no branch.  fp32 rows may end after four of them.
struct At {
  int row, col;    // from the tile's corner
  bool ok, ok2;    // the first and the last four values exist
};
struct Held {  // 8 values (or 8 of two planes) on their way
  uint4 v[2];
};
template <class T>
struct TileMat {
  __amdgpu_buffer_rsrc_t rs;
  int ld;  // bytes
  TRG_DEV TileMat(const T* p, long at, long ld_elts) : ld((int)ld_elts * (int)sizeof(T)) {
    const unsigned long a = (unsigned long)(p + at);
    const unsigned lo = __builtin_amdgcn_readfirstlane((unsigned)a);
    const unsigned hi = __builtin_amdgcn_readfirstlane((unsigned)(a >> 32));
    rs = __builtin_amdgcn_make_buffer_rsrc((void*)((unsigned long)hi << 32 | lo), (short)0, kPast, gg::kRsrcFlags);
  }
  TRG_DEV int off(const At& a) const { return a.row * ld + a.col * (int)sizeof(T); }
  TRG_DEV uint4 raw(int o) const {
    return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rs, o, 0, 0));
  }
  TRG_DEV void raw_st(int o, uint4 v) const {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4v, v), rs, o, 0, 0);
  }
  TRG_DEV void fetch(const At& a, Held& h) const {
    const int o = off(a);
    h.v[0] = raw(a.ok ? o : kPast);
    if constexpr (sizeof(T) == 4) h.v[1] = raw(a.ok2 ? o + 16 : kPast);
  }
  static TRG_DEV void unpack(const Held& h, float (&f)[8]) {
    unpack16<T>(h.v[0], f);
    if constexpr (sizeof(T) == 4) unpack16<T>(h.v[1], f + 4);
  }
  TRG_DEV void load(const At& a, float (&f)[8]) const {
    Held h;
    fetch(a, h);
    unpack(h, f);
  }
  TRG_DEV void store(const At& a, const float (&f)[8]) const {
    const int o = off(a);
    if constexpr (sizeof(T) == 2) {
      raw_st(a.ok ? o : kPast, pack16<uint16_t>(f));
    } else {
      raw_st(a.ok ? o : kPast, pack16<float>(f));
      raw_st(a.ok2 ? o + 16 : kPast, pack16<float>(f + 4));
    }
  }
};

// ---- operand tiles: memory -> LDS, a wave and 1 KiB block at a time ------------
// A tile's resource: under 2^31 bytes (the caller's widths see to that), never
// negative.  All of it is uniform, which the loads' scalar operands rely on: said
// outright, since the compiler may have formed it in vector registers.
TRG_DEV __amdgpu_buffer_rsrc_t tile_rsrc(const char* base, int bytes) {
  const unsigned long p = (unsigned long)base;
  const unsigned lo = __builtin_amdgcn_readfirstlane((unsigned)p);
  const unsigned hi = __builtin_amdgcn_readfirstlane((unsigned)(p >> 32));
  return __builtin_amdgcn_make_buffer_rsrc((void*)((unsigned long)hi << 32 | lo), (short)0,
                                           __builtin_amdgcn_readfirstlane(bytes), gg::kRsrcFlags);
}

// gg::lds_load16 at an LDS byte offset.
TRG_DEV void lds_load16(__amdgpu_buffer_rsrc_t rs, unsigned lds, int voff) {
  unsigned saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %1\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %2, %3, 0 offen lds\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(voff), "s"(rs)
      : "memory");
}

// K-contiguous: block blk holds rows 8 blk .. 8 blk + 7, 128 bytes of each, their
// 16-byte chunks swizzled as gg::load_kc does.  kc_chunk: the byte of those 128
// that a lane takes (the same for every other block); kc_offset: its place from
// the tile's first row on.
TRG_DEV int kc_chunk(int blk, int lane) { return ((lane & 7) ^ (((blk & 1) << 2) | (lane >> 4))) << 4; }
TRG_DEV int kc_offset(int blk, int lane, int ld_bytes) {
  return (blk * 8 + (lane >> 3)) * ld_bytes + kc_chunk(blk, lane);
}

// MN-contiguous: 128 / ES rows of BMN values; the resource starts at the step's
// first row and the tile's first column and ends with the last row.  Chunk c of row
// kr lies at c ^ mn_swizzle: the rows that one fragment read takes at once (four,
// or in fp32 two, four apart) are in different banks.
template <int ES, int BMN>
TRG_DEV int mn_swizzle(int kr) {
  if (ES == 4) return ((kr >> 2) & 1) << 3;
  return BMN == 64 ? ((kr >> 1) & 1) << 2 : (kr & 3) << 2;
}
template <int ES, int BMN>
TRG_DEV int mn_offset(int blk, int lane, int ld_bytes) {
  constexpr int ROWB = BMN * ES;
  const int at = blk * 1024 + lane * 16, kr = at / ROWB;
  return kr * ld_bytes + ((((at % ROWB) >> 4) ^ mn_swizzle<ES, BMN>(kr)) << 4);
}

// ---- fragments: LDS -> registers --------------------------------------------
// 16 bytes of K (slice kk of 4, half lane / 32) of row base + lane % 32.
template <class El, int BMN, bool KC>
TRG_DEV u32x4v frag(const char* s, int base, int kk, int lane) {
  if constexpr (KC) {
    return __builtin_bit_cast(u32x4v, gg::frag_kc(s, base, kk, lane));
  } else if constexpr (El::ES == 2) {
    // as gg::frag_mnc: a transpose read hands 16 lanes a 4 (k) x 16 block of columns
    const int g = lane >> 4, s16 = lane & 15;
    const int col = base + (g & 1) * 16 + (s16 & 3) * 4;
    const int kr = kk * 16 + (g >> 1) * 8 + (s16 >> 2);
    const char* p = s + kr * (BMN * 2) + (((col >> 3) ^ mn_swizzle<2, BMN>(kr)) << 4) + (col & 7) * 2;
    const auto lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((gg::lds_bf16x4_t*)p);
    const auto hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((gg::lds_bf16x4_t*)(p + 4 * (BMN * 2)));
    return __builtin_bit_cast(u32x4v, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
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

// Epi: `auto tile = epi.tile(b, part, m0, n0)` for a tile's corner, then
// tile.fetch(at, held), which loads what the epilogue has to add, and
// tile.apply(at, v, held): 8 consecutive columns of a row, at.col a multiple of 8.
// epi.cols(): how many columns C has in memory (a multiple of four), Epi::kMirror:
// whether C may be symmetric.
//
// 256-wide tiles: 8 waves, two on a SIMD, one of which computes while the other
// waits for LDS; 128-wide ones: 4 waves, and two workgroups on a CU or, where
// there is one at most (the waits are then all there is), 8 and NST = 4 stages,
// three of which are on their way.  64-wide ones, for few or short sums: 4 waves,
// four stages, two workgroups on a CU (8 waves, two sharing a quarter with half of
// every step's slices each, measured 7 % slower).  Four waves
// with 128 x 128 products each (a third fewer LDS reads, every wait covered by
// reading two slices ahead and loading across tiles) measured no better: 8192^3
// bf16 925 us against 885.
template <class El, int BM, int BN, int WM, int WN, int NST, bool AKC, bool BKC, class Epi>
__global__ __launch_bounds__(64 * WM * WN, 2) void dense_kernel(Args g, Epi epi) {
  constexpr int NW = WM * WN, ES = El::ES, KSTEP = 128 / ES;
  constexpr int WTM = BM / WM, WTN = BN / WN, TM = WTM / 32, TN = WTN / 32;
  constexpr int SA = BM * 128, SB = BN * 128, STAGE = SA + SB;
  constexpr int PA = BM / 8 / NW, PB = BN / 8 / NW;  // 1 KiB blocks of a stage a wave loads
  constexpr int SC = WTN, WLDS = 32 * SC * 4;        // epilogue: 32 rows of a wave's columns, in the last stage
  static_assert((SC == 64 || SC == 32) && NW * WLDS <= STAGE, "epilogue staging");
  __shared__ __attribute__((aligned(1024))) char smem[NST * STAGE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const unsigned lds0 = (unsigned)(unsigned long)(gg::lds_void_t*)smem;

  const int total = g.batch * g.nsplit * g.tiles;
  const int xcd = blockIdx.x & 7, nbx = gridDim.x >> 3;
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
    c.nk = max(0, min((g.K - c.k0 + KSTEP - 1) / KSTEP, g.split_steps));
    return c;
  };
  // The loads: a lane's offsets in its wave's blocks, and the next step's place, all
  // of it moved on from step to step (formed anew each time it cost some 300 cycles a
  // step, which nothing hides where a CU has one workgroup).
  static_assert(PA % 2 == 0 && PB % 2 == 0, "kc_chunk by a block's place in its wave");
  int aoff[PA], boff[PB];
#pragma unroll
  for (int i = 0; i < PA; ++i)
    aoff[i] = AKC ? kc_offset(wave * PA + i, lane, lda_b) : mn_offset<ES, BM>(wave * PA + i, lane, lda_b);
#pragma unroll
  for (int i = 0; i < PB; ++i)
    boff[i] = BKC ? kc_offset(wave * PB + i, lane, ldb_b) : mn_offset<ES, BN>(wave * PB + i, lane, ldb_b);
  const char *pa = nullptr, *pb = nullptr;  // K-contiguous: the tile's first row; else the step's
  int lk = 0, lleft = 0, lseg = 0;          // its first k, steps left in this run, run
  auto aim = [&](const Cur& c) {            // at the first step of run lseg
    const long ea = c.at.b * g.a_bs + (g.nseg > 1 && lseg == 0 ? g.a_plane : 0);
    const long eb = c.at.b * g.b_bs + (lseg == 1 ? g.b_plane : 0);
    pa = (const char*)g.A + (AKC ? ea + c.m0 * g.lda : ea + c.k0 * g.lda + c.m0) * ES;
    pb = (const char*)g.B + (BKC ? eb + c.n0 * g.ldb : eb + c.k0 * g.ldb + c.n0) * ES;
    lk = c.k0;
    lleft = c.nk;
  };
  // half HALF (or, 2, all) of this wave's blocks of the next step; the second one moves on
  // (TAIL: it may end a K-contiguous row)
  auto issue = [&](const Cur& c, int stage, auto HALF, auto TAIL) {
    constexpr int half = decltype(HALF)::value, P = PA + PB;
    constexpr int i0 = half == 1 ? P / 2 : 0, i1 = half == 0 ? P / 2 : P;
    const unsigned sA = lds0 + stage * STAGE + wave * (PA * 1024), sB = lds0 + stage * STAGE + SA + wave * (PB * 1024);
    const int past = (g.K - lk) * ES;  // bytes to the end of a K-contiguous row
    const int mn = min(KSTEP, g.K - lk);
    if (i0 < PA) {
      const auto rs = tile_rsrc(pa, AKC ? min(BM, g.M - c.m0) * lda_b : mn * lda_b - c.m0 * ES);
#pragma unroll
      for (int i = i0; i < (i1 < PA ? i1 : PA); ++i)
        lds_load16(rs, sA + i * 1024, !AKC ? aoff[i] : !decltype(TAIL)::value || kc_chunk(i, lane) < past ? aoff[i] + lk * ES : kPast);
    }
    if (i1 > PA) {
      const auto rs = tile_rsrc(pb, BKC ? max(0, min(BN, g.b_rows - c.n0)) * ldb_b : mn * ldb_b - c.n0 * ES);
#pragma unroll
      for (int i = (i0 > PA ? i0 - PA : 0); i < i1 - PA; ++i)
        lds_load16(rs, sB + i * 1024, !BKC ? boff[i] : !decltype(TAIL)::value || kc_chunk(i, lane) < past ? boff[i] + lk * ES : kPast);
    }
    if (half > 0) {
      lk += KSTEP;
      if (!AKC) pa += (long)KSTEP * lda_b;
      if (!BKC) pb += (long)KSTEP * ldb_b;
      if (--lleft == 0 && ++lseg < g.nseg) aim(c);
    }
  };

  // A tile's first NST - 1 steps are loaded into the first stages before the
  // previous tile's epilogue, which stages through the last one.
  auto start = [&](const Cur& c) {
    lseg = 0;
    aim(c);
#pragma unroll
    for (int s = 0; s < NST - 1; ++s)
      if (s < c.nk * g.nseg) issue(c, s, std::integral_constant<int, 2>{}, std::true_type{});
  };
  int t = xcd * per + (blockIdx.x >> 3);
  Cur cur;
  if (t < t_end) {
    cur = decode(t);
    start(cur);
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
    // One step: FULL, one of NST in a row after which NST more exist.  stage: a constant
    // there, so that every LDS address is one of a few registers and an immediate.
    auto step = [&](int it, int steps, auto stage, auto FULL) {
      constexpr bool full = decltype(FULL)::value;
      constexpr int P = PA + PB;
      // (the last step of all is never loaded from a FULL one; of several runs each has its own)
      const std::integral_constant<bool, !full || El::kRuns> TAIL{};
      const int st = stage;
      // this step's loads are done once no more are under way than the later steps'
      // (whatever was issued after those only makes the wait longer)
      const int later = full ? NST - 2 : min(NST - 2, steps - 1 - it);
      if (NST > 2 && later == 2) asm volatile("s_waitcnt vmcnt(%0)" ::"i"(2 * P) : "memory");
      else if (NST > 2 && later == 1) asm volatile("s_waitcnt vmcnt(%0)" ::"i"(P) : "memory");
      else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();  // this step's stage is complete; the one read last is free
      const bool more = full || it + NST - 1 < steps;
      constexpr bool AHEAD = BM == 128 && NST == 2;
      if (AHEAD && more) issue(c, (st + NST - 1) % NST, std::integral_constant<int, 2>{}, TAIL);
      const char* sA = smem + st * STAGE;
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
        // The loads of the step NST - 1 ahead, half of them before each of the first
        // two slices' products: a wave that issues them stalls until the memory
        // pipe takes them (16 cycles each), so all at once leave the matrix unit
        // idle, and later than this they have too little time to land.  8192^3
        // bf16: all ahead of the first slice 885 us, before slices 0 and 1 843, a
        // quarter before each 942, one between every two products 966.
        // (Two workgroups on a CU wait for each other's loads anyway: all ahead, 24.8
        // against 26.3 us for 8 x 1024 x 1024 x 1024 symmetric.)
        if constexpr (!AHEAD && kk < 2)
          if (more) issue(c, (st + NST - 1) % NST, KK, TAIL);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) acc[i][j] = El::mma(bf[fb][j], af[fb][i], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
      });
    };
    const int steps = c.nk * g.nseg;
    int it = 0;
    for (; it + 2 * NST - 1 < steps; it += NST)
      static_for<NST>([&](auto S) { step(it + decltype(S)::value, steps, S, std::true_type{}); });
    for (; it < steps; ++it) step(it, steps, it % NST, std::false_type{});
    __syncthreads();  // every wave is done with the last stage
    if (t + nbx < t_end) {
      cur = decode(t + nbx);
      start(cur);
    }
    // Epilogue, 32 rows of SC columns of a wave at a time: staged in fp32 (straight
    // from the accumulators' registers; 16-byte chunk c of row r at a place XORed with r:
    // neither the rows' writes nor the reads meet in a bank), then a lane takes 8
    // consecutive columns of a row and, for the mirrored tile, 8 rows of a column.
    constexpr int ROWB = SC * 4, CPR = SC / 8;  // staged row; its pieces of 8 columns
    auto place = [&](int r, int c) {
      return r * ROWB + ((c ^ (SC == 64 ? r & 15 : (r >> 1) & 7)) << 4);
    };
    char* wl = smem + (NST - 1) * STAGE + wave * WLDS;
    const auto tile = epi.tile(c.at.b, c.at.part, c.m0, c.n0);
    const auto twin = epi.tile(c.at.b, c.at.part, c.n0, c.m0);
    const int cols = epi.cols() - c.n0, rows = g.M - c.m0;
    const bool mirror = Epi::kMirror && g.sym && c.at.mt != c.at.nt;
    // What it adds is fetched one block of 32 rows ahead, each piece ahead of the
    // current one's store, which it would otherwise wait for.
    constexpr int NS = 32 * CPR / 64, NB = TM * (WTN / SC);
    Held held[NS];
    auto at_of = [&](int ln, int ih, int s) {
      At at{wm * WTM + ih / (WTN / SC) * 32 + s * (64 / CPR) + ln / CPR, wn * WTN + ih % (WTN / SC) * SC + ln % CPR * 8,
            false, false};
      at.ok = at.row < rows && at.col < cols;
      at.ok2 = at.row < rows && at.col + 4 < cols;
      return at;
    };
#pragma unroll
    for (int s = 0; s < NS; ++s) tile.fetch(at_of(lane, 0, s), held[s]);
    static_for<NB>([&](auto IH) {
      constexpr int i = decltype(IH)::value / (WTN / SC), jh = decltype(IH)::value % (WTN / SC);
      int ln = lane;  // a new value to the compiler, or it keeps every block's addresses at once
      asm volatile("" : "+v"(ln));
      const int lrow = ln & 31, lhalf = ln >> 5;
      static_for<SC / 32>([&](auto J) {
        constexpr int j = jh * (SC / 32) + decltype(J)::value;
        static_for<4>([&](auto Q) {
          constexpr int q = decltype(Q)::value;
          const f32x4_t v = {acc[i][j][q * 4], acc[i][j][q * 4 + 1], acc[i][j][q * 4 + 2], acc[i][j][q * 4 + 3]};
          *(f32x4_t*)(wl + place(lrow, decltype(J)::value * 8 + q * 2 + lhalf)) = v;
        });
      });
      __builtin_amdgcn_wave_barrier();
      constexpr int ih = decltype(IH)::value;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int r = s * (64 / CPR) + ln / CPR, c8 = ln % CPR;
        float v[8];
        *(f32x4_t*)v = *(const f32x4_t*)(wl + place(r, c8 * 2));
        *(f32x4_t*)(v + 4) = *(const f32x4_t*)(wl + place(r, c8 * 2 + 1));
        const Held now = held[s];
        if (ih + 1 < NB) tile.fetch(at_of(ln, ih + 1, s), held[s]);
        tile.apply(at_of(ln, ih, s), v, now);
      }
      if constexpr (Epi::kMirror) {
        if (mirror) {
#pragma unroll
          for (int s = 0; s < 4 * SC / 64; ++s) {
            const int col = s * 16 + (ln >> 2), r8 = (ln & 3) * 8;
            float v[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) v[r] = *(const float*)(wl + place(r8 + r, col >> 2) + (col & 3) * 4);
            At at{wn * WTN + jh * SC + col, wm * WTM + i * 32 + r8, false, false};
            at.ok = at.ok2 = at.row < g.M - c.n0 && at.col < epi.cols() - c.m0;
            Held h;
            twin.fetch(at, h);
            twin.apply(at, v, h);
          }
        }
      }
      __builtin_amdgcn_wave_barrier();  // the staging area is rewritten next
    });
  }
}

// One K part's sums: [part][batch][M][ld] fp32, ld a multiple of 8.
struct EpiPart {
  static constexpr bool kMirror = false;
  float* p;
  long ld, mat, all;  // row; one matrix; one part of all matrices
  struct Tile {
    TileMat<float> o;
    TRG_DEV void fetch(const At&, Held&) const {}
    TRG_DEV void apply(const At& a, const float (&v)[8], const Held&) const { o.store(a, v); }
  };
  TRG_DEV int cols() const { return (int)ld; }
  TRG_DEV Tile tile(int b, int part, int m0, int n0) const {
    return {TileMat<float>(p, part * all + b * mat + m0 * ld + n0, ld)};
  }
};

// blockIdx.y, z: 128-row tile and matrix.
template <class Epi>
__global__ __launch_bounds__(256) void join_kernel(EpiPart in, int nsplit, int M, Epi epi) {
  const int chunks = (int)(in.ld / 8), i = blockIdx.x * 256 + threadIdx.x;
  const int m0 = blockIdx.y * 128, b = blockIdx.z;
  At a{i / chunks, 0, false, false};
  a.col = (i - a.row * chunks) * 8;
  a.ok = a.row < 128 && m0 + a.row < M && a.col < epi.cols();
  a.ok2 = a.ok && a.col + 4 < epi.cols();
  const auto tile = epi.tile(b, 0, m0, 0);
  Held held;
  tile.fetch(a, held);
  const float* p = in.p + b * in.mat + (m0 + (a.ok ? a.row : 0)) * in.ld + (a.ok ? a.col : 0);
  float v[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) v[c] = p[c];
  for (int s = 1; s < nsplit; ++s) {
    p += in.all;
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] += p[c];
  }
  tile.apply(a, v, held);
}

// The same for a symmetric product, of which the parts hold what lies on and above
// the diagonal of the product's tiles: blockIdx.x counts pairs of 64-row and
// 64-column tiles on and above it, each written once more across it.
template <class Epi>
__global__ __launch_bounds__(256) void join_sym_kernel(EpiPart in, int nsplit, int M, Epi epi) {
  __shared__ float turn[64][65];
  int i = blockIdx.x, nt = 0;
  while (i > nt) i -= ++nt;
  const int m0 = i * 64, n0 = nt * 64, b = blockIdx.y;
  const auto tile = epi.tile(b, 0, m0, n0);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    At a{h * 32 + (int)threadIdx.x / 8, (int)threadIdx.x % 8 * 8, false, false};
    a.ok = a.ok2 = m0 + a.row < M && n0 + a.col < epi.cols();
    Held held;
    tile.fetch(a, held);
    const float* p = in.p + b * in.mat + (a.ok ? (m0 + a.row) * in.ld + n0 + a.col : 0);
    float v[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = p[c];
    for (int s = 1; s < nsplit; ++s) {
      p += in.all;
#pragma unroll
      for (int c = 0; c < 8; ++c) v[c] += p[c];
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) turn[a.row][a.col + c] = a.ok ? v[c] : 0.f;
    tile.apply(a, v, held);
  }
  if (i == nt) return;
  __syncthreads();
  const auto twin = epi.tile(b, 0, n0, m0);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    At a{h * 32 + (int)threadIdx.x / 8, (int)threadIdx.x % 8 * 8, false, false};
    a.ok = a.ok2 = n0 + a.row < M && m0 + a.col < epi.cols();
    Held held;
    twin.fetch(a, held);
    float v[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = turn[a.col + c][a.row];
    twin.apply(a, v, held);
  }
}

// ---- host: which tiles, how many parts ----------------------------------------
struct Plan {
  int tile;    // 256, 128 or 64
  int nsplit;  // parts of K
  double us;   // the estimate
  size_t part_bytes(int batch, int M, int N) const {
    return nsplit > 1 ? (size_t)nsplit * batch * M * ((N + 7) / 8 * 8) * 4 : 0;
  }
  // of a tile's K steps in LDS, for so many tiles in all (128-wide ones have a CU each or share it)
  int stages(long tiles) const { return tile == 256 || (tile == 128 && tiles > 256) ? 2 : 4; }
};

inline long tiles_of(int M, int N, int tile, bool sym) {
  const long tm = gg::cdiv(M, tile), tn = gg::cdiv(N, tile);
  return sym ? tm * (tm + 1) / 2 : tm * tn;
}

// Tile and parts by an estimate in us, with constants fitted to times of 64 to 16384
// rows, sums of 64 to 16384, all layouts, bf16 and fp32, each with every tile and 1 to 16
// parts, the operands in the caches where they fit.  On 400 other sizes of that range,
// drawn evenly over their logarithms, what it picks takes 2.7 % longer than the best on
// average (fp32 1.4), one in twenty 9 % or more, the worst 48 %: bf16 sums of some
// thousands over 60 to 200 tiles of 64, where four to eight parts of 128-wide ones win.
// It only ranks: batches and sums over more than one run take up to twice its us.
// es: bytes an element; ksteps: 128-byte steps of K, over all runs (run() cuts a single
// one, so of a short K in three runs the last parts may have no steps: they are zeros);
// a part has two at least.
inline Plan plan(int batch, int M, int N, long ksteps, int es, bool sym) {
  const bool f32 = es == 4;
  Plan best{128, 1, 1e300};
  for (int tile = 256; tile >= 64; tile /= 2) {
    if (tile == 256 && f32) continue;
    for (int split = 1; split <= 16 && (split == 1 || ksteps >= 2L * split); ++split) {
      const long wgs = (long)batch * split * tiles_of(M, N, tile, sym), rest = wgs % 512;
      const double steps = (double)gg::cdiv(ksteps, split);
      // rounds of workgroups that share their CU, and one that does not
      auto rounds = [&](double shared, double lone, double each) {
        double t = (double)(wgs / 512) * (steps * shared + each);
        if (rest > 0) t += steps * (rest > 256 ? shared : lone) + each;
        return t;
      };
      double t;
      if (tile == 256) t = 3.5 + (double)gg::cdiv(wgs, 256) * (steps * 1.02 + 5.0);
      else if (tile == 64) t = 2.1 + rounds(f32 ? 0.98 : 0.459, f32 ? 0.554 : 0.175, 1.35);
      else if (wgs <= 256) t = 5.0 + steps * (f32 ? 1.93 : 0.434);  // (four stages)
      else t = 3.5 + rounds(f32 ? 3.9 : 0.742, f32 ? 1.92 : 0.402, 1.6);
      // the sums' way out and in again (a symmetric product's: half as many)
      if (split > 1) t += 4.9 + (sym ? 1.1e-6 : 2.17e-6) * split * batch * (double)M * N;
      if (t < best.us) best = Plan{tile, split, t};
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
  a.tiles = (int)tiles_of(a.M, a.N, p.tile, a.sym);
  a.nsplit = p.nsplit;
  const int ksteps = gg::cdiv(a.K, KSTEP);
  a.split_steps = gg::cdiv(ksteps, p.nsplit);
  const long total = (long)a.tiles * a.nsplit * a.batch;
  const int need = (int)((total + 7) / 8 * 8);
  auto go = [&](const auto& e) {
    if (p.tile == 64) {
      dense_kernel<El, 64, 64, 2, 2, 4, AKC, BKC><<<need < 512 ? need : 512, 256, 0, s>>>(a, e);
    } else if (p.tile == 256) {
      if constexpr (El::ES == 2)
        dense_kernel<El, 256, 256, 2, 4, 2, AKC, BKC><<<need < 256 ? need : 256, 512, 0, s>>>(a, e);
    } else {
      if (p.stages(total) == 4) dense_kernel<El, 128, 128, 2, 4, 4, AKC, BKC><<<need, 512, 0, s>>>(a, e);
      else dense_kernel<El, 128, 128, 2, 2, 2, AKC, BKC><<<need < 512 ? need : 512, 256, 0, s>>>(a, e);
    }
  };
  if (p.nsplit == 1) {
    go(epi);
  } else {
    const long ld = (a.N + 7) / 8 * 8;
    const EpiPart part{parts, ld, a.M * ld, a.batch * (long)a.M * ld};
    go(part);
    if constexpr (Epi::kMirror) {
      if (a.sym) {
        const int side = gg::cdiv(a.N, 64);
        join_sym_kernel<<<dim3(side * (side + 1) / 2, a.batch), 256, 0, s>>>(part, p.nsplit, a.M, epi);
        return hipGetLastError();
      }
    }
    const dim3 grid((unsigned)gg::cdiv(128 * (ld / 8), 256), gg::cdiv(a.M, 128), a.batch);
    join_kernel<<<grid, 256, 0, s>>>(part, p.nsplit, a.M, epi);
  }
  return hipGetLastError();
}

}  // namespace dn
}  // namespace trg
