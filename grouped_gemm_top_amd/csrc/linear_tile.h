// linear_tile.h -- the matrix tile shared by the dense products (linear.hip) and the cross entropy
// (linear_ce.hip): operand layouts, the k-loop, the epilogue's staging and the choice of tile
// (internal, not part of the ABI).
#pragma once

#include "gemm_lds.h"

namespace moe {
namespace ln {

using namespace gk;
using gg::OOB;

constexpr int BK = 64;  // k per LDS stage: a K-contiguous row of a stage is one 128-byte line

// 16 rows x 64 columns of fp32 staged as rows of 256 bytes, 16-byte chunk q of row r at q ^ r
__device__ __forceinline__ void stage_write(char* st, const f32x4* blk, int L) {
  const int c = L & 15, g = L >> 4;
#pragma unroll
  for (int j = 0; j < 4; ++j) *reinterpret_cast<f32x4*>(st + c * 256 + (((4 * j + g) ^ c) << 4)) = blk[j];
}
// columns 8 (L & 7) .. + 7 of row 8 p + (L >> 3)
__device__ __forceinline__ void stage_read(const char* st, int p, int L, f32x4 (&v)[2]) {
  const int r = 8 * p + (L >> 3), q = 2 * (L & 7);
  v[0] = *reinterpret_cast<const f32x4*>(st + r * 256 + ((q ^ r) << 4));
  v[1] = *reinterpret_cast<const f32x4*>(st + r * 256 + (((q + 1) ^ r) << 4));
}
__device__ __forceinline__ u32x4 pack8(const f32x4 (&v)[2]) {
  return u32x4{pk2(v[0][0], v[0][1]), pk2(v[0][2], v[0][3]), pk2(v[1][0], v[1][1]), pk2(v[1][2], v[1][3])};
}

// eight values from element o of p on, in type T
template <typename T>
__device__ __forceinline__ void store8(void* p, size_t o, const f32x4 (&v)[2]) {
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<u32x4*>(static_cast<T*>(p) + o) = pack8(v);
  } else {
    *reinterpret_cast<f32x4*>(static_cast<T*>(p) + o) = v[0];
    *reinterpret_cast<f32x4*>(static_cast<T*>(p) + o + 4) = v[1];
  }
}
// An operand: X rows (K-contiguous) or X columns (K-strided) of a matrix whose rows are ld elements apart
// (a multiple of 8), `bytes` in all planes together; an fp32 operand's parts are `plane` bytes apart.
struct Opnd {
  const void* p;
  int X, ld;
  long long bytes;
  uint32_t plane;
};

// One operand's loads: R rows (K-contiguous) or R columns (K-strided) of a 64-wide k-step, as R / 8
// kilobytes; instruction q of wavefront w fills kilobyte w + NW q, lane L its bytes 16 L .. 16 L + 15.
//  K-contiguous: kilobyte b holds rows 8b .. 8b + 7 of 128 bytes, k-chunk c of row r at c ^ ((r >> 1) & 7)
//  K-strided: k-rows of 2R bytes, column chunk c of k-row k at c ^ mn_f(k)
template <int R, int NW, bool KC>
struct Op {
  static constexpr int NI = R / 8 / NW;
  static_assert(R % (8 * NW) == 0 && NW % 2 == 0 && (KC || R >= 128), "whole kilobytes per wavefront");
  i32x4 r;
  uint32_t v[NI];  // this lane's byte offset at k = 0 (OOB when masked)
  int kl;          // k of this lane inside a step (K-strided: instruction 0's)
  static constexpr int KQ = KC ? 0 : 512 * NW / R;  // and how much further each instruction's is

  // rows or columns x0 .. x0 + R - 1 of d.X
  __device__ __forceinline__ void setup(const Opnd& d, int x0, int w, int L) {
    const int X = d.X;
    const uint32_t ld = (uint32_t)d.ld;
    r = sgpr4(dmadesc(d.p, d.bytes));
#pragma unroll
    for (int q = 0; q < NI; ++q) {
      const int b = w + NW * q;
      if constexpr (KC) {
        const int row = x0 + 8 * b + (L >> 3);
        const int c = (L & 7) ^ ((4 * (w & 1) + (L >> 4)) & 7);
        kl = 8 * c;  // (the same for every q: NW is even)
        v[q] = row < X ? ((uint32_t)row * ld + 8u * c) * 2u : OOB;
      } else {
        constexpr int CPR = R / 8;  // chunks per k-row
        const int k = b * (64 / CPR) + L / CPR;
        const int col = x0 + 8 * ((L % CPR) ^ mn_f(k));
        if (q == 0) kl = k;
        v[q] = col < X ? ((uint32_t)k * ld + (uint32_t)col) * 2u : OOB;
      }
    }
  }
  // Load instruction q of the step at k0 of the plane at byte offset `plane` into the stage area at
  // LDS address m; k >= klim (K; 0 for a step past the last) is masked per lane (K is a multiple of 8
  // where a chunk runs along k).  The uniform advance stays below 2^31, so a masked lane's offset is
  // past the descriptor's range with and without it.
  __device__ __forceinline__ void issue(int q, uint32_t m, int ld, int k0, int klim, uint32_t plane, int w) const {
    const uint32_t adv = plane + (KC ? (uint32_t)k0 * 2u : (uint32_t)k0 * (uint32_t)ld * 2u);
    dma16(r, m + (uint32_t)(w + NW * q) * 1024u, k0 + kl + KQ * q < klim ? v[q] : OOB, (uint32_t)ufl((int)adv));
  }
};

// fragment of 16 rows (or columns) from x0 on, k-half sub of a stage (layouts: Op)
template <int R, bool KC>
struct Frag {
  int o0, ff, bb;
  __device__ __forceinline__ void init(int L) {
    if constexpr (KC) {
      o0 = (L & 15) * 128 + ((((L >> 4) ^ ((L >> 1) & 7)) & 7) << 4);
    } else {
      const int m = L & 15, g = L >> 4;
      o0 = (8 * g + (m >> 2)) * (2 * R) + 8 * (m & 1);
      ff = 2 * ((m >> 2) | ((g & 1) << 2));
      bb = (m >> 1) & 1;
    }
  }
  __device__ __forceinline__ bf16x8 get(const char* op, int x0, int sub) const {
    if constexpr (KC) {
      return *reinterpret_cast<const bf16x8*>(op + x0 * 128 + (o0 ^ (64 * sub)));
    } else {
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      const char* p = op + o0 + sub * (32 * 2 * R) + ((((x0 >> 3) ^ ff) | bb) << 4);
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * 2 * R));
      struct P { s16x4 a, b; } pr{lo, hi};
      return __builtin_bit_cast(bf16x8, pr);
    }
  }
};

// Slice s of S of a contraction of `terms` times `steps` k-steps: how many it has, and the term and the step within it
// of its first one.  (steps is 0 where a count made on the device leaves nothing to sum over.)
struct KSlice { int n, term, step; };
__host__ __device__ constexpr KSlice k_slice(int terms, int steps, int s, int S) {
  const int lo = (int)((long long)terms * steps * s / S), hi = (int)((long long)terms * steps * (s + 1) / S);
  const int term = terms > 1 && steps > 0 ? lo / steps : 0;
  return KSlice{hi - lo, term, lo - term * steps};
}

// C[m0 ..][n0 ..] of a BM x BN tile by WM x WN wavefronts, each (BM / WM) x (BN / WN) in 16 x 16 blocks.
// F32: six terms of three parts an operand; SF: the smallest terms first, which are then rounded to a small sum
// (cross entropy at H = 1880: losses off by 7e-7 in place of 2.1e-6).
template <int BM_, int BN_, int WM_, int WN_, int NST_, bool AKC, bool BKC, bool F32, bool SF = false>
struct Core {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NST = NST_;
  static constexpr int NW = WM * WN, MB = BM / WM / 16, NB = BN / WN / 16;
  static constexpr int OPA = BM * 128, STG = OPA + BN * 128;
  static constexpr int TERMS = F32 ? 6 : 1, PLANES = F32 ? 3 : 1;
  // digits of the terms' parts, A: 0 0 1 1 0 2, B: 0 1 0 1 2 0; SF, A: 1 0 2 0 1 0, B: 1 2 0 1 0 0
  static constexpr uint32_t DA = SF ? 0x010201u : 0x201100u, DB = SF ? 0x001021u : 0x021010u;
  static_assert(NB % 4 == 0, "the epilogue stages 64 columns at a time");
  static_assert(NST * STG >= NW * 4096, "the epilogue's staging");
  static_assert(MB > 1 || NB == 4, "shapes below");

  // A slice's k-steps (of BK each) into acc; the ring is free afterwards.
  // acc[i][j][v] = C[wm (BM / WM) + 16 i + (L & 15)][wn (BN / WN) + 16 j + 4 (L >> 4) + v]
  static __device__ __forceinline__ void run(char* s_ring, const Opnd& A, const Opnd& B, int m0, int n0, int K,
                                             const KSlice& sl, int w, int L, f32x4 (&acc)[MB][NB]) {
    const int nk = sl.n;
    const int wm = w % WM, wn = w / WM;
    Op<BM, NW, AKC> oa;
    Op<BN, NW, BKC> ob;
    oa.setup(A, m0, w, L);
    ob.setup(B, n0, w, L);
    Frag<BM, AKC> fra;
    Frag<BN, BKC> frb;
    fra.init(L);
    frb.init(L);
    const uint32_t ring = lds_addr(s_ring);
    constexpr int NIA = Op<BM, NW, AKC>::NI, NI = NIA + Op<BN, NW, BKC>::NI;
    // the next step to load: its number, k and term (all wavefront-uniform)
    int lc = 0, lt = sl.term, lk = sl.step * BK;
    // its load instruction q into stage st (a step past the last one is all masked)
    auto issue = [&](int q, int st) __attribute__((always_inline)) {
      const uint32_t m = ring + (uint32_t)st * STG;
      const bool live = lc < nk;
      const int k0 = live ? lk : 0, klim = live ? K : 0;
      uint32_t pa = 0u, pb = 0u;
      if constexpr (F32) {
        pa = live ? ((DA >> (4 * lt)) & 3u) * A.plane : 0u;
        pb = live ? ((DB >> (4 * lt)) & 3u) * B.plane : 0u;
      }
      if (q < NIA) oa.issue(q, m, A.ld, k0, klim, pa, w);
      else ob.issue(q - NIA, m + OPA, B.ld, k0, klim, pb, w);
    };
    auto advance = [&]() __attribute__((always_inline)) {
      ++lc;
      lk += BK;
      if (F32 && lk >= K) lk = 0, ++lt;
    };
    auto frag_a = [&](int i, int st, int sub) __attribute__((always_inline)) {
      return fra.get(s_ring + st * STG, wm * (BM / WM) + 16 * i, sub);
    };
    auto frag_b = [&](int j, int st, int sub) __attribute__((always_inline)) {
      return frb.get(s_ring + st * STG + OPA, wn * (BN / WN) + 16 * j, sub);
    };

#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // A k-step is two half-steps of k = 32.  During a half-step's MFMAs the next one's fragments are
    // read: a row block's A fragment is replaced as soon as its MFMAs are issued, B's have a second
    // set.  The step's barrier sits inside its second half-step: by then every wavefront holds all of
    // step kt in registers, so its stage takes the loads of step kt + NST, and step kt + 1 has landed
    // for the reads that follow (its loads had NST - 1 steps; those of the NST - 2 steps after it may
    // still be in flight).
    bf16x8 fa[MB], fb[2][NB];
#pragma unroll
    for (int g = 0; g < NST; ++g) {
#pragma unroll
      for (int q = 0; q < NI; ++q) issue(q, g);
      advance();
    }
    vm_wait_barrier<(NST - 1) * NI>();
#pragma unroll
    for (int j = 0; j < NB; ++j) fb[0][j] = frag_b(j, 0, 0);
#pragma unroll
    for (int i = 0; i < MB; ++i) fa[i] = frag_a(i, 0, 0);
    constexpr int BR = MB > 4 ? 2 : MB > 1 ? 1 : 0;  // row blocks of the second half-step before the barrier
    constexpr int RP = (NB + MB + MB - BR - 1) / (MB - BR);  // fragment reads per row block after it
    constexpr int LP = (NI + MB - BR - 1) / (MB - BR);       // and load instructions
    // (sched_barrier keeps the compiler from gathering the reads at the end of a half-step)
    int st3 = 0;
#pragma unroll 1
    for (int kt = 0; kt < nk; ++kt) {
      // this step's stage and the next one's
      const int st = NST == 2 ? kt & 1 : st3, sn = NST == 2 ? st ^ 1 : (st + 1 == NST ? 0 : st + 1);
#pragma unroll
      for (int i = 0; i < MB; ++i) {
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = mma(fb[0][j], fa[i], acc[i][j]);
        fa[i] = frag_a(i, st, 1);
#pragma unroll
        for (int j = i; j < NB; j += MB) fb[1][j] = frag_b(j, st, 1);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        if (i == BR)
          asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NST - 2) * NI) : "memory");
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = mma(fb[1][j], fa[i], acc[i][j]);
        if (i >= BR) {
#pragma unroll
          for (int q = (i - BR) * LP; q < (i - BR + 1) * LP && q < NI; ++q) issue(q, st);
          // B's fragments first, then A's in order, each after its row block's MFMAs (past the last
          // step they are read and never used)
#pragma unroll
          for (int q = (i - BR) * RP; q < (i - BR + 1) * RP && q < NB + MB; ++q) {
            if (q < NB) fb[0][q] = frag_b(q, sn, 0);
            else fa[q - NB] = frag_a(q - NB, sn, 0);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      st3 = sn;
      advance();
    }
    vm_drain();  // (the masked loads past the last step write zeros into the ring)
    lds_barrier();  // the ring is free: it stages the epilogue
  }
};

// Where workgroup b works: XCD x gets the tiles x per .. (x + 1) per - 1 (workgroups go to XCDs round
// robin), in groups of eight M-tiles so that what one L2 serves at a time is a compact block of C.
// Tile t of nM x nN: its first row and column of tiles.
__device__ __forceinline__ void tile_at(int t, int nM, int nN, int& mt, int& nt) {
  const int gsz = 8 * nN, gr = t / gsz, gm = min(8, nM - 8 * gr), in = t - gr * gsz;
  mt = 8 * gr + in % gm;
  nt = in / gm;
}

// eight fp32 values as their three bf16 parts, part p at dst + p plane (elements)
__device__ __forceinline__ void store_parts(bf16_t* dst, size_t plane, const float (&v)[8]) {
  float h[8], m[8], l[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    h[j] = bf16_to_f32(f32_to_bf16(v[j]));
    const float r = v[j] - h[j];  // exact
    m[j] = bf16_to_f32(f32_to_bf16(r));
    l[j] = r - m[j];
  }
  auto pk = [](const float (&p)[8]) { return make_uint4(pk2(p[0], p[1]), pk2(p[2], p[3]), pk2(p[4], p[5]), pk2(p[6], p[7])); };
  *reinterpret_cast<uint4*>(dst) = pk(h);
  *reinterpret_cast<uint4*>(dst + plane) = pk(m);
  *reinterpret_cast<uint4*>(dst + 2 * plane) = pk(l);
}
__device__ __forceinline__ void load8(const bf16_t* p, float (&v)[8]) {
  load4(p, v[0], v[1], v[2], v[3]);
  load4(p + 4, v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  load4(p, v[0], v[1], v[2], v[3]);
  load4(p + 4, v[4], v[5], v[6], v[7]);
}

// src (n values, a multiple of 8) -> its three parts, planes of n values
static __global__ __launch_bounds__(256) void k_split(const float* __restrict__ src, size_t n, bf16_t* __restrict__ dst) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n / 8; i += (size_t)gridDim.x * 256) {
    float v[8];
    load8(src + 8 * i, v);
    store_parts(dst + 8 * i, n, v);
  }
}

// ------------------------------------------------------------------ host side
enum Kind { K_FWD, K_DX, K_DW };
struct Shape { int big, S; };  // big: 2 = 256 x 256, 1 = 128 x 128, 0 = 64 x 64 (64 x 128 for dx)

// Tile and K slices of a product: the choice with the least estimated time,
//   launch + rounds x (start and epilogue) + steps x max(latency of a step alone, tiles a CU x
//   time of a step when the CU is full) (+ the partial sums' way to memory and back)
// in us.  The constants are fitted to 110 random shapes (65 <= N <= 16384, 64 <= K, O <= 8192) with
// every tile and slice count timed: the choice is on average 0.7 % slower than the best one
// measured, at worst 17 %.  The cross entropy asks outside that range, with V as N or K.  40 random shapes (1 <= N <= 8192, H
// from 128 to 4096, V from 2000 to 107000), each product's tile and slices changed alone, whole calls: bf16 0.6 % (z), 1.1 %
// (dx) and 1.0 % (dW) slower than with the best one, at worst 6 %; fp32 1.1, 2.3 and 0.8 %, at worst 14 % (dx of N = 103,
// H = 1192, V = 37048: 455 us with 16 slices, 400 with 32).
inline Shape choose(Kind kind, int M, int N, int K, int terms, int max_s = 16) {
  const int steps = terms * ((K + BK - 1) / BK);
  struct C { int bm, bn, occ; double fix, lat, thr; };
  const C cs[3] = {kind == K_FWD ? C{64, 64, 3, 3.0, 0.23, 0.26} : C{64, 128, 2, 3.0, 0.32, 0.47},
                   {128, 128, 2, 3.1, 0.75, 0.49}, {256, 256, 1, 6.4, 0.40, 1.20}};
  Shape best{1, 1};
  double tb = 1e30;
  for (int b = kind == K_DW ? 1 : 0; b < 3; ++b) {
    const long long tiles = (long long)((M + cs[b].bm - 1) / cs[b].bm) * ((N + cs[b].bn - 1) / cs[b].bn);
    for (int S = 1; S <= max_s && S <= steps; S *= 2) {
      const double elems = (double)S * M * N;
      if (S > 1 && elems > 64e6) break;  // at most 256 MB of partial sums
      const long long tpc = (tiles * S + 255) / 256, rounds = (tpc + cs[b].occ - 1) / cs[b].occ;
      const double step = cs[b].thr * tpc > cs[b].lat ? cs[b].thr * tpc : cs[b].lat;
      double t = 2.5 + rounds * cs[b].fix + (steps + S - 1) / S * step;
      if (S > 1) t += 2.2 + 2.3e-6 * elems;
      if (t < tb) tb = t, best = Shape{b, S};
    }
  }
  return best;
}

inline size_t up(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace ln
}  // namespace moe
