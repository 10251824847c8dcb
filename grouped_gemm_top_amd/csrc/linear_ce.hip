// linear_ce.hip -- softmax cross entropy with a z-loss over logits that are never kept, and its
// gradient, for gfx950 (bf16, and fp32 at fp32 accuracy).
//
//   z = x W^T,  lse_t = log sum_v e^z[t,v],  loss_t = lse_t - z[t, y_t] + c lse_t^2     x [N,H], W [V,H]
//   dz[t,v] = g_t ((1 + 2 c lse_t) e^(z[t,v] - lse_t) - [v = y_t]),   dx = dz W,   dW = dz^T x
//
// Tokens whose target lies outside [0, V) take no part.  The n others are listed first, in token order, on
// the device; every product then runs on n rows, so tokens without a target cost nothing and what their x
// holds (NaN too) reaches no result.
//
// Forward: one pass of tiles over x W^T.  A tile's logits stay in the accumulators; each row leaves its
// maximum and its sum of exponentials over the tile's columns (8 bytes for 256 logits) and, where it has
// it, its target's logit; a second launch joins the tiles' pairs in tile order.
// Backward: the vocabulary in pieces.  For each piece the tiles form z again, write dz (bf16) of that piece
// alone, and the two other products take it from there while it is in the caches: dW of the piece is
// complete, dx is summed over the pieces in fp32.  Where all three products fill the large tile, dx and dW of a
// piece run in one launch with dz of the next.  Every sum has a fixed order (bitwise reproducible).
// dz is rounded to bf16 as an operand of the matrix cores (the fp32 call: three bf16 parts, see linear.hip): dx and dW
// are off by 0.0021-0.0025 of their norms, 0.0017 of it their own rounding, and by up to 0.0034 where a handful of tokens
// count, whose few large dz do not average.  A second part of dz would double both products.
//
// Measured (bf16).  N = 4096, H = 2048, V = 32000, losses: 414-448 us on 256 x 256 tiles, 1.20-1.30
// PFLOP/s; torch's product alone, which writes z, takes 457.  N = 8192, V = 50021, a tenth of the tokens without target,
// losses and gradients: 4.9-5.2 ms, 1.16-1.24 PFLOP/s over its four products (tiles of a piece apart, a launch
// each, where it took 4.9-5.0: 5.08).
// What bounds these is the chip's power: on zeros the same forward is 15-20 % faster, as the library's products
// are.  N = 300, H = 1024, V = 50021, 180 counted: 170 us in eight launches; z 43 and 38, dx 39 + 5, dW 39, each at
// twice the time of W's 102 MB: a tile waits for loads that only two stages are ahead.  N = 1, V = 130001: 118 us, 532 MB of
// W at 4.5 TB/s.
#include <type_traits>

#include "linear_tile.h"

namespace moe {
namespace ce {

using namespace ln;

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;

struct Args {
  const void* x;    // the counted rows, one behind the other [n, H] (fp32: three planes of N rows)
  const void* w;    // the piece of W: [V, H]
  void* dxo;        // dx [N, H]
  void* dwo;        // the piece of dW [V, H]
  const int* cnt;   // n
  const int* list;  // the counted tokens
  int N, H, V, ldz;
  int v0, nt0;      // the piece's first column and first tile (forward)
  const int* tgt;   // [n] the targets
  // forward
  float2* part;     // [tiles of all pieces][N]
  float* zt;        // [N] the target's logit
  // backward
  const float4* info;  // lse, g (1 + 2 c lse), g
  bf16_t* dz;          // [N, ldz], in fp32 three planes of it
  float* acc;          // [N, H] dx so far
  int first, last;     // piece
  float* slices;       // S > 1: [S][N or V][H]
  int S;
};

__device__ __forceinline__ bool in_vocab(int t, int V) { return (unsigned)t < (unsigned)V; }

// ---- the counted tokens ----
constexpr int GR = 16;  // tokens of a group: one a wavefront

// A workgroup takes `groups` groups of tokens.  It counts the counted ones before them over all targets (a list of
// counts would be another launch; at N = 8192 a workgroup reads 32 KB, and beyond N = 32768 the workgroups are 2048, so
// that all of them together read 4 KB a token at most), then, a group at a time, lists its own with their targets
// (BWD: with what dz needs) and copies their rows of x one behind the other (fp32: as three planes of N rows).  The
// others' loss and lse (BWD: rows of dx, where wanted) are 0.  H = 2048: N = 4096 10.9 us (12.8 with groups of 32,
// 11.0 of 8), N = 8192 14.6 (14.9, 17.4).
template <typename T, bool BWD>
__global__ __launch_bounds__(1024) void k_ce_select(const int* __restrict__ target, const T* __restrict__ x, int N, int H,
                                                   int V, int groups, int* __restrict__ list, int* __restrict__ cnt,
                                                   int* __restrict__ tgt, bf16_t* __restrict__ xc, float* __restrict__ loss,
                                                   float* __restrict__ lse_out, const float* __restrict__ lse,
                                                   const float* __restrict__ dloss, float zc, float4* __restrict__ info,
                                                   T* __restrict__ dx) {
  __shared__ int s_n[16], s_pos[GR];
  const int L = threadIdx.x & 63, w = threadIdx.x >> 6, t_lo = blockIdx.x * groups * GR;
  int c = 0;
  for (int t = threadIdx.x; t < t_lo; t += 4 * 1024) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c += t + 1024 * j < t_lo && in_vocab(target[min(t + 1024 * j, t_lo - 1)], V);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) c += __shfl_xor(c, o);
  if (L == 0) s_n[w] = c;
  __syncthreads();
  int base = 0;
#pragma unroll
  for (int q = 0; q < 16; ++q) base += s_n[q];
  for (int t0 = t_lo; t0 < N && t0 < t_lo + GR * groups; t0 += GR) {
    if (w == 0) {
      const int t = t0 + L;
      const bool mine = L < GR && t < N;
      const int y = mine ? target[t] : -1;
      const unsigned long long live = __ballot(in_vocab(y, V));
      const int p = base + __popcll(live & ((1ull << L) - 1));
      if (L < GR) s_pos[L] = in_vocab(y, V) ? p : -1;
      if (in_vocab(y, V)) {
        list[p] = t;
        tgt[p] = y;
        if constexpr (BWD) {
          const float l = lse[t], g = dloss ? dloss[t] : 1.0f;
          info[p] = make_float4(l, g * (1.0f + 2.0f * zc * l), g, 0.f);
        }
      } else if (!BWD && mine) {
        loss[t] = 0.f;
        lse_out[t] = 0.f;
      }
      base += __popcll(live);
      if (L == 0 && t0 + GR >= N) *cnt = base;
    }
    __syncthreads();
    for (int r = w; r < GR && t0 + r < N; r += 16) {
      const int p = s_pos[r];
      const T* src = x + (size_t)(t0 + r) * H;
      if (p >= 0) {
        bf16_t* dst = xc + (size_t)p * H;
        for (int h0 = 8 * L; h0 < H; h0 += 4 * 512) {  // four loads in flight
          if constexpr (sizeof(T) == 2) {
            uint4 v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = *reinterpret_cast<const uint4*>(src + min(h0 + 512 * q, H - 8));
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (h0 + 512 * q < H) *reinterpret_cast<uint4*>(dst + h0 + 512 * q) = v[q];
          } else {
            float v[4][8];
#pragma unroll
            for (int q = 0; q < 4; ++q) load8(src + min(h0 + 512 * q, H - 8), v[q]);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (h0 + 512 * q < H) store_parts(dst + h0 + 512 * q, (size_t)N * H, v[q]);
          }
        }
      } else if (BWD && dx) {
        for (int h = 8 * L; h < H; h += 512)
#pragma unroll
          for (int q = 0; q < (int)sizeof(T) / 2; ++q)
            *reinterpret_cast<uint4*>(dx + (size_t)(t0 + r) * H + h + q * 16 / sizeof(T)) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    __syncthreads();  // s_pos has been read
  }
}

// The tile of workgroup b among nM x nN (x S slices, slice major); false: none
__device__ __forceinline__ bool my_tile(int b, int nM, int nN, int S, int& mt, int& nt, int& s) {
  const int nT = nM * nN, per = (nT * S + 7) / 8;
  const int t = (b & 7) * per + (b >> 3);
  if ((b >> 3) >= per || t >= nT * S) return false;
  s = t / nT;
  tile_at(t - s * nT, nM, nN, mt, nt);
  return true;
}

enum { LSE = 0, DZ = 1 };

// Core's k-loop over a run of tiles without a pause: the load instructions of a tile's last steps fetch the first
// steps of the next one, which then arrive during the epilogue (whose staging lies outside the ring).  All
// tiles have the same K.
template <int BM, int BN, int WM, int WN, int NST, bool AKC, bool BKC, bool F32>
struct Pipe {
  using C = Core<BM, BN, WM, WN, NST, AKC, BKC, F32, true>;
  typedef Op<BM, C::NW, AKC> OpA;
  typedef Op<BN, C::NW, BKC> OpB;
  static constexpr int MB = C::MB, NB = C::NB, NIA = OpA::NI, NI = NIA + OpB::NI;
  OpA oa;
  OpB ob;
  Frag<BM, AKC> fra;
  Frag<BN, BKC> frb;
  char* s_ring;
  uint32_t ring;
  int w, L, nk, K, gs;           // gs: ring stage of the tile's first step
  int lit, lc, lt, lk;           // the next step to load: its tile (-1: none), number, term and k

  // at(it, m0, n0): origin of this workgroup's tile `it`, false past the last one
  template <typename AT>
  __device__ __forceinline__ void point(const Opnd& A, const Opnd& B, AT at) {
    int m0, n0;
    lc = lt = lk = 0;
    if (at(lit, m0, n0)) {
      oa.setup(A, m0, w, L);
      ob.setup(B, n0, w, L);
    } else {
      lit = -1;
    }
  }
  __device__ __forceinline__ void issue(const Opnd& A, const Opnd& B, int q, int st) {
    const uint32_t m = ring + (uint32_t)st * C::STG;
    const bool live = lit >= 0;
    const int k0 = live ? lk : 0, klim = live ? K : 0;
    uint32_t pa = 0u, pb = 0u;
    if constexpr (F32) {
      pa = live ? ((C::DA >> (4 * lt)) & 3u) * A.plane : 0u;
      pb = live ? ((C::DB >> (4 * lt)) & 3u) * B.plane : 0u;
    }
    if (q < NIA) oa.issue(q, m, A.ld, k0, klim, pa, w);
    else ob.issue(q - NIA, m + C::OPA, B.ld, k0, klim, pb, w);
  }
  template <typename AT>
  __device__ __forceinline__ void advance(const Opnd& A, const Opnd& B, AT at) {
    if (lit < 0) return;
    lk += BK;
    if (F32 && lk >= K) lk = 0, ++lt;
    if (++lc == nk) {
      ++lit;
      point(A, B, at);
    }
  }
  template <typename AT>
  __device__ __forceinline__ void start(char* r, const Opnd& A, const Opnd& B, int K_, int w_, int L_, AT at) {
    s_ring = r;
    ring = lds_addr(r);
    w = w_;
    L = L_;
    K = K_;
    nk = C::TERMS * ((K_ + BK - 1) / BK);
    gs = 0;
    lit = 0;
    fra.init(L);
    frb.init(L);
    point(A, B, at);
#pragma unroll
    for (int g = 0; g < NST; ++g) {
#pragma unroll
      for (int q = 0; q < NI; ++q) issue(A, B, q, g);
      advance(A, B, at);
    }
  }
  // one tile into acc; a barrier must follow before anything but the loads in flight writes to the ring
  template <typename AT>
  __device__ __forceinline__ void tile(const Opnd& A, const Opnd& B, f32x4 (&acc)[MB][NB], AT at) {
    const int wm = w % WM, wn = w / WM;
    auto frag_a = [&](int i, int st, int sub) __attribute__((always_inline)) {
      return fra.get(s_ring + st * C::STG, wm * (BM / WM) + 16 * i, sub);
    };
    auto frag_b = [&](int j, int st, int sub) __attribute__((always_inline)) {
      return frb.get(s_ring + st * C::STG + C::OPA, wn * (BN / WN) + 16 * j, sub);
    };
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // (the loop is Core's: see there; what the epilogue before has queued is younger than this tile's first steps)
    bf16x8 fa[MB], fb[2][NB];
    vm_wait_barrier<(NST - 1) * NI>();
    int st = gs;
#pragma unroll
    for (int j = 0; j < NB; ++j) fb[0][j] = frag_b(j, st, 0);
#pragma unroll
    for (int i = 0; i < MB; ++i) fa[i] = frag_a(i, st, 0);
    constexpr int BR = MB > 4 ? 2 : MB > 1 ? 1 : 0;
    constexpr int RP = (NB + MB + MB - BR - 1) / (MB - BR);
    constexpr int LP = (NI + MB - BR - 1) / (MB - BR);
#pragma unroll 1
    for (int kt = 0; kt < nk; ++kt) {
      const int sn = st + 1 == NST ? 0 : st + 1;
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
          for (int q = (i - BR) * LP; q < (i - BR + 1) * LP && q < NI; ++q) issue(A, B, q, st);
#pragma unroll
          for (int q = (i - BR) * RP; q < (i - BR + 1) * RP && q < NB + MB; ++q) {
            if (q < NB) fb[0][q] = frag_b(q, sn, 0);
            else fa[q - NB] = frag_a(q - NB, sn, 0);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      st = sn;
      advance(A, B, at);
    }
    gs = st;
  }
};

// x W^T by tiles, and from the accumulators either the rows' (maximum, sum of exponentials) or dz.  XCD x takes a
// contiguous run of the tile list (tile_at's order), workgroup b of G every (G / 8)th tile of it.
// s_stage: 2 KB a wavefront.
template <int BM, int BN, int WM, int WN, int NST, int EPI, bool F32>
__device__ __forceinline__ void z_tiles(const Args& a, int b, int G, char* s_ring, char* s_stage) {
  using P = Pipe<BM, BN, WM, WN, NST, true, true, F32>;
  using C = typename P::C;
  constexpr int MB = C::MB, NB = C::NB;
  static_assert(BM * WN * 8 <= C::NW * 2048, "the staging holds the tile's pairs");
  const int L = threadIdx.x & 63, w = ufl(threadIdx.x >> 6);
  const int wm = w % WM, wn = w / WM;
  const int n = ufl(*a.cnt);
  const int nM = (n + BM - 1) / BM, nN = (a.V + BN - 1) / BN, nT = nM * nN, per = (nT + 7) / 8;
  const int xcd = b & 7, slot = b >> 3, step = G >> 3;
  auto at = [&](int it, int& m0, int& n0) __attribute__((always_inline)) {
    const int q = slot + it * step, t = xcd * per + q;
    if (q >= per || t >= nT) return false;
    int mt, nt;
    tile_at(t, nM, nN, mt, nt);
    m0 = mt * BM;
    n0 = nt * BN;
    return true;
  };
  int m0, n0;
  if (!at(0, m0, n0)) return;
  const Opnd A{a.x, n, a.H, (long long)C::PLANES * a.N * a.H * 2, (uint32_t)a.N * (uint32_t)a.H * 2u};
  const Opnd B{a.w, a.V, a.H, (long long)C::PLANES * a.V * a.H * 2, (uint32_t)a.V * (uint32_t)a.H * 2u};
  P pipe;
  pipe.start(s_ring, A, B, a.H, w, L, at);
  const int c = L & 15, g = L >> 4;
#pragma unroll 1
  for (int it = 0; at(it, m0, n0); ++it) {
    f32x4 acc[MB][NB];
    // Lane (g, c) gets columns 16 j + 4 g + v of row 16 i + c; of those rows: the target's place among its columns
    const int c0 = n0 + wn * (BN / WN), r0 = m0 + wm * (BM / WM) + c;
    int y[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) y[i] = a.tgt[min(r0 + 16 * i, n - 1)];
    pipe.tile(A, B, acc, at);
#pragma unroll
    for (int i = 0; i < MB; ++i) y[i] -= a.v0 + c0 + 4 * g;
    const bool ragged = n0 + BN > a.V;
    if constexpr (EPI == LSE) {
      // (columns past the piece count as -inf)
      if (ragged) {
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (c0 + 16 * j + 4 * g + v >= a.V) {
#pragma unroll
              for (int i = 0; i < MB; ++i) acc[i][j][v] = -INFINITY;
            }
      }
      float m[MB], sum[MB];
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        m[i] = -INFINITY;
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v) m[i] = fmaxf(m[i], acc[i][j][v]);
      }
#pragma unroll
      for (int i = 0; i < MB; ++i) m[i] = fmaxf(m[i], __shfl_xor(m[i], 16));
#pragma unroll
      for (int i = 0; i < MB; ++i) m[i] = fmaxf(m[i], __shfl_xor(m[i], 32));
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const float ms = m[i] == -INFINITY ? 0.f : m[i];
        sum[i] = 0.f;
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v) sum[i] += __builtin_amdgcn_exp2f((acc[i][j][v] - ms) * kLog2e);
      }
#pragma unroll
      for (int i = 0; i < MB; ++i) sum[i] += __shfl_xor(sum[i], 16);
#pragma unroll
      for (int i = 0; i < MB; ++i) sum[i] += __shfl_xor(sum[i], 32);
      float2* s_part = reinterpret_cast<float2*>(s_stage);  // [BM][WN]
      if (g == 0) {
#pragma unroll
        for (int i = 0; i < MB; ++i) s_part[(wm * (BM / WM) + 16 * i + c) * WN + wn] = make_float2(m[i], sum[i]);
      }
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        if (y[i] >= 0 && y[i] < 16 * NB && (y[i] & 15) < 4 && r0 + 16 * i < n) {
#pragma unroll
          for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v)
              if (y[i] == 16 * j + v) a.zt[r0 + 16 * i] = acc[i][j][v];
        }
      }
      lds_barrier();
      // (the next tile's k-loop has a barrier behind these reads)
      for (int r = threadIdx.x; r < BM; r += 64 * WM * WN) {
        if (m0 + r >= n) break;
        float2 p[WN];
        float mm = -INFINITY;
#pragma unroll
        for (int q = 0; q < WN; ++q) {
          p[q] = s_part[r * WN + q];
          mm = fmaxf(mm, p[q].x);
        }
        const float ms = mm == -INFINITY ? 0.f : mm;
        float tot = 0.f;
#pragma unroll
        for (int q = 0; q < WN; ++q) tot += p[q].y * __builtin_amdgcn_exp2f((p[q].x - ms) * kLog2e);
        a.part[(size_t)(a.nt0 + n0 / BN) * a.N + m0 + r] = make_float2(mm, tot);
      }
    } else {
      // dz in the accumulators' layout, then as bf16 (fp32: part by part) through LDS, rows of 128 bytes with 16-byte
      // chunk q of row r at q ^ (r & 7), so that eight lanes store a row's 64 columns.  Columns from V to ldz get
      // zeros.  A row's lse and gradient are loaded while the row before is worked on.
      char* sg = s_stage + w * 2048;
      float4 f = a.info[min(r0, n - 1)];
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const float4 cur = f;
        if (i + 1 < MB) f = a.info[min(r0 + 16 * (i + 1), n - 1)];
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            acc[i][j][v] = cur.y * __builtin_amdgcn_exp2f((acc[i][j][v] - cur.x) * kLog2e);
        if (y[i] >= 0 && y[i] < 16 * NB && (y[i] & 15) < 4) {
#pragma unroll
          for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[i][j][v] -= y[i] == 16 * j + v ? cur.z : 0.f;
        }
        if (ragged) {
#pragma unroll
          for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v)
              if (c0 + 16 * j + 4 * g + v >= a.V) acc[i][j][v] = 0.f;
        }
#pragma unroll
        for (int q = 0; q < C::PLANES; ++q) {
#pragma unroll
          for (int h = 0; h < NB / 4; ++h) {
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
              f32x4& d = acc[i][4 * h + jj];
              const u32x2 b = {pk2(d[0], d[1]), pk2(d[2], d[3])};
              *reinterpret_cast<u32x2*>(sg + c * 128 + (((2 * jj + (g >> 1)) ^ (c & 7)) << 4) + 8 * (g & 1)) = b;
              if (q + 1 < C::PLANES)  // what the part leaves, exactly
                d -= f32x4{__uint_as_float(b[0] << 16), __uint_as_float(b[0] & 0xFFFF0000u), __uint_as_float(b[1] << 16),
                           __uint_as_float(b[1] & 0xFFFF0000u)};
            }
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const int r = 8 * p + (L >> 3), m = m0 + wm * (BM / WM) + 16 * i + r, col = c0 + 64 * h + 8 * (L & 7);
              const u32x4 v = *reinterpret_cast<const u32x4*>(sg + r * 128 + (((L & 7) ^ (r & 7)) << 4));
              if (m < n && col < a.ldz)
                *reinterpret_cast<u32x4*>(a.dz + (size_t)q * a.N * a.ldz + (size_t)m * a.ldz + col) = v;
            }
          }
        }
      }
    }
  }
  vm_drain();  // (the masked loads past the last tile write zeros into the ring)
}
template <int BM, int BN, int WM, int WN, int NST, int EPI, bool F32>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_ce_z(Args a) {
  using C = Core<BM, BN, WM, WN, NST, true, true, F32, true>;
  __shared__ __attribute__((aligned(1024))) char s_ring[NST * C::STG];
  __shared__ __attribute__((aligned(256))) char s_stage[C::NW * 2048];
  z_tiles<BM, BN, WM, WN, NST, EPI, F32>(a, blockIdx.x, gridDim.x, s_ring, s_stage);
}

// The tiles' pairs joined, in one order: 16 rows a workgroup, 64 groups of tiles each.
__global__ __launch_bounds__(1024) void k_ce_loss(const float2* __restrict__ part, const float* __restrict__ zt,
                                                  const int* __restrict__ list, const int* __restrict__ cnt, int N,
                                                  int tiles, float zc, float* __restrict__ loss,
                                                  float* __restrict__ lse) {
  __shared__ float2 s[64][16];
  const int c = threadIdx.x & 15, g = threadIdx.x >> 4, r = blockIdx.x * 16 + c, n = *cnt;
  if ((int)blockIdx.x * 16 >= n) return;
  float m = -INFINITY, sum = 0.f;
  if (r < n) {
    for (int t = g; t < tiles; t += 256) {
      float2 p[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        p[q] = t + 64 * q < tiles ? part[(size_t)(t + 64 * q) * N + r] : make_float2(-INFINITY, 0.f);
      const float mn = fmaxf(fmaxf(fmaxf(m, p[0].x), fmaxf(p[1].x, p[2].x)), p[3].x);
      const float ms = mn == -INFINITY ? 0.f : mn;
      sum *= __builtin_amdgcn_exp2f((m - ms) * kLog2e);
#pragma unroll
      for (int q = 0; q < 4; ++q) sum += p[q].y * __builtin_amdgcn_exp2f((p[q].x - ms) * kLog2e);
      m = mn;
    }
  }
  s[g][c] = make_float2(m, sum);
  __syncthreads();
  if (g > 0 || r >= n) return;
  float mm = m;
#pragma unroll 8
  for (int q = 1; q < 64; ++q) mm = fmaxf(mm, s[q][c].x);
  const float ms = mm == -INFINITY ? 0.f : mm;
  float tot = 0.f;
#pragma unroll 8
  for (int q = 0; q < 64; ++q) {
    const float2 p = s[q][c];
    tot += p.y * __builtin_amdgcn_exp2f((p.x - ms) * kLog2e);
  }
  const float l = ms + __logf(tot);
  const int t = list[r];
  lse[t] = l;
  loss[t] = l - zt[r] + zc * l * l;
}

// dx = dz W of a piece: straight, or (S > 1) fp32 slices of its K range
template <int BM, int BN, int WM, int WN, int NST, bool PART, bool F32>
__device__ __forceinline__ void dx_tile(const Args& a, int b, char* s_ring) {
  using C = Core<BM, BN, WM, WN, NST, true, false, F32, true>;
  typedef typename std::conditional<F32, float, bf16_t>::type T;
  constexpr int MB = C::MB, NB = C::NB;
  const int L = threadIdx.x & 63, w = ufl(threadIdx.x >> 6);
  const int wm = w % WM, wn = w / WM;
  const int n = ufl(*a.cnt);
  int mt, nt, s;
  if (!my_tile(b, (n + BM - 1) / BM, (a.H + BN - 1) / BN, PART ? a.S : 1, mt, nt, s)) return;
  const int m0 = mt * BM, n0 = nt * BN;
  const KSlice sl = k_slice(C::TERMS, (a.V + BK - 1) / BK, s, PART ? a.S : 1);
  const Opnd A{a.dz, n, a.ldz, (long long)C::PLANES * a.N * a.ldz * 2, (uint32_t)a.N * (uint32_t)a.ldz * 2u};
  const Opnd B{a.w, a.H, a.H, (long long)C::PLANES * a.V * a.H * 2, (uint32_t)a.V * (uint32_t)a.H * 2u};
  f32x4 acc[MB][NB];
  C::run(s_ring, A, B, m0, n0, a.V, sl, w, L, acc);
  char* sg = s_ring + w * 4096;
#pragma unroll
  for (int h = 0; h < NB / 4; ++h) {
    const int col = n0 + wn * (BN / WN) + 64 * h + 8 * (L & 7), mr = m0 + wm * (BM / WM) + (L >> 3);
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      stage_write(sg, &acc[i][4 * h], L);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        f32x4 v[2];
        stage_read(sg, p, L, v);
        const int m = mr + 16 * i + 8 * p;
        if (m >= n || col >= a.H) continue;
        const size_t o = (size_t)m * a.H + col;
        if constexpr (PART) {
          store8<float>(a.slices, (size_t)s * a.N * a.H + o, v);
        } else {
          if (!a.first) {
            v[0] += *reinterpret_cast<const f32x4*>(a.acc + o);
            v[1] += *reinterpret_cast<const f32x4*>(a.acc + o + 4);
          }
          if (a.last) store8<T>(a.dxo, (size_t)a.list[m] * a.H + col, v);
          else store8<float>(a.acc, o, v);
        }
      }
    }
  }
}

template <int BM, int BN, int WM, int WN, int NST, bool PART, bool F32>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_ce_dx(Args a) {
  __shared__ __attribute__((aligned(1024))) char s_ring[NST * Core<BM, BN, WM, WN, NST, true, false, F32, true>::STG];
  dx_tile<BM, BN, WM, WN, NST, PART, F32>(a, blockIdx.x, s_ring);
}

// dx's slices added in slice order
template <typename T>
__global__ __launch_bounds__(256) void k_ce_dx_sum(Args a) {
  const int cpr = a.H / 8;
  const size_t nv = (size_t)*a.cnt * cpr, slice = (size_t)a.N * a.H;
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < nv; i += (size_t)gridDim.x * 256) {
    const int m = (int)(i / cpr), col = (int)(i % cpr) * 8;
    f32x4 v[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
    if (!a.first) {
      v[0] = *reinterpret_cast<const f32x4*>(a.acc + 8 * i);
      v[1] = *reinterpret_cast<const f32x4*>(a.acc + 8 * i + 4);
    }
#pragma unroll 16
    for (int s = 0; s < a.S; ++s) {
      const float* p = a.slices + (size_t)s * slice + 8 * i;
      v[0] += *reinterpret_cast<const f32x4*>(p);
      v[1] += *reinterpret_cast<const f32x4*>(p + 4);
    }
    if (a.last) store8<T>(a.dxo, (size_t)a.list[m] * a.H + col, v);
    else store8<float>(a.acc, 8 * i, v);
  }
}

// dW = dz^T x of a piece, a workgroup its share of the tiles (PART: of fp32 slices of the tokens, one tile each)
template <int BM, int BN, int WM, int WN, int NST, bool PART, bool F32>
__device__ __forceinline__ void dw_tiles(const Args& a, int b, int G, char* s_ring, char* s_stage) {
  using P = Pipe<BM, BN, WM, WN, NST, false, false, F32>;
  using C = typename P::C;
  typedef typename std::conditional<F32, float, bf16_t>::type T;
  constexpr int MB = C::MB, NB = C::NB;
  const int L = threadIdx.x & 63, w = ufl(threadIdx.x >> 6);
  const int wm = w % WM, wn = w / WM;
  const int n = ufl(*a.cnt), S = PART ? a.S : 1;
  const int nM = (a.V + BM - 1) / BM, nN = (a.H + BN - 1) / BN, nT = nM * nN, per = (nT * S + 7) / 8;
  const int xcd = b & 7, slot = b >> 3, step = G >> 3;
  int s = 0;
  auto at = [&](int it, int& m0, int& n0) __attribute__((always_inline)) {
    const int q = slot + it * step, t = xcd * per + q;
    if (q >= per || t >= nT * S || (PART && it > 0)) return false;
    if (PART) s = t / nT;
    int mt, nt;
    tile_at(t - (PART ? s * nT : 0), nM, nN, mt, nt);
    m0 = mt * BM;
    n0 = nt * BN;
    return true;
  };
  int m0, n0;
  if (!at(0, m0, n0)) return;
  const Opnd A{a.dz, a.V, a.ldz, (long long)C::PLANES * a.N * a.ldz * 2, (uint32_t)a.N * (uint32_t)a.ldz * 2u};
  const Opnd B{a.x, a.H, a.H, (long long)C::PLANES * a.N * a.H * 2, (uint32_t)a.N * (uint32_t)a.H * 2u};
  f32x4 acc[MB][NB];
  P pipe;
  if constexpr (PART) {
    C::run(s_ring, A, B, m0, n0, n, k_slice(C::TERMS, (n + BK - 1) / BK, s, S), w, L, acc);
  } else {
    pipe.start(s_ring, A, B, n, w, L, at);
  }
#pragma unroll 1
  for (int it = 0; at(it, m0, n0); ++it) {
    if constexpr (!PART) pipe.tile(A, B, acc, at);
    char* sg = s_stage + w * 4096;
#pragma unroll
    for (int h = 0; h < NB / 4; ++h) {
      const int col = n0 + wn * (BN / WN) + 64 * h + 8 * (L & 7), mr = m0 + wm * (BM / WM) + (L >> 3);
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        stage_write(sg, &acc[i][4 * h], L);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          f32x4 v[2];
          stage_read(sg, p, L, v);
          const int m = mr + 16 * i + 8 * p;
          if (m >= a.V || col >= a.H) continue;
          const size_t o = (size_t)m * a.H + col;
          if constexpr (PART) store8<float>(a.slices, (size_t)s * a.V * a.H + o, v);
          else store8<T>(a.dwo, o, v);
        }
      }
    }
  }
  if (!PART) vm_drain();
}
template <int BM, int BN, int WM, int WN, int NST, bool PART, bool F32>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_ce_dw(Args a) {
  using C = Core<BM, BN, WM, WN, NST, false, false, F32, true>;
  __shared__ __attribute__((aligned(1024))) char s_ring[NST * C::STG];
  __shared__ __attribute__((aligned(256))) char s_stage[C::NW * 4096];
  dw_tiles<BM, BN, WM, WN, NST, PART, F32>(a, blockIdx.x, gridDim.x, s_ring, s_stage);
}

// dx and dW of piece p and, in the same launch, dz of the piece behind it (z, dz in the other buffer): the three
// products' tiles fill the chip without a badly filled last round each.  The long ones come first, the
// many short ones fill what they leave.
template <bool F32>
__global__ __launch_bounds__(512, 2) void k_ce_piece(Args p, Args z, int b_dx, int b_dw) {
  __shared__ __attribute__((aligned(1024))) char s_ring[2 * Core<256, 256, 2, 4, 2, true, true, F32, true>::STG];
  __shared__ __attribute__((aligned(256))) char s_stage[8 * 4096];
  const int b = blockIdx.x;
  if (b < b_dx) dx_tile<256, 256, 2, 4, 2, false, F32>(p, b, s_ring);
  else if (b < b_dx + b_dw) dw_tiles<256, 256, 2, 4, 2, false, F32>(p, b - b_dx, b_dw, s_ring, s_stage);
  else z_tiles<256, 256, 2, 4, 2, DZ, F32>(z, b - b_dx - b_dw, gridDim.x - b_dx - b_dw, s_ring, s_stage);
}

template <typename T>
__global__ __launch_bounds__(256) void k_ce_dw_sum(Args a) {
  const size_t slice = (size_t)a.V * a.H, nv = slice / 8;
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < nv; i += (size_t)gridDim.x * 256) {
    f32x4 v[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll 16
    for (int s = 0; s < a.S; ++s) {
      const float* p = a.slices + (size_t)s * slice + 8 * i;
      v[0] += *reinterpret_cast<const f32x4*>(p);
      v[1] += *reinterpret_cast<const f32x4*>(p + 4);
    }
    store8<T>(a.dwo, 8 * i, v);
  }
}

__global__ __launch_bounds__(256) void k_ce_zero(uint4* __restrict__ p, size_t n) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256)
    p[i] = make_uint4(0u, 0u, 0u, 0u);
}

// ------------------------------------------------------------------ host side
constexpr long long kDesc = 0x7FFFFFFF;

int tile_n(int big) { return big == 2 ? 256 : big == 1 ? 128 : 64; }

// groups that a workgroup of k_ce_select takes
int select_groups(int N) { return (N + 2048 * GR - 1) / (2048 * GR); }
unsigned select_grid(int N) { return (unsigned)((N + GR * select_groups(N) - 1) / (GR * select_groups(N))); }

// The tile of x W^T: choose's, without K slices (the epilogue needs whole sums); for up to 64 tokens 3 = 64 x 128
// with three stages in place of 128 x 128 with two, as W's way from memory is the time then and twice as much of it is
// on its way (N = 1, H = 2048, losses alone: V = 130001 118 us, 134 with two; V = 50021 55, 59; V <= 32000 equal).
constexpr int kZm[4] = {64, 128, 256, 64}, kZn[4] = {64, 128, 256, 128};
int z_tile(int N, int H, int V, int terms) {
  const int b = choose(K_FWD, N, V, H, terms, 1).big;
  if (b == 1 && N <= 64) return 3;
  return b < 2 && (long long)((N + 63) / 64) * ((V + 63) / 64) > 1 << 20 ? 2 : b;
}

// Columns of a forward piece: all of them, unless a descriptor (2 GiB) or, in fp32, the workspace's copy of
// the piece in three parts (512 MB) does not hold them.
int fwd_piece(bool f, int H, int V) {
  const long long most = f ? (512LL << 20) / (6LL * H) : kDesc / (2LL * H);
  if (most >= V) return V;
  return most < 256 ? 256 : (int)(most / 256 * 256);
}

// Columns of a backward piece: at most 64 M elements of dz (fp32: 32 M), pieces of one size
int bwd_piece(bool f, int N, int H, int V) {
  long long most = (f ? 32LL : 64LL) * (1 << 20) / (N > 0 ? N : 1);
  const long long desc = f ? (1LL << 30) / (6LL * H) : kDesc / (2LL * H);
  if (desc < most) most = desc;
  if (most >= V) return V;
  most = most < 256 ? 256 : most / 256 * 256;
  const long long np = (V + most - 1) / most;
  return (int)((V + np * 256 - 1) / (np * 256) * 256);
}

struct FwdWs {
  size_t list, tgt, cnt, zt, part, xp, wp;
  int vc, tile, tiles;
  FwdWs(bool f, int N, int H, int V) {
    vc = fwd_piece(f, H, V);
    tile = z_tile(N, H, vc, f ? 6 : 1);
    const int bn = kZn[tile];
    tiles = (V + bn - 1) / bn;  // (a piece is a multiple of 256 unless it is the last)
    list = tgt = zt = up((size_t)N * 4);
    cnt = 256;
    part = up((size_t)tiles * N * 8);
    xp = up((size_t)N * H * (f ? 6 : 2));
    wp = f ? up((size_t)vc * H * 6) : 0;
  }
  size_t total() const { return 256 + list + tgt + cnt + zt + part + xp + wp; }
};

// Tile and K slices of dx and dW: the sum runs over a whole vocabulary or a whole batch while the output may be a
// tile or two, so more than 16 slices as long as they go once into the chip (loss and gradients: N = 1, H = 96, V = 60011
// fp32 121 us, 220 with 16; N = 100, H = 512, V = 100000 140, 151; N = 100000, H = 64, V = 100 178, 213; beyond that
// the partial sums cost more: N = 300, H = 1024, V = 50021 188 with 32, 179).
Shape sliced(Kind kind, int M, int N, int K, int terms) {
  const long long tiles = (long long)((M + 127) / 128) * ((N + 127) / 128);
  return choose(kind, M, N, K, terms, tiles <= 4 ? 64 : tiles <= 8 ? 32 : 16);
}

// whether all products of a piece run on the large tile without K slices
bool mixes(int N, int H, int v, int terms) {
  const Shape dx = sliced(K_DX, N, H, v, terms), dw = sliced(K_DW, v, H, N, terms);
  return dx.big == 2 && dx.S == 1 && dw.big == 2 && dw.S == 1 && z_tile(N, H, v, terms) == 2;
}

struct BwdWs {
  size_t list, tgt, cnt, info, xc, dz, acc, slices, wp;
  int vc;
  bool two;  // two pieces in work at once: dz, and in fp32 W's parts, have two buffers
  BwdWs(bool f, int N, int H, int V) {
    const int terms = f ? 6 : 1;
    vc = bwd_piece(f, N, H, V);
    list = tgt = up((size_t)N * 4);
    cnt = 256;
    info = up((size_t)N * 16);
    xc = up((size_t)N * H * (f ? 6 : 2));
    two = vc < V && mixes(N, H, vc, terms);
    dz = up((size_t)N * ((vc + 7) / 8 * 8) * (f ? 6 : 2));
    acc = vc < V ? up((size_t)N * H * 4) : 0;
    wp = f ? up((size_t)vc * H * 6) : 0;
    slices = 0;
    const int sizes[2] = {vc, V % vc};
    for (int p : sizes) {
      if (p == 0) continue;
      const Shape dx = sliced(K_DX, N, H, p, terms), dw = sliced(K_DW, p, H, N, terms);
      const size_t a = dx.S > 1 ? up((size_t)dx.S * N * H * 4) : 0, b = dw.S > 1 ? up((size_t)dw.S * p * H * 4) : 0;
      if (a > slices) slices = a;
      if (b > slices) slices = b;
    }
  }
  size_t total() const { return 256 + list + tgt + cnt + info + xc + acc + slices + (two ? 2 : 1) * (dz + wp); }
};

unsigned grid8(long long tiles) { return (unsigned)((tiles + 7) / 8 * 8); }
long long n_tiles(int M, int N, int bm, int bn) { return (long long)((M + bm - 1) / bm) * ((N + bn - 1) / bn); }

template <int EPI, bool F>
void launch_z(const Args& a, int tile, hipStream_t s) {
  const int room = tile == 2 ? 256 : 512;  // workgroups that fit at once
  const unsigned all = grid8(n_tiles(a.N, a.V, kZm[tile], kZn[tile]));
  const dim3 g(all < (unsigned)room ? all : (unsigned)room);
  if (tile == 2) hipLaunchKernelGGL((k_ce_z<256, 256, 2, 4, 2, EPI, F>), g, dim3(512), 0, s, a);
  else if (tile == 1) hipLaunchKernelGGL((k_ce_z<128, 128, 2, 2, 2, EPI, F>), g, dim3(256), 0, s, a);
  else if (tile == 3) hipLaunchKernelGGL((k_ce_z<64, 128, 2, 2, 3, EPI, F>), g, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_ce_z<64, 64, 4, 1, 3, EPI, F>), g, dim3(256), 0, s, a);
}
template <bool PART, bool F>
void launch_dx_tiles(const Args& a, int big, hipStream_t s) {
  const int bm = tile_n(big), bn = big == 0 ? 128 : bm;
  const dim3 g(grid8(n_tiles(a.N, a.H, bm, bn) * a.S));
  if (big == 2) hipLaunchKernelGGL((k_ce_dx<256, 256, 2, 4, 2, PART, F>), g, dim3(512), 0, s, a);
  else if (big == 1) hipLaunchKernelGGL((k_ce_dx<128, 128, 2, 2, 2, PART, F>), g, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_ce_dx<64, 128, 2, 2, 3, PART, F>), g, dim3(256), 0, s, a);
}
template <bool PART, bool F>
void launch_dw_tiles(const Args& a, int big, hipStream_t s) {
  const int b = tile_n(big), room = big == 2 ? 256 : 512;  // workgroups that fit at once
  const unsigned all = grid8(n_tiles(a.V, a.H, b, b) * a.S);
  const dim3 g(PART || all < (unsigned)room ? all : (unsigned)room);
  if (big == 2) hipLaunchKernelGGL((k_ce_dw<256, 256, 2, 4, 2, PART, F>), g, dim3(512), 0, s, a);
  else hipLaunchKernelGGL((k_ce_dw<128, 128, 2, 2, 2, PART, F>), g, dim3(256), 0, s, a);
}
unsigned grid_sum(size_t nv) { return (unsigned)(nv / 256 + 1 < 2048 ? nv / 256 + 1 : 2048); }

template <typename T>
hipError_t fwd(const T* x, const T* w, const int* target, int N, int H, int V, float zc, float* loss, float* lse,
               void* ws, hipStream_t s) {
  constexpr bool F = sizeof(T) == 4;
  const FwdWs b(F, N, H, V);
  char* p = static_cast<char*>(ws);
  auto take = [&](size_t n) { char* q = p; p += n; return q; };
  int* list = (int*)take(b.list);
  int* tgt = (int*)take(b.tgt);
  int* cnt = (int*)take(b.cnt);
  Args a{};
  a.zt = (float*)take(b.zt);
  a.part = (float2*)take(b.part);
  bf16_t* xp = (bf16_t*)take(b.xp);
  bf16_t* wp = (bf16_t*)take(b.wp);
  hipLaunchKernelGGL((k_ce_select<T, false>), dim3(select_grid(N)), dim3(1024), 0, s, target, x, N, H, V,
                     select_groups(N), list, cnt, tgt,
                     xp, loss, lse, (const float*)nullptr, (const float*)nullptr, zc, (float4*)nullptr, (T*)nullptr);
  a.cnt = cnt;
  a.tgt = tgt;
  a.N = N;
  a.H = H;
  a.x = xp;
  for (int v0 = 0; v0 < V; v0 += b.vc) {
    a.v0 = v0;
    a.V = V - v0 < b.vc ? V - v0 : b.vc;
    a.nt0 = v0 / kZn[b.tile];
    a.w = w + (size_t)v0 * H;
    if (F) {
      const size_t n = (size_t)a.V * H;
      hipLaunchKernelGGL(k_split, dim3(grid_sum(n / 8)), dim3(256), 0, s, (const float*)a.w, n, wp);
      a.w = wp;
    }
    launch_z<LSE, F>(a, b.tile, s);
  }
  hipLaunchKernelGGL(k_ce_loss, dim3((N + 15) / 16), dim3(1024), 0, s, a.part, a.zt, list, cnt, N, b.tiles, zc, loss,
                     lse);
  return hipGetLastError();
}

template <typename T>
hipError_t bwd(const float* dloss, const T* x, const T* w, const int* target, const float* lse, int N, int H, int V,
               float zc, T* dx, T* dw, void* ws, hipStream_t s) {
  constexpr bool F = sizeof(T) == 4;
  const int terms = F ? 6 : 1;
  const BwdWs b(F, N, H, V);
  char* p = static_cast<char*>(ws);
  auto take = [&](size_t n) { char* q = p; p += n; return q; };
  int* list = (int*)take(b.list);
  int* tgt = (int*)take(b.tgt);
  int* cnt = (int*)take(b.cnt);
  Args a{};
  a.tgt = tgt;
  float4* info = (float4*)take(b.info);
  bf16_t* xc = (bf16_t*)take(b.xc);
  a.acc = (float*)take(b.acc);
  a.slices = (float*)take(b.slices);
  bf16_t *dz[2], *wp[2];
  for (int i = 0; i < 2; ++i) {
    dz[i] = i && !b.two ? dz[0] : (bf16_t*)take(b.dz);
    wp[i] = i && !b.two ? wp[0] : (bf16_t*)take(b.wp);
  }
  hipLaunchKernelGGL((k_ce_select<T, true>), dim3(select_grid(N)), dim3(1024), 0, s, target, x, N, H, V,
                     select_groups(N), list, cnt, tgt,
                     xc, (float*)nullptr, (float*)nullptr, lse, dloss, zc, info, dx);
  a.info = info;
  a.cnt = cnt;
  a.list = list;
  a.N = N;
  a.H = H;
  a.x = xc;
  a.dxo = dx;
  // piece i from column v0 on, its part of W split where it is fp32
  auto piece = [&](int v0, int i) {
    Args q = a;
    q.v0 = v0;
    q.V = V - v0 < b.vc ? V - v0 : b.vc;
    q.ldz = (q.V + 7) / 8 * 8;
    q.first = v0 == 0;
    q.last = v0 + q.V == V;
    q.w = w + (size_t)v0 * H;
    q.dz = dz[i & 1];
    q.dwo = dw + (size_t)v0 * H;
    if (F) {
      const size_t n = (size_t)q.V * H;
      hipLaunchKernelGGL(k_split, dim3(grid_sum(n / 8)), dim3(256), 0, s, (const float*)q.w, n, wp[i & 1]);
      q.w = wp[i & 1];
    }
    return q;
  };
  Args c = piece(0, 0);
  launch_z<DZ, F>(c, z_tile(N, H, c.V, terms), s);
  for (int i = 0, v0 = 0;; ++i) {
    v0 += c.V;
    const bool more = v0 < V;
    Args nx{};
    if (more && b.two) nx = piece(v0, i + 1);
    if (more && b.two && dx && dw && mixes(N, H, c.V, terms)) {
      const unsigned g_dx = grid8(n_tiles(N, H, 256, 256)), g_dw = grid8(n_tiles(c.V, H, 256, 256));
      const unsigned g_z = grid8(n_tiles(N, nx.V, 256, 256));
      hipLaunchKernelGGL((k_ce_piece<F>), dim3(g_dx + g_dw + g_z), dim3(512), 0, s, c, nx, (int)g_dx, (int)g_dw);
    } else {
      if (dx) {
        const Shape h = sliced(K_DX, N, H, c.V, terms);
        c.S = h.S;
        if (h.S > 1) {
          launch_dx_tiles<true, F>(c, h.big, s);
          hipLaunchKernelGGL(k_ce_dx_sum<T>, dim3(grid_sum((size_t)N * H / 8)), dim3(256), 0, s, c);
        } else {
          launch_dx_tiles<false, F>(c, h.big, s);
        }
      }
      if (dw) {
        const Shape h = sliced(K_DW, c.V, H, N, terms);
        c.S = h.S;
        if (h.S > 1) {
          launch_dw_tiles<true, F>(c, h.big, s);
          hipLaunchKernelGGL(k_ce_dw_sum<T>, dim3(grid_sum((size_t)c.V * H / 8)), dim3(256), 0, s, c);
        } else {
          launch_dw_tiles<false, F>(c, h.big, s);
        }
      }
      if (more) {
        if (!b.two) nx = piece(v0, i + 1);
        launch_z<DZ, F>(nx, z_tile(N, H, nx.V, terms), s);
      }
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !more) return e;
    c = nx;
  }
}

}  // namespace ce

size_t linear_ce_fwd_ws_bytes(moe_dtype dt, int N, int H, int V) { return ce::FwdWs(dt == MOE_F32, N, H, V).total(); }
size_t linear_ce_bwd_ws_bytes(moe_dtype dt, int N, int H, int V) { return ce::BwdWs(dt == MOE_F32, N, H, V).total(); }

hipError_t launch_linear_ce_fwd(moe_dtype dt, const void* x, const void* w, const int32_t* target, int N, int H, int V,
                                float zc, float* loss, float* lse, void* ws, hipStream_t s) {
  if (N == 0) return hipSuccess;
  if (dt == MOE_F32) return ce::fwd((const float*)x, (const float*)w, target, N, H, V, zc, loss, lse, ws, s);
  return ce::fwd((const bf16_t*)x, (const bf16_t*)w, target, N, H, V, zc, loss, lse, ws, s);
}

hipError_t launch_linear_ce_bwd(moe_dtype dt, const float* dloss, const void* x, const void* w, const int32_t* target,
                                const float* lse, int N, int H, int V, float zc, void* dx, void* dw, void* ws,
                                hipStream_t s) {
  if (N == 0) {  // W's gradient is zero (a fill kernel, so that the call can be captured)
    if (dw)
      hipLaunchKernelGGL(ce::k_ce_zero, dim3(1024), dim3(256), 0, s, (uint4*)dw,
                         (size_t)V * H / (dt == MOE_F32 ? 4 : 8));
    return hipGetLastError();
  }
  if (dt == MOE_F32)
    return ce::bwd(dloss, (const float*)x, (const float*)w, target, lse, N, H, V, zc, (float*)dx, (float*)dw, ws, s);
  return ce::bwd(dloss, (const bf16_t*)x, (const bf16_t*)w, target, lse, N, H, V, zc, (bf16_t*)dx, (bf16_t*)dw, ws, s);
}

}  // namespace moe
