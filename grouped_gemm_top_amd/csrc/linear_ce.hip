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
// complete, dx is summed over the pieces in fp32.  Every sum has a fixed order (bitwise reproducible).
// dz is rounded to bf16 as an operand of the matrix cores (the fp32 call: three bf16 parts, see linear.hip).
#include <type_traits>

#include "linear_tile.h"

namespace moe {
namespace ce {

using namespace ln;

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;

struct Args {
  const void* x;    // [., H]; the operand's rows are x's rows `rows` (NULL: 0 .. n - 1)
  const void* w;    // the piece of W: [V, H]
  const int* rows;
  const int* cnt;   // n
  const int* list;  // the counted tokens
  int N, H, V, ldz;
  int v0, nt0;      // the piece's first column and first tile (forward)
  int xrows;        // rows that x's storage holds
  // forward
  const int* tgt;
  float2* part;     // [tiles of all pieces][N]
  float* zt;        // [N] the target's logit
  // backward
  const float4* info;  // lse, g (1 + 2 c lse), g, target
  bf16_t* dz;          // [N, ldz], in fp32 three planes of it
  const void* xc;      // [n, H], K-strided operand of dW
  float* acc;          // [N, H] dx so far
  int first, last;     // piece
  void* out;           // dx [N, H] or the piece of dW [V, H]
  float* slices;       // S > 1: [S][N or V][H]
  int S;
};

__device__ __forceinline__ bool in_vocab(int t, int V) { return (unsigned)t < (unsigned)V; }

// ---- the counted tokens ----
// exclusive prefix of c over the 1024 threads; *total: the sum
__device__ __forceinline__ int scan1024(int c, int* s_w, int* total) {
  const int L = threadIdx.x & 63, w = threadIdx.x >> 6;
  int x = c;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(x, o);
    if (L >= o) x += y;
  }
  if (L == 63) s_w[w] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const int v = s_w[q];
    before += q < w ? v : 0;
    all += v;
  }
  __syncthreads();
  *total = all;
  return before + x - c;
}

// The list of the counted tokens, with their targets (BWD: with what dz needs), by one workgroup, 4096 tokens a turn.
// Forward: the others' loss and lse are 0.
template <bool BWD>
__global__ __launch_bounds__(1024) void k_ce_rows(const int* __restrict__ target, int N, int V, int* __restrict__ list,
                                                  int* __restrict__ cnt, int* __restrict__ tgt, float* __restrict__ loss,
                                                  float* __restrict__ lse_out, const float* __restrict__ lse,
                                                  const float* __restrict__ dloss, float zc, float4* __restrict__ info) {
  __shared__ int s_w[16];
  int base = 0;
  for (int t0 = 0; t0 < N; t0 += 4096) {
    const int t = t0 + 4 * threadIdx.x;
    int y[4], c = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[j] = t + j < N ? target[t + j] : -1;
      c += in_vocab(y[j], V);
    }
    int total;
    int p = base + scan1024(c, s_w, &total);
    base += total;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (in_vocab(y[j], V)) {
        list[p] = t + j;
        if constexpr (BWD) {
          const float l = lse[t + j], g = dloss ? dloss[t + j] : 1.0f;
          info[p] = make_float4(l, g * (1.0f + 2.0f * zc * l), g, __int_as_float(y[j]));
        } else {
          tgt[p] = y[j];
        }
        ++p;
      } else if (!BWD && t + j < N) {
        loss[t + j] = 0.f;
        lse_out[t + j] = 0.f;
      }
    }
  }
  if (threadIdx.x == 0) *cnt = base;
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  load4(p, v[0], v[1], v[2], v[3]);
  load4(p + 4, v[4], v[5], v[6], v[7]);
}

// The counted rows of x, one behind the other (fp32: as three planes of N rows), and zeros in the rows of
// dx whose token takes no part (out NULL: no such rows); a wavefront per row.
template <typename T>
__global__ __launch_bounds__(256) void k_ce_gather(const T* __restrict__ x, const int* __restrict__ list,
                                                   const int* __restrict__ cnt, const int* __restrict__ target, int N,
                                                   int H, int V, bf16_t* __restrict__ xc, T* __restrict__ out) {
  const int L = threadIdx.x & 63, n = *cnt;
  for (int r = blockIdx.x * 4 + (threadIdx.x >> 6); r < N; r += 4 * gridDim.x) {
    if (xc && r < n) {
      const T* src = x + (size_t)list[r] * H;
      bf16_t* dst = xc + (size_t)r * H;
      for (int h = 8 * L; h < H; h += 512) {
        if constexpr (sizeof(T) == 2) {
          *reinterpret_cast<uint4*>(dst + h) = *reinterpret_cast<const uint4*>(src + h);
        } else {
          float v[8];
          load8(src + h, v);
          store_parts(dst + h, (size_t)N * H, v);
        }
      }
    }
    if (out && !in_vocab(target[r], V))
      for (int h = 8 * L; h < H; h += 512)
#pragma unroll
        for (int q = 0; q < (int)sizeof(T) / 2; ++q)
          *reinterpret_cast<uint4*>(out + (size_t)r * H + h + q * 16 / sizeof(T)) = make_uint4(0u, 0u, 0u, 0u);
  }
}

// a piece of W as its three parts, planes of n values (a multiple of 8)
__global__ __launch_bounds__(256) void k_ce_split(const float* __restrict__ src, size_t n, bf16_t* __restrict__ dst) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n / 8; i += (size_t)gridDim.x * 256) {
    float v[8];
    load8(src + 8 * i, v);
    store_parts(dst + 8 * i, n, v);
  }
}

// The tile of this workgroup among nM x nN (x S slices, slice major); false: none
__device__ __forceinline__ bool my_tile(int nM, int nN, int S, int& mt, int& nt, int& s) {
  const int nT = nM * nN, per = (nT * S + 7) / 8;
  const int t = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per || t >= nT * S) return false;
  s = t / nT;
  tile_at(t - s * nT, nM, nN, mt, nt);
  return true;
}

enum { LSE = 0, DZ = 1 };

// x W^T on one tile, and from the accumulators either the rows' (maximum, sum of exponentials) or dz
template <int BM, int BN, int WM, int WN, int NST, int EPI, bool F32>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_ce_z(Args a) {
  using C = Core<BM, BN, WM, WN, NST, true, true, F32>;
  constexpr int MB = C::MB, NB = C::NB;
  __shared__ __attribute__((aligned(1024))) char s_ring[NST * C::STG];
  const int L = threadIdx.x & 63, w = ufl(threadIdx.x >> 6);
  const int wm = w % WM, wn = w / WM;
  const int n = ufl(*a.cnt);
  int mt, nt, s;
  if (!my_tile((n + BM - 1) / BM, (a.V + BN - 1) / BN, 1, mt, nt, s)) return;
  const int m0 = mt * BM, n0 = nt * BN;
  const int steps = (a.H + BK - 1) / BK;
  const Opnd A{a.x, n, a.H, (long long)C::PLANES * a.xrows * a.H * 2, (uint32_t)a.xrows * (uint32_t)a.H * 2u, a.rows};
  const Opnd B{a.w, a.V, a.H, (long long)C::PLANES * a.V * a.H * 2, (uint32_t)a.V * (uint32_t)a.H * 2u, nullptr};
  f32x4 acc[MB][NB];
  C::run(s_ring, A, B, m0, n0, a.H, steps, 0, C::TERMS * steps, w, L, acc);

  const int c = L & 15, g = L >> 4, c0 = n0 + wn * (BN / WN);
  if constexpr (EPI == LSE) {
    // Lane (g, c) holds columns 16 j + 4 g + v of row 16 i + c.  Columns past the piece count as -inf.
    float2* s_part = reinterpret_cast<float2*>(s_ring);  // [BM][WN]
    const bool ragged = n0 + BN > a.V;
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int row = wm * (BM / WM) + 16 * i + c;
      if (ragged) {
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (c0 + 16 * j + 4 * g + v >= a.V) acc[i][j][v] = -INFINITY;
      }
      const int y = m0 + row < n ? a.tgt[m0 + row] - a.v0 - c0 - 4 * g : -1;
      if (y >= 0 && y < 16 * NB && (y & 15) < 4) {
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (y == 16 * j + v) a.zt[m0 + row] = acc[i][j][v];
      }
      float m = -INFINITY;
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) m = fmaxf(m, acc[i][j][v]);
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      const float ms = m == -INFINITY ? 0.f : m;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) sum += __builtin_amdgcn_exp2f((acc[i][j][v] - ms) * kLog2e);
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (g == 0) s_part[row * WN + wn] = make_float2(m, sum);
    }
    __syncthreads();
    for (int r = threadIdx.x; r < BM; r += 64 * WM * WN) {
      if (m0 + r >= n) break;
      float2 p[WN];
      float m = -INFINITY;
#pragma unroll
      for (int q = 0; q < WN; ++q) {
        p[q] = s_part[r * WN + q];
        m = fmaxf(m, p[q].x);
      }
      const float ms = m == -INFINITY ? 0.f : m;
      float sum = 0.f;
#pragma unroll
      for (int q = 0; q < WN; ++q) sum += p[q].y * __builtin_amdgcn_exp2f((p[q].x - ms) * kLog2e);
      a.part[(size_t)(a.nt0 + nt) * a.N + m0 + r] = make_float2(m, sum);
    }
  } else {
    // dz of the tile, eight columns a lane; columns from V to ldz get zeros
    char* sg = s_ring + w * 4096;
#pragma unroll
    for (int h = 0; h < NB / 4; ++h) {
      const int col = c0 + 64 * h + 8 * (L & 7), mr = m0 + wm * (BM / WM) + (L >> 3);
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        stage_write(sg, &acc[i][4 * h], L);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          f32x4 v[2];
          stage_read(sg, p, L, v);
          const int m = mr + 16 * i + 8 * p;
          if (m >= n || col >= a.ldz) continue;
          const float4 f = a.info[m];
          const int y = __float_as_int(f.w) - a.v0 - col;
          float d[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            d[q] = f.y * __builtin_amdgcn_exp2f((v[q >> 2][q & 3] - f.x) * kLog2e);
            if (q == y) d[q] -= f.z;
            if (col + q >= a.V) d[q] = 0.f;
          }
          bf16_t* o = a.dz + (size_t)m * a.ldz + col;
          if constexpr (F32)
            store_parts(o, (size_t)a.N * a.ldz, d);
          else
            *reinterpret_cast<u32x4*>(o) = u32x4{pk2(d[0], d[1]), pk2(d[2], d[3]), pk2(d[4], d[5]), pk2(d[6], d[7])};
        }
      }
    }
  }
}

// The tiles' pairs joined in tile order: 64 rows a workgroup, 16 groups of tiles each.
__global__ __launch_bounds__(1024) void k_ce_loss(const float2* __restrict__ part, const float* __restrict__ zt,
                                                  const int* __restrict__ list, const int* __restrict__ cnt, int N,
                                                  int tiles, float zc, float* __restrict__ loss,
                                                  float* __restrict__ lse) {
  __shared__ float2 s[16][64];
  const int r = blockIdx.x * 64 + (threadIdx.x & 63), g = threadIdx.x >> 6, n = *cnt;
  if ((int)blockIdx.x * 64 >= n) return;
  float m = -INFINITY, sum = 0.f;
  if (r < n) {
    for (int t = g; t < tiles; t += 64) {
      float2 p[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        p[q] = t + 16 * q < tiles ? part[(size_t)(t + 16 * q) * N + r] : make_float2(-INFINITY, 0.f);
      const float mn = fmaxf(fmaxf(fmaxf(m, p[0].x), fmaxf(p[1].x, p[2].x)), p[3].x);
      const float ms = mn == -INFINITY ? 0.f : mn;
      sum *= __builtin_amdgcn_exp2f((m - ms) * kLog2e);
#pragma unroll
      for (int q = 0; q < 4; ++q) sum += p[q].y * __builtin_amdgcn_exp2f((p[q].x - ms) * kLog2e);
      m = mn;
    }
  }
  s[g][threadIdx.x & 63] = make_float2(m, sum);
  __syncthreads();
  if (g > 0 || r >= n) return;
  float mm = m;
  for (int q = 1; q < 16; ++q) mm = fmaxf(mm, s[q][threadIdx.x].x);
  const float ms = mm == -INFINITY ? 0.f : mm;
  float tot = 0.f;
  for (int q = 0; q < 16; ++q) {
    const float2 p = s[q][threadIdx.x];
    tot += p.y * __builtin_amdgcn_exp2f((p.x - ms) * kLog2e);
  }
  const float l = ms + __logf(tot);
  const int t = list[r];
  lse[t] = l;
  loss[t] = l - zt[r] + zc * l * l;
}

// dx = dz W of a piece: straight, or (S > 1) fp32 slices of its K range
template <int BM, int BN, int WM, int WN, int NST, bool PART, bool F32>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_ce_dx(Args a) {
  using C = Core<BM, BN, WM, WN, NST, true, false, F32>;
  typedef typename std::conditional<F32, float, bf16_t>::type T;
  constexpr int MB = C::MB, NB = C::NB;
  __shared__ __attribute__((aligned(1024))) char s_ring[NST * C::STG];
  const int L = threadIdx.x & 63, w = ufl(threadIdx.x >> 6);
  const int wm = w % WM, wn = w / WM;
  const int n = ufl(*a.cnt);
  int mt, nt, s;
  if (!my_tile((n + BM - 1) / BM, (a.H + BN - 1) / BN, PART ? a.S : 1, mt, nt, s)) return;
  const int m0 = mt * BM, n0 = nt * BN;
  const int steps = (a.V + BK - 1) / BK;
  const int S = PART ? a.S : 1;
  const int k_lo = (int)((long long)C::TERMS * steps * s / S);
  const int nk = (int)((long long)C::TERMS * steps * (s + 1) / S) - k_lo;
  const Opnd A{a.dz, n, a.ldz, (long long)C::PLANES * a.N * a.ldz * 2, (uint32_t)a.N * (uint32_t)a.ldz * 2u, nullptr};
  const Opnd B{a.w, a.H, a.H, (long long)C::PLANES * a.V * a.H * 2, (uint32_t)a.V * (uint32_t)a.H * 2u, nullptr};
  f32x4 acc[MB][NB];
  C::run(s_ring, A, B, m0, n0, a.V, steps, k_lo, nk, w, L, acc);
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
          if (a.last) store8<T>(a.out, (size_t)a.list[m] * a.H + col, v);
          else store8<float>(a.acc, o, v);
        }
      }
    }
  }
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
#pragma unroll 4
    for (int s = 0; s < a.S; ++s) {
      const float* p = a.slices + (size_t)s * slice + 8 * i;
      v[0] += *reinterpret_cast<const f32x4*>(p);
      v[1] += *reinterpret_cast<const f32x4*>(p + 4);
    }
    if (a.last) store8<T>(a.out, (size_t)a.list[m] * a.H + col, v);
    else store8<float>(a.acc, 8 * i, v);
  }
}

// dW = dz^T x of a piece
template <int BM, int BN, int WM, int WN, int NST, bool PART, bool F32>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_ce_dw(Args a) {
  using C = Core<BM, BN, WM, WN, NST, false, false, F32>;
  typedef typename std::conditional<F32, float, bf16_t>::type T;
  constexpr int MB = C::MB, NB = C::NB;
  __shared__ __attribute__((aligned(1024))) char s_ring[NST * C::STG];
  const int L = threadIdx.x & 63, w = ufl(threadIdx.x >> 6);
  const int wm = w % WM, wn = w / WM;
  const int n = ufl(*a.cnt), S = PART ? a.S : 1;
  int mt, nt, s;
  if (!my_tile((a.V + BM - 1) / BM, (a.H + BN - 1) / BN, S, mt, nt, s)) return;
  const int m0 = mt * BM, n0 = nt * BN;
  const int steps = (n + BK - 1) / BK;
  const int k_lo = (int)((long long)C::TERMS * steps * s / S);
  const int nk = (int)((long long)C::TERMS * steps * (s + 1) / S) - k_lo;
  const Opnd A{a.dz, a.V, a.ldz, (long long)C::PLANES * a.N * a.ldz * 2, (uint32_t)a.N * (uint32_t)a.ldz * 2u, nullptr};
  const Opnd B{a.xc, a.H, a.H, (long long)C::PLANES * a.N * a.H * 2, (uint32_t)a.N * (uint32_t)a.H * 2u, nullptr};
  f32x4 acc[MB][NB];
  C::run(s_ring, A, B, m0, n0, n, steps, k_lo, nk, w, L, acc);
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
        if (m >= a.V || col >= a.H) continue;
        const size_t o = (size_t)m * a.H + col;
        if constexpr (PART) store8<float>(a.slices, (size_t)s * a.V * a.H + o, v);
        else store8<T>(a.out, o, v);
      }
    }
  }
}

template <typename T>
__global__ __launch_bounds__(256) void k_ce_dw_sum(Args a) {
  const size_t slice = (size_t)a.V * a.H, nv = slice / 8;
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < nv; i += (size_t)gridDim.x * 256) {
    f32x4 v[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll 4
    for (int s = 0; s < a.S; ++s) {
      const float* p = a.slices + (size_t)s * slice + 8 * i;
      v[0] += *reinterpret_cast<const f32x4*>(p);
      v[1] += *reinterpret_cast<const f32x4*>(p + 4);
    }
    store8<T>(a.out, 8 * i, v);
  }
}

__global__ __launch_bounds__(256) void k_ce_zero(uint4* __restrict__ p, size_t n) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256)
    p[i] = make_uint4(0u, 0u, 0u, 0u);
}

// ------------------------------------------------------------------ host side
constexpr long long kDesc = 0x7FFFFFFF;

int tile_n(int big) { return big == 2 ? 256 : big == 1 ? 128 : 64; }

// the tile of x W^T: no K slices (the epilogue needs whole sums)
int z_tile(int N, int H, int V, int terms) {
  const int b = choose(K_FWD, N, V, H, terms, 1).big;
  return b < 2 && (long long)((N + 63) / 64) * ((V + 63) / 64) > 1 << 20 ? 2 : b;
}

// Columns of a forward piece: all of them, unless a descriptor (2 GiB) or, in fp32, the workspace's copy of
// the piece in three parts (512 MB) does not hold them.
int fwd_piece(bool f, int H, int V) {
  const long long most = f ? (512LL << 20) / (6LL * H) : kDesc / (2LL * H);
  if (most >= V) return V;
  return most < 256 ? 256 : (int)(most / 256 * 256);
}

// Columns of a backward piece.
int bwd_piece(bool f, int N, int H, int V) {
  long long most = (f ? 32LL : 64LL) * (1 << 20) / (N > 0 ? N : 1);
  const long long desc = f ? (1LL << 30) / (6LL * H) : kDesc / (2LL * H);
  if (desc < most) most = desc;
  if (most >= V) return V;
  const int nH = (H + 255) / 256;
  const long long unit = 256LL * (nH < 256 ? 256 / nH : 1);
  if (most >= unit) return (int)(most / unit * unit);
  return most < 256 ? 256 : (int)(most / 256 * 256);
}

struct FwdWs {
  size_t list, tgt, cnt, zt, part, xp, wp;
  int vc, tile, tiles;
  FwdWs(bool f, int N, int H, int V) {
    vc = fwd_piece(f, H, V);
    tile = z_tile(N, H, vc, f ? 6 : 1);
    const int bn = tile_n(tile);
    tiles = (V + bn - 1) / bn;  // (a piece is a multiple of 256 unless it is the last)
    list = tgt = zt = up((size_t)N * 4);
    cnt = 256;
    part = up((size_t)tiles * N * 8);
    xp = f ? up((size_t)N * H * 6) : 0;
    wp = f ? up((size_t)vc * H * 6) : 0;
  }
  size_t total() const { return 256 + list + tgt + cnt + zt + part + xp + wp; }
};

struct BwdWs {
  size_t list, cnt, info, xc, dz, acc, slices, wp;
  int vc;
  BwdWs(bool f, int N, int H, int V) {
    const int terms = f ? 6 : 1;
    vc = bwd_piece(f, N, H, V);
    list = up((size_t)N * 4);
    cnt = 256;
    info = up((size_t)N * 16);
    xc = up((size_t)N * H * (f ? 6 : 2));
    dz = up((size_t)N * ((vc + 7) / 8 * 8) * (f ? 6 : 2));
    acc = vc < V ? up((size_t)N * H * 4) : 0;
    wp = f ? up((size_t)vc * H * 6) : 0;
    slices = 0;
    const int sizes[2] = {vc, V % vc};
    for (int p : sizes) {
      if (p == 0) continue;
      const Shape dx = choose(K_DX, N, H, p, terms), dw = choose(K_DW, p, H, N, terms);
      const size_t a = dx.S > 1 ? up((size_t)dx.S * N * H * 4) : 0, b = dw.S > 1 ? up((size_t)dw.S * p * H * 4) : 0;
      if (a > slices) slices = a;
      if (b > slices) slices = b;
    }
  }
  size_t total() const { return 256 + list + cnt + info + xc + dz + acc + slices + wp; }
};

unsigned grid8(long long tiles) { return (unsigned)((tiles + 7) / 8 * 8); }
long long n_tiles(int M, int N, int bm, int bn) { return (long long)((M + bm - 1) / bm) * ((N + bn - 1) / bn); }

template <int EPI, bool F>
void launch_z(const Args& a, int tile, hipStream_t s) {
  const int b = tile_n(tile);
  const dim3 g(grid8(n_tiles(a.N, a.V, b, b)));
  if (tile == 2) hipLaunchKernelGGL((k_ce_z<256, 256, 2, 4, 2, EPI, F>), g, dim3(512), 0, s, a);
  else if (tile == 1) hipLaunchKernelGGL((k_ce_z<128, 128, 2, 2, 2, EPI, F>), g, dim3(256), 0, s, a);
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
  const int b = tile_n(big);
  const dim3 g(grid8(n_tiles(a.V, a.H, b, b) * a.S));
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
  hipLaunchKernelGGL(k_ce_rows<false>, dim3(1), dim3(1024), 0, s, target, N, V, list, cnt, tgt, loss, lse,
                     (const float*)nullptr, (const float*)nullptr, zc, (float4*)nullptr);
  a.cnt = cnt;
  a.tgt = tgt;
  a.N = N;
  a.H = H;
  a.xrows = N;
  if (F) {
    hipLaunchKernelGGL(k_ce_gather<T>, dim3((unsigned)(N / 4 + 1 < 4096 ? N / 4 + 1 : 4096)), dim3(256), 0, s, x, list,
                       cnt, target, N, H, V, xp, (T*)nullptr);
    a.x = xp;
  } else {
    a.x = x;
    a.rows = list;
  }
  for (int v0 = 0; v0 < V; v0 += b.vc) {
    a.v0 = v0;
    a.V = V - v0 < b.vc ? V - v0 : b.vc;
    a.nt0 = v0 / tile_n(b.tile);
    a.w = w + (size_t)v0 * H;
    if (F) {
      const size_t n = (size_t)a.V * H;
      hipLaunchKernelGGL(k_ce_split, dim3(grid_sum(n / 8)), dim3(256), 0, s, (const float*)a.w, n, wp);
      a.w = wp;
    }
    launch_z<LSE, F>(a, b.tile, s);
  }
  hipLaunchKernelGGL(k_ce_loss, dim3((N + 63) / 64), dim3(1024), 0, s, a.part, a.zt, list, cnt, N, b.tiles, zc, loss,
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
  int* cnt = (int*)take(b.cnt);
  Args a{};
  float4* info = (float4*)take(b.info);
  bf16_t* xc = (bf16_t*)take(b.xc);
  a.dz = (bf16_t*)take(b.dz);
  a.acc = (float*)take(b.acc);
  a.slices = (float*)take(b.slices);
  bf16_t* wp = (bf16_t*)take(b.wp);
  hipLaunchKernelGGL(k_ce_rows<true>, dim3(1), dim3(1024), 0, s, target, N, V, list, cnt, (int*)nullptr,
                     (float*)nullptr, (float*)nullptr, lse, dloss, zc, info);
  hipLaunchKernelGGL(k_ce_gather<T>, dim3((unsigned)(N / 4 + 1 < 4096 ? N / 4 + 1 : 4096)), dim3(256), 0, s, x, list,
                     cnt, target, N, H, V, xc, dx);
  a.info = info;
  a.cnt = cnt;
  a.list = list;
  a.N = N;
  a.H = H;
  a.x = xc;
  a.xc = xc;
  a.xrows = N;
  for (int v0 = 0; v0 < V; v0 += b.vc) {
    a.v0 = v0;
    a.V = V - v0 < b.vc ? V - v0 : b.vc;
    a.ldz = (a.V + 7) / 8 * 8;
    a.first = v0 == 0;
    a.last = v0 + a.V == V;
    a.w = w + (size_t)v0 * H;
    if (F) {
      const size_t n = (size_t)a.V * H;
      hipLaunchKernelGGL(k_ce_split, dim3(grid_sum(n / 8)), dim3(256), 0, s, (const float*)a.w, n, wp);
      a.w = wp;
    }
    launch_z<DZ, F>(a, z_tile(N, H, a.V, terms), s);
    if (dx) {
      const Shape c = choose(K_DX, N, H, a.V, terms);
      a.S = c.S;
      a.out = dx;
      if (c.S > 1) {
        launch_dx_tiles<true, F>(a, c.big, s);
        hipLaunchKernelGGL(k_ce_dx_sum<T>, dim3(grid_sum((size_t)N * H / 8)), dim3(256), 0, s, a);
      } else {
        launch_dx_tiles<false, F>(a, c.big, s);
      }
    }
    if (dw) {
      const Shape c = choose(K_DW, a.V, H, N, terms);
      a.S = c.S;
      a.out = dw + (size_t)v0 * H;
      if (c.S > 1) {
        launch_dw_tiles<true, F>(a, c.big, s);
        hipLaunchKernelGGL(k_ce_dw_sum<T>, dim3(grid_sum((size_t)a.V * H / 8)), dim3(256), 0, s, a);
      } else {
        launch_dw_tiles<false, F>(a, c.big, s);
      }
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
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
