// few.hip -- the whole expert layer for a few tokens (N <= 64: decoding steps, draft verification), for
// gfx950: bf16 or fp32 weights, or MX-FP8 weights under bf16 activations.
//
//   z = x W_r + b;  the k largest z of a token (z descending, expert ascending);  w = softmax over them
//   out_t = sum_e w[t,e] W_d[e] (silu(W_g[e] x_t) * (W_u[e] x_t))
//
// With so few tokens each weight is used once or a handful of times: the layer is one pass over the matrices
// of the experts that any token names, E (1 - (1 - k/E)^N) of them, and everything else has to hide behind
// that stream.  Launches:
//  1. router product, sliced along H (fp32 on the vector units: 2 N H E operations are nothing here);
//  2. gate/up: every workgroup joins the slices and chooses the experts itself (a few hundred logits: cheaper
//     than a launch that hands the choice on), then takes tasks (expert, 16 columns of I).  Its eight wavefronts
//     split H, weights go straight from memory into registers as the matrix instruction's operand, and the
//     sums meet in LDS; a' = w silu(g) u is rounded once, as the next product's operand;
//  3. down: a workgroup owns 16 outputs of every token.  The other operand's columns are the tokens, zero for
//     those that do not name the expert, so the sum over the experts is the matrix instruction's own
//     accumulation: no scatter, no atomics, one fixed order.
#include <type_traits>

#include "gemm_lds.h"

namespace moe {
namespace fw {

using namespace gk;

constexpr int MAXN = MOE_FEW_MAX_TOKENS, MAXK = MOE_FEW_MAX_K, MAXE = 1024;
constexpr int NW = 8, NT = 64 * NW;  // wavefronts and threads of the two product kernels

struct Args {
  const void* x;
  const float* wr;
  const float* bias;
  const void *wg, *wu, *wd;
  const uint8_t *gs, *us, *ds;  // MX-FP8: scale codes
  int N, H, I, E, k;
  int S, hs;      // slices of the router product and their length
  float* part;    // [S, N, E]
  void* act;      // a' [N k, I]: rows by expert, then token
  int32_t* idx;   // [N, k]
  float* w;       // [N, k]
  void* out;      // [N, H]
};

// ------------------------------------------------------------------ router product
// Slice s of H, 64 experts (a lane each), 16 tokens: part[s][t][e] = sum over the slice of x[t,h] w_r[h,e].
template <typename T>
__global__ __launch_bounds__(256) void k_few_router(Args a) {
  __shared__ __attribute__((aligned(16))) float s_x[16][256];
  __shared__ float s_p[4][16][64];
  const int L = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int s = blockIdx.x, e = blockIdx.y * 64 + L, t0 = blockIdx.z * 16;
  const int lo = s * a.hs, len = max(0, min(a.hs, a.H - lo));
  const int nt = min(16, a.N - t0);
  for (int q = threadIdx.x; q < 16 * 256; q += 256) {
    const int t = q >> 8, h = q & 255;
    s_x[t][h] = t < nt && h < len ? to_f32<T>(static_cast<const T*>(a.x)[(size_t)(t0 + t) * a.H + lo + h]) : 0.f;
  }
  __syncthreads();
  float acc[16];
#pragma unroll
  for (int t = 0; t < 16; ++t) acc[t] = 0.f;
  const float* wp = a.wr + (size_t)lo * a.E + min(e, a.E - 1);
  for (int h = 4 * w; h < len; h += 16) {
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = h + j < len ? wp[(size_t)(h + j) * a.E] : 0.f;
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      if (t >= nt) break;
      const float4 xv = *reinterpret_cast<const float4*>(&s_x[t][h]);
      acc[t] = __builtin_fmaf(xv.x, v[0], acc[t]);
      acc[t] = __builtin_fmaf(xv.y, v[1], acc[t]);
      acc[t] = __builtin_fmaf(xv.z, v[2], acc[t]);
      acc[t] = __builtin_fmaf(xv.w, v[3], acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < 16; ++t) s_p[w][t][L] = acc[t];
  __syncthreads();
  for (int t = w; t < nt; t += 4)
    if (e < a.E)
      a.part[((size_t)s * a.N + t0 + t) * a.E + e] = (s_p[0][t][L] + s_p[1][t][L]) + (s_p[2][t][L] + s_p[3][t][L]);
}

// ------------------------------------------------------------------ choice of the experts
template <int CTRL>
__device__ __forceinline__ float dpp_f(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float lane_f(float v, int l) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}
// the wavefront's maximum in every lane: quad permutations, half-row and row mirrors, then the four rows
__device__ __forceinline__ float wave_max(float x) {
  x = fmaxf(x, dpp_f<0xB1>(x));
  x = fmaxf(x, dpp_f<0x4E>(x));
  x = fmaxf(x, dpp_f<0x141>(x));
  x = fmaxf(x, dpp_f<0x140>(x));
  return fmaxf(fmaxf(lane_f(x, 0), lane_f(x, 16)), fmaxf(lane_f(x, 32), lane_f(x, 48)));
}

struct Lists {  // in LDS
  unsigned long long mask[MAXE];  // the tokens that name an expert
  int exp[MAXE], row[MAXE];       // active experts, ascending, and the first row of a' of each
  int idx[MAXN * MAXK];
  float w[MAXN * MAXK];
  int scan[NW];
  int n;                          // active experts
};

// Experts and weights of every token, a wavefront per token.  A NaN logit counts as -inf; weights of
// experts at -inf are 0 (all of a token's, where it has no other).
template <int PL>  // experts per lane: E <= 64 PL
__device__ __forceinline__ void choose_experts(const Args& a, Lists& s, int w, int L) {
  for (int t = w; t < a.N; t += NW) {
    float z[PL];
    uint32_t avail = 0;
#pragma unroll
    for (int q = 0; q < PL; ++q) {
      const int e = L + 64 * q, ec = min(e, a.E - 1);
      const float* p = a.part + (size_t)t * a.E + ec;
      float v = 0.f;
#pragma unroll 8
      for (int i = 0; i < a.S; ++i) v += p[(size_t)i * a.N * a.E];
      if (a.bias) v += a.bias[ec];
      z[q] = v == v ? v : -INFINITY;
      if (e < a.E) avail |= 1u << q;
    }
    float myz = -INFINITY, z0 = 0.f;
    int mye = 0;
    for (int j = 0; j < a.k; ++j) {
      float m = -INFINITY;
#pragma unroll
      for (int q = 0; q < PL; ++q)
        if ((avail >> q) & 1u) m = fmaxf(m, z[q]);
      m = wave_max(m);
      int e = 0;  // the lowest expert that has it (-0 and +0 tie)
#pragma unroll
      for (int q = PL - 1; q >= 0; --q) {
        const unsigned long long b = __ballot(((avail >> q) & 1u) && z[q] == m);
        if (b) e = 64 * q + __builtin_ctzll(b);
      }
      if ((e & 63) == L) avail &= ~(1u << (e >> 6));
      if (L == j) myz = m, mye = e;
      if (j == 0) z0 = m;
    }
    const float zm = z0 == -INFINITY ? 0.f : z0;
    const float ex = L < a.k ? expf(myz - zm) : 0.f;
    float sum = ex;
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
    if (L < a.k) {
      s.idx[t * a.k + L] = mye;
      s.w[t * a.k + L] = sum == 0.f ? 0.f : ex / sum;
    }
  }
}

// From s.idx: each expert's tokens, the active experts and the rows of a'.  Ends with a barrier.
__device__ __forceinline__ void make_lists(const Args& a, Lists& s, int w, int L) {
  const int tid = threadIdx.x;
  for (int e = tid; e < MAXE; e += NT) s.mask[e] = 0;
  __syncthreads();
  for (int p = tid; p < a.N * a.k; p += NT) atomicOr(&s.mask[s.idx[p]], 1ull << (p / a.k));
  __syncthreads();
  const unsigned long long m0 = s.mask[2 * tid], m1 = s.mask[2 * tid + 1];
  // (active experts, rows) before this thread's two, packed
  const int c0 = (m0 ? 1 << 16 : 0) + __popcll(m0), c1 = (m1 ? 1 << 16 : 0) + __popcll(m1);
  int v = c0 + c1;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(v, o);
    if (L >= o) v += y;
  }
  if (L == 63) s.scan[w] = v;
  __syncthreads();
  int before = v - c0 - c1;
#pragma unroll
  for (int q = 0; q < NW; ++q) before += q < w ? s.scan[q] : 0;
  if (m0) s.exp[before >> 16] = 2 * tid, s.row[before >> 16] = before & 0xFFFF;
  before += c0;
  if (m1) s.exp[before >> 16] = 2 * tid + 1, s.row[before >> 16] = before & 0xFFFF;
  if (tid == NT - 1) s.n = (before + c1) >> 16;
  __syncthreads();
}

// the r-th set bit of m (r < popcount)
__device__ __forceinline__ int nth_bit(unsigned long long m, int r) {
  for (; r > 0; --r) m &= m - 1;
  return __builtin_ctzll(m);
}

// ------------------------------------------------------------------ operands
// A 128-byte line of a weight row per k-step: lane (g, r) takes bytes 16 g and 64 + 16 g of row r, as
// fragments for the matrix instruction, with the other operand's values at the same k.
//  T = bf16: k = 64, two fragments;  fp32: k = 32, eight one-k instructions;  MX-FP8: k = 128, four
//  fragments (codes times their scale, exact in bf16), the scale word of the line beside it.
template <typename T, bool F8> struct Line;
template <> struct Line<bf16_t, false> {
  static constexpr int K = 64;
  u32x4 v[2];
  __device__ __forceinline__ void load(const char* row, const uint8_t*, int k0, int K_, int g) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = k0 + 32 * h + 8 * g;
      v[h] = k < K_ ? *reinterpret_cast<const u32x4*>(row + 2 * (size_t)k) : u32x4{0u, 0u, 0u, 0u};
    }
  }
};
template <> struct Line<float, false> {
  static constexpr int K = 32;
  u32x4 v[2];
  __device__ __forceinline__ void load(const char* row, const uint8_t*, int k0, int K_, int g) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = k0 + 16 * h + 4 * g;
      v[h] = k < K_ ? *reinterpret_cast<const u32x4*>(row + 4 * (size_t)k) : u32x4{0u, 0u, 0u, 0u};
    }
  }
};
template <> struct Line<bf16_t, true> {
  static constexpr int K = 128;
  u32x4 v[2];
  uint32_t s;
  __device__ __forceinline__ void load(const char* row, const uint8_t* sc, int k0, int K_, int g) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = k0 + 64 * h + 16 * g;
      v[h] = k < K_ ? *reinterpret_cast<const u32x4*>(row + k) : u32x4{0u, 0u, 0u, 0u};
    }
    s = k0 < K_ ? *reinterpret_cast<const uint32_t*>(sc + k0 / 32) : 0u;
  }
};
// the other operand's values of a k-step: row p of type T (NULL: zeros)
template <typename T, bool F8> struct Vec {
  static constexpr int NV = F8 ? 4 : 2;
  u32x4 v[NV];
  __device__ __forceinline__ void load(const T* p, int k0, int K_, int g) {
#pragma unroll
    for (int h = 0; h < NV; ++h) {
      const int k = F8 ? k0 + 64 * (h >> 1) + 16 * g + 8 * (h & 1) : k0 + (int)(64 / sizeof(T)) * h + (int)(16 / sizeof(T)) * g;
      v[h] = p && k < K_ ? *reinterpret_cast<const u32x4*>(p + k) : u32x4{0u, 0u, 0u, 0u};
    }
  }
};
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
template <typename T, bool F8>
__device__ __forceinline__ f32x4 line_mma(const Line<T, F8>& w, const Vec<T, F8>& x, f32x4 acc, int g) {
  if constexpr (F8) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // block 2 h + (g >> 1) of the line's four; a power of two
      const int c = (int)((w.s >> (16 * h + 8 * (g >> 1))) & 255u);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t f[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t u = w.v[h][2 * q + j];
          const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)u, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)u, true);
          f[2 * j] = pk2(__builtin_amdgcn_ldexpf(lo.x, c - 127), __builtin_amdgcn_ldexpf(lo.y, c - 127));
          f[2 * j + 1] = pk2(__builtin_amdgcn_ldexpf(hi.x, c - 127), __builtin_amdgcn_ldexpf(hi.y, c - 127));
        }
        acc = mma(__builtin_bit_cast(bf16x8, u32x4{f[0], f[1], f[2], f[3]}), __builtin_bit_cast(bf16x8, x.v[2 * h + q]), acc);
      }
    }
  } else if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h) acc = mma(__builtin_bit_cast(bf16x8, w.v[h]), __builtin_bit_cast(bf16x8, x.v[h]), acc);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w.v[h][j]), __uint_as_float(x.v[h][j]), acc, 0, 0, 0);
  }
  return acc;
}

__device__ __forceinline__ float silu(float g) { return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

// ------------------------------------------------------------------ gate / up
// TB: blocks of 16 tokens (N <= 16 TB)
template <typename T, bool F8, int PL, int TB>
__global__ __launch_bounds__(NT, 2) void k_few_gateup(Args a) {
  using Ln = Line<T, F8>;
  constexpr int U = F8 ? 2 : 4;  // k-steps in flight
  __shared__ Lists s;
  __shared__ f32x4 s_sum[NW][2][64];
  const int L = threadIdx.x & 63, w = ufl(threadIdx.x >> 6);
  const int r = L & 15, g = L >> 4;
  choose_experts<PL>(a, s, w, L);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int p = threadIdx.x; p < a.N * a.k; p += NT) {
      a.idx[p] = s.idx[p];
      a.w[p] = s.w[p];
    }
  make_lists(a, s, w, L);
  const int IB = (a.I + 15) / 16, tasks = ufl(s.n) * IB;
  const int KS = 4 * ((a.H + 127) / 128);
  constexpr size_t ES = F8 ? 1 : sizeof(T);
  for (int task = blockIdx.x; task < tasks; task += gridDim.x) {
    const int ai = task / IB, i0 = (task - ai * IB) * 16, e = ufl(s.exp[ai]);
    const unsigned long long m = s.mask[e];
    const int cnt = __popcll(m), nb = ufl((cnt + 15) / 16);
    const size_t row = (size_t)e * a.I + min(i0 + r, a.I - 1);
    const char* pg = static_cast<const char*>(a.wg) + row * a.H * ES;
    const char* pu = static_cast<const char*>(a.wu) + row * a.H * ES;
    const uint8_t* sg = F8 ? a.gs + row * KS : nullptr;
    const uint8_t* su = F8 ? a.us + row * KS : nullptr;
    const T* px[TB];
#pragma unroll
    for (int b = 0; b < TB; ++b)
      px[b] = static_cast<const T*>(a.x) + (size_t)nth_bit(m, min(16 * b + r, cnt - 1)) * a.H;
    f32x4 ag[TB], au[TB];
#pragma unroll
    for (int b = 0; b < TB; ++b) ag[b] = au[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int k0 = w * Ln::K; k0 < a.H; k0 += U * NW * Ln::K) {
      Ln lg[U], lu[U];
      Vec<T, F8> xv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * NW * Ln::K;
        lg[u].load(pg, sg, k, a.H, g);
        lu[u].load(pu, su, k, a.H, g);
        xv[u].load(px[0], k, a.H, g);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        ag[0] = line_mma(lg[u], xv[u], ag[0], g);
        au[0] = line_mma(lu[u], xv[u], au[0], g);
      }
#pragma unroll
      for (int b = 1; b < TB; ++b) {
        if (b >= nb) break;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          Vec<T, F8> xb;
          xb.load(px[b], k0 + u * NW * Ln::K, a.H, g);
          ag[b] = line_mma(lg[u], xb, ag[b], g);
          au[b] = line_mma(lu[u], xb, au[b], g);
        }
      }
    }
    // the wavefronts' sums in wavefront order; lane l of wavefront 0: columns i0 + 4 (l >> 4) + v, token slot l & 15
#pragma unroll
    for (int b = 0; b < TB; ++b) {
      if (b >= nb) break;
      s_sum[w][0][L] = ag[b];
      s_sum[w][1][L] = au[b];
      __syncthreads();
      if (w == 0) {
        f32x4 G = s_sum[0][0][L], Uv = s_sum[0][1][L];
#pragma unroll
        for (int q = 1; q < NW; ++q) {
          G += s_sum[q][0][L];
          Uv += s_sum[q][1][L];
        }
        const int slot = 16 * b + r, i = i0 + 4 * g;
        if (slot < cnt && i < a.I) {
          const int t = nth_bit(m, slot);
          float wt = 0.f;
          for (int j = 0; j < a.k; ++j)
            if (s.idx[t * a.k + j] == e) wt = s.w[t * a.k + j];
          T* o = static_cast<T*>(a.act) + (size_t)(s.row[ai] + slot) * a.I + i;
          store4(o, wt * silu(G[0]) * Uv[0], wt * silu(G[1]) * Uv[1], wt * silu(G[2]) * Uv[2], wt * silu(G[3]) * Uv[3]);
        }
      }
      __syncthreads();
    }
  }
}

// ------------------------------------------------------------------ down
template <typename T, bool F8, int TB>
__global__ __launch_bounds__(NT, 2) void k_few_down(Args a) {
  using Ln = Line<T, F8>;
  constexpr int U = F8 ? 2 : 4;
  __shared__ Lists s;
  __shared__ f32x4 s_sum[NW][TB][64];
  const int L = threadIdx.x & 63, w = ufl(threadIdx.x >> 6);
  const int r = L & 15, g = L >> 4;
  for (int p = threadIdx.x; p < a.N * a.k; p += NT) s.idx[p] = a.idx[p];
  __syncthreads();
  make_lists(a, s, w, L);
  const int h0 = blockIdx.x * 16;
  const int KS = 4 * ((a.I + 127) / 128), steps = (a.I + Ln::K - 1) / Ln::K, units = ufl(s.n) * steps;
  constexpr size_t ES = F8 ? 1 : sizeof(T);
  const int hr = min(h0 + r, a.H - 1);
  f32x4 acc[TB];
#pragma unroll
  for (int b = 0; b < TB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int u0 = w; u0 < units; u0 += U * NW) {
    Ln l[U];
    Vec<T, F8> v[U][TB];
    bool has[U][TB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int un = u0 + u * NW, ai = min(un / steps, s.n - 1);
      const int k0 = un < units ? (un - ai * steps) * Ln::K : a.I;
      const int e = ufl(s.exp[ai]);
      const unsigned long long m = s.mask[e];
      const size_t row = (size_t)e * a.H + hr;
      l[u].load(static_cast<const char*>(a.wd) + row * a.I * ES, F8 ? a.ds + row * KS : nullptr, k0, a.I, g);
#pragma unroll
      for (int b = 0; b < TB; ++b) {
        const int t = 16 * b + r;
        has[u][b] = (m >> t) & 1ull;
        const T* p = static_cast<const T*>(a.act) + (size_t)(s.row[ai] + __popcll(m & ((1ull << t) - 1))) * a.I;
        v[u][b].load(has[u][b] ? p : nullptr, k0, a.I, g);
      }
    }
    // (a step's products are added only where the token names the expert: an infinity or NaN among another
    // expert's weights, times its zeros, would spoil every token)
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int b = 0; b < TB; ++b) {
        const f32x4 d = line_mma(l[u], v[u][b], f32x4{0.f, 0.f, 0.f, 0.f}, g);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[b][j] += has[u][b] ? d[j] : 0.f;
      }
  }
#pragma unroll
  for (int b = 0; b < TB; ++b) s_sum[w][b][L] = acc[b];
  __syncthreads();
  for (int b = w; b < TB; b += NW) {
    f32x4 o = s_sum[0][b][L];
#pragma unroll
    for (int q = 1; q < NW; ++q) o += s_sum[q][b][L];
    const int t = 16 * b + r, h = h0 + 4 * g;
    if (t < a.N && h < a.H) store4(static_cast<T*>(a.out) + (size_t)t * a.H + h, o[0], o[1], o[2], o[3]);
  }
}

// ------------------------------------------------------------------ host side
size_t up(size_t n) { return (n + 255) / 256 * 256; }

// slices of the router product: about 128 workgroups, 32 to 256 of H each
void slices(int N, int H, int E, int& S, int& hs) {
  const int others = ((E + 63) / 64) * (N > 16 ? (N + 15) / 16 : 1);
  S = 128 / others;
  if (S > 32) S = 32;
  if (S > H / 32) S = H / 32;
  if (S < 1) S = 1;
  if (S < (H + 255) / 256) S = (H + 255) / 256;
  hs = ((H + S - 1) / S + 15) / 16 * 16;
}

template <typename T, bool F8, int PL, int TB>
hipError_t run(const Args& a, hipStream_t s) {
  const dim3 gr(a.S, (a.E + 63) / 64, (a.N + 15) / 16);
  hipLaunchKernelGGL(k_few_router<T>, gr, dim3(256), 0, s, a);
  const long long act = a.E < a.N * a.k ? a.E : a.N * a.k, tasks = act * ((a.I + 15) / 16);
  hipLaunchKernelGGL((k_few_gateup<T, F8, PL, TB>), dim3((unsigned)(tasks < 512 ? tasks : 512)), dim3(NT), 0, s, a);
  hipLaunchKernelGGL((k_few_down<T, F8, TB>), dim3((a.H + 15) / 16), dim3(NT), 0, s, a);
  return hipGetLastError();
}
template <typename T, bool F8, int PL>
hipError_t run_tb(const Args& a, hipStream_t s) {
  if (a.N <= 16) return run<T, F8, PL, 1>(a, s);
  if (a.N <= 32) return run<T, F8, PL, 2>(a, s);
  return run<T, F8, PL, 4>(a, s);
}
template <typename T, bool F8>
hipError_t run_pl(const Args& a, hipStream_t s) {
  if (a.E <= 128) return run_tb<T, F8, 2>(a, s);
  if (a.E <= 256) return run_tb<T, F8, 4>(a, s);
  return run_tb<T, F8, 16>(a, s);
}

}  // namespace fw

size_t layer_few_ws_bytes(moe_dtype dt, int N, int E, int k, int H, int I) {
  int S, hs;
  fw::slices(N, H, E, S, hs);
  return 256 + fw::up((size_t)S * N * E * 4) + fw::up((size_t)N * k * I * (dt == MOE_BF16 ? 2 : 4));
}

hipError_t launch_layer_few(moe_dtype dt, const void* x, const float* wr, const float* bias, const void* wg,
                            const void* gs, const void* wu, const void* us, const void* wd, const void* ds, int N,
                            int H, int I, int E, int k, void* out, int32_t* idx, float* w, void* ws, hipStream_t s) {
  using namespace fw;
  if (N == 0) return hipSuccess;
  Args a{};
  a.x = x; a.wr = wr; a.bias = bias; a.wg = wg; a.wu = wu; a.wd = wd;
  a.gs = (const uint8_t*)gs; a.us = (const uint8_t*)us; a.ds = (const uint8_t*)ds;
  a.N = N; a.H = H; a.I = I; a.E = E; a.k = k; a.out = out; a.idx = idx; a.w = w;
  slices(N, H, E, a.S, a.hs);
  a.part = (float*)ws;
  a.act = (char*)ws + up((size_t)a.S * N * E * 4);
  if (gs) return run_pl<bf16_t, true>(a, s);
  return dt == MOE_BF16 ? run_pl<bf16_t, false>(a, s) : run_pl<float, false>(a, s);
}

}  // namespace moe
