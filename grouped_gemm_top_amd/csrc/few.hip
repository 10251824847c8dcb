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
//  2. gate/up: for a single token every workgroup joins the slices and chooses the experts itself (for more a launch
//     of its own does, a workgroup per token), then takes tasks (expert, 16 columns of I).  Its eight wavefronts split
//     H (fewer, with several tasks at a time, where H is short), weights go straight from memory into registers as
//     the matrix instruction's operand, and the sums meet in LDS; a' = w silu(g) u is rounded once, as the next
//     product's operand (bf16: out is then off by 0.0023-0.0025 of its norm, 0.0017 of it its own rounding);
//  3. down: a workgroup owns 8 to 16 outputs of every token, or a part of the experts for them; its
//     wavefronts take the experts in turn and add each one's products to their tokens' sums in LDS.  No
//     floating-point atomics, one fixed order.
// One launch for 2 and 3, whose workgroups draw their tasks from a counter and where those of the down product wait
// for gate/up's, took 57 us at N = 1 against 18: some hundred draws from one address, 40 ns each, are the time.
//
// Measured (E = 128, H = 2048, I = 512, k = 8): N = 1 20.7 us a call, launches 3.3 + 11.7 + 5.8.  51 MB take 10 us
// at copy rate; the rest are three starts (2.7 each with nothing to do) and the choice (2).  N = 16, E = 256: 644 MB in
// 115 us, 5.5 TB/s.  fp32, N = 61, E = 64, H = 1432, I = 520, k = 4: 562 MB in 148-155; N = 1 as above: 38.  MX-FP8: N = 1 19,
// N = 24, E = 256, H = 4096, I = 256: 447 MB in 112.  Beyond a token or two what is above the stream is the router and the choice (12 us)
// and gate/up's last round of tasks (2112 over 512 workgroups: four rounds and an eighth); cutting that round's tasks along
// H, with their parts joined by a ticket, cost 2 to 10 % on most shapes.
#include <type_traits>

#include "gemm_lds.h"

namespace moe {
namespace fw {

using namespace gk;

constexpr int MAXN = MOE_FEW_MAX_TOKENS, MAXK = MOE_FEW_MAX_K, MAXE = 1024;
constexpr int NW = 8, NT = 64 * NW;  // wavefronts and threads of the two product kernels
constexpr int MAXP = 4;  // parts of the down product

struct Args {
  const void* x;
  const float* wr;
  const float* bias;
  const void *wg, *wu, *wd;
  const uint8_t *gs, *us, *ds;  // MX-FP8: scale codes
  int N, H, I, E, k;
  int S, hs;         // slices of the router product and their length
  int ws;            // wavefronts that share a gate/up task
  int rb, P;         // outputs of a down workgroup (8 to 16) and parts of its sum
  float* part;       // [S, N, E]
  void* act;         // a' [N k, I]: rows by expert, then token (N = 1: by slot)
  float* dpart;      // P > 1: [H / rb, P, N, 16]
  unsigned* ticket;  // P > 1: [H / rb], zeroed by the router's launch
  int32_t* idx;      // [N, k]
  float* w;          // [N, k]
  void* out;         // [N, H]
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
  if (a.ticket && blockIdx.y == 0 && blockIdx.z == 0)
    for (int q = s * 256 + threadIdx.x; q < (a.H + a.rb - 1) / a.rb; q += 256 * a.S) a.ticket[q] = 0;
  // sixteen rows of w_r in flight, the first ones before x is staged
  const float* wp = a.wr + (size_t)lo * a.E + min(e, a.E - 1);
  float v[16];
  auto fetch = [&](int h) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = h + j < len ? wp[(size_t)(h + j) * a.E] : 0.f;
  };
  fetch(16 * w);
  // eight values of x a thread, two turns at most (a row's share ends with zeros: H and hs are multiples of 8)
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int q = threadIdx.x + 256 * u, t = q >> 5, h = (q & 31) * 8;
    if (t < nt) {
      float4 p[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
      if (h < len) {
        const T* src = static_cast<const T*>(a.x) + (size_t)(t0 + t) * a.H + lo + h;
        load4(src, p[0].x, p[0].y, p[0].z, p[0].w);
        load4(src + 4, p[1].x, p[1].y, p[1].z, p[1].w);
      }
      *reinterpret_cast<float4*>(&s_x[t][h]) = p[0];
      *reinterpret_cast<float4*>(&s_x[t][h + 4]) = p[1];
    }
  }
  __syncthreads();
  float acc[16];
#pragma unroll
  for (int t = 0; t < 16; ++t) acc[t] = 0.f;
  for (int h = 16 * w; h < len; h += 64) {
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      if (t >= nt) break;
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        const float4 xv = *reinterpret_cast<const float4*>(&s_x[t][h + j]);
        acc[t] = __builtin_fmaf(xv.x, v[j], acc[t]);
        acc[t] = __builtin_fmaf(xv.y, v[j + 1], acc[t]);
        acc[t] = __builtin_fmaf(xv.z, v[j + 2], acc[t]);
        acc[t] = __builtin_fmaf(xv.w, v[j + 3], acc[t]);
      }
    }
    if (h + 64 < len) fetch(h + 64);
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

// A token by one wavefront, from z[q] = the logit (without its bias) of expert L + 64 q: lane j < k gets slot j's
// expert and weight.  A NaN logit counts as -inf; weights of experts at -inf are 0 (all of a token's, where it
// has no other).
template <int PL>  // experts per lane: E <= 64 PL
__device__ __forceinline__ void choose_experts(const Args& a, float (&z)[PL], int L, int& my_e, float& my_w) {
  uint32_t avail = 0;
#pragma unroll
  for (int q = 0; q < PL; ++q) {
    if (L + 64 * q < a.E) avail |= 1u << q;
    if (a.bias) z[q] += a.bias[min(L + 64 * q, a.E - 1)];
    z[q] = z[q] == z[q] ? z[q] : -INFINITY;
  }
  float myz = -INFINITY, z0 = 0.f;
  my_e = 0;
#pragma unroll 1
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
    if (L == j) myz = m, my_e = e;
    if (j == 0) z0 = m;
  }
  const float zm = z0 == -INFINITY ? 0.f : z0;
  const float ex = L < a.k ? expf(myz - zm) : 0.f;
  float sum = ex;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
  my_w = sum == 0.f ? 0.f : ex / sum;
}
// z[q] += the slices s0, s0 + step, ... of token t
template <int PL>
__device__ __forceinline__ void join_slices(const Args& a, int t, int s0, int step, int L, float (&z)[PL]) {
  constexpr int B = PL <= 2 ? 16 : PL <= 4 ? 8 : 4;  // in flight
#pragma unroll 1
  for (int i0 = s0; i0 < a.S; i0 += step * B) {
    float v[PL][B];
#pragma unroll
    for (int q = 0; q < PL; ++q)
#pragma unroll
      for (int i = 0; i < B; ++i)
        v[q][i] = a.part[((size_t)min(i0 + step * i, a.S - 1) * a.N + t) * a.E + min(L + 64 * q, a.E - 1)];
#pragma unroll
    for (int q = 0; q < PL; ++q)
#pragma unroll
      for (int i = 0; i < B; ++i) z[q] += i0 + step * i < a.S ? v[q][i] : 0.f;
  }
}

// The choice as a launch of its own (more than one token): a workgroup per token, whose four wavefronts share the
// slices.  (Made in every gate/up workgroup instead: N = 8, H = 4096, I = 256, E = 256, k = 2 43 us, 38 with the
// launch; N = 4, H = 2048, I = 512, E = 128, k = 8 51.4, 51.8; N = 2 35.5, 35.9.)
template <int PL>
__global__ __launch_bounds__(256) void k_few_choose(Args a) {
  __shared__ float s_z[4][64 * PL];
  const int t = blockIdx.x, w = threadIdx.x >> 6, L = threadIdx.x & 63;
  float z[PL], wt;
#pragma unroll
  for (int q = 0; q < PL; ++q) z[q] = 0.f;
  join_slices<PL>(a, t, w, 4, L, z);
#pragma unroll
  for (int q = 0; q < PL; ++q) s_z[w][L + 64 * q] = z[q];
  __syncthreads();
  if (w > 0) return;
#pragma unroll
  for (int q = 0; q < PL; ++q) z[q] = (z[q] + s_z[1][L + 64 * q]) + (s_z[2][L + 64 * q] + s_z[3][L + 64 * q]);
  int e;
  choose_experts<PL>(a, z, L, e, wt);
  if (L < a.k) {
    a.idx[t * a.k + L] = e;
    a.w[t * a.k + L] = wt;
  }
}

// A single token: the eight wavefronts share the slices, then every expert's rank is counted against the others
// (z descending, expert ascending), which takes no rounds one after the other.
struct One {  // in LDS
  __attribute__((aligned(16))) float z[NW][MAXE];
  int rank[MAXE];
  int e[MAXK];
};
template <int PL>
__device__ __forceinline__ void choose_one(const Args& a, One& s, int w, int L) {
  constexpr int EP = 64 * PL;
  const int tid = threadIdx.x;
  float z[PL];
#pragma unroll
  for (int q = 0; q < PL; ++q) z[q] = 0.f;
  join_slices<PL>(a, 0, w, NW, L, z);
#pragma unroll
  for (int q = 0; q < PL; ++q) s.z[w][L + 64 * q] = z[q];
  for (int e = tid; e < EP; e += NT) s.rank[e] = 0;
  __syncthreads();
  for (int e = tid; e < EP; e += NT) {
    float v = s.z[0][e];
#pragma unroll
    for (int q = 1; q < NW; ++q) v += s.z[q][e];
    if (a.bias && e < a.E) v += a.bias[e];
    s.z[0][e] = v == v && e < a.E ? v : -INFINITY;
  }
  __syncthreads();
  constexpr int PARTS = EP >= NT ? 1 : NT / EP, PER = EP / PARTS;
  for (int q = tid; q < EP * PARTS; q += NT) {
    const int e = q % EP, f0 = q / EP * PER;
    const float ze = s.z[0][e];
    int c = 0;
    // (| and &: no branches.  What stands behind the last expert is -inf and behind everything.)
#pragma unroll 4
    for (int f = f0; f < f0 + PER; f += 4) {
      const float4 v = *reinterpret_cast<const float4*>(&s.z[0][f]);
      c += (int)((v.x > ze) | ((v.x == ze) & (f < e)));
      c += (int)((v.y > ze) | ((v.y == ze) & (f + 1 < e)));
      c += (int)((v.z > ze) | ((v.z == ze) & (f + 2 < e)));
      c += (int)((v.w > ze) | ((v.w == ze) & (f + 3 < e)));
    }
    if (PARTS == 1) s.rank[e] = c;
    else atomicAdd(&s.rank[e], c);
  }
  __syncthreads();
  for (int e = tid; e < a.E; e += NT)
    if (s.rank[e] < a.k) s.e[s.rank[e]] = e;
  __syncthreads();
}
// slot L's weight (lanes < k), from what choose_one left
__device__ __forceinline__ float weight_one(const Args& a, const One& s, int L) {
  const float z0 = s.z[0][s.e[0]], zm = z0 == -INFINITY ? 0.f : z0;
  const float ex = L < a.k ? expf(s.z[0][s.e[L < a.k ? L : 0]] - zm) : 0.f;
  float sum = ex;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
  return sum == 0.f ? 0.f : ex / sum;
}

struct Lists {  // in LDS
  unsigned long long mask[MAXE];  // the tokens that name an expert
  uint16_t exp[MAXE];             // active experts, ascending
  uint16_t row[MAXE];             // an expert's first row of a'
  uint16_t idx[MAXN * MAXK];      // [N, k]
  uint8_t tok[MAXN * MAXK];       // a row's token
  int scan[NW];
  int n;                          // active experts
};

// From s.idx (behind a barrier): the experts' tokens and rows.  Ends with a barrier.
__device__ __forceinline__ void make_lists(const Args& a, Lists& s, int w, int L) {
  const int tid = threadIdx.x, np = a.N * a.k;
  for (int e = tid; e < MAXE; e += NT) s.mask[e] = 0;
  __syncthreads();
  for (int p = tid; p < np; p += NT) atomicOr(&s.mask[s.idx[p]], 1ull << (p / a.k));
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
  if (m0) s.exp[before >> 16] = (uint16_t)(2 * tid), s.row[2 * tid] = (uint16_t)before;
  before += c0;
  if (m1) s.exp[before >> 16] = (uint16_t)(2 * tid + 1), s.row[2 * tid + 1] = (uint16_t)before;
  if (tid == NT - 1) s.n = (before + c1) >> 16;
  __syncthreads();
  for (int p = tid; p < np; p += NT) {
    const int t = p / a.k, e = s.idx[p];
    s.tok[s.row[e] + __popcll(s.mask[e] & ((1ull << t) - 1))] = (uint8_t)t;
  }
  __syncthreads();
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
// two e4m3 codes (the low or the high half of w) times the power of two x, in bf16
template <bool HI>
__device__ __forceinline__ uint32_t mx2(uint32_t w, float x) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, x, HI));
}
template <typename T, bool F8>
__device__ __forceinline__ f32x4 line_mma(const Line<T, F8>& w, const Vec<T, F8>& x, f32x4 acc, int g) {
  if constexpr (F8) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // block 2 h + (g >> 1) of the line's four
      const float c = __uint_as_float(((w.s >> (16 * h + 8 * (g >> 1))) & 255u) << 23);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t u0 = w.v[h][2 * q], u1 = w.v[h][2 * q + 1];
        const u32x4 f = {mx2<false>(u0, c), mx2<true>(u0, c), mx2<false>(u1, c), mx2<true>(u1, c)};
        acc = mma(__builtin_bit_cast(bf16x8, f), __builtin_bit_cast(bf16x8, x.v[2 * h + q]), acc);
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
// k-steps in flight: as many as 128 registers hold, for two workgroups a compute unit are worth more than longer bursts
// (N = 24 on MX-FP8 weights: 59 us with one step, 74 with four in twice the registers; N = 61 in fp32: 79 and 98)
constexpr int lines_ahead(bool f8, int TB) { return f8 ? (TB > 1 ? 1 : 2) : TB > 2 ? 1 : 4; }

// TB: blocks of 16 tokens (N <= 16 TB; 0: N = 1).  PL: experts per lane of the choice, which is made here for a single
// token (0: it was made before).  GRP: a.ws wavefronts share a task and a workgroup takes NW / a.ws of them at a time (see
// shares()); else all of them one.
template <typename T, bool F8, int PL, int TB_, bool GRP>
__global__ __launch_bounds__(NT, PL == 16 ? 2 : 4) void k_few_gateup(Args a) {
  using Ln = Line<T, F8>;
  constexpr bool ONE = TB_ == 0;
  constexpr int TB = ONE ? 1 : TB_;
  constexpr int U = lines_ahead(F8, TB);
  __shared__ typename std::conditional<ONE, One, Lists>::type s;
  __shared__ f32x4 s_sum[NW][2][64];
  __shared__ float s_w[MAXN * MAXK];
  const int L = threadIdx.x & 63, w = ufl(threadIdx.x >> 6);
  const int r = L & 15, g = L >> 4;
  int n = a.k;
  if constexpr (ONE) {
    choose_one<PL>(a, s, w, L);
  } else {
    for (int p = threadIdx.x; p < a.N * a.k; p += NT) {
      s.idx[p] = (uint16_t)a.idx[p];
      s_w[p] = a.w[p];
    }
    __syncthreads();
    make_lists(a, s, w, L);
    n = ufl(s.n);
  }
  const int IB = (a.I + 15) / 16, tasks = n * IB;
  const int KS = 4 * ((a.H + 127) / 128);
  constexpr size_t ES = F8 ? 1 : sizeof(T);
  const int WS = GRP ? a.ws : NW, per = GRP ? NW / WS : 1, sub = GRP ? w / WS : 0, wi = GRP ? w - sub * WS : w;
  for (int first = blockIdx.x * per; first < tasks; first += (int)gridDim.x * per) {
    const bool on = !GRP || first + sub < tasks;  // (a wavefront without a task takes the last one and stores nothing)
    const int task = GRP ? min(first + sub, tasks - 1) : first;
    const int ai = task / IB, i0 = (task - ai * IB) * 16;
    int e, row0, cnt, nb;
    if constexpr (ONE) {
      e = ufl(s.e[ai]);
      row0 = ai;
      cnt = nb = 1;
    } else {
      e = ufl(s.exp[ai]);
      row0 = ufl(s.row[e]);
      cnt = ufl(__popcll(s.mask[e]));
      nb = (cnt + 15) / 16;
    }
    const size_t row = (size_t)e * a.I + min(i0 + r, a.I - 1);
    const char* pg = static_cast<const char*>(a.wg) + row * a.H * ES;
    const char* pu = static_cast<const char*>(a.wu) + row * a.H * ES;
    const uint8_t* sg = F8 ? a.gs + row * KS : nullptr;
    const uint8_t* su = F8 ? a.us + row * KS : nullptr;
    auto x_row = [&](int b) __attribute__((always_inline)) {
      const T* p = static_cast<const T*>(a.x);
      if constexpr (!ONE) p += (size_t)s.tok[row0 + min(16 * b + r, cnt - 1)] * a.H;
      return p;
    };
    const T* px = x_row(0);
    f32x4 ag[TB], au[TB];
#pragma unroll
    for (int b = 0; b < TB; ++b) ag[b] = au[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int k0 = wi * Ln::K; k0 < a.H; k0 += U * WS * Ln::K) {
      Ln lg[U], lu[U];
      Vec<T, F8> xv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * WS * Ln::K;
        lg[u].load(pg, sg, k, a.H, g);
        lu[u].load(pu, su, k, a.H, g);
        xv[u].load(px, k, a.H, g);
      }
      if constexpr (ONE) {  // the weights, while the first lines are on their way
        if (w == 0 && k0 == 0 && task == (int)blockIdx.x) {
          const float wt = weight_one(a, s, L);
          if (L < a.k) {
            s_w[L] = wt;
            if (blockIdx.x == 0) {
              a.idx[L] = s.e[L];
              a.w[L] = wt;
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        ag[0] = line_mma(lg[u], xv[u], ag[0], g);
        au[0] = line_mma(lu[u], xv[u], au[0], g);
      }
#pragma unroll
      for (int b = 1; b < TB; ++b) {
        if (b >= nb) break;
        const T* pb = x_row(b);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          Vec<T, F8> xb;
          xb.load(pb, k0 + u * WS * Ln::K, a.H, g);
          ag[b] = line_mma(lg[u], xb, ag[b], g);
          au[b] = line_mma(lu[u], xb, au[b], g);
        }
      }
    }
    // the wavefronts' sums in wavefront order; lane l of a task's first: columns i0 + 4 (l >> 4) + v, token slot l & 15
#pragma unroll
    for (int b = 0; b < TB; ++b) {
      if (GRP ? 16 * b >= a.N : b >= nb) break;  // (the same for all wavefronts)
      s_sum[w][0][L] = ag[b];
      s_sum[w][1][L] = au[b];
      __syncthreads();
      if (wi == 0 && on) {
        f32x4 G = s_sum[w][0][L], Uv = s_sum[w][1][L];
#pragma unroll
        for (int q = 1; q < NW; ++q) {
          if (GRP && q >= WS) break;
          G += s_sum[w + q][0][L];
          Uv += s_sum[w + q][1][L];
        }
        const int slot = 16 * b + r, i = i0 + 4 * g;
        if (slot < cnt && i < a.I) {
          float wt = 0.f;
          if constexpr (ONE) {
            wt = s_w[ai];
          } else {
            const int t = s.tok[row0 + slot];
            for (int j = 0; j < a.k; ++j)
              if (s.idx[t * a.k + j] == e) wt = s_w[t * a.k + j];
          }
          T* o = static_cast<T*>(a.act) + (size_t)(row0 + slot) * a.I + i;
          store4(o, wt * silu(G[0]) * Uv[0], wt * silu(G[1]) * Uv[1], wt * silu(G[2]) * Uv[2], wt * silu(G[3]) * Uv[3]);
        }
      }
      __syncthreads();
    }
  }
}

// ------------------------------------------------------------------ down
// Part p of the outputs h0 .. h0 + rb - 1 of all tokens.  A unit is an expert's share of k-steps (all of them,
// unless there are fewer experts than wavefronts); a wavefront takes every eighth unit of its part and adds each
// unit's products to its own [token][output] sums in LDS; the wavefronts' and the parts' sums meet in order.
template <typename T, bool F8, int TB_>
__global__ __launch_bounds__(NT, 4) void k_few_down(Args a) {
  using Ln = Line<T, F8>;
  constexpr bool ONE = TB_ == 0;
  constexpr int TB = ONE ? 1 : TB_;
  constexpr int U = F8 || TB > 2 ? 2 : 4;  // k-steps in flight
  __shared__ typename std::conditional<ONE, int, Lists>::type s;
  __shared__ __attribute__((aligned(16))) float s_acc[NW][16 * TB][16];
  __shared__ int s_last;
  const int L = threadIdx.x & 63, w = ufl(threadIdx.x >> 6);
  const int r = L & 15, g = L >> 4;
  for (int q = L; q < 16 * TB * 4; q += 64) *reinterpret_cast<f32x4*>(&s_acc[w][0][4 * q]) = f32x4{0.f, 0.f, 0.f, 0.f};
  int n = a.k;
  if constexpr (!ONE) {
    for (int p = threadIdx.x; p < a.N * a.k; p += NT) s.idx[p] = (uint16_t)a.idx[p];
    __syncthreads();
    make_lists(a, s, w, L);
    n = ufl(s.n);
  }
  const int hb = blockIdx.x / a.P, p = blockIdx.x - hb * a.P, h0 = hb * a.rb;
  const int KS = 4 * ((a.I + 127) / 128), steps = (a.I + Ln::K - 1) / Ln::K;
  const int split = max(1, min(steps, (NW * a.P + n - 1) / n)), units = n * split;
  const int u_hi = (int)((long long)units * (p + 1) / a.P);
  constexpr size_t ES = F8 ? 1 : sizeof(T);
  const bool mine = r < a.rb && h0 + r < a.H;  // (rb < 16: the other lanes load nothing, and their sums are not used)
  for (int un = (int)((long long)units * p / a.P) + w; un < u_hi; un += NW) {
    const int ai = un / split, sp = un - ai * split;
    int e, row0, cnt, nb;
    if constexpr (ONE) {
      e = ufl(a.idx[ai]);
      row0 = ai;
      cnt = nb = 1;
    } else {
      e = ufl(s.exp[ai]);
      row0 = ufl(s.row[e]);
      cnt = ufl(__popcll(s.mask[e]));
      nb = (cnt + 15) / 16;
    }
    const int k_lo = steps * sp / split * Ln::K, k_hi = min(a.I, steps * (sp + 1) / split * Ln::K);
    const size_t row = (size_t)e * a.H + h0 + (mine ? r : 0);
    const char* pw = static_cast<const char*>(a.wd) + row * a.I * ES;
    const uint8_t* sw = F8 ? a.ds + row * KS : nullptr;
    const T* pa = static_cast<const T*>(a.act) + (size_t)(row0 + min(r, cnt - 1)) * a.I;
    f32x4 d[TB];
#pragma unroll
    for (int b = 0; b < TB; ++b) d[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int k0 = k_lo; k0 < k_hi; k0 += U * Ln::K) {
      Ln l[U];
      Vec<T, F8> v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        l[u].load(pw, sw, k0 + u * Ln::K, mine ? k_hi : 0, g);
        v[u].load(pa, k0 + u * Ln::K, k_hi, g);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) d[0] = line_mma(l[u], v[u], d[0], g);
#pragma unroll
      for (int b = 1; b < TB; ++b) {
        if (b >= nb) break;
        const T* pb = static_cast<const T*>(a.act) + (size_t)(row0 + min(16 * b + r, cnt - 1)) * a.I;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          Vec<T, F8> vb;
          vb.load(pb, k0 + u * Ln::K, k_hi, g);
          d[b] = line_mma(l[u], vb, d[b], g);
        }
      }
    }
    // d[b][v] = output h0 + 4 g + v of the expert's token slot 16 b + r
#pragma unroll
    for (int b = 0; b < TB; ++b) {
      if (16 * b + r < cnt) {
        int t = 0;
        if constexpr (!ONE) t = s.tok[row0 + 16 * b + r];
        f32x4* q = reinterpret_cast<f32x4*>(&s_acc[w][t][4 * g]);
        *q = *q + d[b];
      }
    }
  }
  __syncthreads();
  for (int q = threadIdx.x; q < a.N * 16; q += NT) {
    const int t = q >> 4, o = q & 15;
    float v = s_acc[0][t][o];
#pragma unroll
    for (int i = 1; i < NW; ++i) v += s_acc[i][t][o];
    if (a.P == 1) {
      if (o < a.rb && h0 + o < a.H) static_cast<T*>(a.out)[(size_t)t * a.H + h0 + o] = from_f32<T>(v);
    } else {
      __hip_atomic_store(&a.dpart[((size_t)blockIdx.x * a.N + t) * 16 + o], v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  if (a.P == 1) return;
  // The part that arrives last adds the parts in order.  Each share was stored with device scope and has
  // arrived (the wait) before the workgroup's ticket is drawn, and is read with device scope.
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0)
    s_last = __hip_atomic_fetch_add(a.ticket + hb, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (unsigned)a.P - 1;
  __syncthreads();
  if (!s_last) return;
  for (int q = threadIdx.x; q < a.N * 16; q += NT) {
    const int t = q >> 4, o = q & 15;
    float v = 0.f, b[MAXP];
#pragma unroll
    for (int i = 0; i < MAXP; ++i)
      b[i] = __hip_atomic_load(&a.dpart[(((size_t)hb * a.P + min(i, a.P - 1)) * a.N + t) * 16 + o], __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
    for (int i = 0; i < MAXP; ++i) v += i < a.P ? b[i] : 0.f;
    if (o < a.rb && h0 + o < a.H) static_cast<T*>(a.out)[(size_t)t * a.H + h0 + o] = from_f32<T>(v);
  }
}

// ------------------------------------------------------------------ host side
size_t up(size_t n) { return (n + 255) / 256 * 256; }

// slices of the router product: 32 to 256 of H each, and no more than a lane joins with one round of loads
void slices(int N, int H, int E, int& S, int& hs) {
  const int most = N > 1 ? 64 : E <= 128 ? 32 : 16;
  S = H / 32;
  if (S > most) S = most;
  if (S < 1) S = 1;
  if (S < (H + 255) / 256) S = (H + 255) / 256;
  hs = ((H + S - 1) / S + 15) / 16 * 16;
}

// Wavefronts that share a gate/up task: eight, unless H has no U lines for each and there are tasks for all workgroups
// all the same (MX-FP8, H = 160, N = 43, E = 190, I = 1120, k = 7: the call 73 us, 99 with eight; H = 224, N = 37, E = 133,
// I = 1536: 80, 105).  tasks: at most, U: lines in flight, K: values of a line
int shares(int H, long long tasks, int U, int K) {
  const int lines = (H + K - 1) / K;
  int n = NW;
  while (n > 1 && U * n / 2 >= lines && tasks * n >= 512 * NW * 2) n /= 2;
  return n;
}

// The down product's workgroups.  Few tokens, where the launch is a matter of latency and a join of parts costs 3
// us: 8 outputs each, parts only where that leaves half the chip idle.  Else the outputs (8 to 16) and parts (up to
// MAXP) with the least time of the fullest compute unit: its share of the matrices at 20 KB a us, and 4 us for each
// turn of two workgroups (its lists, its join); where equal, the most workgroups, and then the most outputs, as a lane
// without one loads nothing (H = 1432, N = 61: 480 workgroups of 12 outputs in four parts 59 us, 480 of 9 in three 69,
// 360 of 16 67; H = 2048, N = 16, E = 256: 16 outputs in four parts 35, 8 in two 46; little to read, H = 3160, N = 26,
// E = 9, I = 104: the call 29 us with 488 workgroups, 37 with 1264).
// row: the bytes that an output takes from all experts' matrices
void parts(int N, int H, double row, int& rb, int& P) {
  if (N <= 2) {
    rb = H < 4096 ? 8 : 16;
    const int hb = (H + rb - 1) / rb;
    P = hb >= 128 ? 1 : (128 + hb - 1) / hb;
    if (P > MAXP) P = MAXP;
    return;
  }
  double best = 1e30;
  long long most = 0;
  for (int p = MAXP; p >= 1; --p)
    for (int r = 16; r >= 8; --r) {
      const long long wg = (long long)((H + r - 1) / r) * p;
      const double t = (double)((wg + 255) / 256) * r / p * row / 20e3 + 4.0 * (double)((wg + 511) / 512);
      if (t < best || (t == best && wg > most)) best = t, most = wg, rb = r, P = p;
    }
}

template <typename T, bool F8, int PL, int TB>
hipError_t run(Args a, hipStream_t s) {
  const dim3 gr(a.S, (a.E + 63) / 64, (a.N + 15) / 16);
  hipLaunchKernelGGL(k_few_router<T>, gr, dim3(256), 0, s, a);
  const long long act = a.E < a.N * a.k ? a.E : a.N * a.k, tasks = act * ((a.I + 15) / 16);
  const dim3 gg((unsigned)(tasks < 512 ? tasks : 512));
  if constexpr (TB == 0) {
    hipLaunchKernelGGL((k_few_gateup<T, F8, PL, 0, false>), gg, dim3(NT), 0, s, a);
  } else {
    hipLaunchKernelGGL(k_few_choose<PL>, dim3(a.N), dim3(256), 0, s, a);
    a.ws = shares(a.H, tasks, lines_ahead(F8, TB), Line<T, F8>::K);
    if (a.ws < NW) hipLaunchKernelGGL((k_few_gateup<T, F8, 0, TB, true>), gg, dim3(NT), 0, s, a);
    else hipLaunchKernelGGL((k_few_gateup<T, F8, 0, TB, false>), gg, dim3(NT), 0, s, a);
  }
  hipLaunchKernelGGL((k_few_down<T, F8, TB>), dim3((a.H + a.rb - 1) / a.rb * a.P), dim3(NT), 0, s, a);
  return hipGetLastError();
}
template <typename T, bool F8, int PL>
hipError_t run_tb(const Args& a, hipStream_t s) {
  if (a.N == 1) return run<T, F8, PL, 0>(a, s);
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

struct Ws {
  int S, hs, rb, P;
  size_t part, act, dpart, ticket;
  Ws(moe_dtype dt, int N, int E, int k, int H, int I) {
    slices(N, H, E, S, hs);
    // (MX-FP8 weights count as bf16's, so that one workspace serves both)
    parts(N, H, (double)(E < N * k ? E : N * k) * I * (dt == MOE_BF16 ? 2 : 4), rb, P);
    const int hb = (H + rb - 1) / rb;
    part = up((size_t)S * N * E * 4);
    act = up((size_t)N * k * I * (dt == MOE_BF16 ? 2 : 4));
    dpart = P > 1 ? up((size_t)hb * P * N * 64) : 0;
    ticket = P > 1 ? up((size_t)hb * 4) : 0;
  }
  size_t total() const { return 256 + part + act + dpart + ticket; }
};

}  // namespace fw

size_t layer_few_ws_bytes(moe_dtype dt, int N, int E, int k, int H, int I) { return fw::Ws(dt, N, E, k, H, I).total(); }

hipError_t launch_layer_few(moe_dtype dt, const void* x, const float* wr, const float* bias, const void* wg,
                            const void* gs, const void* wu, const void* us, const void* wd, const void* ds, int N,
                            int H, int I, int E, int k, void* out, int32_t* idx, float* w, void* ws, hipStream_t s) {
  using namespace fw;
  if (N == 0) return hipSuccess;
  const Ws b(dt, N, E, k, H, I);
  Args a{};
  a.x = x; a.wr = wr; a.bias = bias; a.wg = wg; a.wu = wu; a.wd = wd;
  a.gs = (const uint8_t*)gs; a.us = (const uint8_t*)us; a.ds = (const uint8_t*)ds;
  a.N = N; a.H = H; a.I = I; a.E = E; a.k = k; a.out = out; a.idx = idx; a.w = w;
  a.S = b.S; a.hs = b.hs; a.rb = b.rb; a.P = b.P;
  char* p = static_cast<char*>(ws);
  a.part = (float*)p;
  a.act = p + b.part;
  a.dpart = (float*)(p + b.part + b.act);
  a.ticket = b.P > 1 ? (unsigned*)(p + b.part + b.act + b.dpart) : nullptr;
  if (gs) return run_pl<bf16_t, true>(a, s);
  return dt == MOE_BF16 ? run_pl<bf16_t, false>(a, s) : run_pl<float, false>(a, s);
}

}  // namespace moe
