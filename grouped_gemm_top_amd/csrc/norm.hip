// norm.hip -- residual addition with RMS norm, its MX-FP8 output and its backward, for gfx950.
//
//   s = x + res (fp32),  h = s rounded to the residual stream's type
//   r = (sum_c s_c^2 / H + eps)^(-1/2),  y_c = s_c r w_c
//   MX-FP8 output: y (fp32, before any rounding) in blocks of 32 values along the row, each with
//   the smallest power of two X that has max |y| <= 448 X as its scale, the codes e4m3(y / X).
//   The codes come from the fp32 y rather than from the rounded y: one rounding instead of two.
//
//   backward, from the stored h:  r = (sum_c h_c^2 / H + eps)^(-1/2),  a_c = dy_c w_c,
//   dh_c = r a_c - r^3 (sum_c a_c h_c / H) h_c + dh_in_c,   dw_c = sum_t dy_tc h_tc r_t
//   (r is taken again from h: the row is read anyway and both sums leave in one reduction, so
//   nothing has to be kept from the forward and the gradient is that of the norm at the stored h)
//
// Both are streaming kernels bound by HBM: each input is read once and each output written once,
// a row stays in registers between the reduction and the result.  Measured on one MI355X, beside a copy
// that moves as many bytes: forward with codes 95 us (copy 98) for 520 MB (N = 16383, H = 2880, fp32 stream) and
// 14.1 us (10.9: part of it stays in the 256 MB cache) for 76 MB (N = 4096, H = 2048); backward 170 + 5 us (177)
// for 940 MB (N = 16384, H = 4096, fp32 stream) and 15.0 + 4 us (9.9) for 67 MB (N = 4096, H = 2048); the second
// launch adds dw's partial rows.  One row (N = 1, H = 2048) is 3 us: a launch and two trips to memory.
// Narrow rows leave lanes idle, a wavefront holds one row: N = 131072, H = 128 forward 51, backward 69 us (26.5);
// N = 32768, H = 64 11 and 19 us (4.0); from H = 512 on all lanes work (N = 32768: 24.4 and 25.4 us, 26.6).
//
// Lane l of the WR wavefronts that share a row holds the 8-value chunks l, l + 64 WR, ... (V of
// them): 16-byte accesses in bf16, two in fp32, and an MX-FP8 block is four neighbouring lanes.
#include "common.h"

namespace moe {
namespace nm {

// eight consecutive values as fp32 (16-byte aligned)
__device__ __forceinline__ void ld8(const bf16_t* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void ld8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pk2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
__device__ __forceinline__ void st8(bf16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pk2(v[0], v[1]), pk2(v[2], v[3]), pk2(v[4], v[5]), pk2(v[6], v[7]));
}
__device__ __forceinline__ void st8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}
// maximum over each group of four neighbouring lanes (quad permutations)
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xF, 0xF, false)));
  return fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xF, 0xF, false)));
}

struct FwdArgs {
  const void* x;
  const void* res;     // NULL: none
  const float* w;      // NULL: ones
  void* h;             // NULL: not written (may be res: every element is read before it is written)
  void* y;             // NULL: not written
  uint8_t* q;          // NULL: not written
  uint8_t* sc;
  long long N;
  int H;
  float eps;
};

// WR wavefronts per row, V chunks of 8 values per lane (H <= 512 WR V), 4 / WR rows per workgroup
// of 256 threads (one row per workgroup of 64 WR threads where WR > 4).
template <typename T, typename R, int WR, int V>
__global__ __launch_bounds__(WR > 4 ? 64 * WR : 256) void k_add_rmsnorm(FwdArgs a) {
  constexpr int RPB = WR > 4 ? 1 : 4 / WR;
  __shared__ float red[RPB][WR];
  const int wv = threadIdx.x >> 6, g = wv / WR, ww = wv % WR, L = threadIdx.x & 63;
  const long long row = (long long)blockIdx.x * RPB + g;
  const bool live = row < a.N;
  const int H = a.H, nc = H >> 3;
  const long long base = row * H;
  const T* x = static_cast<const T*>(a.x) + base;
  const R* res = a.res ? static_cast<const R*>(a.res) + base : nullptr;
  float s[V][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = L + 64 * (ww + WR * i);
    if (live && c < nc) {
      ld8(x + 8 * c, s[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] = 0.f;
    }
  }
  if (res) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = L + 64 * (ww + WR * i);
      if (live && c < nc) {
        float v[8];
        ld8(res + 8 * c, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[i][j] += v[j];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) ss += s[i][j] * s[i][j];
  ss = wave_sum(ss);
  if constexpr (WR > 1) {
    if (L == 0) red[g][ww] = ss;
    __syncthreads();
    ss = 0.f;
#pragma unroll
    for (int q = 0; q < WR; ++q) ss += red[g][q];
  }
  if (!live) return;
  const float r = 1.0f / sqrtf(ss / (float)H + a.eps);
  R* h = a.h ? static_cast<R*>(a.h) + base : nullptr;
  T* y = a.y ? static_cast<T*>(a.y) + base : nullptr;
  const int KS = 4 * ((H + 127) / 128);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = L + 64 * (ww + WR * i);
    if (c >= nc) continue;
    if (h) st8(h + 8 * c, s[i]);
    float o[8];
    if (a.w) {
      ld8(a.w + 8 * c, o);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = s[i][j] * r * o[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = s[i][j] * r;
    }
    if (y) st8(y + 8 * c, o);
    if (a.q) {  // H is a multiple of 32: the four lanes of a block are all here
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(o[j]));
      const int e = mx_scale_exp(quad_max(m));
      *reinterpret_cast<uint2*>(a.q + base + 8 * c) =
          make_uint2(mx_pack4(o[0], o[1], o[2], o[3], e), mx_pack4(o[4], o[5], o[6], o[7], e));
      if ((L & 3) == 0) a.sc[row * KS + (c >> 2)] = (uint8_t)(e + 127);
    }
  }
  // the scale row's padding entries
  if (a.q && ww == 0 && L < KS - H / 32) a.sc[row * KS + H / 32 + L] = 0;
}

struct BwdArgs {
  const void* dy;
  const void* h;
  const void* dh_in;  // NULL: zeros
  const float* w;     // NULL: ones
  void* dh;           // (may be dh_in)
  void* dx;           // NULL: not written; dh in the type of x
  float* part;        // [gridDim.x, H] column sums of dy h r over this workgroup's rows; NULL: not wanted
  long long N;
  int H;
  float eps;
};

// RG rows per workgroup of 64 WR RG threads at a time, WR wavefronts on each: rows blockIdx.x RG + g,
// then gridDim.x RG further on.  The column sums of dw stay in registers over a workgroup's rows
// and its RG groups' sums are added in order through LDS.
template <typename T, typename R, int WR, int V, int RG>
__global__ __launch_bounds__(64 * WR * RG) void k_add_rmsnorm_bwd(BwdArgs a) {
  __shared__ float2 red[2][RG][WR];
  __shared__ float4 s_dw[RG > 1 ? 64 * WR * V * 2 : 1];
  const int g = threadIdx.x / (64 * WR), tr = threadIdx.x % (64 * WR);
  const int ww = tr >> 6, L = threadIdx.x & 63;
  const int H = a.H, nc = H >> 3;
  float w[V][8], dw[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = tr + 64 * WR * i;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[i][j] = 1.f, dw[i][j] = 0.f;
    if (a.w && c < nc) ld8(a.w + 8 * c, w[i]);
  }
  int par = 0;
  // (every group makes the same number of turns: the barrier inside meets all wavefronts)
  for (long long r0 = (long long)blockIdx.x * RG; r0 < a.N; r0 += (long long)gridDim.x * RG, par ^= 1) {
    const long long row = r0 + g;
    const bool live = row < a.N;
    const long long base = row * H;
    const T* dy = static_cast<const T*>(a.dy) + base;
    const R* h = static_cast<const R*>(a.h) + base;
    const R* din = a.dh_in ? static_cast<const R*>(a.dh_in) + base : nullptr;
    float vh[V][8], vd[V][8], vi[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tr + 64 * WR * i;
#pragma unroll
      for (int j = 0; j < 8; ++j) vh[i][j] = 0.f, vd[i][j] = 0.f, vi[i][j] = 0.f;
      if (live && c < nc) {
        ld8(h + 8 * c, vh[i]);
        ld8(dy + 8 * c, vd[i]);
        if (din) ld8(din + 8 * c, vi[i]);
      }
    }
    float2 p = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p.x += vh[i][j] * vh[i][j];
        p.y += vd[i][j] * w[i][j] * vh[i][j];
      }
    p.x = wave_sum(p.x);
    p.y = wave_sum(p.y);
    if constexpr (WR > 1) {
      // two slots by turn: a wavefront writes a slot again only after the next turn's barrier
      if (L == 0) red[par][g][ww] = p;
      __syncthreads();
      p = make_float2(0.f, 0.f);
#pragma unroll
      for (int q = 0; q < WR; ++q) {
        const float2 t = red[par][g][q];
        p.x += t.x;
        p.y += t.y;
      }
    }
    const float r = 1.0f / sqrtf(p.x / (float)H + a.eps);
    const float m = r * r * (p.y / (float)H);
    if (!live) continue;  // (its wavefronts' sums took part in no other row)
    R* dh = static_cast<R*>(a.dh) + base;
    T* dx = a.dx ? static_cast<T*>(a.dx) + base : nullptr;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tr + 64 * WR * i;
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        o[j] = r * (vd[i][j] * w[i][j] - m * vh[i][j]) + vi[i][j];
        dw[i][j] += vd[i][j] * (vh[i][j] * r);
      }
      if (c < nc) {
        st8(dh + 8 * c, o);
        if (dx) st8(dx + 8 * c, o);
      }
    }
  }
  if (!a.part) return;
  if constexpr (RG > 1) {
    for (int q = 1; q < RG; ++q) {
      __syncthreads();
      if (g == q) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          s_dw[(i * 2) * 64 * WR + tr] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
          s_dw[(i * 2 + 1) * 64 * WR + tr] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
        }
      }
      __syncthreads();
      if (g == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float4 u = s_dw[(i * 2) * 64 * WR + tr], v = s_dw[(i * 2 + 1) * 64 * WR + tr];
          dw[i][0] += u.x; dw[i][1] += u.y; dw[i][2] += u.z; dw[i][3] += u.w;
          dw[i][4] += v.x; dw[i][5] += v.y; dw[i][6] += v.z; dw[i][7] += v.w;
        }
      }
    }
  }
  if (g == 0) {
    float* part = a.part + (size_t)blockIdx.x * H;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tr + 64 * WR * i;
      if (c < nc) st8(part + 8 * c, dw[i]);
    }
  }
}

// The column sums of G partial rows [G, H] (H a multiple of 4): a workgroup owns 32 columns; thread (g, c) sums the rows g,
// g + 128, ... of four columns, then the 128 sums are added in a fixed order.
__global__ __launch_bounds__(1024) void k_sum_rows(const float* __restrict__ part, int G, int H,
                                                    float* __restrict__ dw) {
  __shared__ float4 s[128][8];
  const int c = threadIdx.x & 7, g = threadIdx.x >> 3;
  const int col = blockIdx.x * 32 + 4 * c;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < H) {
#pragma unroll 4
    for (int q = g; q < G; q += 128) {
      const float4 u = *reinterpret_cast<const float4*>(part + (size_t)q * H + col);
      v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
    }
  }
#pragma unroll
  for (int n = 128; n > 8; n /= 4) {
    s[g][c] = v;
    __syncthreads();
    if (g < n / 4)
      for (int q = 1; q < 4; ++q) {
        const float4 u = s[g + q * (n / 4)][c];
        v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
      }
    __syncthreads();
  }
  // eight rows are left (128 / 4 / 4)
  if (g < 8) s[g][c] = v;
  __syncthreads();
  if (g == 0 && col < H) {
    for (int q = 1; q < 8; ++q) {
      const float4 u = s[q][c];
      v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
    }
    *reinterpret_cast<float4*>(dw + col) = v;
  }
}

__global__ __launch_bounds__(256) void k_fill0(float* __restrict__ p, int n) {
  for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) p[i] = 0.f;
}

// Wavefronts per row: as few values a lane as the row allows, so that a row's own latency is short.
// N = 16383, H = 2880, fp32 stream: 8 wavefronts of one chunk a lane 95 us, 4 of two 99, 2 of four
// 104, 1 of eight 115, 16 of one (two thirds idle) 126.  N = 1, H = 2048: 4 of one 3.0, 2 of two 3.6, 1 of four 4.5;
// at N = 4096 all three 12.1 - 12.4.
template <typename T, typename R>
void fwd(const FwdArgs& a, hipStream_t s) {
  const int nc = a.H / 8;
#define NORM_FWD(WR, V)                                                                              \
  hipLaunchKernelGGL((k_add_rmsnorm<T, R, WR, V>), dim3((unsigned)((a.N + (WR > 4 ? 1 : 4 / WR) - 1) / \
                                                                    (WR > 4 ? 1 : 4 / WR))),          \
                     dim3(WR > 4 ? 64 * WR : 256), 0, s, a)
  if (nc <= 64) NORM_FWD(1, 1);
  else if (nc <= 128) NORM_FWD(1, 2);
  else if (nc <= 256) NORM_FWD(4, 1);
  else if (nc <= 512) NORM_FWD(8, 1);
  else if (nc <= 1024) NORM_FWD(8, 2);
  else NORM_FWD(16, 2);
#undef NORM_FWD
}

template <typename T, typename R, int WR, int V, int RG>
void bwd1(const BwdArgs& a, int G, hipStream_t s) {
  hipLaunchKernelGGL((k_add_rmsnorm_bwd<T, R, WR, V, RG>), dim3(G), dim3(64 * WR * RG), 0, s, a);
}
// Rows per workgroup (bf16 us, fp32 stream in brackets): two of 4 wavefronts against one up to H =
// 2048 (N = 4096, H = 2048: 17.0 and 18.1; N = 16384: 54.4 and 60.3), one of 8 against two beyond
// (N = 4096, H = 2880: 24.6 and 28.4 [36.7 and 40.3]; N = 16384, H = 4096: 103.6 and 105.8 [175 and 172]).
template <typename T, typename R>
void bwd(const BwdArgs& a, int G, hipStream_t s) {
  const int nc = a.H / 8;
  if (nc <= 64) bwd1<T, R, 1, 1, 4>(a, G, s);
  else if (nc <= 128) bwd1<T, R, 2, 1, 4>(a, G, s);
  else if (nc <= 256) bwd1<T, R, 4, 1, 2>(a, G, s);
  else if (nc <= 512) bwd1<T, R, 8, 1, 1>(a, G, s);
  else if (nc <= 1024) bwd1<T, R, 8, 2, 1>(a, G, s);
  else bwd1<T, R, 16, 2, 1>(a, G, s);
}

// Workgroups of the backward.  Each leaves one partial row of dw: more of them hide more latency, but
// write and add more (N = 4096, H = 2048: 256 take 18.9 us, 512 17.0, 1024 19.5, 2048 23.7; N =
// 8192, H = 2880: 256 58.0, 512 41.9, 768 48.7, 1024 45.1).
int bwd_groups(long long N) { return (int)(N < 512 ? (N < 1 ? 1 : N) : 512); }

}  // namespace nm

void launch_sum_rows(const float* part, int G, int H, float* out, hipStream_t s) {
  hipLaunchKernelGGL(nm::k_sum_rows, dim3((unsigned)((H + 31) / 32)), dim3(1024), 0, s, part, G, H, out);
}

size_t add_rmsnorm_bwd_ws_bytes(int N, int H) { return (size_t)nm::bwd_groups(N) * H * 4; }

hipError_t launch_add_rmsnorm(moe_dtype dt, moe_dtype rdt, const void* x, const void* res, const float* w, float eps,
                              int N, int H, void* h, void* y, uint8_t* q, uint8_t* scales, hipStream_t s) {
  if (N == 0) return hipSuccess;
  // at most 2^21 rows a launch: 1024 threads a row stay below the 2^32 threads that one may have
  const long long slab = 1 << 21;
  const size_t xs = dt == MOE_F32 ? 4 : 2, rs = rdt == MOE_F32 ? 4 : 2, KS = 4 * ((H + 127) / 128);
  for (long long r0 = 0; r0 < N; r0 += slab) {
    auto at = [&](auto* p, size_t row_bytes) { return p ? (decltype(p))((uintptr_t)p + r0 * row_bytes) : p; };
    const nm::FwdArgs a{at(x, H * xs), at(res, H * rs), w, at(h, H * rs), at(y, H * xs), at(q, H), at(scales, KS),
                        N - r0 < slab ? N - r0 : slab, H, eps};
    if (dt == MOE_F32) nm::fwd<float, float>(a, s);
    else if (rdt == MOE_F32) nm::fwd<bf16_t, float>(a, s);
    else nm::fwd<bf16_t, bf16_t>(a, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_add_rmsnorm_bwd(moe_dtype dt, moe_dtype rdt, const void* dy, const void* h, const void* dh_in,
                                  const float* w, float eps, int N, int H, void* dh, void* dx, float* dw, void* ws,
                                  hipStream_t s) {
  if (N == 0) {
    if (dw) hipLaunchKernelGGL(nm::k_fill0, dim3(16), dim3(256), 0, s, dw, H);
    return hipGetLastError();
  }
  const int G = nm::bwd_groups(N);
  // one workgroup's column sums are dw itself
  float* part = dw ? (G == 1 ? dw : static_cast<float*>(ws)) : nullptr;
  const nm::BwdArgs a{dy, h, dh_in, w, dh, dx, part, N, H, eps};
  if (dt == MOE_F32) nm::bwd<float, float>(a, G, s);
  else if (rdt == MOE_F32) nm::bwd<bf16_t, float>(a, G, s);
  else nm::bwd<bf16_t, bf16_t>(a, G, s);
  if (dw && G > 1) launch_sum_rows(part, G, H, dw, s);
  return hipGetLastError();
}

}  // namespace moe
