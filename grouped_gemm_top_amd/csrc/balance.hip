// balance.hip -- the router's balance loss and z-loss with per-expert counts, and their gradient.
//
// Tokens seq_ptr[b] .. seq_ptr[b+1] - 1 that the mask leaves form sequence b, n_b of them, n in all.
// With z = logits + bias, p = softmax(z) over the experts, lse = log sum exp z, and c[b,e] the
// selections of expert e by sequence b's tokens:
//   L0 = alpha / B  sum_b  E / (k n_b^2)  sum_e c[b,e] sum_t p[t,e],      L1 = beta / n  sum_t lse_t^2
//   g[b,e] = alpha E c[b,e] / (B k n_b^2)      (dL0 / dp[t,e]; counts carry no gradient)
//   dz[t,m] = d0 p_m (g[b,m] - sum_e g[b,e] p_e) + d1 (2 beta / n) lse_t p_m
//
// Both directions read the logits once and are bound by that stream, small calls by launches.
// Measured on one MI355X (a copy moves 5.1 - 5.3 TB/s there): N = 65536, E = 256, k = 8, ragged and masked,
// forward 23.6 us + 5.8 us in k_balance_sum for 69 MB, gradient 27.4 us for 134 MB (4.9 TB/s); N = 4096, E = 128:
// 6.8 + 5.6 and 5.1 us, chains of a few dependent trips to memory; N = 64, E = 8: 5.1 and 2.5 us.
// A group of LP lanes holds one token's logits in registers (VW consecutive values per lane, Q
// times), so maximum, sum and dot product are a few lane exchanges and no LDS.
//
// Forward: workgroup i takes the tokens i T .. (i + 1) T - 1, whatever sequences they belong to,
// so ragged batches are balanced by construction.  It leaves one partial row of sums and counts
// per (workgroup i, sequence b) it meets, in slot i + b: along the batch neither i nor b decreases and
// at each new pair one of them or both grow, so slots are distinct.  k_balance_sum adds a sequence's slots in
// order (no floating-point atomics: bitwise reproducible), and its last workgroup, known by a
// ticket, adds the loss.  A call small enough for one workgroup finishes in one launch.
#include "common.h"

namespace moe {
namespace bl {

constexpr int NT = 256;

// ---- exchanges inside a group of LP lanes: every lane gets the group's result, in one fixed tree
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, false));
}
struct Add { __device__ static __forceinline__ float op(float a, float b) { return a + b; } };
struct Max { __device__ static __forceinline__ float op(float a, float b) { return fmaxf(a, b); } };
template <int LP, class O>
__device__ __forceinline__ float group(float v) {
  if constexpr (LP >= 2) v = O::op(v, dpp<0xB1>(v));    // lane ^ 1
  if constexpr (LP >= 4) v = O::op(v, dpp<0x4E>(v));    // lane ^ 2
  if constexpr (LP >= 8) v = O::op(v, dpp<0x141>(v));   // the other quad of eight lanes
  if constexpr (LP >= 16) v = O::op(v, dpp<0x140>(v));  // the other eight of sixteen
  if constexpr (LP >= 32) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = O::op(__uint_as_float(s[0]), __uint_as_float(s[1]));
  }
  if constexpr (LP >= 64) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = O::op(__uint_as_float(s[0]), __uint_as_float(s[1]));
  }
  return v;
}
// sum over the groups of a wavefront (lanes of equal position in their group)
template <int LP>
__device__ __forceinline__ float across(float v) {
#pragma unroll
  for (int off = LP; off < 64; off <<= 1) v += __shfl_xor(v, off);
  return v;
}

// e^x for x <= 0 as 2^(x log2 e), the part that the rounded product loses (its own rounding and log2 e's,
// up to |x| 2^-24) carried as a first-order factor: 5 units of 2^-24 at any x, where the product alone is off
// by up to 44 at x = -64.  Below -200, at -infinity too, it is 0; a NaN stays one.  Forward and gradient at
// N = 65536, E = 256 (one sequence, the same tensors again and again) take 29.9 + 23.7 us, with the product
// alone 29.1 + 23.1.
__device__ __forceinline__ float exp_neg(float x) {
  x = __builtin_elementwise_maximum(x, -200.f);
  const float c = 1.44269502162933349609f, c_lo = 1.92596299e-8f;  // log2 e = c + c_lo
  const float t = x * c;
  const float e = __builtin_fmaf(x, c_lo, __builtin_fmaf(x, c, -t));
  const float r = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(r, e * 0.6931471805599453f, r);
}

// The logits of one token, LP lanes: element (q LP + l) VW + v.  Positions past E hold -inf.
template <int VW, int LP, int Q>
__device__ __forceinline__ void load_row(const float* __restrict__ p, int E, int l, float fill, float (&z)[Q][VW]) {
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int e = (q * LP + l) * VW;
    if constexpr (VW == 4) {
      float4 u = make_float4(fill, fill, fill, fill);
      if (e < E) u = *reinterpret_cast<const float4*>(p + e);  // E is a multiple of 4 here
      z[q][0] = u.x; z[q][1] = u.y; z[q][2] = u.z; z[q][3] = u.w;
    } else {
      z[q][0] = e < E ? p[e] : fill;
    }
  }
}

// z -> e^(z - max) in place; the caller gets 1 / sum and the token's log sum exp (hardware
// reciprocal and logarithm, one unit in the last place each).  A token whose logits are all -inf has
// 1 / sum = 0 and lse = 0; one with a NaN or +inf has NaN for both (some z - max is NaN, so the sum is).
template <int VW, int LP, int Q>
__device__ __forceinline__ float2 softmax(float (&z)[Q][VW], const float (&b)[Q][VW]) {
  float m = -__builtin_inff();
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int v = 0; v < VW; ++v) {
      z[q][v] += b[q][v];
      m = fmaxf(m, z[q][v]);
    }
  m = group<LP, Max>(m);
  m = m == -__builtin_inff() ? 0.f : m;
  float s = 0.f;
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int v = 0; v < VW; ++v) {
      z[q][v] = exp_neg(z[q][v] - m);
      s += z[q][v];
    }
  s = group<LP, Add>(s);
  const bool none = s == 0.f;
  return make_float2(none ? 0.f : __builtin_amdgcn_rcpf(s),
                     none ? 0.f : __builtin_fmaf(__builtin_amdgcn_logf(s), 0.6931471805599453f, m));
}

// The first sequence b in [0, B) that ends behind token t (ptr[b+1] > t), or B: 64 probes a round.
// Called by whole wavefronts with equal arguments.
__device__ __forceinline__ int find_seq(const int32_t* __restrict__ ptr, int B, int t) {
  if (!ptr) return 0;
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = B;  // the answer is in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 63) / 64;
    const int at = min(lo + (lane + 1) * step, hi) - 1;
    const unsigned long long m = __ballot(ptr[at + 1] > t);
    if (!m) return hi;
    const int f = __builtin_ctzll(m);
    const int nlo = lo + f * step, nhi = min(nlo + step, hi) - 1;  // ptr[nhi + 1] > t
    lo = nlo;
    hi = nhi;
  }
  return lo;
}

struct Args {
  const float* logits;
  const float* bias;       // NULL: zeros
  const int32_t* idx;      // [N, k]
  const uint8_t* mask;     // [N], 0 leaves a token out; NULL: none
  const int32_t* ptr;      // [B + 1]; NULL: one sequence of all tokens
  int N, E, k, B, T;       // T tokens per workgroup
  float c0, beta;          // alpha E / (B k)
  float* loss;             // [2]
  int32_t* counts;         // [B, E]
  float* saved;            // [B, E] g, then 2 beta / n
  // workspace (more than one workgroup)
  float* psum;             // [slots, E]
  int32_t* cnt;            // [slots, E]
  int32_t* ns;             // [slots] tokens
  float* zc;               // [workgroups] sums of lse^2
  int32_t* nc;             // [workgroups] tokens
  float* part;             // [workgroups of k_balance_sum] shares of L0
  unsigned* ticket;
};

__device__ __forceinline__ int seq_lo(const Args& a, int b) { return a.ptr ? min(max(a.ptr[b], 0), a.N) : 0; }
__device__ __forceinline__ int seq_hi(const Args& a, int b, int lo) {
  return a.ptr ? min(max(a.ptr[b + 1], lo), a.N) : a.N;
}

// The expert of this lane's pair of the wavefront's next 64 / k tokens from t0 on (k <= 64), -1 for
// none.  Its load is issued well before count_pairs needs the value.
__device__ __forceinline__ int load_pair(const Args& a, int t0, int te) {
  const int L = threadIdx.x & 63, k = a.k, tpw = 64 / k, tt = L / k, t = t0 + tt;
  return tt < tpw && t < te && (!a.mask || a.mask[t]) ? a.idx[(size_t)t * k + (L - tt * k)] : -1;
}

// Counts the pairs of tokens [ts, te) into the LDS histogram: an index outside [0, E) and a second
// naming of an expert by one token count nothing (they make no row of a plan either).  e: the
// lane's first pair (load_pair at the wavefront's first token; k <= 64).
__device__ __forceinline__ void count_pairs(const Args& a, int ts, int te, int e, int* hist, uint32_t (*bits)[32]) {
  const int wv = threadIdx.x >> 6, L = threadIdx.x & 63, k = a.k, E = a.E;
  if (k <= 64) {
    const int tpw = 64 / k, j = L % k;  // tokens per wavefront at a time
    for (int t0 = ts + wv * tpw; t0 < te; t0 += 4 * tpw) {
      const int next = load_pair(a, t0 + 4 * tpw, te);
      bool ok = e >= 0 && e < E;
      for (int d = 1; d < k; ++d) {
        const int o = __shfl_up(e, d);
        if (j >= d && o == e) ok = false;
      }
      if (ok) atomicAdd(&hist[e], 1);
      e = next;
    }
  } else {
    for (int t = ts + wv; t < te; t += 4) {
      if (a.mask && !a.mask[t]) continue;
      if (L < 32) bits[wv][L] = 0;
      __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
      __builtin_amdgcn_wave_barrier();
      for (int j = L; j < k; j += 64) {
        const int x = a.idx[(size_t)t * k + j];
        if (x < 0 || x >= E) continue;
        const uint32_t bit = 1u << (x & 31);
        if (!(atomicOr(&bits[wv][x >> 5], bit) & bit)) atomicAdd(&hist[x], 1);
      }
      __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  }
}

// sum of one value per thread over the workgroup, in a fixed tree; every thread gets it
__device__ __forceinline__ float block_sum(float v, float* s) {
  v = group<64, Add>(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  float r = 0.f;
  for (int q = 0; q < (int)(blockDim.x >> 6); ++q) r += s[q];
  return r;
}
__device__ __forceinline__ int block_sum(int v, int* s) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  int r = 0;
  for (int q = 0; q < (int)(blockDim.x >> 6); ++q) r += s[q];
  return r;
}

// ONE: the only workgroup; it writes the results itself.
template <int VW, int LP, int Q, bool ONE>
__global__ __launch_bounds__(NT) void k_balance(Args a) {
  constexpr int SL = NT / LP, EP = LP * Q * VW;         // token slots; padded row
  constexpr int U = Q * VW >= 8 ? 1 : 2;  // tokens in flight per slot
  __shared__ float s_sum[4][EP];
  __shared__ int s_hist[EP];
  __shared__ uint32_t s_bits[4][32];
  __shared__ float s_f[4];
  __shared__ int s_i[4];
  const int L = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int slot = threadIdx.x / LP, l = threadIdx.x % LP;
  const int E = a.E;
  const int t0 = ONE ? 0 : blockIdx.x * a.T;
  const int t1 = ONE ? a.N : min(a.N, t0 + a.T);  // (T blocks cover N: no overflow past t0 + T < 2^31)
  float bias[Q][VW];
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int v = 0; v < VW; ++v) {
      const int e = (q * LP + l) * VW + v;
      bias[q][v] = a.bias && e < E ? a.bias[e] : 0.f;
    }
  if (!ONE && blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;  // read by the next launch
  float zsum = 0.f, l0 = 0.f;  // zsum: lane l == 0 of each slot counts
  int nsum = 0;
  for (int b = ONE ? 0 : find_seq(a.ptr, a.B, t0); b < a.B; ++b) {
    const int lo = seq_lo(a, b);
    if (!ONE && lo >= t1) break;
    const int ts = max(lo, t0), te = min(seq_hi(a, b, lo), t1);
    if (!ONE && ts >= te) continue;
    const int pair = a.k <= 64 ? load_pair(a, ts + wv * (64 / a.k), te) : -1;
    for (int e = threadIdx.x; e < EP; e += NT) s_hist[e] = 0;
    __syncthreads();  // (the previous sequence's readers of s_sum and s_hist are done as well)
    float acc[Q][VW];
    int nt = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int v = 0; v < VW; ++v) acc[q][v] = 0.f;
    // The next U tokens' loads are issued before this turn's are used.
    float z[U][Q][VW];
    int mk[U];
    auto load = [&](int tb) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = min(tb + u * SL + slot, te - 1);
        load_row<VW, LP, Q>(a.logits + (size_t)t * E, E, l, -__builtin_inff(), z[u]);
        mk[u] = a.mask ? a.mask[t] : 1;
      }
    };
    if (ts < te) load(ts);
    for (int tb = ts; tb < te; tb += U * SL) {
      float c[U][Q][VW];
      bool live[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
          for (int v = 0; v < VW; ++v) c[u][q][v] = z[u][q][v];
        live[u] = tb + u * SL + slot < te && mk[u] != 0;
      }
      if (tb + U * SL < te) load(tb + U * SL);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float2 il = softmax<VW, LP, Q>(c[u], bias);  // 1 / sum, lse
        if (live[u]) {  // (a token left out may hold anything: nothing of it is added)
#pragma unroll
          for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int v = 0; v < VW; ++v) acc[q][v] += c[u][q][v] * il.x;
          if (l == 0) zsum += il.y * il.y, ++nt;
        }
      }
    }
    count_pairs(a, ts, te, pair, s_hist, s_bits);
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int v = 0; v < VW; ++v) {
        const float s = across<LP>(acc[q][v]);
        if (L < LP) s_sum[wv][(q * LP + l) * VW + v] = s;
      }
    nsum += nt;
    const int nb = block_sum(nt, s_i);  // (its barriers publish s_sum and s_hist)
    if constexpr (ONE) {
      const float cb = nb > 0 ? a.c0 / (float)nb / (float)nb : 0.f;
      for (int e = threadIdx.x; e < E; e += NT) {
        const int c = s_hist[e];
        const float g = cb * (float)c;
        a.counts[(size_t)b * E + e] = c;
        a.saved[(size_t)b * E + e] = g;
        l0 += g * ((s_sum[0][e] + s_sum[1][e]) + (s_sum[2][e] + s_sum[3][e]));
      }
    } else {
      const size_t o = (size_t)(blockIdx.x + b);
      for (int e = threadIdx.x; e < E; e += NT) {
        a.psum[o * E + e] = (s_sum[0][e] + s_sum[1][e]) + (s_sum[2][e] + s_sum[3][e]);
        a.cnt[o * E + e] = s_hist[e];
      }
      if (threadIdx.x == 0) a.ns[o] = nb;
    }
    __syncthreads();
  }
  const float zs = block_sum(zsum, s_f);
  const int n = block_sum(nsum, s_i);
  if constexpr (ONE) {
    l0 = block_sum(l0, s_f);
    if (threadIdx.x == 0) {
      a.loss[0] = l0;
      a.loss[1] = n > 0 ? a.beta * (zs / (float)n) : 0.f;
      a.saved[(size_t)a.B * E] = n > 0 ? 2.f * a.beta / (float)n : 0.f;
    }
  } else if (threadIdx.x == 0) {
    a.zc[blockIdx.x] = zs;
    a.nc[blockIdx.x] = n;
  }
}

// Workgroup b nE + x, nE = ceil(E / 64): experts 64 x .. 64 x + 63 of sequence b; thread (g, e) adds the slots of
// workgroups first + g, first + g + 16, ..., then the 16 sums are added in order.
__global__ __launch_bounds__(1024) void k_balance_sum(Args a, int nch) {
  __shared__ float s_p[16][64];
  __shared__ int s_c[16][64];
  __shared__ float s_f[16];
  __shared__ int s_i[16];
  __shared__ unsigned s_last;
  const int E = a.E, nE = (E + 63) / 64, b = blockIdx.x / nE, xe = blockIdx.x - b * nE;
  const int x = threadIdx.x & 63, g = threadIdx.x >> 6, e = xe * 64 + x;
  const int lo = seq_lo(a, b), hi = seq_hi(a, b, lo);
  const int c0 = lo / a.T, c1 = hi > lo ? (hi - 1) / a.T : c0 - 1;
  float p = 0.f;
  int c = 0, nt = 0;
  if (e < E) {
#pragma unroll 4
    for (int i = c0 + g; i <= c1; i += 16) {
      p += a.psum[(size_t)(i + b) * E + e];
      c += a.cnt[(size_t)(i + b) * E + e];
    }
  }
  for (int i = c0 + (int)threadIdx.x; i <= c1; i += 1024) nt += a.ns[i + b];
  s_p[g][x] = p;
  s_c[g][x] = c;
  const int nb = block_sum(nt, s_i);
  float l0 = 0.f;
  if (g == 0 && e < E) {
    for (int q = 1; q < 16; ++q) {
      p += s_p[q][x];
      c += s_c[q][x];
    }
    const float gv = nb > 0 ? a.c0 / (float)nb / (float)nb * (float)c : 0.f;
    a.counts[(size_t)b * E + e] = c;
    a.saved[(size_t)b * E + e] = gv;
    l0 = gv * p;
  }
  l0 = group<64, Add>(l0);  // wavefront 0 holds them all
  if (blockIdx.x == 0) {  // the z-loss
    float zs = 0.f;
    int n = 0;
    for (int i = threadIdx.x; i < nch; i += 1024) zs += a.zc[i], n += a.nc[i];
    zs = block_sum(zs, s_f);
    n = block_sum(n, s_i);
    if (threadIdx.x == 0) {
      a.loss[1] = n > 0 ? a.beta * (zs / (float)n) : 0.f;
      a.saved[(size_t)a.B * E] = n > 0 ? 2.f * a.beta / (float)n : 0.f;
    }
  }
  // The last workgroup to come adds the shares of L0, in their order.  Each share is stored with
  // device scope (past this XCD's L2) and has arrived before its ticket is drawn (the wait); the
  // last one reads them with device scope.  So nothing else needs to leave the L2s: a device-scope
  // fence, which writes back every dirty line there, made this kernel 3 us longer at N = 4096, E = 128.
  const unsigned total = gridDim.x;
  if (threadIdx.x == 0) {
    __hip_atomic_store(&a.part[blockIdx.x], l0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    s_last = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == total - 1;
  }
  __syncthreads();
  if (!s_last) return;
  float v = 0.f;
  for (unsigned i = threadIdx.x; i < total; i += 1024)
    v += __hip_atomic_load(&a.part[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  v = block_sum(v, s_f);
  if (threadIdx.x == 0) a.loss[0] = v;
}

// no tokens: everything is zero
__global__ __launch_bounds__(NT) void k_balance_zero(Args a) {
  const size_t n = (size_t)a.B * a.E;
  for (size_t i = (size_t)blockIdx.x * NT + threadIdx.x; i <= n; i += (size_t)gridDim.x * NT) {
    a.saved[i] = 0.f;
    if (i < n) a.counts[i] = 0;
  }
  if (blockIdx.x == 0 && threadIdx.x < 2) a.loss[threadIdx.x] = 0.f;
}

struct BwdArgs {
  const float* logits;
  const float* bias;
  const uint8_t* mask;
  const int32_t* ptr;
  const float* saved;
  const float* dloss;  // [2]; NULL: ones
  const float* din;    // NULL: zeros (may be dz)
  float* dz;
  int N, E, B;
  long long first;  // this launch's first token
};

template <int VW, int LP, int Q>
__global__ __launch_bounds__(NT) void k_balance_bwd(BwdArgs a) {
  constexpr int SL = NT / LP;
  constexpr int U = Q * VW >= 16 ? 1 : (Q * VW >= 8 ? 2 : 4);
  const int slot = threadIdx.x / LP, l = threadIdx.x % LP;
  const int E = a.E, N = a.N;
  const long long tb = a.first + (long long)blockIdx.x * (SL * U);
  const int tl = (int)min(tb + SL * U, (long long)N) - 1;  // the workgroup's last token
  float bias[Q][VW];
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int v = 0; v < VW; ++v) {
      const int e = (q * LP + l) * VW + v;
      bias[q][v] = a.bias && e < E ? a.bias[e] : 0.f;
    }
  float z[U][Q][VW], di[U][Q][VW];
  int mk[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int t = (int)min(tb + u * SL + slot, (long long)tl);
    load_row<VW, LP, Q>(a.logits + (size_t)t * E, E, l, -__builtin_inff(), z[u]);
    mk[u] = a.mask ? a.mask[t] : 1;
    if (a.din) {
      load_row<VW, LP, Q>(a.din + (size_t)t * E, E, l, 0.f, di[u]);
    } else {
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int v = 0; v < VW; ++v) di[u][q][v] = 0.f;
    }
  }
  const float d0 = a.dloss ? a.dloss[0] : 1.f;
  const float d1 = (a.dloss ? a.dloss[1] : 1.f) * a.saved[(size_t)a.B * E];
  const int b0 = find_seq(a.ptr, a.B, (int)tb), b1 = a.ptr ? find_seq(a.ptr, a.B, tl) : 0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long tw = tb + u * SL + slot;
    if (tw > tl) continue;
    const int t = (int)tw;
    int lo = b0, hi = b1;  // the first sequence that ends behind t
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (a.ptr[mid + 1] > t) hi = mid; else lo = mid + 1;
    }
    const bool in = mk[u] != 0 && lo < a.B && (!a.ptr || a.ptr[lo] <= t);
    float o[Q][VW];
    if (in) {
      float gr[Q][VW];
      load_row<VW, LP, Q>(a.saved + (size_t)lo * E, E, l, 0.f, gr);
      const float2 il = softmax<VW, LP, Q>(z[u], bias);  // 1 / sum, lse
      float dot = 0.f;
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int v = 0; v < VW; ++v) dot += gr[q][v] * z[u][q][v];
      dot = group<LP, Add>(dot) * il.x;
      const float zc = d1 * il.y;
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int v = 0; v < VW; ++v) o[q][v] = di[u][q][v] + z[u][q][v] * il.x * (d0 * (gr[q][v] - dot) + zc);
    } else {
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int v = 0; v < VW; ++v) o[q][v] = di[u][q][v];
    }
    float* dz = a.dz + (size_t)t * E;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int e = (q * LP + l) * VW;
      if (e < E) {
        if constexpr (VW == 4)
          *reinterpret_cast<float4*>(dz + e) = make_float4(o[q][0], o[q][1], o[q][2], o[q][3]);
        else
          dz[e] = o[q][0];
      }
    }
  }
}

// N E up to here: one workgroup and one launch (N = 64, E = 8, one sequence: 5.6 us, 11.0 by two launches;
// N = 64, E = 128, four: 15.1 and 16.7; at N E = 32768, N = 256, four: 23.6 and 14.0)
constexpr int ONE_MAX = 1 << 13;
// Tokens per workgroup of the forward, for about 1024 workgroups, four a CU (N = 65536, E = 256, 37 ragged masked
// sequences: 256 of them 37.9 us, 512 29.4, 1024 28.2, 2048 31.4, 4096 36.6; one sequence, where k_balance_sum
// adds all rows in few workgroups: 32.6, 28.4, 30.4, 37.3, 52.4; N = 16384 ragged: 22.7, 20.4, 20.7, 20.7, 20.8)
int chunk_tokens(int N) {
  const int t = (int)(((long long)N + 1023) / 1024);
  return t < 16 ? 16 : (t + 15) / 16 * 16;
}
size_t up(size_t n) { return (n + 255) / 256 * 256; }

// f(VW, LP, Q) for E experts; vec: rows of 16-byte vectors.  Fewer lanes a token share each lane
// exchange among more tokens, more lanes leave fewer values in each.  Forward and gradient at N = 65536,
// E = 256, ragged: 64 lanes 30.4 + 31.6 us, 32 28.2 + 28.5, 16 31.2 + 30.9; E = 128, one sequence: 32 lanes 25.3 + 16.4,
// 16 25.0 + 14.7.
#define BL_SHAPES(vec, E, F) \
  if (vec) {                 \
    if (E <= 8) F(4, 2, 1); \
    else if (E <= 16) F(4, 4, 1); \
    else if (E <= 32) F(4, 8, 1); \
    else if (E <= 64) F(4, 16, 1); \
    else if (E <= 128) F(4, 16, 2); \
    else if (E <= 256) F(4, 32, 2); \
    else if (E <= 512) F(4, 32, 4); \
    else F(4, 64, 4); \
  } else { \
    if (E <= 8) F(1, 8, 1); \
    else if (E <= 32) F(1, 32, 1); \
    else if (E <= 64) F(1, 64, 1); \
    else if (E <= 128) F(1, 64, 2); \
    else if (E <= 256) F(1, 64, 4); \
    else if (E <= 512) F(1, 64, 8); \
    else F(1, 64, 16); \
  }

bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace bl

size_t balance_loss_ws_bytes(int N, int E, int B) {
  const size_t nch = ((size_t)N + bl::chunk_tokens(N) - 1) / bl::chunk_tokens(N), slots = nch + B;
  return 2 * bl::up(slots * E * 4) + bl::up(slots * 4) + 2 * bl::up(nch * 4) +
         bl::up((size_t)B * ((E + 63) / 64) * 4) + 256;
}

hipError_t launch_balance_loss(const float* logits, const float* bias, const int32_t* idx, const uint8_t* mask,
                               const int32_t* ptr, int B, int N, int E, int k, float alpha, float beta, float* loss,
                               int32_t* counts, float* saved, void* ws, hipStream_t s) {
  using namespace bl;
  const int T = chunk_tokens(N), nch = (N + T - 1) / T;
  const size_t slots = (size_t)nch + B;
  char* w = static_cast<char*>(ws);
  auto take = [&](size_t bytes) { char* p = w; w += up(bytes); return p; };
  Args a{};
  a.logits = logits; a.bias = bias; a.idx = idx; a.mask = mask; a.ptr = ptr;
  a.N = N; a.E = E; a.k = k; a.B = B; a.T = T;
  a.c0 = (float)((double)alpha * E / ((double)B * k));
  a.beta = beta;
  a.loss = loss; a.counts = counts; a.saved = saved;
  a.psum = reinterpret_cast<float*>(take(slots * E * 4));
  a.cnt = reinterpret_cast<int32_t*>(take(slots * E * 4));
  a.ns = reinterpret_cast<int32_t*>(take(slots * 4));
  a.zc = reinterpret_cast<float*>(take((size_t)nch * 4));
  a.nc = reinterpret_cast<int32_t*>(take((size_t)nch * 4));
  a.part = reinterpret_cast<float*>(take((size_t)B * ((E + 63) / 64) * 4));
  a.ticket = reinterpret_cast<unsigned*>(take(256));
  if (N == 0) {
    hipLaunchKernelGGL(k_balance_zero, dim3(64), dim3(NT), 0, s, a);
    return hipGetLastError();
  }
  const bool vec = E % 4 == 0 && al16(logits);
  // one workgroup walks all sequences in turn, so it takes few of them
  const bool one = (long long)N * E <= ONE_MAX && B <= 16;
#define BL_FWD(VW, LP, Q)                                                                     \
  do {                                                                                        \
    if (one) hipLaunchKernelGGL((k_balance<VW, LP, Q, true>), dim3(1), dim3(NT), 0, s, a);    \
    else hipLaunchKernelGGL((k_balance<VW, LP, Q, false>), dim3(nch), dim3(NT), 0, s, a);     \
  } while (0)
  BL_SHAPES(vec, E, BL_FWD)
#undef BL_FWD
  if (!one) hipLaunchKernelGGL(k_balance_sum, dim3((unsigned)((E + 63) / 64) * (unsigned)B), dim3(1024), 0, s, a, nch);
  return hipGetLastError();
}

hipError_t launch_balance_loss_bwd(const float* logits, const float* bias, const uint8_t* mask, const int32_t* ptr,
                                   int B, int N, int E, const float* saved, const float* dloss, const float* din,
                                   float* dz, hipStream_t s) {
  using namespace bl;
  if (N == 0) return hipSuccess;
  BwdArgs a{logits, bias, mask, ptr, saved, dloss, din, dz, N, E, B, 0};
  const bool vec = E % 4 == 0 && al16(logits) && al16(saved) && al16(din) && al16(dz);
#define BL_BWD(VW, LP, Q)                                                                                  \
  do {                                                                                                     \
    constexpr int per = (NT / LP) * (Q * VW >= 16 ? 1 : (Q * VW >= 8 ? 2 : 4));                             \
    hipLaunchKernelGGL((k_balance_bwd<VW, LP, Q>), dim3((unsigned)((n + per - 1) / per)), dim3(NT), 0, s, a); \
  } while (0)
  // at most 2^22 tokens a launch (a multiple of every `per`): 64 threads a token stay below the 2^32
  // threads that one may have
  for (; a.first < N; a.first += 1 << 22) {
    const long long n = N - a.first < (1 << 22) ? N - a.first : 1 << 22;
    BL_SHAPES(vec, E, BL_BWD)
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
#undef BL_BWD
  return hipSuccess;
}

}  // namespace moe
