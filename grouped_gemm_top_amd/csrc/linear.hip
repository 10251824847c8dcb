// linear.hip -- the dense product with bias, activation and residual in its epilogue, and its
// backward, for gfx950 (bf16, and fp32 at fp32 accuracy).
//
//   z = x W^T + b,   out = act(z) + res,  z kept where asked             x [N,K], W [O,K], out [N,O]
//   dz = dout act'(z),   dx = dz W,   dW = dz^T x,   db = sum_t dz
//
// The three products are one kernel, C[m][n] = sum_k A(m,k) B(n,k), in three layouts: forward with
// both operands K-contiguous, dx with B K-strided (W read along its rows), dW with both K-strided.
// Accumulation, bias, activation and residual are fp32; each output is rounded once.  In bf16, where
// there is an activation, dz is rounded to bf16 before its two products, as an operand of the matrix
// cores, and db sums it unrounded.  dx and dW are then off by 0.0023 in the 2-norm, where their own rounding
// alone makes 0.0017; a second bf16 part of dz would save the difference and double both products, 240 of
// 264 us at N = 8192, K = 2048, O = 4096.  The fp32 call keeps dz whole.
//
// fp32 operands are split into three bf16 parts, v = v0 + v1 + v2 (8 significant bits each; exact from
// 2^-109 on, below to 2^-134), and the product is the sum of the part products (0,0) (0,1) (1,0) (1,1) (0,2) (2,0); the
// others are below 2^-24 of the leading one.  The kernel walks those six terms as one contraction
// six times as long: a term only moves the two operands' plane offsets.  The matrix cores' fp32
// instructions would take 16 times as long as one bf16 term, these six take 6 times.
//
// What bounds it, on one MI355X (the library behind torch's bf16 product reaches 1600 TFLOP/s there
// on 16384^3 and 1440 on 8192^3):
//  * large products: a 64-wide step of the 256 x 256 tile takes 1.38 - 1.48 us, 1450 - 1560 TFLOP/s over
//    the chip while the loop runs.  The loop without its loads takes 1.19 us, without its LDS
//    reads too 1.11; without its LDS reads but with the loads 1.42.  So it is the 64 KB a CU loads in a
//    step.  N = 8192, K = O = 4096: forward 210 - 222 us, dx 206 - 215, dW 204 - 211 (library in the same runs 180 -
//    219, 204 - 243, 225 - 268); with bias, tanh gelu, residual and z, 134 MB more, 237 - 244.
//  * products of few tiles: one CU's loads and the launch, 17.7 us for N = 333, K = 2880, O = 2056.
//  * few tokens: W's stream, 8.7 us for 34 MB (N = 1, K = O = 4096; library 12.5).
//  * fp32: six bf16 terms, 1234 - 1282 us for N = 8192, K = O = 4096 (library 1813 - 1835), dx 1242, dW 1293 (1826,
//    1805), 116 - 122 for 2048^3 (126 - 130); the split's own pass costs most where the product is small, 46 us
//    for 1000^3 (24).
#include <type_traits>

#include "gemm_lds.h"

namespace moe {
namespace ln {

using namespace gk;
using gg::OOB;

constexpr int BK = 64;  // k per LDS stage: a K-contiguous row of a stage is one 128-byte line

enum Act { NONE = MOE_ACT_NONE, RELU = MOE_ACT_RELU, SILU = MOE_ACT_SILU, GELU = MOE_ACT_GELU,
           GELU_TANH = MOE_ACT_GELU_TANH };

// Activations and their slopes, compiled in: one dispatch serves eight values, which then run
// interleaved.  Exponential and reciprocal are the hardware's, about one unit in the last place each; the
// exponent's own roundings cost |exponent| units of 2^-24 more, where the result is small.  In all, against
// 64 bits, in units of 2^-24 of the value: within 4 for |z| <= 1, 6 (silu) and 20 - 35 (gelus) at z = -5, 16
// (silu) at z = -12; bf16 rounds by 2^16 of them.
// 1 / (1 + E) and E / (1 + E) for E = 2^-t; t = v log2 e: sigmoid(v) and 1 - sigmoid(v), which 1 - s would
// leave with an error of 2^-24 (times v, in the slopes).  E = infinity makes E s NaN, for which fminf gives 1.
struct Sig { float s, q; };
__device__ __forceinline__ Sig sig2_scaled(float t) {
  const float E = __builtin_amdgcn_exp2f(-t), s = __builtin_amdgcn_rcpf(1.0f + E);
  return Sig{s, fminf(E * s, 1.0f)};
}
__device__ __forceinline__ float sig_scaled(float t) { return sig2_scaled(t).s; }
constexpr float kLog2e = 1.44269504088896340736f;
// gelu_tanh: (1 + tanh u) / 2 = sigmoid(2u), u = kG (v + kG3 v^3), kG = sqrt(2 / pi)
constexpr float kG = 0.7978845608028654f, kG3 = 0.044715f;
// gelu: Phi(v) = (1 + erf(v / sqrt 2)) / 2, with e = e^(-v^2 / 2), which the slope takes as well.
// 1 + erf would cancel for v < 0 (no digit left at v = -5.5), so the smaller tail is computed itself:
//   |v| < 1:  Phi = 1/2 + v Q(v^2)
//   else:     Phi(-|v|) = e w P(w), w = 1 / (1 + 0.4 |v|);  Phi(|v|) = 1 - Phi(-|v|)
// P and Q are least-maximum fits of relative error 2^-27 and below (P on 1 <= |v| <= 13.4, past which e is 0
// in fp32).  Relative error: 5 units of 2^-24 and, of e, what v^2 / 2 loses in its roundings, 1.5 v^2
// units.  8192 x 4096 x 4096 with its full epilogue: 247 us (253 with erff; without an activation 236).
struct Gauss { float cdf, e; };
__device__ __forceinline__ Gauss gauss(float v) {
  const float a = fabsf(v), s = v * v;
  const float e = __builtin_amdgcn_exp2f((-0.5f * kLog2e) * s);
  const float w = __builtin_amdgcn_rcpf(__builtin_fmaf(0.4f, a, 1.0f));
  float p = -0.056554921f;
  p = __builtin_fmaf(p, w, 0.189746842f);
  p = __builtin_fmaf(p, w, -0.201070011f);
  p = __builtin_fmaf(p, w, 0.0237784851f);
  p = __builtin_fmaf(p, w, 0.00688937446f);
  p = __builtin_fmaf(p, w, 0.0837814957f);
  p = __builtin_fmaf(p, w, 0.134175435f);
  p = __builtin_fmaf(p, w, 0.159548461f);
  p = __builtin_fmaf(p, w, 0.159578457f);
  const float t = p * w * e;
  float q = -7.65420828e-06f;
  q = __builtin_fmaf(q, s, 0.000113486371f);
  q = __builtin_fmaf(q, s, -0.00118632999f);
  q = __builtin_fmaf(q, s, 0.00997332297f);
  q = __builtin_fmaf(q, s, -0.0664903596f);
  q = __builtin_fmaf(q, s, 0.398942292f);
  return Gauss{a < 1.0f ? __builtin_fmaf(v, q, 0.5f) : (v < 0.f ? t : 1.0f - t), e};
}
template <int ACT>
__device__ __forceinline__ float act_fwd1(float v) {
  if constexpr (ACT == RELU) return v > 0.f ? v : (v != v ? v : 0.f);
  else if constexpr (ACT == SILU) return v * sig_scaled(kLog2e * v);
  else if constexpr (ACT == GELU) return v * gauss(v).cdf;
  else if constexpr (ACT == GELU_TANH)
    return v * sig_scaled(v * (2.0f * kG * kLog2e + (2.0f * kG * kG3 * kLog2e) * (v * v)));
  else return v;
}
template <int ACT>
__device__ __forceinline__ float act_bwd1(float v) {
  if constexpr (ACT == RELU) {
    return v > 0.f ? 1.f : (v != v ? v : 0.f);
  } else if constexpr (ACT == SILU) {
    const Sig g = sig2_scaled(kLog2e * v);
    return g.s * (1.0f + v * g.q);
  } else if constexpr (ACT == GELU) {
    const Gauss g = gauss(v);
    return g.cdf + v * 0.3989422804014327f * g.e;
  } else if constexpr (ACT == GELU_TANH) {
    if (fabsf(v) > 16.f) return v > 0.f ? 1.f : 0.f;  // exact there, and v^2 may overflow further out
    const Sig g = sig2_scaled(v * (2.0f * kG * kLog2e + (2.0f * kG * kG3 * kLog2e) * (v * v)));
    return g.s + v * g.s * g.q * (2.0f * kG + (6.0f * kG * kG3) * (v * v));
  } else {
    return 1.f;
  }
}
// v = act(v)
template <int ACT>
__device__ __forceinline__ void act_all(f32x4 (&v)[2]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j >> 2][j & 3] = act_fwd1<ACT>(v[j >> 2][j & 3]);
}
__device__ __forceinline__ void act_fwd8(f32x4 (&v)[2], int act) {
  switch (act) {
    case RELU: act_all<RELU>(v); break;
    case SILU: act_all<SILU>(v); break;
    case GELU: act_all<GELU>(v); break;
    case GELU_TANH: act_all<GELU_TANH>(v); break;
    default: break;
  }
}

struct Args {
  const void* A;  // K-contiguous [M, K] or K-strided [K, M]
  const void* B;  // K-contiguous [N, K] or K-strided [K, N]
  int M, N, K;
  int nM, nN, S, per;  // tiles along M and N, K slices, workgroups per XCD
  float* part;         // S > 1: [S, M, N]
  void* out;           // [M, N]
  void* z;             // forward: [M, N] or NULL
  const float* bias;   // forward: [N] or NULL
  const void* res;     // forward: [M, N] or NULL
  int act;
};

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
template <typename T> struct Res8 { u32x4 r; };           // eight values as they are stored
template <> struct Res8<float> { f32x4 r[2]; };
__device__ __forceinline__ void load_res(const void* p, size_t o, Res8<bf16_t>& r) {
  r.r = *reinterpret_cast<const u32x4*>(static_cast<const bf16_t*>(p) + o);
}
__device__ __forceinline__ void load_res(const void* p, size_t o, Res8<float>& r) {
  r.r[0] = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + o);
  r.r[1] = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + o + 4);
}
__device__ __forceinline__ void add_res(f32x4 (&v)[2], const Res8<bf16_t>& r) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j >> 1][2 * (j & 1)] += __uint_as_float(r.r[j] << 16);
    v[j >> 1][2 * (j & 1) + 1] += __uint_as_float(r.r[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void add_res(f32x4 (&v)[2], const Res8<float>& r) {
  v[0] += r.r[0];
  v[1] += r.r[1];
}

// the epilogue of eight neighbouring columns: element o of the outputs, b their bias, r the residual's
// values (read by the caller, before)
template <typename T>
__device__ __forceinline__ void finish8(const Args& a, size_t o, f32x4 (&v)[2], const f32x4 (&b)[2],
                                        const Res8<T>& r) {
  v[0] += b[0];
  v[1] += b[1];
  if (a.z) store8<T>(a.z, o, v);
  act_fwd8(v, a.act);
  if (a.res) add_res(v, r);
  store8<T>(a.out, o, v);
}
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

  // rows or columns x0 .. x0 + R - 1 of X; ld: row length in elements
  __device__ __forceinline__ void setup(const void* p, int X, int K, int planes, int x0, int w, int L) {
    r = sgpr4(dmadesc(p, (long long)planes * X * K * 2));
#pragma unroll
    for (int q = 0; q < NI; ++q) {
      const int b = w + NW * q;
      if constexpr (KC) {
        const int row = x0 + 8 * b + (L >> 3);
        const int c = (L & 7) ^ ((4 * (w & 1) + (L >> 4)) & 7);
        kl = 8 * c;  // (the same for every q: NW is even)
        v[q] = row < X ? ((uint32_t)row * (uint32_t)K + 8u * c) * 2u : OOB;
      } else {
        constexpr int CPR = R / 8;  // chunks per k-row
        const int k = b * (64 / CPR) + L / CPR;
        const int col = x0 + 8 * ((L % CPR) ^ mn_f(k));
        if (q == 0) kl = k;
        v[q] = col < X ? ((uint32_t)k * (uint32_t)X + (uint32_t)col) * 2u : OOB;
      }
    }
  }
  // Load instruction q of the step at k0 of the plane at byte offset `plane` into the stage area at
  // LDS address m; k >= klim (K; 0 for a step past the last) is masked per lane (K is a multiple of 8
  // where a chunk runs along k).  The uniform advance stays below 2^31, so a masked lane's offset is
  // past the descriptor's range with and without it.
  __device__ __forceinline__ void issue(int q, uint32_t m, int X, int k0, int klim, uint32_t plane, int w) const {
    const uint32_t adv = plane + (KC ? (uint32_t)k0 * 2u : (uint32_t)k0 * (uint32_t)X * 2u);
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

enum Epi { FWD = 0, PLAIN = 1, PART = 2 };

// A BM x BN tile by WM x WN wavefronts, each (BM / WM) x (BN / WN) in 16 x 16 blocks.
template <int BM, int BN, int WM, int WN, int NST, bool AKC, bool BKC, int EPI, bool F32>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_linear(Args a) {
  constexpr int NW = WM * WN, MB = BM / WM / 16, NB = BN / WN / 16;
  constexpr int OPA = BM * 128, STG = OPA + BN * 128;
  static_assert(NB % 4 == 0, "the epilogue stages 64 columns at a time");
  static_assert(NST * STG >= NW * 4096, "the epilogue's staging");
  static_assert(MB > 1 || NB == 4, "shapes below");
  __shared__ __attribute__((aligned(1024))) char s_ring[NST * STG];
  const int L = threadIdx.x & 63, w = ufl(threadIdx.x >> 6);
  const int wm = w % WM, wn = w / WM;
  // XCD x gets the tiles x per .. (x + 1) per - 1 (workgroups go to XCDs round robin), in groups of
  // eight M-tiles so that what one L2 serves at a time is a compact block of C
  const int t = (blockIdx.x & 7) * a.per + (blockIdx.x >> 3);
  const int nT = a.nM * a.nN;
  if ((int)(blockIdx.x >> 3) >= a.per || t >= nT * a.S) return;
  const int s = t / nT, tt = t - s * nT;
  const int gsz = 8 * a.nN, gr = tt / gsz, gm = min(8, a.nM - 8 * gr), in = tt - gr * gsz;
  const int m0 = (8 * gr + in % gm) * BM, n0 = (in / gm) * BN;
  constexpr int TERMS = F32 ? 6 : 1, PLANES = F32 ? 3 : 1;
  const int steps = (a.K + BK - 1) / BK;  // of one term
  const int k_lo = (int)((long long)TERMS * steps * s / a.S);
  const int nk = (int)((long long)TERMS * steps * (s + 1) / a.S) - k_lo;

  Op<BM, NW, AKC> oa;
  Op<BN, NW, BKC> ob;
  oa.setup(a.A, a.M, a.K, PLANES, m0, w, L);
  ob.setup(a.B, a.N, a.K, PLANES, n0, w, L);
  Frag<BM, AKC> fra;
  Frag<BN, BKC> frb;
  fra.init(L);
  frb.init(L);
  const uint32_t ring = lds_addr(s_ring);
  constexpr int NIA = Op<BM, NW, AKC>::NI, NI = NIA + Op<BN, NW, BKC>::NI;
  // the next step to load: its number, k and term (all wavefront-uniform)
  int lc = 0, lt = F32 ? k_lo / steps : 0, lk = (k_lo - lt * steps) * BK;
  const uint32_t planeA = (uint32_t)a.M * (uint32_t)a.K * 2u, planeB = (uint32_t)a.N * (uint32_t)a.K * 2u;
  // its load instruction q into stage st (a step past the last one is all masked)
  auto issue = [&](int q, int st) __attribute__((always_inline)) {
    const uint32_t m = ring + (uint32_t)st * STG;
    const bool live = lc < nk;
    const int k0 = live ? lk : 0, klim = live ? a.K : 0;
    uint32_t pa = 0u, pb = 0u;
    if constexpr (F32) {  // digits of the terms' parts, A: 0 0 1 1 0 2, B: 0 1 0 1 2 0
      pa = live ? ((0x201100u >> (4 * lt)) & 3u) * planeA : 0u;
      pb = live ? ((0x021010u >> (4 * lt)) & 3u) * planeB : 0u;
    }
    if (q < NIA) oa.issue(q, m, a.M, k0, klim, pa, w);
    else ob.issue(q - NIA, m + OPA, a.N, k0, klim, pb, w);
  };
  auto advance = [&]() __attribute__((always_inline)) {
    ++lc;
    lk += BK;
    if (F32 && lk >= a.K) lk = 0, ++lt;
  };
  auto frag_a = [&](int i, int st, int sub) __attribute__((always_inline)) {
    return fra.get(s_ring + st * STG, wm * (BM / WM) + 16 * i, sub);
  };
  auto frag_b = [&](int j, int st, int sub) __attribute__((always_inline)) {
    return frb.get(s_ring + st * STG + OPA, wn * (BN / WN) + 16 * j, sub);
  };

  f32x4 acc[MB][NB];
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

  // acc[i][j][v] = C[wm.. + 16 i + (L & 15)][wn.. + 16 j + 4 (L >> 4) + v]; through LDS a lane gets
  // columns 8 (L & 7) .. + 7 of row 8 p + (L >> 3), so eight lanes cover a row's 128-byte line.  The
  // residual of the whole 64-column strip is in flight before the first block needs it (bf16; in fp32
  // it would take twice the registers, and is read block by block).
  typedef typename std::conditional<F32, float, bf16_t>::type T;
  char* sg = s_ring + w * 4096;
#pragma unroll
  for (int h = 0; h < NB / 4; ++h) {
    const int n = n0 + wn * (BN / WN) + 64 * h + 8 * (L & 7), mr = m0 + wm * (BM / WM) + (L >> 3);
    Res8<T> res[F32 ? 1 : MB][2];
    f32x4 bv[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
    if constexpr (EPI == FWD) {
      if (a.bias && n < a.N) {
        bv[0] = *reinterpret_cast<const f32x4*>(a.bias + n);
        bv[1] = *reinterpret_cast<const f32x4*>(a.bias + n + 4);
      }
      if (!F32 && a.res) {
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const int m = mr + 16 * i + 8 * p;
            if (m < a.M && n < a.N) load_res(a.res, (size_t)m * a.N + n, res[F32 ? 0 : i][p]);
          }
      }
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      stage_write(sg, &acc[i][4 * h], L);
      if constexpr (EPI == PART) {  // fp32: sixteen lanes cover a row's 256 bytes
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const int r = 4 * p + (L >> 4), q = L & 15;
          const f32x4 v = *reinterpret_cast<const f32x4*>(sg + r * 256 + ((q ^ r) << 4));
          const int m = m0 + wm * (BM / WM) + 16 * i + r, nn = n0 + wn * (BN / WN) + 64 * h + 4 * q;
          if (m < a.M && nn < a.N) *reinterpret_cast<f32x4*>(a.part + ((size_t)s * a.M + m) * a.N + nn) = v;
        }
        continue;
      }
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        f32x4 v[2];
        stage_read(sg, p, L, v);
        const int m = mr + 16 * i + 8 * p;
        const size_t o = (size_t)m * a.N + n;
        if (m < a.M && n < a.N) {
          if constexpr (EPI == FWD) {
            if (F32 && a.res) load_res(a.res, o, res[0][p]);
            finish8<T>(a, o, v, bv, res[F32 ? 0 : i][p]);
          } else {
            store8<T>(a.out, o, v);
          }
        }
      }
    }
  }
}

// Split K: the slices' partial sums added in slice order, then the epilogue.
template <typename T, int EPI>
__global__ __launch_bounds__(256) void k_linear_sum(Args a) {
  const size_t nv = (size_t)a.M * a.N / 8, slice = (size_t)a.M * a.N;
  const int cpr = a.N / 8;
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < nv; i += (size_t)gridDim.x * 256) {
    const int n = (int)(i % cpr) * 8;
    Res8<T> r;
    f32x4 b[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
    if constexpr (EPI == FWD) {
      if (a.res) load_res(a.res, 8 * i, r);
      if (a.bias) {
        b[0] = *reinterpret_cast<const f32x4*>(a.bias + n);
        b[1] = *reinterpret_cast<const f32x4*>(a.bias + n + 4);
      }
    }
    f32x4 v[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll 4
    for (int s = 0; s < a.S; ++s) {
      const float* p = a.part + (size_t)s * slice + 8 * i;
      v[0] += *reinterpret_cast<const f32x4*>(p);
      v[1] += *reinterpret_cast<const f32x4*>(p + 4);
    }
    if constexpr (EPI == FWD) finish8<T>(a, 8 * i, v, b, r);
    else store8<T>(a.out, 8 * i, v);
  }
}

// Few tokens (M <= 16 NT): the product is one pass over W, so it streams W straight into registers.
// A workgroup owns 16 outputs; its KW wavefronts take k-steps of 128 bytes a W row in turn (lane
// (g, r) the 16 bytes g and g + 4 of row r), with the 16-token blocks of x as the other operand, and
// their sums meet in LDS in wavefront order.  U k-steps' loads are in flight.  fp32 runs on the fp32
// matrix instruction, which takes one k per lane group: the four k of a lane's 16 bytes are four
// instructions, the same four of both operands.
template <typename T, int NT, int KW, int U>
__global__ __launch_bounds__(64 * KW) void k_linear_few(Args a) {
  __shared__ f32x4 s_sum[KW][NT][64];
  constexpr int EPC = 16 / (int)sizeof(T), SK = 8 * EPC;  // values of 16 bytes, k of a step
  const int L = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int o0 = blockIdx.x * 16, K = a.K;
  const int r = L & 15, g = L >> 4;
  const T* wp = static_cast<const T*>(a.B) + (size_t)min(o0 + r, a.N - 1) * K;
  const T* xp[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) xp[i] = static_cast<const T*>(a.A) + (size_t)min(16 * i + r, a.M - 1) * K;
  f32x4 acc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const u32x4 zero = {0u, 0u, 0u, 0u};
  for (int k0 = w * SK; k0 < K; k0 += U * KW * SK) {
    u32x4 fw[U][2], fx[U][NT][2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = k0 + u * KW * SK + 4 * EPC * h + EPC * g;
        const bool in = k < K;  // K is a multiple of 8
        fw[u][h] = in ? *reinterpret_cast<const u32x4*>(wp + k) : zero;
#pragma unroll
        for (int i = 0; i < NT; ++i) fx[u][i][h] = in ? *reinterpret_cast<const u32x4*>(xp[i] + k) : zero;
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          if constexpr (sizeof(T) == 2) {
            acc[i] = mma(__builtin_bit_cast(bf16x8, fw[u][h]), __builtin_bit_cast(bf16x8, fx[u][i][h]), acc[i]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(fw[u][h][j]),
                                                            __uint_as_float(fx[u][i][h][j]), acc[i], 0, 0, 0);
          }
        }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) s_sum[w][i][L] = acc[i];
  __syncthreads();
  // s_sum[..][l][v] = C[token 16 i + (l & 15)][output o0 + 4 (l >> 4) + v]: lane L finishes the eight
  // outputs 8 (L >> 4) .. + 7 of token L & 15, lanes l and l + 16 with l = 32 (L >> 4) + (L & 15)
  if (g < 2) {
    for (int i = w; i < NT; i += KW) {
      const int m = 16 * i + r, n = o0 + 8 * g;
      if (m >= a.M || n >= a.N) continue;
      const size_t o = (size_t)m * a.N + n;
      f32x4 v[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
      f32x4 b[2] = {v[0], v[0]};
      Res8<T> res;
      if (a.res) load_res(a.res, o, res);
      if (a.bias) {
        b[0] = *reinterpret_cast<const f32x4*>(a.bias + n);
        b[1] = *reinterpret_cast<const f32x4*>(a.bias + n + 4);
      }
#pragma unroll
      for (int q = 0; q < KW; ++q) {
        v[0] += s_sum[q][i][32 * g + r];
        v[1] += s_sum[q][i][32 * g + 16 + r];
      }
      finish8<T>(a, o, v, b, res);
    }
  }
}

template <int ACT>
__device__ __forceinline__ void times_slope(float (&d)[8], const float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) d[j] *= act_bwd1<ACT>(v[j]);
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
__global__ __launch_bounds__(256) void k_linear_split(const float* __restrict__ src, size_t n, bf16_t* __restrict__ dst) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n / 8; i += (size_t)gridDim.x * 256) {
    float v[8];
    load8(src + 8 * i, v);
    store_parts(dst + 8 * i, n, v);
  }
}

// dz = dout act'(z) as the products take it: rounded to bf16, or in fp32 its three parts (dz NULL: not
// written; act NONE: dz is dout), and the column sums of the unrounded dz over this workgroup's rows
// (part NULL: not wanted).  A workgroup owns 512 columns (64 threads of 8) and the rows g, g + 4
// gridDim.y, ... (four at a time).
template <typename T>
__global__ __launch_bounds__(256) void k_linear_dz(const T* __restrict__ dout, const T* __restrict__ z, int N, int O,
                                                   int act, bf16_t* __restrict__ dz, float* __restrict__ part) {
  __shared__ float s[3][64][8];
  const int c = threadIdx.x & 63, g = threadIdx.x >> 6;
  const int col = blockIdx.x * 512 + 8 * c;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (col < O) {
#pragma unroll 2
    for (int t = blockIdx.y * 4 + g; t < N; t += 4 * gridDim.y) {
      const size_t o = (size_t)t * O + col;
      float d[8], v[8];
      load8(dout + o, d);
      if (act != NONE) load8(z + o, v);
      switch (act) {
        case RELU: times_slope<RELU>(d, v); break;
        case SILU: times_slope<SILU>(d, v); break;
        case GELU: times_slope<GELU>(d, v); break;
        case GELU_TANH: times_slope<GELU_TANH>(d, v); break;
        default: break;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += d[j];
      if (dz) {
        if constexpr (sizeof(T) == 2)
          *reinterpret_cast<uint4*>(dz + o) = make_uint4(pk2(d[0], d[1]), pk2(d[2], d[3]), pk2(d[4], d[5]), pk2(d[6], d[7]));
        else
          store_parts(dz + o, (size_t)N * O, d);
      }
    }
  }
  if (!part) return;
  if (g > 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) s[g - 1][c][j] = sum[j];
  }
  __syncthreads();
  if (g == 0 && col < O) {
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] = (sum[j] + s[0][c][j]) + (s[1][c][j] + s[2][c][j]);
    float* p = part + (size_t)blockIdx.y * O + col;
    *reinterpret_cast<float4*>(p) = make_float4(sum[0], sum[1], sum[2], sum[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(sum[4], sum[5], sum[6], sum[7]);
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
// measured, at worst 17 %.
Shape choose(Kind kind, int M, int N, int K, int terms) {
  const int steps = terms * ((K + BK - 1) / BK);
  struct C { int bm, bn, occ; double fix, lat, thr; };
  const C cs[3] = {kind == K_FWD ? C{64, 64, 3, 3.0, 0.23, 0.26} : C{64, 128, 2, 3.0, 0.32, 0.47},
                   {128, 128, 2, 3.1, 0.75, 0.49}, {256, 256, 1, 6.4, 0.40, 1.20}};
  Shape best{1, 1};
  double tb = 1e30;
  for (int b = kind == K_DW ? 1 : 0; b < 3; ++b) {
    const long long tiles = (long long)((M + cs[b].bm - 1) / cs[b].bm) * ((N + cs[b].bn - 1) / cs[b].bn);
    for (int S = 1; S <= 16 && S <= steps; S *= 2) {
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

size_t up(size_t n) { return (n + 255) / 256 * 256; }
size_t part_bytes(Kind kind, int M, int N, int K, int terms) {
  const Shape c = choose(kind, M, N, K, terms);
  return c.S > 1 ? up((size_t)c.S * M * N * 4) : 0;
}

template <int BM, int BN, int WM, int WN, int NST, bool AKC, bool BKC, bool F32>
void launch(Args& a, int S, hipStream_t s) {
  a.nM = (a.M + BM - 1) / BM;
  a.nN = (a.N + BN - 1) / BN;
  a.S = S;
  const long long T = (long long)a.nM * a.nN * S;
  a.per = (int)((T + 7) / 8);
  const dim3 g((unsigned)(8 * a.per)), b(64 * WM * WN);
  if (S > 1)
    hipLaunchKernelGGL((k_linear<BM, BN, WM, WN, NST, AKC, BKC, PART, F32>), g, b, 0, s, a);
  else  // (both operands K-contiguous: the forward)
    hipLaunchKernelGGL((k_linear<BM, BN, WM, WN, NST, AKC, BKC, AKC && BKC ? FWD : PLAIN, F32>), g, b, 0, s, a);
}

// the product; bf16 operands, or (T float) three-part planes of them
template <typename T>
hipError_t product(Kind kind, Args a, void* ws, hipStream_t s) {
  constexpr bool F = sizeof(T) == 4;
  const Shape c = choose(kind, a.M, a.N, a.K, F ? 6 : 1);
  a.part = static_cast<float*>(ws);
  if (kind == K_FWD) {
    if (c.big == 2) launch<256, 256, 2, 4, 2, true, true, F>(a, c.S, s);
    else if (c.big == 1) launch<128, 128, 2, 2, 2, true, true, F>(a, c.S, s);
    else launch<64, 64, 4, 1, 3, true, true, F>(a, c.S, s);
  } else if (kind == K_DX) {
    if (c.big == 2) launch<256, 256, 2, 4, 2, true, false, F>(a, c.S, s);
    else if (c.big == 1) launch<128, 128, 2, 2, 2, true, false, F>(a, c.S, s);
    else launch<64, 128, 2, 2, 3, true, false, F>(a, c.S, s);
  } else {
    if (c.big == 2) launch<256, 256, 2, 4, 2, false, false, F>(a, c.S, s);
    else launch<128, 128, 2, 2, 2, false, false, F>(a, c.S, s);
  }
  if (c.S > 1) {
    const size_t nv = (size_t)a.M * a.N / 8;
    const unsigned g = (unsigned)((nv + 255) / 256 < 2048 ? (nv + 255) / 256 : 2048);
    if (kind == K_FWD) hipLaunchKernelGGL((k_linear_sum<T, FWD>), dim3(g), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_linear_sum<T, PLAIN>), dim3(g), dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

void split(const void* src, size_t n, bf16_t* dst, hipStream_t s) {
  const size_t b = (n / 8 + 255) / 256;
  hipLaunchKernelGGL(k_linear_split, dim3((unsigned)(b < 4096 ? b : 4096)), dim3(256), 0, s, (const float*)src, n, dst);
}

// Calls whose W is streamed into registers (k_linear_few) rather than tiled.  Measured, us (few /
// tiles): K = O = 2048: N = 1 5.5 / 7.8, 16 6.9 / 8.4, 32 8.9 / 8.8; K = O = 4096: N = 1 8.6 / 13.5,
// 16 11.6 / 10.7, 32 14.6 / 10.9; K = 512, O = 4096: N = 32 4.4 / 5.5.
// (fp32 tiles would first split all of W.)  The rule does not look at O, and a narrow, deep W pays for it:
// K = 16384, O = 128 runs on 8 workgroups, 20 us at N = 1 and 31 at N = 16, where tiles with K slices take
// 10.6 at N = 17.
bool few_tokens(bool f32, int N, int K) { return N <= 16 || (N <= 32 && (f32 || K <= 2048)); }

// row groups of the dz kernel: one (its column sums are dbias) for few rows
int dz_groups(int N) { return N <= 64 ? 1 : (N >= 2048 ? 128 : (N + 15) / 16); }

__global__ __launch_bounds__(256) void k_zero16(uint4* __restrict__ p, size_t n) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256)
    p[i] = make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace ln

size_t linear_fwd_ws_bytes(moe_dtype dt, int N, int K, int O) {
  using namespace ln;
  const bool f = dt == MOE_F32;
  if (few_tokens(f, N, K)) return 256;
  const size_t planes = f ? up((size_t)N * K * 6) + up((size_t)O * K * 6) : 0;
  return 256 + planes + part_bytes(K_FWD, N, O, K, f ? 6 : 1);
}

namespace ln {

template <typename T>
hipError_t fwd(Args a, void* ws, hipStream_t s) {
  if (few_tokens(sizeof(T) == 4, a.M, a.K)) {
    const dim3 g((unsigned)((a.N + 15) / 16));
    if (a.M <= 16) hipLaunchKernelGGL((k_linear_few<T, 1, 8, 4>), g, dim3(512), 0, s, a);
    else hipLaunchKernelGGL((k_linear_few<T, 2, 8, 2>), g, dim3(512), 0, s, a);
    return hipGetLastError();
  }
  char* p = static_cast<char*>(ws);
  if constexpr (sizeof(T) == 4) {
    const size_t nx = (size_t)a.M * a.K, nw = (size_t)a.N * a.K;
    bf16_t* xp = reinterpret_cast<bf16_t*>(p);
    bf16_t* wp = reinterpret_cast<bf16_t*>(p + up(nx * 6));
    p += up(nx * 6) + up(nw * 6);
    split(a.A, nx, xp, s);
    split(a.B, nw, wp, s);
    a.A = xp;
    a.B = wp;
  }
  return product<T>(K_FWD, a, p, s);
}

// the backward's workspace: dz, the column sums, x's and W's parts (fp32), partial sums
struct BwdWs {
  size_t dz, dbp, xp, wp, part;
  BwdWs(bool f, int N, int K, int O) {
    const int terms = f ? 6 : 1;
    dz = up((size_t)N * O * (f ? 6 : 2));
    dbp = up((size_t)dz_groups(N) * O * 4);
    xp = f ? up((size_t)N * K * 6) : 0;
    wp = f ? up((size_t)O * K * 6) : 0;
    const size_t dx = part_bytes(K_DX, N, K, O, terms), dw = part_bytes(K_DW, O, K, N, terms);
    part = dx > dw ? dx : dw;
  }
  size_t total() const { return 256 + dz + dbp + xp + wp + part; }
};

template <typename T>
hipError_t bwd(const T* dout, const T* x, const T* w, const T* z, int act, int N, int K, int O, void* dx, void* dw,
               float* db, void* ws, hipStream_t s) {
  constexpr bool F = sizeof(T) == 4;
  const BwdWs b(F, N, K, O);
  char* p = static_cast<char*>(ws);
  bf16_t* dz = reinterpret_cast<bf16_t*>(p);
  float* dbp = reinterpret_cast<float*>(p + b.dz);
  bf16_t* xp = reinterpret_cast<bf16_t*>(p + b.dz + b.dbp);
  bf16_t* wp = reinterpret_cast<bf16_t*>(p + b.dz + b.dbp + b.xp);
  void* part = p + b.dz + b.dbp + b.xp + b.wp;
  const bool make = (F || act != NONE) && (dx || dw);  // (bf16 without an activation: dz is dout)
  if (make || db) {
    const int G = dz_groups(N);
    float* sums = db ? (G == 1 ? db : dbp) : nullptr;
    hipLaunchKernelGGL(k_linear_dz<T>, dim3((O + 511) / 512, G), dim3(256), 0, s, dout, z, N, O, act,
                       make ? dz : nullptr, sums);
    if (db && G > 1) launch_sum_rows(dbp, G, O, db, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  Args a{};
  const void* d = make ? static_cast<const void*>(dz) : dout;
  if (dx) {
    if (F) split(w, (size_t)O * K, wp, s);
    a.A = d; a.B = F ? static_cast<const void*>(wp) : w; a.M = N; a.N = K; a.K = O; a.out = dx;
    hipError_t e = product<T>(K_DX, a, part, s);
    if (e != hipSuccess) return e;
  }
  if (dw) {
    if (F) split(x, (size_t)N * K, xp, s);
    a.A = d; a.B = F ? static_cast<const void*>(xp) : x; a.M = O; a.N = K; a.K = N; a.out = dw;
    return product<T>(K_DW, a, part, s);
  }
  return hipSuccess;
}

}  // namespace ln

hipError_t launch_linear_fwd(moe_dtype dt, const void* x, const void* w, const float* bias, int act, const void* res,
                             int N, int K, int O, void* out, void* z, void* ws, hipStream_t s) {
  using namespace ln;
  if (N == 0) return hipSuccess;
  Args a{};
  a.A = x; a.B = w; a.M = N; a.N = O; a.K = K;
  a.out = out; a.z = z; a.bias = bias; a.res = res; a.act = act;
  return dt == MOE_F32 ? fwd<float>(a, ws, s) : fwd<bf16_t>(a, ws, s);
}

size_t linear_bwd_ws_bytes(moe_dtype dt, int N, int K, int O) { return ln::BwdWs(dt == MOE_F32, N, K, O).total(); }

hipError_t launch_linear_bwd(moe_dtype dt, const void* dout, const void* x, const void* w, const void* z, int act,
                             int N, int K, int O, void* dx, void* dw, float* db, void* ws, hipStream_t s) {
  using namespace ln;
  if (N == 0) {  // the parameters' gradients are zero (a fill kernel, so that the call can be captured)
    const size_t nw = (size_t)O * K / (dt == MOE_F32 ? 4 : 8);
    if (dw) hipLaunchKernelGGL(k_zero16, dim3(1024), dim3(256), 0, s, (uint4*)dw, nw);
    if (db) hipLaunchKernelGGL(k_zero16, dim3(16), dim3(256), 0, s, (uint4*)db, (size_t)O / 4);
    return hipGetLastError();
  }
  if (dt == MOE_F32)
    return bwd((const float*)dout, (const float*)x, (const float*)w, (const float*)z, act, N, K, O, dx, dw, db, ws, s);
  return bwd((const bf16_t*)dout, (const bf16_t*)x, (const bf16_t*)w, (const bf16_t*)z, act, N, K, O, dx, dw, db, ws, s);
}

}  // namespace moe
