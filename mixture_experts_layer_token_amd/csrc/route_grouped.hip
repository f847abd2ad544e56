// Grouped routing: per-token top-k_t by score plus balance bias inside the best
// groups of experts.  Per token, from the float32 logits l of the routing
// contract (float64 sum of exact products, one rounding):
//   s_e = 1 / (1 + exp(-l_e))  or  exp(l_e - max l) / sum exp(l - max l)   (float64)
//   c_e = s_e + b_e                                                      (float64)
//   an expert with c_e = -inf or NaN is out of service and is never chosen
//   V_g = the largest c of group g, or the sum of its two largest
//   kept = the topk_group groups of largest V (ties: lower group)
//   chosen = the k_t largest c in kept groups (ties: lower expert)
//   w = scale * s (/ sum of the chosen s)
// A token with fewer than k_t experts to choose from fills the rest of its slots
// with id -1 and weight 0, which moe_permute and moe_combine skip.
#include "common.h"
#include "launch.h"
#include "screen.h"
#include "select.h"

namespace moe {

namespace {

// Order-preserving image of a float64 key; 0 marks an expert that cannot be
// chosen (out of service, or in a group that is not kept).
__device__ __forceinline__ uint64_t score_key(double c) {
  if (!(c > -INFINITY)) return 0;  // -inf or NaN
  if (c == 0.0) c = 0.0;           // -0 -> +0
  const uint64_t u = (uint64_t)__double_as_longlong(c);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}
__device__ __forceinline__ double key_score(uint64_t k) {
  return __longlong_as_double((long long)((k >> 63) ? (k & ~(1ull << 63)) : ~k));
}

__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ uint64_t shfl_xor_u64(uint64_t v, int m) {
  return (uint64_t)__shfl_xor((unsigned long long)v, m, 64);
}
__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = fmax(v, __shfl_xor(v, off, 64));
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {  // fixed order: every lane gets the same bits
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// The two largest of two pairs of keys (a1 >= a2, b1 >= b2).
__device__ __forceinline__ void merge2(uint64_t& a1, uint64_t& a2, uint64_t b1, uint64_t b2) {
  const uint64_t hi = a1 > b1 ? a1 : b1, lo = a1 > b1 ? b1 : a1;
  const uint64_t s = a2 > b2 ? a2 : b2;
  a1 = hi;
  a2 = lo > s ? lo : s;
}

// The k largest keys (1 <= k <= keys > 0): sel marks them.  Radix search from
// the top bit that stops as soon as exactly k keys reach the trial value; ties
// at the last key go to the lower expert.
template <int KPL>
__device__ __forceinline__ void select_u64(const uint64_t (&key)[KPL], int k, bool (&sel)[KPL]) {
  const int lane = threadIdx.x & 63;
  uint64_t prefix = 0;
  int got = -1;
  for (int b = 63; b >= 0 && got != k; --b) {
    const uint64_t trial = prefix | (1ull << b);
    int c = 0;
#pragma unroll
    for (int s = 0; s < KPL; ++s) c += __popcll(__ballot(key[s] >= trial));
    if (c >= k) {
      prefix = trial;
      got = c;
    }
  }
  if (got == k) {
#pragma unroll
    for (int s = 0; s < KPL; ++s) sel[s] = key[s] >= prefix;
    return;
  }
  int need = k;
#pragma unroll
  for (int s = 0; s < KPL; ++s) {
    sel[s] = key[s] > prefix;
    need -= __popcll(__ballot(sel[s]));
  }
  const uint64_t below = (1ull << lane) - 1ull;
#pragma unroll
  for (int s = 0; s < KPL; ++s) {
    const uint64_t eq = __ballot(key[s] == prefix);
    if (need > 0 && key[s] == prefix && __popcll(eq & below) < need) sel[s] = true;
    need -= min(need, (int)__popcll(eq));
  }
}

// Scores of the token's experts from their logits.
template <int KPL>
__device__ __forceinline__ void scores(const double (&l)[KPL], int E, int softmax, double (&s)[KPL]) {
  const int lane = threadIdx.x & 63;
  if (!softmax) {
#pragma unroll
    for (int q = 0; q < KPL; ++q) s[q] = 1.0 / (1.0 + exp(-l[q]));
    return;
  }
  double m = -INFINITY;
  bool nan = false;
#pragma unroll
  for (int q = 0; q < KPL; ++q)
    if (lane + 64 * q < E) {
      m = fmax(m, l[q]);
      nan |= l[q] != l[q];
    }
  m = wave_max(m);
  if (__ballot(nan)) m = NAN;  // a logit that is no number leaves no score of the token a number
  double t = 0.0;
#pragma unroll
  for (int q = 0; q < KPL; ++q) {
    s[q] = lane + 64 * q < E ? exp(l[q] - m) : 0.0;
    t += s[q];
  }
  t = wave_sum(t);
#pragma unroll
  for (int q = 0; q < KPL; ++q) s[q] /= t;
}

}  // namespace

// ---------------------------------------------------------------------------
// Partial logits in float64 on the matrix cores: v_mfma_f64_16x16x4_f64 is a
// float64 fused multiply-add over 4 of K, so products of float32 or bf16 values
// stay exact and only the accumulation rounds, as the routing contract asks.
// A wave takes 16 ME experts x 16 NT tokens of a slice of K; a lane's 16-byte
// load of row l % 16 holds LE values of K from LE * (l / 16) on, and instruction
// i of a step multiplies value i of each lane group (any order of K will do, as
// long as both operands have the same).  The four waves of a workgroup take
// quarters of the slice and are added in wave order; slices are added by the
// selection kernel.  One more slice (z = S) holds the token-offset scan.
typedef double f64x4_t __attribute__((ext_vector_type(4)));

template <typename T>
__device__ __forceinline__ void widen(const u32x4_t& v, double* o) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      o[2 * i] = (double)__uint_as_float(v[i] << 16);
      o[2 * i + 1] = (double)__uint_as_float(v[i] & 0xffff0000u);
    } else {
      o[i] = (double)__uint_as_float(v[i]);
    }
  }
}

template <typename T, int ME, int NT>
__global__ __launch_bounds__(256) void logits_f64_kernel(const T* __restrict__ x, const T* __restrict__ w, int T_,
                                                         int d, int E, double* __restrict__ part,
                                                         const int32_t* __restrict__ k, int k_max, BudgetPolicy pol,
                                                         int32_t* __restrict__ tok_off, int32_t* __restrict__ status) {
  constexpr int LE = 16 / (int)sizeof(T), KS = 4 * LE;
  constexpr int TE = 16 * ME, TT = 16 * NT, LD = TE + 1;
  __shared__ double red[4 * TT * LD];
  const int S = gridDim.z - 1;
  if ((int)blockIdx.z == S) {
    if (blockIdx.x == 0 && blockIdx.y == 0) {
      int32_t* sc = reinterpret_cast<int32_t*>(red);
      token_offsets_block<256>(k, T_, k_max, pol, tok_off, status, sc, sc + 8);
    }
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, lg = lane >> 4;
  const int e0 = blockIdx.x * TE, t0 = blockIdx.y * TT;
  const int steps = d / KS, nq = S * 4, q = blockIdx.z * 4 + wave;
  const int s0 = (int)((long long)steps * q / nq), s1 = (int)((long long)steps * (q + 1) / nq);
  const T* wr[ME];
  const T* xr[NT];
#pragma unroll
  for (int m = 0; m < ME; ++m) wr[m] = w + (size_t)min(e0 + 16 * m + l16, E - 1) * d + lg * LE;
#pragma unroll
  for (int n = 0; n < NT; ++n) xr[n] = x + (size_t)min(t0 + 16 * n + l16, T_ - 1) * d + lg * LE;
  f64x4_t acc[ME][NT];
#pragma unroll
  for (int m = 0; m < ME; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = f64x4_t{0.0, 0.0, 0.0, 0.0};
  // one step ahead in registers
  constexpr int U = ME * NT <= 2 ? 4 : 2;
  u32x4_t wv[U][ME], xv[U][NT];
  auto load = [&](int u, int s) {
    if (s >= s1) return;
#pragma unroll
    for (int m = 0; m < ME; ++m) wv[u][m] = *reinterpret_cast<const u32x4_t*>(wr[m] + (size_t)s * KS);
#pragma unroll
    for (int n = 0; n < NT; ++n) xv[u][n] = *reinterpret_cast<const u32x4_t*>(xr[n] + (size_t)s * KS);
  };
#pragma unroll
  for (int u = 0; u < U; ++u) load(u, s0 + u);
  for (int s = s0; s < s1; s += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s + u >= s1) break;
      double wd[ME][LE], xd[NT][LE];
#pragma unroll
      for (int m = 0; m < ME; ++m) widen<T>(wv[u][m], wd[m]);
#pragma unroll
      for (int n = 0; n < NT; ++n) widen<T>(xv[u][n], xd[n]);
      load(u, s + u + U);
#pragma unroll
      for (int i = 0; i < LE; ++i)
#pragma unroll
        for (int m = 0; m < ME; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            acc[m][n] = __builtin_amdgcn_mfma_f64_16x16x4f64(wd[m][i], xd[n][i], acc[m][n], 0, 0, 0);
    }
  }
  // acc[m][n][i]: expert 16 m + 4 i + lg, token 16 n + l16
#pragma unroll
  for (int m = 0; m < ME; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[(wave * TT + 16 * n + l16) * LD + 16 * m + 4 * i + lg] = acc[m][n][i];
  __syncthreads();
  double* const out = part + (size_t)blockIdx.z * T_ * E;
  for (int i = threadIdx.x; i < TT * TE; i += 256) {
    const int t = i / TE, e = i % TE;
    if (t0 + t >= T_ || e0 + e >= E) continue;
    const double* r = red + t * LD + e;
    out[(size_t)(t0 + t) * E + e0 + e] = (r[0] + r[TT * LD]) + (r[2 * TT * LD] + r[3 * TT * LD]);
  }
}

// Tile: 16 x 16 for a batch of one tile, 16 x 32 while the batch is small, 32 x
// 64 (half the operand traffic) where the tiles alone fill the chip.
static int f64_tile(int T, int E) {
  if (T <= 16) return 0;
  return (long long)((T + 63) / 64) * ((E + 31) / 32) >= 256 ? 2 : 1;
}
int logits_f64_splits(int T, int d, int E, int dtype) {
  const int te = f64_tile(T, E) == 2 ? 32 : 16, tt = f64_tile(T, E) == 2 ? 64 : (f64_tile(T, E) == 1 ? 32 : 16);
  const long long tiles = (long long)((max(T, 1) + tt - 1) / tt) * ((E + te - 1) / te);
  const int steps = d / (dtype == DT_BF16 ? 32 : 16);
  return (int)max(1LL, min(min((256 + tiles - 1) / tiles, 16LL), (long long)steps / 8));
}

template <typename T>
static void launch_logits_f64_t(const T* x, const T* w, const int32_t* k, int T_, int d, int E, int k_max,
                                BudgetPolicy pol, int S, double* part, int32_t* tok_off, int32_t* status,
                                hipStream_t st) {
#define MOE_LF(ME, NT)                                                                                             \
  hipLaunchKernelGGL((logits_f64_kernel<T, ME, NT>),                                                               \
                     dim3((E + 16 * ME - 1) / (16 * ME), max(1, (T_ + 16 * NT - 1) / (16 * NT)), S + 1), dim3(256), 0, \
                     st, x, w, T_, d, E, part, k, k_max, pol, tok_off, status)
  switch (T_ == 0 ? -1 : f64_tile(T_, E)) {
    case -1:  // the token scan alone
      hipLaunchKernelGGL((logits_f64_kernel<T, 1, 1>), dim3(1, 1, 1), dim3(256), 0, st, x, w, T_, d, E, part, k, k_max,
                         pol, tok_off, status);
      break;
    case 0: MOE_LF(1, 1); break;
    case 1: MOE_LF(1, 2); break;
    default: MOE_LF(2, 4); break;
  }
#undef MOE_LF
}

hipError_t launch_logits_f64(int dtype, const void* x, const void* w, const int32_t* k, int T, int d, int E, int k_max,
                             BudgetPolicy pol, int S, double* part, int32_t* tok_off, int32_t* status, hipStream_t st) {
  if (dtype == DT_BF16)
    launch_logits_f64_t<bf16_t>((const bf16_t*)x, (const bf16_t*)w, k, T, d, E, k_max, pol, S, part, tok_off, status, st);
  else
    launch_logits_f64_t<float>((const float*)x, (const float*)w, k, T, d, E, k_max, pol, S, part, tok_off, status, st);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Large bf16 batches: logits from bf16 matrix instructions, close enough that
// few have to be computed again.  A workgroup of 8 waves covers 64 tokens x 256
// experts of one slice of K, 64 of K at a time through an LDS ring of whole
// 128-byte lines (the schedule of the screened router); wave w multiplies
// experts [32 w, 32 w + 32) with the 64 tokens.  The float32 accumulators start
// from zero at every stage and are added to float64 ones at its end, so that a
// float32 sum has at most 64 products: with u = 2^-22 for each addition (the
// margin of the screened router), a logit is off by at most
//   r = (64 * 2^-22 + 2^-24) * |x|_2 * max_e |w_e|_2 + d * 2^-126
// (sum |x_i w_i| <= |x| |w|; 2^-24: the slices are stored in float32), which is
// 1/28 of what one float32 sum over a slice of 1,792 would leave.  The norms'
// squares are summed beside the products, by the slices: xn[S][T], wn[S][E].
typedef float f32x16_t __attribute__((ext_vector_type(16)));
constexpr int RG_NW = 8, RG_TOK = 64, RG_EXP = 256, RG_STG = 3;
constexpr int RG_XB = RG_TOK * 128, RG_SB = RG_XB + RG_EXP * 128;  // 8 KB + 32 KB a stage

__device__ __forceinline__ float square8(const u32x4_t& v, float s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = __uint_as_float(v[i] << 16), b = __uint_as_float(v[i] & 0xffff0000u);
    s = fmaf(b, b, fmaf(a, a, s));
  }
  return s;
}

__global__ __launch_bounds__(64 * RG_NW) void logits_tile_kernel(
    const bf16_t* __restrict__ x, const bf16_t* __restrict__ w, int T, int d, int E, float* __restrict__ part,
    float* __restrict__ xn, float* __restrict__ wn, const int32_t* __restrict__ k, int k_max, BudgetPolicy pol,
    int32_t* __restrict__ tok_off, int32_t* __restrict__ status) {
  __shared__ __attribute__((aligned(1024))) char lds[RG_STG * RG_SB];
  if (blockIdx.z == gridDim.z - 1) {
    if (blockIdx.x == 0 && blockIdx.y == 0) {
      int32_t* sc = reinterpret_cast<int32_t*>(lds);
      token_offsets_block<64 * RG_NW>(k, T, k_max, pol, tok_off, status, sc, sc + RG_NW);
    }
    return;
  }
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, lh = lane >> 5;
  const int S = gridDim.z - 1, z = blockIdx.z;
  const int t0 = blockIdx.x * RG_TOK, e0 = blockIdx.y * RG_EXP;
  const int chunks = d / 64;
  const int k_beg = (int)(((long long)z * chunks) / S) * 64;
  const int k_end = (int)(((long long)(z + 1) * chunks) / S) * 64;
  const int nk = (k_end - k_beg) / 64;  // >= 1: S <= chunks

  // DMA sources (rows clamped in range; clamped rows are not stored)
  const int rsub = lane >> 3;
  const bf16_t* xsrc;
  {
    const int r = 8 * wave + rsub;
    xsrc = x + (size_t)min(t0 + r, T - 1) * d + k_beg + ((lane & 7) ^ lds_swz(r)) * 8;
  }
  const bf16_t* wsrc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = 8 * (j * RG_NW + wave) + rsub;
    wsrc[j] = w + (size_t)min(e0 + r, E - 1) * d + k_beg + ((lane & 7) ^ lds_swz(r)) * 8;
  }
  auto issue = [&](int st) {
    char* sb = lds + (st % RG_STG) * RG_SB;
    const int ko = st * 64;
    __builtin_amdgcn_global_load_lds((gbl_ptr_t)(xsrc + ko), (lds_ptr_t)(sb + wave * 1024), 16, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      __builtin_amdgcn_global_load_lds((gbl_ptr_t)(wsrc[j] + ko), (lds_ptr_t)(sb + RG_XB + (j * RG_NW + wave) * 1024),
                                       16, 0, 0);
  };
  constexpr int PER = 5;  // DMA instructions per wave per stage

  f32x16_t acc[2];
  double sum[2][16];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      acc[i][e] = 0.f;
      sum[i][e] = 0.0;
    }
  u32x4_t fw[2], fx[2][2];
  auto load_frags = [&](int kt, int s, int slot) {
    const char* sb = lds + (kt % RG_STG) * RG_SB;
    fw[slot] = *reinterpret_cast<const u32x4_t*>(sb + RG_XB + lds_off(32 * wave + l32, 2 * s + lh));
#pragma unroll
    for (int i = 0; i < 2; ++i) fx[slot][i] = *reinterpret_cast<const u32x4_t*>(sb + lds_off(32 * i + l32, 2 * s + lh));
  };
  // squares: thread tid has 16 bytes of x row tid / 8 and of w rows tid / 8 + 64 j
  float xs = 0.f, wsq[4] = {0.f, 0.f, 0.f, 0.f};
  const bool do_x = blockIdx.y == 0, do_w = blockIdx.x == 0;
#pragma unroll
  for (int p = 0; p < RG_STG; ++p)
    if (p < nk) issue(p);
  vm_wait_dyn<PER * (RG_STG - 1)>(PER * min(RG_STG - 1, nk - 1));  // stage 0 landed
  compiler_fence();
  __builtin_amdgcn_s_barrier();
  compiler_fence();
  load_frags(0, 0, 0);
  for (int kt = 0; kt < nk; ++kt) {
    const char* sb = lds + (kt % RG_STG) * RG_SB;
    if (do_x) xs = square8(*reinterpret_cast<const u32x4_t*>(sb + tid * 16), xs);
    if (do_w) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        wsq[j] = square8(*reinterpret_cast<const u32x4_t*>(sb + RG_XB + j * 8192 + tid * 16), wsq[j]);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s + 1 < 4) {
        load_frags(kt, s + 1, (s + 1) & 1);
      } else {
        // stage kt+1 landed (stages up to kt + RG_STG - 1 may be in flight) and this
        // wave's reads of stage kt are complete; on the last stage the reads
        // below touch a buffer whose values are never used
        vm_wait_dyn<PER * (RG_STG - 2)>(kt + 1 < nk ? PER * min(RG_STG - 2, nk - 2 - kt) : 0);
        lgkm_wait0();
        compiler_fence();
        __builtin_amdgcn_s_barrier();
        compiler_fence();
        if (kt + RG_STG < nk) issue(kt + RG_STG);
        load_frags(kt + 1, 0, 0);
      }
      const int slot = s & 1;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, fw[slot]),
                                                         __builtin_bit_cast(bf16x8_t, fx[slot][i]), acc[i], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        sum[i][e] += (double)acc[i][e];
        acc[i][e] = 0.f;
      }
  }
  // element e of sum[i]: expert e0 + 32 * wave + 8 * (e / 4) + 4 * lh + e % 4,
  // token t0 + 32 * i + l32
  float* const ap = part + (size_t)z * T * E;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = t0 + 32 * i + l32;
    if (t >= T) continue;
#pragma unroll
    for (int e4 = 0; e4 < 4; ++e4) {
      const int e = e0 + 32 * wave + 8 * e4 + 4 * lh;
      if ((E & 3) == 0 && e + 3 < E) {
        *reinterpret_cast<float4*>(ap + (size_t)t * E + e) =
            make_float4((float)sum[i][4 * e4], (float)sum[i][4 * e4 + 1], (float)sum[i][4 * e4 + 2],
                        (float)sum[i][4 * e4 + 3]);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (e + r < E) ap[(size_t)t * E + e + r] = (float)sum[i][4 * e4 + r];
      }
    }
  }
  // the eight threads of a row
#pragma unroll
  for (int off = 1; off < 8; off <<= 1) {
    xs += __shfl_xor(xs, off, 64);
#pragma unroll
    for (int j = 0; j < 4; ++j) wsq[j] += __shfl_xor(wsq[j], off, 64);
  }
  if ((tid & 7) == 0) {
    const int r = tid >> 3;
    if (do_x && t0 + r < T) xn[(size_t)z * T + t0 + r] = xs;
    if (do_w) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (e0 + r + 64 * j < E) wn[(size_t)z * E + e0 + r + 64 * j] = wsq[j];
    }
  }
}

// Slices: a workgroup for every CU.
int logits_tile_splits(int T, int d, int E) {
  const long long wgs = (long long)max(1, (T + RG_TOK - 1) / RG_TOK) * ((E + RG_EXP - 1) / RG_EXP);
  return (int)max(1LL, min(min((256 + wgs - 1) / wgs, 32LL), (long long)d / 64));
}

hipError_t launch_logits_tile(const void* x, const void* w, const int32_t* k, int T, int d, int E, int k_max,
                              BudgetPolicy pol, int S, float* part, float* xn, float* wn, int32_t* tok_off,
                              int32_t* status, hipStream_t st) {
  if (d % 64) return hipErrorInvalidValue;  // d is a multiple of 128 for any valid descriptor
  const dim3 grid(max(1, (T + RG_TOK - 1) / RG_TOK), (E + RG_EXP - 1) / RG_EXP, T == 0 ? 1 : S + 1);
  hipLaunchKernelGGL(logits_tile_kernel, grid, dim3(64 * RG_NW), 0, st, (const bf16_t*)x, (const bf16_t*)w, T, d, E,
                     part, xn, wn, k, k_max, pol, tok_off, status);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Scores, groups, top-k_t and weights; one wave per token.
//
// SCREEN: the logits come from logits_tile_kernel and may be off by r.  A score
// may then be off by R (sigmoid: r / 4; softmax: a factor within exp(+-2 r)),
// and two keys whose distance is over 2 R are in their true order.  Only what is
// closer and decides something is computed again, exactly:
//  - groups whose value is within 2 R (top2: 4 R) of the last one kept or of the
//    first one dropped: those of their experts that may be among the counted
//    ones.  Every other group is certainly kept or certainly dropped.
//  - then chosen experts and, of the kept groups, experts within 2 R of a chosen
//    one.  An expert that is further from every chosen one is on its true side
//    of each, and of anything that takes a chosen one's place.
// So the ids are those of exact logits, whatever the rounding did.  Where r is
// large (or no number) every logit of the token is computed exactly.
// The softmax's sum keeps its screened terms: it scales all scores alike, so
// the order needs select_bias to be absent (the host takes float64 otherwise).
struct ScreenIn {
  const bf16_t *x, *w;
  const float *part, *xn, *wn;
  int d;
};

// LDS words (8 bytes) of one wave.
__host__ __device__ constexpr int rg_words(int E, bool screen) { return 2 * E + (screen ? SEL_GRP * 64 + E + E : 0); }

// Group values of the keys (0: no expert in service), this lane's group in
// `grp` (lanes of a group: lpg), and its second largest key in `second`.
template <int KPL>
__device__ __forceinline__ uint64_t group_value(const uint64_t (&key)[KPL], int E, const GroupRule& g, int lpg,
                                                uint64_t* lds, uint64_t* second) {
  const int lane = threadIdx.x & 63, per = E / g.n_group, grp = lane / lpg, sub = lane % lpg;
#pragma unroll
  for (int s = 0; s < KPL; ++s)
    if (lane + 64 * s < E) lds[lane + 64 * s] = key[s];
  wave_sync();
  uint64_t m1 = 0, m2 = 0;
  if (grp < g.n_group)
    for (int i = sub; i < per; i += lpg) merge2(m1, m2, lds[grp * per + i], 0);
  for (int off = 1; off < lpg; off <<= 1) {
    const uint64_t b1 = shfl_xor_u64(m1, off), b2 = shfl_xor_u64(m2, off);
    merge2(m1, m2, b1, b2);
  }
  wave_sync();
  *second = g.top2 && m2 ? m2 : m1;
  // two keys above -inf never add to an empty key
  return g.top2 && m1 && m2 ? score_key(key_score(m1) + key_score(m2)) : m1;
}
// Place of this lane's group among the groups (ties: lower group first).
__device__ __forceinline__ int group_rank(uint64_t val, int n_group, int lpg) {
  const int grp = (threadIdx.x & 63) / lpg;
  int rank = 0;
  for (int j = 0; j < n_group; ++j) {
    const uint64_t vj = (uint64_t)__shfl((unsigned long long)val, j * lpg, 64);
    rank += (vj > val || (vj == val && j < grp)) ? 1 : 0;
  }
  return rank;
}

template <int KPL, bool SCREEN>
__global__ __launch_bounds__(256) void route_grouped_kernel(const double* __restrict__ part, int S, ScreenIn in,
                                                            const float* __restrict__ bias,
                                                            const float* __restrict__ sel_bias,
                                                            const int32_t* __restrict__ tok_off, int T_, int E,
                                                            GroupRule rule, float scale, int32_t* __restrict__ ids,
                                                            float* __restrict__ wts) {
  extern __shared__ uint64_t rg_lds[];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int t = blockIdx.x * (blockDim.x >> 6) + wv;
  if (t >= T_) return;
  uint64_t* const lds = rg_lds + (size_t)wv * rg_words(E, SCREEN);
  const int base = tok_off[t];
  const int kt = tok_off[t + 1] - base;
  const uint64_t below = (1ull << lane) - 1ull;
  // slices are added in ascending order, G of them in flight
  constexpr int G = 32 / KPL;
  const size_t qstride = (size_t)T_ * E;
  double l[KPL], sc[KPL];
#pragma unroll
  for (int s = 0; s < KPL; ++s) l[s] = 0.0;
  for (int q0 = 0; q0 < S; q0 += G) {
    double v[KPL][G];
#pragma unroll
    for (int s = 0; s < KPL; ++s) {
      const size_t at = (size_t)t * E + min(lane + 64 * s, E - 1);
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const size_t o = at + (size_t)(q0 + i) * qstride;
        v[s][i] = q0 + i < S ? (SCREEN ? (double)in.part[o] : part[o]) : 0.0;
      }
    }
#pragma unroll
    for (int s = 0; s < KPL; ++s)
#pragma unroll
      for (int i = 0; i < G; ++i) l[s] += v[s][i];
  }
  if (kt == 0) return;
  float bs[KPL], sb[KPL];
#pragma unroll
  for (int s = 0; s < KPL; ++s) {
    const int e = lane + 64 * s;
    bs[s] = bias && e < E ? bias[e] : 0.f;
    sb[s] = sel_bias && e < E ? sel_bias[e] : 0.f;
    l[s] += (double)bs[s];
    if (!SCREEN) l[s] = (double)(float)l[s];
  }

  double R2 = 0.0;  // twice the radius of a score
  bool exact[KPL];  // slots whose logit is exact
#pragma unroll
  for (int s = 0; s < KPL; ++s) exact[s] = !SCREEN;
  auto rescore = [&](uint64_t (&key)[KPL]) {
    scores<KPL>(l, E, rule.softmax, sc);
#pragma unroll
    for (int s = 0; s < KPL; ++s)
      key[s] = lane + 64 * s < E ? score_key(sel_bias ? sc[s] + (double)sb[s] : sc[s]) : 0;
  };
  // exact logits of the marked slots
  auto refine = [&](const bool (&mark)[KPL]) -> bool {
    int32_t* const list = reinterpret_cast<int32_t*>(lds + 2 * E + SEL_GRP * 64);
    double* const val = reinterpret_cast<double*>(lds + 2 * E + SEL_GRP * 64 + E);
    int n = 0, at[KPL];
#pragma unroll
    for (int s = 0; s < KPL; ++s) {
      const bool want = mark[s] && !exact[s] && lane + 64 * s < E;
      const uint64_t m = __ballot(want);
      at[s] = want ? n + __popcll(m & below) : -1;
      if (want) list[at[s]] = lane + 64 * s;
      n += __popcll(m);
    }
    if (n == 0) return false;
    wave_sync();
    exact_dots<4, false, SEL_GRP>(
        in.x + (size_t)t * in.d, in.d, n, [&](int c) { return in.w + (size_t)list[c] * in.d; },
        reinterpret_cast<double*>(lds + 2 * E), [&](int c, double v) { val[c] = v; });
#pragma unroll
    for (int s = 0; s < KPL; ++s)
      if (at[s] >= 0) {
        l[s] = (double)(float)(val[at[s]] + (double)bs[s]);
        exact[s] = true;
      }
    wave_sync();
    return true;
  };

  uint64_t key[KPL];
  if constexpr (SCREEN) {
    double xx = 0.0, ww = 0.0, lm = 0.0;
    for (int q = 0; q < S; ++q) xx += (double)in.xn[(size_t)q * T_ + t];
#pragma unroll
    for (int s = 0; s < KPL; ++s) {
      const int e = min(lane + 64 * s, E - 1);
      double a = 0.0;
      for (int q = 0; q < S; ++q) a += (double)in.wn[(size_t)q * E + e];
      ww = a > ww || a != a ? a : ww;
      lm = fmax(lm, fabs(l[s]));
    }
    const bool nan = __ballot(ww != ww) != 0;
    // 1.01: the float32 sums of the squares (at most 65,536 terms of 2^-24 each)
    const double prod = 1.01 * sqrt(xx) * sqrt(wave_max(ww));
    const double r = prod * (64.0 * 0x1p-22 + 0x1p-24) + in.d * 0x1p-126;
    const double rl = r + (wave_max(lm) + r) * 0x1p-24 + 0x1p-149;  // and the one rounding of the exact logit
    rescore(key);
    bool all[KPL];
#pragma unroll
    for (int s = 0; s < KPL; ++s) all[s] = true;
    if (nan || !(rl < 0.0625)) {
      if (refine(all)) rescore(key);
    } else if (rule.softmax) {
      double sm = 0.0;
#pragma unroll
      for (int s = 0; s < KPL; ++s)
        if (lane + 64 * s < E) sm = fmax(sm, sc[s]);
      R2 = 2.0 * expm1(2.0 * rl) * wave_max(sm) + 0x1p-50;
    } else {
      R2 = 0.5 * rl + 0x1p-50;
    }
  } else {
    rescore(key);
  }

  // groups
  if (rule.topk_group < rule.n_group) {
    int gp = 1;
    while (gp < rule.n_group) gp *= 2;
    const int lpg = 64 / gp, per = E / rule.n_group, grp = lane / lpg;
    uint64_t second;
    uint64_t val = group_value<KPL>(key, E, rule, lpg, lds, &second);
    int rank = group_rank(val, rule.n_group, lpg);
    if constexpr (SCREEN) {
      // values of the last group kept and the first dropped
      const bool mine = grp < rule.n_group;
      const uint64_t ml = __ballot(mine && rank == rule.topk_group - 1), mf = __ballot(mine && rank == rule.topk_group);
      const uint64_t vl = (uint64_t)__shfl((unsigned long long)val, __builtin_ctzll(ml), 64);
      const uint64_t vf = (uint64_t)__shfl((unsigned long long)val, __builtin_ctzll(mf), 64);
      const double z2 = rule.top2 ? 2.0 * R2 : R2;
      // a group without experts in service is last, whatever the scores
      if (vf != 0 && !(key_score(vl) - key_score(vf) > z2)) {
        const double v = key_score(val);
        const bool zone = mine && val != 0 && (!(fabs(v - key_score(vl)) > z2) || !(fabs(v - key_score(vf)) > z2));
        const uint64_t zones = __ballot(zone);
        bool mark[KPL];
#pragma unroll
        for (int s = 0; s < KPL; ++s) {
          const int e = lane + 64 * s, first = (min(e, E - 1) / per) * lpg;
          const uint64_t sec = (uint64_t)__shfl((unsigned long long)second, first, 64);
          mark[s] = e < E && key[s] != 0 && ((zones >> first) & 1ull) && !(key_score(sec) - key_score(key[s]) > R2);
        }
        if (refine(mark)) {
          rescore(key);
          val = group_value<KPL>(key, E, rule, lpg, lds, &second);
          rank = group_rank(val, rule.n_group, lpg);
        }
      }
    }
    const uint64_t kept = __ballot(grp < rule.n_group && rank < rule.topk_group);
#pragma unroll
    for (int s = 0; s < KPL; ++s) {
      const int e = lane + 64 * s;
      if (e < E && !((kept >> ((e / per) * lpg)) & 1ull)) sb[s] = -INFINITY;  // out of this token's reach
      if (sb[s] == -INFINITY) key[s] = 0;
    }
  }
  int avail = 0;
#pragma unroll
  for (int s = 0; s < KPL; ++s) avail += __popcll(__ballot(key[s] != 0));
  const int k = min(kt, avail);

  // the chosen, listed in ascending expert order
  bool sel[KPL];
  int slot[KPL];
  auto choose = [&]() {
#pragma unroll
    for (int s = 0; s < KPL; ++s) sel[s] = false;
    if (k > 0) select_u64<KPL>(key, k, sel);
    int n = 0;
#pragma unroll
    for (int s = 0; s < KPL; ++s) {
      const uint64_t m = __ballot(sel[s]);
      slot[s] = sel[s] ? n + __popcll(m & below) : -1;
      if (sel[s]) lds[slot[s]] = key[s];
      n += __popcll(m);
    }
    wave_sync();
  };
  choose();
  if constexpr (SCREEN) {
    int32_t* const near = reinterpret_cast<int32_t*>(lds + E);
    for (int j = lane; j < k; j += 64) near[j] = 0;
    wave_sync();
    bool mark[KPL];
    bool any = false;
#pragma unroll
    for (int s = 0; s < KPL; ++s) {
      mark[s] = false;
      if (key[s] == 0) continue;
      const double c = key_score(key[s]);
      for (int j = 0; j < k; ++j)
        if (j != slot[s] && !(fabs(c - key_score(lds[j])) > R2)) {
          mark[s] = true;
          near[j] = 1;
        }
      any |= mark[s];
    }
    if (__ballot(any)) {
      wave_sync();
#pragma unroll
      for (int s = 0; s < KPL; ++s)
        if (sel[s] && near[slot[s]]) mark[s] = true;
      if (refine(mark)) {
        uint64_t nk[KPL];
        rescore(nk);
#pragma unroll
        for (int s = 0; s < KPL; ++s) key[s] = key[s] != 0 ? nk[s] : 0;
        choose();
      }
    }
  }
  // each one's place: the chosen keys that are larger, or equal with a lower expert
  double* const ps = reinterpret_cast<double*>(lds + E);
#pragma unroll
  for (int s = 0; s < KPL; ++s) {
    if (!sel[s]) continue;
    int r = 0;
    for (int j = 0; j < k; ++j) {
      const uint64_t kj = lds[j];
      r += (kj > key[s] || (kj == key[s] && j < slot[s])) ? 1 : 0;
    }
    slot[s] = r;
    ps[r] = sc[s];
    ids[base + r] = lane + 64 * s;
  }
  wave_sync();
  double total = 1.0;
  if (rule.renorm) {
    double p = 0.0;
    for (int j = lane; j < k; j += 64) p += ps[j];
    total = wave_sum(p);
  }
#pragma unroll
  for (int s = 0; s < KPL; ++s)
    if (sel[s]) wts[base + slot[s]] = total > 0.0 ? (float)((double)scale * (sc[s] / total)) : 0.f;
  for (int j = k + lane; j < kt; j += 64) {
    ids[base + j] = -1;
    wts[base + j] = 0.f;
  }
}

template <bool SCREEN>
static hipError_t launch_rg(const double* part, int S, const ScreenIn& in, const float* bias, const float* sel_bias,
                            const int32_t* tok_off, int T, int E, const GroupRule& rule, float scale, int32_t* ids,
                            float* wts, hipStream_t st) {
  if (T == 0) return hipSuccess;
  // waves of a workgroup: as many as 64 KB of LDS hold, at most four
  const size_t per = (size_t)rg_words(E, SCREEN) * sizeof(uint64_t);
  const int nw = (int)max((size_t)1, min((size_t)4, (size_t)65536 / per));
  const dim3 grid((T + nw - 1) / nw);
#define MOE_RG(KPL)                                                                                               \
  hipLaunchKernelGGL((route_grouped_kernel<KPL, SCREEN>), grid, dim3(64 * nw), per * nw, st, part, S, in, bias,   \
                     sel_bias, tok_off, T, E, rule, scale, ids, wts)
  if (E <= 64) MOE_RG(1);
  else if (E <= 128) MOE_RG(2);
  else if (E <= 256) MOE_RG(4);
  else if (E <= 512) MOE_RG(8);
  else MOE_RG(16);
#undef MOE_RG
  return hipGetLastError();
}

hipError_t launch_route_grouped(const double* part, int S, const float* bias, const float* sel_bias,
                                const int32_t* tok_off, int T, int E, const GroupRule& rule, float scale,
                                int32_t* ids, float* wts, hipStream_t st) {
  return launch_rg<false>(part, S, ScreenIn{}, bias, sel_bias, tok_off, T, E, rule, scale, ids, wts, st);
}

hipError_t launch_route_grouped_screen(const float* part, const float* xn, const float* wn, int S, const void* x,
                                       const void* w, int d, const float* bias, const float* sel_bias,
                                       const int32_t* tok_off, int T, int E, const GroupRule& rule, float scale,
                                       int32_t* ids, float* wts, hipStream_t st) {
  return launch_rg<true>(nullptr, S, ScreenIn{(const bf16_t*)x, (const bf16_t*)w, part, xn, wn, d}, bias, sel_bias,
                         tok_off, T, E, rule, scale, ids, wts, st);
}

}  // namespace moe
