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

// Keys of the groups that are not kept become 0.  `lds`: E words of this wave
// (the keys by expert).  LPG = 64 / (n_group rounded up to a power of two)
// lanes scan one group and merge their two largest keys.
template <int KPL>
__device__ __forceinline__ void keep_groups(uint64_t (&key)[KPL], int E, const GroupRule& g, uint64_t* lds) {
  if (g.topk_group >= g.n_group) return;
  const int lane = threadIdx.x & 63;
  const int per = E / g.n_group;
#pragma unroll
  for (int s = 0; s < KPL; ++s)
    if (lane + 64 * s < E) lds[lane + 64 * s] = key[s];
  wave_sync();
  int gp = 1;
  while (gp < g.n_group) gp *= 2;
  const int lpg = 64 / gp, grp = lane / lpg, sub = lane % lpg;
  uint64_t m1 = 0, m2 = 0;
  if (grp < g.n_group)
    for (int i = sub; i < per; i += lpg) merge2(m1, m2, lds[grp * per + i], 0);
  for (int off = 1; off < lpg; off <<= 1) {
    const uint64_t b1 = shfl_xor_u64(m1, off), b2 = shfl_xor_u64(m2, off);
    merge2(m1, m2, b1, b2);
  }
  uint64_t val = m1;
  if (g.top2 && m1 && m2) val = score_key(key_score(m1) + key_score(m2));
  // +inf plus a finite key is +inf; two keys above -inf never add to NaN or to
  // an empty key other than by -inf + ..., which cannot occur here
  int rank = 0;
  for (int j = 0; j < g.n_group; ++j) {
    const uint64_t vj = (uint64_t)__shfl((unsigned long long)val, j * lpg, 64);
    rank += (vj > val || (vj == val && j < grp)) ? 1 : 0;
  }
  const uint64_t kept_lanes = __ballot(grp < g.n_group && rank < g.topk_group && sub == 0);
#pragma unroll
  for (int s = 0; s < KPL; ++s) {
    const int e = lane + 64 * s;
    if (e < E && !((kept_lanes >> ((e / per) * lpg)) & 1ull)) key[s] = 0;
  }
  wave_sync();
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

// One wave per token.  `part`: float64 partial logits [S][T][E], added in
// ascending slice order.  LDS per wave: E words (keys by expert, then the list
// of the chosen, then their scores).
template <int KPL>
__global__ __launch_bounds__(256) void route_grouped_kernel(const double* __restrict__ part, int S,
                                                            const float* __restrict__ bias,
                                                            const float* __restrict__ sel_bias,
                                                            const int32_t* __restrict__ tok_off, int T_, int E,
                                                            GroupRule rule, float scale, int32_t* __restrict__ ids,
                                                            float* __restrict__ wts) {
  extern __shared__ uint64_t rg_lds[];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int t = blockIdx.x * (blockDim.x >> 6) + wv;
  if (t >= T_) return;
  uint64_t* const lds = rg_lds + (size_t)wv * 2 * E;
  const int base = tok_off[t];
  const int kt = tok_off[t + 1] - base;
  constexpr int G = 32 / KPL;
  const size_t qstride = (size_t)T_ * E;
  double l[KPL], sc[KPL];
#pragma unroll
  for (int s = 0; s < KPL; ++s) l[s] = 0.0;
  for (int q0 = 0; q0 < S; q0 += G) {
    double v[KPL][G];
#pragma unroll
    for (int s = 0; s < KPL; ++s) {
      const int e = lane + 64 * s;
      const double* pe = part + (size_t)t * E + (e < E ? e : 0);
#pragma unroll
      for (int i = 0; i < G; ++i) v[s][i] = (q0 + i < S) ? pe[(size_t)(q0 + i) * qstride] : 0.0;
    }
#pragma unroll
    for (int s = 0; s < KPL; ++s)
#pragma unroll
      for (int i = 0; i < G; ++i) l[s] += v[s][i];
  }
  if (kt == 0) return;
#pragma unroll
  for (int s = 0; s < KPL; ++s) {
    const int e = lane + 64 * s;
    if (bias && e < E) l[s] += (double)bias[e];
    l[s] = (double)(float)l[s];
  }
  scores<KPL>(l, E, rule.softmax, sc);
  uint64_t key[KPL];
#pragma unroll
  for (int s = 0; s < KPL; ++s) {
    const int e = lane + 64 * s;
    key[s] = e < E ? score_key(sel_bias ? sc[s] + (double)sel_bias[e] : sc[s]) : 0;
  }
  keep_groups<KPL>(key, E, rule, lds);
  int avail = 0;
#pragma unroll
  for (int s = 0; s < KPL; ++s) avail += __popcll(__ballot(key[s] != 0));
  const int k = min(kt, avail);
  bool sel[KPL];
#pragma unroll
  for (int s = 0; s < KPL; ++s) sel[s] = false;
  if (k > 0) select_u64<KPL>(key, k, sel);
  // the chosen in ascending expert order, then each one's place: the number of
  // chosen keys that are larger, or equal with a lower expert (listed before)
  const uint64_t below = (1ull << lane) - 1ull;
  int n = 0, slot[KPL];
#pragma unroll
  for (int s = 0; s < KPL; ++s) {
    const uint64_t m = __ballot(sel[s]);
    slot[s] = sel[s] ? n + __popcll(m & below) : -1;
    if (sel[s]) lds[slot[s]] = key[s];
    n += __popcll(m);
  }
  wave_sync();
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

hipError_t launch_route_grouped(const double* part, int S, const float* bias, const float* sel_bias,
                                const int32_t* tok_off, int T, int E, const GroupRule& rule, float scale,
                                int32_t* ids, float* wts, hipStream_t st) {
  if (T == 0) return hipSuccess;
  const dim3 grid((T + 3) / 4);
  const size_t lds = (size_t)4 * 2 * E * sizeof(uint64_t);
#define MOE_RG(KPL)                                                                                              \
  hipLaunchKernelGGL(route_grouped_kernel<KPL>, grid, dim3(256), lds, st, part, S, bias, sel_bias, tok_off, T, E, \
                     rule, scale, ids, wts)
  if (E <= 64) MOE_RG(1);
  else if (E <= 128) MOE_RG(2);
  else if (E <= 256) MOE_RG(4);
  else if (E <= 512) MOE_RG(8);
  else MOE_RG(16);
#undef MOE_RG
  return hipGetLastError();
}

}  // namespace moe
