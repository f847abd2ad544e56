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

#include <type_traits>

namespace moe {

namespace {

// Workgroups of at most 256 threads in x and, behind 2^23 of them, in y: a launch
// holds less than 2^32 threads a dimension.
constexpr int BLOCKS_X = 1 << 23;
dim3 grid_of(int blocks, int z = 1) { return dim3(min(blocks, BLOCKS_X), (blocks - 1) / BLOCKS_X + 1, z); }
__device__ __forceinline__ int grid_block() { return (int)(blockIdx.y * gridDim.x + blockIdx.x); }

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

// The same for a float32 score.
__device__ __forceinline__ uint32_t score_key32(float c) {
  if (!(c > -INFINITY)) return 0;
  return logit_key(c);
}

__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// v of one lane, the same for all.
__device__ __forceinline__ uint64_t read_lane(uint64_t v, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)v, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
  return ((uint64_t)hi << 32) | lo;
}
// Reductions over the wave by DPP (a shuffle through LDS takes several times as
// long): rows of 16 lanes, then the rows; lane 63 has the result, in a fixed order.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float old, float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp((int)__float_as_uint(old), (int)__float_as_uint(v), CTRL,
                                                               ROWS, 0xf, false));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double old, double v) {
  const uint64_t o = (uint64_t)__double_as_longlong(old), u = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp((int)(uint32_t)o, (int)(uint32_t)u, CTRL, ROWS, 0xf, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp((int)(o >> 32), (int)(u >> 32), CTRL, ROWS, 0xf, false);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
template <class F>
__device__ __forceinline__ F last_lane(F v) {
  if constexpr (sizeof(F) == 4) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
  } else {
    return __longlong_as_double((long long)read_lane((uint64_t)__double_as_longlong(v), 63));
  }
}
template <class F>
__device__ __forceinline__ F fmaxx(F a, F b) {
  if constexpr (sizeof(F) == 4) return fmaxf(a, b);
  else return fmax(a, b);
}
template <class F>
__device__ __forceinline__ F wave_max(F v) {
  v = fmaxx(v, dpp<0x111, 0xf>(v, v));  // row_shr 1, 2, 4, 8
  v = fmaxx(v, dpp<0x112, 0xf>(v, v));
  v = fmaxx(v, dpp<0x114, 0xf>(v, v));
  v = fmaxx(v, dpp<0x118, 0xf>(v, v));
  v = fmaxx(v, dpp<0x142, 0xa>(v, v));  // row_bcast 15, 31
  v = fmaxx(v, dpp<0x143, 0xc>(v, v));
  return last_lane(v);
}
template <class F>
__device__ __forceinline__ F wave_sum(F v) {
  v += dpp<0x111, 0xf>((F)0, v);
  v += dpp<0x112, 0xf>((F)0, v);
  v += dpp<0x114, 0xf>((F)0, v);
  v += dpp<0x118, 0xf>((F)0, v);
  v += dpp<0x142, 0xa>((F)0, v);
  v += dpp<0x143, 0xc>((F)0, v);
  return last_lane(v);
}

// The two largest of two pairs of keys (a1 >= a2, b1 >= b2).
template <class K>
__device__ __forceinline__ void merge2(K& a1, K& a2, K b1, K b2) {
  const K hi = a1 > b1 ? a1 : b1, lo = a1 > b1 ? b1 : a1;
  const K s = a2 > b2 ? a2 : b2;
  a1 = hi;
  a2 = lo > s ? lo : s;
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
// Bound by the f64 matrix rate (a loop of these instructions alone reaches 70
// TFLOP/s): 128 tokens x 7168 x 256 take 14 us against 6.7 us at that rate (the
// rest is the first loads and the sum over the waves), 4,096 tokens 269 us against
// 215 (float32 batches; bf16 ones take the kernel below), one token 4 us.  The
// split-K kernel of the plain router, vector float64 through LDS, takes 24 us for
// one token and 750 us for 4,096.
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
  // expert tiles of a token tile next to each other
  const int ntile = (E + TE - 1) / TE, tile = grid_block();
  const int e0 = (tile % ntile) * TE, t0 = (tile / ntile) * TT;
  if (t0 >= T_) return;  // the same for the whole workgroup
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
                     grid_of(((E + 16 * ME - 1) / (16 * ME)) * ((T_ + 16 * NT - 1) / (16 * NT)), S + 1), dim3(256), 0,  \
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
// float32 sum has at most 64 products: with 2^-23 of the running sum for each
// addition (the instruction may truncate), a logit is off by at most
//   r = (66 * 2^-23 + 2^-24) * |x|_2 * max_e |w_e|_2 + d * 2^-126
// (sum |x_i w_i| <= |x| |w|; 66 for 64 covers the second-order terms; 2^-24: the
// slices are stored in float32).  One float32 sum over a slice of 1,792 would
// leave 28 times as much.  The norms'
// squares are summed beside the products, by the slices: xn[S][T], wn[S][E]; those
// below float32's normal range count as d * 2^-126 more.
// 4,096 tokens x 7168 x 256: 43 us, against 12 us for reading x at 4.9 TB/s and 12
// us of bf16 products at 1,200 TFLOP/s.  It moves 290 MB from the L2 into LDS (a
// workgroup re-reads its 256 router rows for every 64 tokens) and stores 17 MB of
// slices; its last 7 us are the scan, whose workgroup finds no CU before the tiles
// end.
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
// A pass runs the steps in float32 first: two values further apart than the
// radius of both are in their true order, and where nothing closer decides, the
// result stands.  The radius is that of the logits (SCREEN: they come from
// logits_tile_kernel and may be off by r, so a sigmoid by r / 4, a softmax by a
// factor within exp(+-2 r); nothing for exact ones) plus what float32 rounds off,
// 2^-20 of the largest score and of the values compared.  What is closer is looked at again:
//  - inexact logits are computed exactly: of the groups whose value is within two
//    radii of the last one kept or the first one dropped, the experts that may be
//    among the counted ones (every other group is certainly kept or dropped);
//    then the chosen, and the experts of kept groups, that are within two radii
//    of another one across the border of the choice or within the chosen (one that
//    is further off is on its true side of all of these, whichever is chosen);
//  - what remains close although its logits are exact takes the same pass in
//    float64, where exact logits decide by definition.
// So the ids are those of exact logits and float64 scores.  Where r is large (or
// no number) every logit is computed exactly.  The softmax's sum keeps screened
// terms: it scales all scores alike, so the order needs select_bias to be absent
// (the host takes float64 logits otherwise, and the pass starts in float64).
//
// The weights of what the first pass decides keep screened logits: a choice, as exact
// ones would be k more rows of exact sums a token.  They are off by r at most and in
// effect by no more than a float32 rounding (4,096 x 7168 x 256: 2.8e-8 against 2.8e-8).
//
// A token whose radius is 1/16 or more, or no number, has every logit computed exactly,
// by its own wave: a batch of such tokens (4,096 x 7168 x 256) takes 1,385 us against
// 290 with MOE_ROUTER_FLOAT64 and 83 for ordinary ones.
//
// What bounds it: instructions.  A token takes some 1,740 vector and 1,115 scalar
// ones (counters, 4,096 tokens, 256 experts in 8 groups), 13 us of issue for the
// batch; its waves are resident at once, three quarters end after 16 us, and the
// tokens with open decisions (one in six) end last: 40 us.  A few tokens take 9-11
// us, of which a wave that runs alone spends most waiting for its own instructions,
// so the common pass is short, reductions go by DPP and the chosen are compared in
// pairs of lanes.
struct ScreenIn {
  const bf16_t *x, *w;
  const float *part, *xn, *wn;
  int d;
};

// LDS words (8 bytes) of one wave: keys (between passes: exact sums); logits;
// experts and places of the chosen; with SCREEN the experts of the exact sums.
__host__ __device__ constexpr int rg_words(int E, bool screen) { return 3 * E + (screen ? (E + 1) / 2 : 0); }

__device__ __forceinline__ uint64_t to_key(double c) { return score_key(c); }
__device__ __forceinline__ uint32_t to_key(float c) { return score_key32(c); }
__device__ __forceinline__ double to_score(uint64_t k) { return key_score(k); }
__device__ __forceinline__ float to_score(uint32_t k) { return key_logit(k); }
__device__ __forceinline__ uint64_t key_lane(uint64_t v, int lane) { return read_lane(v, lane); }
__device__ __forceinline__ uint32_t key_lane(uint32_t v, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}
__device__ __forceinline__ uint32_t shfl_key(uint32_t v, int lane) { return __shfl(v, lane, 64); }
__device__ __forceinline__ uint64_t shfl_key(uint64_t v, int lane) {
  return (uint64_t)__shfl((unsigned long long)v, lane, 64);
}

// The k-th largest key's value or a lower one that exactly k keys reach (1 <= k <=
// keys > 0), by a radix search of two bits a step (three independent counts take
// little longer than one); *got is how many keys reach it.
template <int KPL, class K>
__device__ __forceinline__ K kth_key(const K (&key)[KPL], int k, int* got) {
  K v = 0;
  int g = -1;
#pragma unroll 1
  for (int b = 8 * (int)sizeof(K) - 2; b >= 0 && g != k; b -= 2) {
    int c[3] = {0, 0, 0};
#pragma unroll
    for (int s = 0; s < KPL; ++s)
#pragma unroll
      for (int i = 0; i < 3; ++i) c[i] += __popcll(__ballot(key[s] >= (v | ((K)(i + 1) << b))));
    const int i = c[2] >= k ? 3 : (c[1] >= k ? 2 : (c[0] >= k ? 1 : 0));
    if (i) {
      v |= (K)i << b;
      g = c[2] >= k ? c[2] : (c[1] >= k ? c[1] : c[0]);
    }
  }
  *got = g;
  return v;
}

// Exact dot products of the token's row x with n rows (row_of(c), c < n): exact
// products, float64 sums, sink(c, sum) on every lane with the sum.  Two rows at a
// time against one reading of x, four steps of 512 elements in flight; the lanes
// are added by DPP.  (At 4,096 tokens, d = 7168, the tokens with open decisions end
// last: 48 us for this kernel with one row after the other and LDS sums, or with
// four rows, whose registers spill; 38 us so.)
template <class RowOf, class Sink>
__device__ __forceinline__ void wave_dots(const bf16_t* __restrict__ x, int d, int n, RowOf row_of, Sink sink) {
  constexpr int CB = 2, RING = 4;
  const int lane = threadIdx.x & 63;
  const int steps = (d + 511) / 512;
#pragma unroll 1
  for (int c0 = 0; c0 < n; c0 += CB) {
    const bf16_t* row[CB];
#pragma unroll
    for (int c = 0; c < CB; ++c) row[c] = row_of(min(c0 + c, n - 1));
    u32x4_t xv[RING], wv[RING][CB];
    double acc[CB] = {};
    auto load = [&](int q, int s) {
      const uint32_t off = (uint32_t)min(s * 512 + 8 * lane, d - 8);
      xv[q] = *reinterpret_cast<const u32x4_t*>(x + off);
#pragma unroll
      for (int c = 0; c < CB; ++c) wv[q][c] = *reinterpret_cast<const u32x4_t*>(row[c] + off);
    };
#pragma unroll
    for (int q = 0; q < RING; ++q) load(q, q);
#pragma unroll 1
    for (int s0 = 0; s0 < steps; s0 += RING) {
#pragma unroll
      for (int q = 0; q < RING; ++q) {
        const bool in = (s0 + q) * 512 + 8 * lane < d;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t xw = in ? xv[q][i] : 0u;
          const double x0 = (double)__uint_as_float(xw << 16), x1 = (double)__uint_as_float(xw & 0xffff0000u);
#pragma unroll
          for (int c = 0; c < CB; ++c) {
            const uint32_t ww = in ? wv[q][c][i] : 0u;
            acc[c] = fma(x0, (double)__uint_as_float(ww << 16), acc[c]);
            acc[c] = fma(x1, (double)__uint_as_float(ww & 0xffff0000u), acc[c]);
          }
        }
        load(q, s0 + q + RING);
      }
    }
#pragma unroll
    for (int c = 0; c < CB; ++c) {
      const double v = wave_sum(acc[c]);
      if (c0 + c < n) sink(c0 + c, v);
    }
  }
}

// What the selection of a token keeps between its passes, by slot s of a lane
// (expert lane + 64 s), as bits of one word.
struct Marks {
  uint32_t there, exact, mark;
};

// p = exp(l - top) (softmax) or exp(-l) in float64, through this wave's E words of
// LDS so that the long code of the exponential exists once and one slot's
// temporaries live at a time (four in parallel held 128 registers more).
template <int KPL>
__device__ __forceinline__ void exp_by_lds(const double (&l)[KPL], bool softmax, double top, double* buf, int E,
                                           double (&p)[KPL]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int s = 0; s < KPL; ++s)
    if (lane + 64 * s < E) buf[lane + 64 * s] = softmax ? l[s] - top : -l[s];
#pragma unroll 1
  for (int e = lane; e < E; e += 64) buf[e] = exp(buf[e]);
#pragma unroll
  for (int s = 0; s < KPL; ++s) p[s] = buf[min(lane + 64 * s, E - 1)];
  wave_sync();
}

// One pass in F (float or double).  Returns 0: decided (k chosen: chosen, ls =
// their logits, place), 1: m.mark asks for exact logits, 2: float32 cannot tell.
// r2: two radii of scores of inexact logits, per unit of the softmax's 1 / sum.
template <class F, int KPL>
__device__ __forceinline__ int route_pass(const double (&l)[KPL], const float (&sb)[KPL], bool biased, int E, int kt,
                                          const GroupRule& rule, double rl, Marks& m, uint64_t* lds, double* ls,
                                          int32_t* chosen, int32_t* place, int* k_out, double* top_out) {
  using K = typename std::conditional<sizeof(F) == 4, uint32_t, uint64_t>::type;
  constexpr bool F32 = sizeof(F) == 4;
  constexpr F tiny = F32 ? (F)0x1p-20 : (F)0;
  // opaque to the compiler: what follows from the lane is not worth a register
  // for the whole loop of passes
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  K key[KPL];
  F p[KPL], unit = 0, inv = 1;
  const bool softmax = rule.softmax;
  double topd = 0.0;
  if (softmax) {
    bool nan = false;
    topd = -INFINITY;
#pragma unroll
    for (int s = 0; s < KPL; ++s)
      if ((m.there >> s) & 1u) {
        topd = fmax(topd, l[s]);
        nan |= l[s] != l[s];
      }
    topd = wave_max(topd);
    if (__ballot(nan)) topd = NAN;  // a logit that is no number leaves no score of the token a number
  }
  F sum = 0;
  if constexpr (!F32) exp_by_lds<KPL>(l, softmax, topd, ls, E, p);
#pragma unroll
  for (int s = 0; s < KPL; ++s) {
    if constexpr (F32) p[s] = expf((float)(softmax ? l[s] - topd : -l[s]));
    sum += (m.there >> s) & 1u ? p[s] : (F)0;
  }
  if (softmax) inv = (F)1 / wave_sum(sum);
  *top_out = topd;
#pragma unroll
  for (int s = 0; s < KPL; ++s) {
    const F sc = softmax ? p[s] * inv : (F)1 / ((F)1 + p[s]);
    const F c = biased ? sc + (F)sb[s] : sc;
    key[s] = (m.there >> s) & 1u ? to_key(c) : 0;
    if constexpr (F32) {
      // float32: a few roundings of the score, |a| half steps of the exponent's
      // argument
      const float a = fminf(fabsf((float)(softmax ? l[s] - topd : l[s])), 1e4f);
      unit = fmaxf(unit, key[s] ? sc * (1.f + 0.125f * a) : 0.f);
    }
  }
  // two radii: of exact logits, and of inexact ones (expm1(2 rl) <= 2.2 rl); in
  // float32 a comparison adds what rounding the two values themselves may do, so
  // that one very large bias does not blur the others
  const F r0 = F32 ? tiny * wave_max(unit) + (F)0x1p-120 : (F)0;
  const F r1 = r0 + (F)(softmax ? 4.5 * rl * (double)inv : 0.51 * rl);
  auto far = [&](F a, F b, F mag, F r) { return F32 ? fabs(a - b) > r + tiny * mag : fabs(a - b) > r; };
  auto apart = [&](F a, F b, bool both_exact) {  // certainly in order
    return F32 || !both_exact ? far(a, b, (F)(fabs(a) + fabs(b)), both_exact ? r0 : r1) : true;
  };

  if (rule.topk_group < rule.n_group) {
    int gp = 1;
    while (gp < rule.n_group) gp *= 2;
    const int lpg = 64 / gp, per = E / rule.n_group, grp = lane / lpg, sub = lane % lpg;
    K* const kl = reinterpret_cast<K*>(lds);
    const float per_inv = (float)rule.n_group / (float)E;
    int first[KPL];  // first lane of a slot's group (E <= 1024: the quotient is exact)
#pragma unroll
    for (int s = 0; s < KPL; ++s) {
      const int e = min(lane + 64 * s, E - 1);
      first[s] = (int)(((float)e + 0.5f) * per_inv) * lpg;
      if ((m.there >> s) & 1u) kl[e] = key[s];
    }
    wave_sync();
    const bool mine = grp < rule.n_group;
    K m1 = 0, m2 = 0;
    if (mine) {
#pragma unroll 4
      for (int i = sub; i < per; i += lpg) merge2<K>(m1, m2, kl[grp * per + i], (K)0);
    }
#pragma unroll 1
    for (int off = 1; off < lpg; off <<= 1) {
      const K b1 = shfl_key(m1, lane ^ off), b2 = shfl_key(m2, lane ^ off);
      merge2<K>(m1, m2, b1, b2);
    }
    wave_sync();
    // two keys above -inf never add to an empty key
    const K val = rule.top2 && m1 && m2 ? to_key(to_score(m1) + to_score(m2)) : m1;
    // place of the lane's group: each of its lpg lanes compares with every lpg-th
    int rank = 0;
    if (mine && sub == 0) kl[grp] = val;
    wave_sync();
    for (int j = sub; j < rule.n_group; j += lpg) {
      const K vj = kl[j];
      rank += (vj > val || (vj == val && j < grp)) ? 1 : 0;
    }
#pragma unroll 1
    for (int off = 1; off < lpg; off <<= 1) rank += __shfl_xor(rank, off, 64);
    wave_sync();
    const uint64_t ml = __ballot(mine && rank == rule.topk_group - 1), mf = __ballot(mine && rank == rule.topk_group);
    // a float32 sum beyond the type's lowest value says nothing of the group
    if (F32 && __ballot(mine && m1 != 0 && val == 0)) return 2;
    const int ll = __builtin_ctzll(ml), lf = __builtin_ctzll(mf);
    const K vl = key_lane(val, ll), vf = key_lane(val, lf);
    const F z = rule.top2 ? (F)2 : (F)1;
    // what the rounding of a group's value goes by: the keys that are added
    const F mag = (F)(fabs(m1 ? to_score(m1) : (F)0) + fabs(rule.top2 && m2 ? to_score(m2) : (F)0));
    const F magl = to_score(key_lane(to_key(mag), ll)), magf = to_score(key_lane(to_key(mag), lf));
    // a group without experts in service is last, whatever the scores
    if (vf != 0 && !far(to_score(vl), to_score(vf), magl + magf, z * r1 + r0)) {
      const F v = to_score(val);
      const bool zone = mine && val != 0 && (!far(v, to_score(vl), mag + magl, z * r1 + r0) ||
                                             !far(v, to_score(vf), mag + magf, z * r1 + r0));
      const uint64_t zones = __ballot(zone);
      const K second = rule.top2 && m2 ? m2 : m1;
      m.mark = 0;
#pragma unroll
      for (int s = 0; s < KPL; ++s) {
        const K sec = shfl_key(second, first[s]);
        if (key[s] != 0 && ((zones >> first[s]) & 1ull) && !(to_score(sec) > to_score(key[s]) &&
              far(to_score(sec), to_score(key[s]), (F)(fabs(to_score(sec)) + fabs(to_score(key[s]))), r1)))
          m.mark |= 1u << s;
      }
      m.mark &= ~m.exact;
      if (__ballot(m.mark != 0)) return 1;
      if (F32 && !far(to_score(vl), to_score(vf), magl + magf, (z + 1) * r0)) return 2;
    }
    const uint64_t in_kept = __ballot(mine && rank < rule.topk_group);
#pragma unroll
    for (int s = 0; s < KPL; ++s)
      if (!((in_kept >> first[s]) & 1ull)) key[s] = 0;
  }

  int avail = 0;
#pragma unroll
  for (int s = 0; s < KPL; ++s) avail += __popcll(__ballot(key[s] != 0));
  const int k = min(kt, avail);
  *k_out = k;
  if (k == 0) return 0;
  int got;
  const K v = kth_key<KPL, K>(key, k, &got);
  // experts on either side of v, within the radius of it
  const F pv = to_score(v);
  uint32_t near = 0, near0 = 0, above = 0;
#pragma unroll
  for (int s = 0; s < KPL; ++s) {
    const F c = to_score(key[s]), m2 = (F)(fabs(c) + fabs(pv));
    if (key[s] != 0 && !far(c, pv, m2, r1)) near |= 1u << s;
    if (F32 && key[s] != 0 && !far(c, pv, m2, r0)) near0 |= 1u << s;
    if (key[s] >= v) above |= 1u << s;
  }
  m.mark = 0;
  if (got != k || (__ballot((near & above) != 0) && __ballot((near & ~above) != 0))) m.mark = near & ~m.exact;
  if (F32 && !__ballot(m.mark != 0) &&
      (got != k || (__ballot((near0 & above) != 0) && __ballot((near0 & ~above) != 0))))
    return 2;
  // the chosen, listed in ascending expert order: the keys above v, then equal
  // ones from the lower expert on until there are k
  const uint64_t below = (1ull << lane) - 1ull;
  int n = 0, need = k;
  if (got != k) {
#pragma unroll
    for (int s = 0; s < KPL; ++s) need -= __popcll(__ballot(key[s] > v));
  }
  int slot[KPL];
  K* const kl = reinterpret_cast<K*>(lds);
#pragma unroll
  for (int s = 0; s < KPL; ++s) {
    bool sel = key[s] != 0 && key[s] >= v;
    if (got != k) {
      const uint64_t eq = __ballot(key[s] == v);
      sel = key[s] > v || (key[s] == v && __popcll(eq & below) < need);
      need -= min(need, (int)__popcll(eq));
    }
    const uint64_t b = __ballot(sel);
    slot[s] = sel ? n + __popcll(b & below) : -1;
    if (sel) {
      kl[slot[s]] = key[s];
      ls[slot[s]] = l[s];
      chosen[slot[s]] = lane + 64 * s;
      place[slot[s]] = (m.exact >> s) & 1u;  // for the loop below
    }
    n += __popcll(b);
  }
  wave_sync();
  // a chosen one's place is the number of chosen keys that are larger, or equal
  // with a lower expert: lanes hold pairs (i, j), P = 2^lp lanes for each i
  bool unsure = false;
  int lp = 0;
  while ((1 << lp) < k && lp < 6) ++lp;
  const int per_pass = 64 >> lp, pj = lane & ((1 << lp) - 1);
#pragma unroll 1
  for (int i0 = 0; i0 < k; i0 += per_pass) {
    const int i = i0 + (lane >> lp);
    const K ki = kl[min(i, k - 1)];
    const F ci = to_score(ki);
    const bool xi = place[min(i, k - 1)] & 1;
    int r = 0;
    bool close = false;
#pragma unroll 1
    for (int j0 = 0; j0 < k; j0 += 64) {
      const int j = j0 + pj;
      const bool pair = i < k && j < k;
      const K kj = kl[min(j, k - 1)];
      const bool xj = place[min(j, k - 1)] & 1;
      const bool touch = pair && i != j && !apart(ci, to_score(kj), xi && xj);
      unsure |= touch && xi && xj;
      const uint64_t first_lanes = (lp == 6 ? ~0ull : (1ull << (1 << lp)) - 1) << (lane & ~((1 << lp) - 1));
      r += __popcll(__ballot(pair && (kj > ki || (kj == ki && j < i))) & first_lanes);
      close |= (__ballot(touch && !xi) & first_lanes) != 0;
    }
    wave_sync();
    if (i < k && pj == 0) place[i] = (xi ? 1 : 0) | (r << 2) | (close ? 2 : 0);
    wave_sync();
  }
#pragma unroll
  for (int s = 0; s < KPL; ++s)
    if (slot[s] >= 0 && (place[slot[s]] & 2)) m.mark |= 1u << s;
  m.mark &= ~m.exact;
  if (__ballot(m.mark != 0)) return 1;
  return F32 && __ballot(unsure) ? 2 : 0;
}

template <int KPL, bool SCREEN>
__global__ __launch_bounds__(256, KPL <= 4 ? 4 : 1) void route_grouped_kernel(const double* __restrict__ part, int S, ScreenIn in,
                                                            const float* __restrict__ bias,
                                                            const float* __restrict__ sel_bias,
                                                            const int32_t* __restrict__ tok_off, int T_, int E,
                                                            GroupRule rule, float scale, int32_t* __restrict__ ids,
                                                            float* __restrict__ wts) {
  extern __shared__ uint64_t rg_lds[];
  // wv is uniform: with it in a scalar register so are the token and its addresses
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = grid_block() * (int)(blockDim.x >> 6) + wv;
  if (t >= T_) return;
  uint64_t* const lds = rg_lds + (size_t)wv * rg_words(E, SCREEN);
  double* const ls = reinterpret_cast<double*>(lds + E);
  int32_t* const chosen = reinterpret_cast<int32_t*>(lds + 2 * E);
  int32_t* const place = chosen + E;
  const int base = tok_off[t];
  const int kt = tok_off[t + 1] - base;
  // slices are added in ascending order, G of them in flight (the last one's
  // address again behind the end: no branch between the loads)
  constexpr int G = KPL <= 4 ? (SCREEN ? 4 : 8) : 2;
  double l[KPL];
  float wn[KPL], bs[KPL], sb[KPL], xx = 0.f;
  Marks m{0u, 0u, 0u};
#pragma unroll
  for (int s = 0; s < KPL; ++s) {
    const uint32_t e = (uint32_t)min(lane + 64 * s, E - 1);
    l[s] = 0.0;
    wn[s] = 0.f;
    bs[s] = bias ? bias[e] : 0.f;
    sb[s] = sel_bias ? sel_bias[e] : 0.f;
    if (lane + 64 * s < E) m.there |= 1u << s;
  }
  if constexpr (SCREEN) xx = lane < S ? in.xn[(size_t)lane * T_ + t] : 0.f;  // S <= 32
#pragma unroll 1
  for (int q0 = 0; q0 < S; q0 += G) {
    typename std::conditional<SCREEN, float, double>::type v[KPL][G];
    float n[KPL][G];
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const size_t q = (size_t)min(q0 + i, S - 1);
#pragma unroll
      for (int s = 0; s < KPL; ++s) {
        const uint32_t e = (uint32_t)min(lane + 64 * s, E - 1);
        if constexpr (SCREEN) {
          v[s][i] = (in.part + (q * T_ + t) * E)[e];
          n[s][i] = (in.wn + q * E)[e];
        } else {
          v[s][i] = (part + (q * T_ + t) * E)[e];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < G; ++i) {
      if (q0 + i >= S) break;
#pragma unroll
      for (int s = 0; s < KPL; ++s) {
        l[s] += (double)v[s][i];
        if constexpr (SCREEN) wn[s] += n[s][i];
      }
    }
  }
  if (kt == 0) return;
#pragma unroll
  for (int s = 0; s < KPL; ++s) {
    l[s] += (double)bs[s];
    if (!SCREEN) l[s] = (double)(float)l[s];
  }
  if (!SCREEN) m.exact = m.there;
  double rl = 0.0;  // how far a logit may be off
  bool wide = rule.softmax && sel_bias;
  bool all = false;
  if constexpr (SCREEN) {
    float ww = 0.f, lm = 0.f;
    bool nan = false;
#pragma unroll
    for (int s = 0; s < KPL; ++s) {
      // a bias that is not finite decides its logit whatever the products are: it says
      // nothing of the others' (-inf at one of 256 experts, 4,096 tokens: 84 us a call
      // where every logit computed exactly takes 1,383)
      const bool decided = !(fabsf(bs[s]) < INFINITY);
      nan |= wn[s] != wn[s] || (l[s] != l[s] && !decided);
      ww = fmaxf(ww, wn[s]);
      lm = fmaxf(lm, decided ? 0.f : fabsf((float)l[s]));
    }
    // 1.01: the float32 sums of the squares (at most 65,536 terms of 2^-24 each); each
    // square below the normal range may be short of 2^-126
    const float low = (float)in.d * 0x1p-126f;
    const double prod = 1.01 * (double)sqrtf(wave_sum(xx) + low) * (double)sqrtf(wave_max(ww) + low);
    const double r = prod * (66.0 * 0x1p-23 + 0x1p-24) + in.d * 0x1p-126;
    rl = r + ((double)wave_max(lm) + r) * 0x1.1p-24 + 0x1p-149;  // and the one rounding of the exact logit
    all = __ballot(nan) != 0 || !(rl < 0.0625);
    if (all) {
      m.mark = m.there;
      rl = 0.0;
    }
  }

  int k = 0, state = all ? 1 : 0;
  double top = 0.0;
#pragma unroll 1
  for (;;) {
    if (!all) {
      if (!wide) {
        state = route_pass<float, KPL>(l, sb, sel_bias != nullptr, E, kt, rule, rl, m, lds, ls, chosen, place, &k, &top);
        wide = state == 2;
      }
      if (wide)
        state = route_pass<double, KPL>(l, sb, sel_bias != nullptr, E, kt, rule, rl, m, lds, ls, chosen, place, &k, &top);
      if (state == 0) break;
    }
    all = false;
    if constexpr (SCREEN) {  // exact logits of the marked slots
      int32_t* const list = reinterpret_cast<int32_t*>(lds + 3 * E);
      double* const val = reinterpret_cast<double*>(lds);
      const uint64_t below = (1ull << lane) - 1ull;
      int n = 0, at[KPL];
#pragma unroll
      for (int s = 0; s < KPL; ++s) {
        const bool want = (m.mark >> s) & 1u;
        const uint64_t b = __ballot(want);
        at[s] = n + __popcll(b & below);
        if (want) list[at[s]] = lane + 64 * s;
        n += __popcll(b);
      }
      wave_sync();
      wave_dots(
          in.x + (size_t)t * in.d, in.d, n,
          [&](int c) { return in.w + (size_t)__builtin_amdgcn_readfirstlane(list[c]) * in.d; },
          [&](int c, double v) {
            if (lane == 0) val[c] = v;
          });
      wave_sync();
#pragma unroll
      for (int s = 0; s < KPL; ++s)
        if ((m.mark >> s) & 1u) l[s] = (double)(float)(val[at[s]] + (double)bs[s]);
      m.exact |= m.mark;
      m.mark = 0;
      wave_sync();
    }
  }

  // ids and weights: the chosen's scores in float64 from their logits (a softmax's
  // sum cancels where the weights are renormalised)
  double p = 0.0, denom = 1.0;
  if (rule.softmax && !rule.renorm) {
    double pe[KPL];
    exp_by_lds<KPL>(l, true, top, reinterpret_cast<double*>(lds), E, pe);
#pragma unroll
    for (int s = 0; s < KPL; ++s) p += (m.there >> s) & 1u ? pe[s] : 0.0;
    denom = wave_sum(p);
    p = 0.0;
  }
#pragma unroll 1
  for (int i = lane; i < k; i += 64) {
    const double a = ls[i], q = exp(rule.softmax ? a - top : -a);
    ls[i] = (rule.softmax ? q : 1.0) / (rule.softmax ? denom : 1.0 + q);
    p += ls[i];
    ids[base + (place[i] >> 2)] = chosen[i];
  }
  const double total = rule.renorm ? wave_sum(p) : 1.0;
#pragma unroll 1
  for (int i = lane; i < k; i += 64)
    wts[base + (place[i] >> 2)] = total > 0.0 ? (float)((double)scale * (ls[i] / total)) : 0.f;
#pragma unroll 1
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
  const dim3 grid = grid_of((T + nw - 1) / nw);
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
