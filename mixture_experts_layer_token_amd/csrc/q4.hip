// 4-bit weights with group scales: quantising, re-laying, widening, and the product
// with few rows (moe_q4_pack, moe_q4_tile, moe_q4_unpack, moe_q4_linear).  rowtile.h
// has the order of the codes and the product's arithmetic.
#include "common.h"
#include "launch.h"
#include "rowtile.h"

namespace moe {

// ------------------------------------------------------------------- quantising
// A group of GROUP inputs of a row has the scale
//   s = ELT(max |w| / 7), codes 8 + rne(w / s)               without zero points
//   s = ELT((hi - lo) / 15), z = rne(-lo / s), codes z + rne(w / s)   with,
// lo and hi the group's range with 0 in it, codes held in [1, 15] or [0, 15].  The
// codes are those of the stored scale; rne takes the exact quotient, ties to even.
// The quotient is w times 1 / s in float32, within 4e-6 of the exact one (no value exceeds
// 16 of them).  For float32 weights the remainder w - s r, whose sign and comparison with
// s / 2 are exact in one fused step, then puts right an r on the wrong side of a tie.  For
// bf16 weights a quotient that is no tie lies 2^-10 or more from each (both mantissas have
// 8 bits, a tie is an odd number of halves), so that rounding to 2^-12 first leaves ties
// exactly on theirs and nothing else; that saves the half of pack's time that ties, frequent
// in bf16, took.
// A group whose values are all 0 (or whose scale rounds to 0) has scale 0; one with a
// value that is no finite number has scale NaN.

// rne(w / s) of q = w * (1 / s), s not below 2^-100.
__device__ __forceinline__ float q4_rne(float w, float s, float q) {
  const float r = rintf(q), e = fmaf(-s, r, w), h = 0.5f * s, up = e > 0.f ? 1.f : -1.f;
  if (fabsf(e) > h) return r + up;
  return fabsf(e) == h && ((int)r & 1) ? r + up : r;
}

// The largest of a group's GROUP / 8 threads (neighbours), in each of them.
template <int GROUP, class F>
__device__ __forceinline__ uint32_t q4_all(uint32_t v, F f) {
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0xB1, 0xF, 0xF, false));   // lane ^ 1
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x4E, 0xF, 0xF, false));   // lane ^ 2
  if (GROUP > 32) v = f(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x141, 0xF, 0xF, false));  // halves of 8
  if (GROUP > 64) v = f(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x140, 0xF, 0xF, false));  // of 16
  return v;
}

// Eight elements of a row (16-byte aligned), read once: past the caches.
__device__ __forceinline__ void q4_load8(const bf16_t* p, float (&v)[8]) {
  const u32x4_t u = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void q4_load8(const float* p, float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x4_t u = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(p) + h);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * h + i] = u[i];
  }
}

// One thread quantises the 8 inputs of a code word; the GROUP / 8 threads of a group agree
// on its range.  A workgroup takes 16 rows x QP_T tiles of 128 inputs (256 threads: row
// tid / 16, word tid % 16 of each tile), whose loads are in flight together, and writes the
// codes through LDS in the tile's order.  Bound by memory: 8 matrices of 14336 x 4096 bf16 in 218
// .. 260 us, 4.6 .. 5.4 TB/s of reads and writes (a copy makes 4.9); with a division an element
// and one tile a workgroup 400.
constexpr int QP_T = 4;

template <typename T, int GROUP, bool ZEROS>
__global__ __launch_bounds__(256) void q4_pack_kernel(const T* __restrict__ w, int G, int N, int K, int kt_n, int nt_n,
                                                      uint32_t* __restrict__ codes, T* __restrict__ scales,
                                                      uint8_t* __restrict__ zeros) {
  __shared__ uint32_t buf[QP_T][256];
  constexpr int NG = Q4_K / GROUP;
  const int tid = threadIdx.x, r = tid >> 4, c = tid & 15, kq = ceil_div(kt_n, QP_T);
  const int kt0 = blockIdx.x % kq * QP_T, nt = blockIdx.x / kq, tiles = min(QP_T, kt_n - kt0);
  const int n = nt * TILE_N + r, k0 = kt0 * Q4_K + 8 * c;
  const int Np = nt_n * TILE_N;
  for (int g = blockIdx.y; g < G; g += gridDim.y) {
    const T* const row = w + ((size_t)g * N + n) * K + k0;
    float v[QP_T][8];
#pragma unroll
    for (int i = 0; i < QP_T; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
      if (n < N && k0 + i * Q4_K < K) q4_load8(row + i * Q4_K, v[i]);
    }
#pragma unroll
    for (int i = 0; i < QP_T; ++i) {
      // |w| as integers: their order, infinities and NaN behind the numbers
      uint32_t top = 0;
      float lo = 0.f, hi = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        top = max(top, __float_as_uint(v[i][j]) & 0x7fffffffu);
        if (ZEROS) lo = fminf(lo, v[i][j]), hi = fmaxf(hi, v[i][j]);
      }
      top = q4_all<GROUP>(top, [](uint32_t a, uint32_t b) { return max(a, b); });
      float s32;
      if (ZEROS) {
        lo = __uint_as_float(q4_all<GROUP>(__float_as_uint(lo), [](uint32_t a, uint32_t b) {
          return __float_as_uint(fminf(__uint_as_float(a), __uint_as_float(b))); }));
        hi = __uint_as_float(q4_all<GROUP>(__float_as_uint(hi), [](uint32_t a, uint32_t b) {
          return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b))); }));
        s32 = (float)(((double)hi - (double)lo) / 15.0);
      } else {
        s32 = __uint_as_float(top) / 7.f;
      }
      const T st = Elt<T>::from_f32(top >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : s32);
      const float s = Elt<T>::to_f32(st);
      const bool live = s > 0.f && s < INFINITY;
      // tiny scales and their weights 2^64 times larger, for 1 / s to exist and w - s r to be exact
      const float lift = s < 0x1p-100f ? 0x1p64f : 1.f, sl = s * lift, inv = live ? 1.f / sl : 0.f;
      const float z = !ZEROS ? 8.f : live ? fminf(fmaxf(q4_rne(-lo * lift, sl, -lo * lift * inv), 0.f), 15.f) : 0.f;
      const float least = ZEROS ? -z : -7.f, most = ZEROS ? 15.f - z : 7.f;
      float q[8];
      bool clear = true;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (sizeof(T) == 2) {
          q[j] = fmaf(v[i][j] * lift, inv, 0x1.8p11f) - 0x1.8p11f;
        } else {
          q[j] = v[i][j] * lift * inv;
          clear &= fabsf(q[j] - rintf(q[j])) < 0.49999f;
        }
      }
      if (sizeof(T) == 4 && !clear) {
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = q4_rne(v[i][j] * lift, sl, q[j]);
      }
      // 1.5 * 2^23 + q rounds q to even and has it in its low bits; the constants' sum goes out again
      uint32_t word = 0, base = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = 4 * (j >> 1) + 16 * (j & 1);
        word += __float_as_uint(fminf(fmaxf(q[j], least), most) + 0x1.8p23f) << at;
        base += 0x4b400000u << at;
      }
      word = (live ? word - base : 0u) + (uint32_t)z * 0x11111111u;
      // word c of row r: instruction c / 4, lane group c % 4
      buf[i][((c & 3) * 16 + r) * 4 + (c >> 2)] = word;
      if (i < tiles && (c & (GROUP / 8 - 1)) == 0) {
        const size_t o = (((size_t)g * kt_n + kt0 + i) * NG + c / (GROUP / 8)) * Np + n;
        scales[o] = n < N ? st : T(0);
        if (ZEROS) zeros[o] = (uint8_t)z;
      }
    }
    __syncthreads();
    // 16 bytes a thread: tiles in a row
    if (tid < 64 * tiles)
      __builtin_nontemporal_store(reinterpret_cast<const u32x4_t*>(buf)[tid],
                                  reinterpret_cast<u32x4_t*>(codes + (((size_t)g * nt_n + nt) * kt_n + kt0) * 256) + tid);
    __syncthreads();
  }
}

// Re-lays row-major codes (input 2 j in the low half of byte j), scales and zero points
// [G][N][groups]; threads and tiles as in packing.  Bound by memory: 256 matrices of 2048 x
// 7168, groups of 64 with zero points, in 770 .. 800 us, 5.2 TB/s (one tile a workgroup: 1,930 ..
// 2,040).
template <typename T, int GROUP, bool ZEROS>
__global__ __launch_bounds__(256) void q4_tile_kernel(const uint8_t* __restrict__ src, const T* __restrict__ s_in,
                                                      const uint8_t* __restrict__ z_in, int G, int N, int K, int kt_n,
                                                      int nt_n, uint32_t* __restrict__ codes, T* __restrict__ scales,
                                                      uint8_t* __restrict__ zeros) {
  __shared__ uint32_t buf[QP_T][256];
  constexpr int NG = Q4_K / GROUP;
  const int tid = threadIdx.x, r = tid >> 4, c = tid & 15, kq = ceil_div(kt_n, QP_T);
  const int kt0 = blockIdx.x % kq * QP_T, nt = blockIdx.x / kq, tiles = min(QP_T, kt_n - kt0);
  const int n = nt * TILE_N + r, k0 = kt0 * Q4_K + 8 * c;
  const int Np = nt_n * TILE_N, ng = ceil_div(K, GROUP);
  for (int g = blockIdx.y; g < G; g += gridDim.y) {
    const uint8_t* const row = src + (((size_t)g * N + n) * K + k0) / 2;
    uint32_t u[QP_T];
#pragma unroll
    for (int i = 0; i < QP_T; ++i)
      u[i] = n < N && k0 + i * Q4_K < K ? *reinterpret_cast<const uint32_t*>(row + i * (Q4_K / 2)) : 0u;
#pragma unroll
    for (int i = 0; i < QP_T; ++i) {
      uint32_t word = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) word |= ((u[i] >> (4 * j)) & 15u) << (4 * (j >> 1) + 16 * (j & 1));
      buf[i][((c & 3) * 16 + r) * 4 + (c >> 2)] = word;
    }
    // scales: of one group, 16 rows side by side (they are written so)
    for (int e = tid; e < tiles * NG * TILE_N; e += 256) {
      const int gi = kt0 * NG + e / TILE_N, m = nt * TILE_N + e % TILE_N;
      const size_t o = ((size_t)g * kt_n * NG + gi) * Np + m, i = ((size_t)g * N + m) * ng + gi;
      const bool in = m < N && gi < ng;
      scales[o] = in ? s_in[i] : T(0);
      if (ZEROS) zeros[o] = in ? z_in[i] : 0;
    }
    __syncthreads();
    if (tid < 64 * tiles)
      __builtin_nontemporal_store(reinterpret_cast<const u32x4_t*>(buf)[tid],
                                  reinterpret_cast<u32x4_t*>(codes + (((size_t)g * nt_n + nt) * kt_n + kt0) * 256) + tid);
    __syncthreads();
  }
}

// The values s (q - z), rounded once to the element type; threads and tiles as in packing.
// The same matrices back in 190 .. 225 us, 5.2 .. 6.2 TB/s (one tile a workgroup, cached stores: 345).
template <typename T, int GROUP, bool ZEROS>
__global__ __launch_bounds__(256) void q4_unpack_kernel(const uint32_t* __restrict__ codes,
                                                        const T* __restrict__ scales,
                                                        const uint8_t* __restrict__ zeros, int G, int N, int K,
                                                        int kt_n, int nt_n, T* __restrict__ w) {
  __shared__ uint32_t buf[QP_T][256];
  constexpr int NG = Q4_K / GROUP;
  const int tid = threadIdx.x, r = tid >> 4, c = tid & 15, kq = ceil_div(kt_n, QP_T);
  const int kt0 = blockIdx.x % kq * QP_T, nt = blockIdx.x / kq, tiles = min(QP_T, kt_n - kt0);
  const int n = nt * TILE_N + r, k0 = kt0 * Q4_K + 8 * c;
  const int Np = nt_n * TILE_N;
  for (int g = blockIdx.y; g < G; g += gridDim.y) {
    if (tid < 64 * tiles)
      reinterpret_cast<u32x4_t*>(buf)[tid] = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4_t*>(codes + (((size_t)g * nt_n + nt) * kt_n + kt0) * 256) + tid);
    float s[QP_T];
    int z[QP_T];
#pragma unroll
    for (int i = 0; i < QP_T; ++i) {
      const size_t o = (((size_t)g * kt_n + min(kt0 + i, kt_n - 1)) * NG + c / (GROUP / 8)) * Np + n;
      s[i] = Elt<T>::to_f32(scales[o]);
      z[i] = ZEROS ? zeros[o] : 8;
    }
    __syncthreads();
    T* const row = w + ((size_t)g * N + n) * K + k0;
#pragma unroll
    for (int i = 0; i < QP_T; ++i)
      if (n < N && k0 + i * Q4_K < K) {
        const uint32_t word = buf[i][((c & 3) * 16 + r) * 4 + (c >> 2)];
        f32x4_t v[2];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[j >> 2][j & 3] = s[i] * (float)((int)((word >> (4 * (j >> 1) + 16 * (j & 1))) & 15u) - z[i]);
        T* const p = row + i * Q4_K;
        if constexpr (sizeof(T) == 2) {
          u32x4_t o;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            o[j] = (uint32_t)f32_to_bf16(v[j >> 1][2 * (j & 1)]) | ((uint32_t)f32_to_bf16(v[j >> 1][2 * (j & 1) + 1]) << 16);
          __builtin_nontemporal_store(o, reinterpret_cast<u32x4_t*>(p));
        } else {
          __builtin_nontemporal_store(v[0], reinterpret_cast<f32x4_t*>(p));
          __builtin_nontemporal_store(v[1], reinterpret_cast<f32x4_t*>(p) + 1);
        }
      }
    __syncthreads();
  }
}

// -------------------------------------------------------------- few-row product
// y[r][n] = sum_k x[r][k] W[n][k].  A workgroup takes NT tiles of 16 outputs and R blocks of
// 16 rows, its waves a share of K each, and adds their sums in LDS.  One row of 7168 inputs to
// 2048 outputs takes 6.9 us, floor 1.1 (7.6 MB at 7.2 TB/s): latency of a launch, of two rounds
// of loads and of the code's fetch (four steps a round 7.1, one 6.7; 4096 inputs 6.9, 5.3 with two
// and with one; 8192 outputs of them 12.8, 7.8 with two, 9.3 with one).
template <class Op, int R, int NT, int U, int NW>
__global__ __launch_bounds__(64 * NW) void q4_linear_kernel(const typename Op::elt* __restrict__ x, RowWeights w,
                                                            int rows, int N, int K,
                                                            typename Op::elt* __restrict__ y) {
  typedef typename Op::elt T;
  __shared__ f32x4_t red[NT][NW * 64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, col = lane & 15;
  const int n0 = blockIdx.x * (NT * TILE_N), r0 = blockIdx.y * (16 * R);
  const int steps = ceil_div(K, Q4_K);
  const int beg = steps * wave / NW, end = steps * (wave + 1) / NW;
  const T* const x0 = x + (size_t)r0 * K;
  uint32_t xrow[R];
#pragma unroll
  for (int r = 0; r < R; ++r)  // rows behind the last repeat it; their sums are not used
    xrow[r] = (uint32_t)min(16 * r + col, rows - 1 - r0) * K * (uint32_t)sizeof(T);
  f32x4_t acc[NT][R];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < R; ++r) acc[t][r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  typename Op::Src src[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t)  // tiles behind the last repeat it
    src[t] = Op::tile(w, 0, min(n0 + t * TILE_N, ceil_div(N, TILE_N) * TILE_N - TILE_N), N, K);
#pragma unroll 1
  for (int s = beg; s < end; s += U) {
    typename Op::W v[U][NT];
    typename Op::X xv[U][R];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = min(s + u, end - 1);
#pragma unroll
      for (int t = 0; t < NT; ++t) v[u][t] = Op::load(src[t], at);
#pragma unroll
      for (int r = 0; r < R; ++r) xv[u][r] = Op::load_x(x0, xrow[r], at, K);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + u < end) {
        Op::template step<4>(acc, v[u], xv[u]);
      }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      settle(acc[t][r]);
      red[t][wave * 64 + lane] = acc[t][r];
    }
    __syncthreads();
#pragma unroll 1
    for (int i = threadIdx.x; i < NT * 256; i += 64 * NW) {
      // output j of row c of the block
      const int j = i % (NT * 16), c = i / (NT * 16), n = n0 + j, row = r0 + 16 * r + c;
      const float* q = reinterpret_cast<const float*>(red[j >> 4]) + ((c >> 2) * 16 + (j & 15)) * 4 + (c & 3);
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < NW; ++k) sum += q[k * 256];
      const bool mine = row < rows && n < N;
      redo_not_finite(sum, mine, c, [&](int l, bool& nan) {
        const int e = i - lane + l;
        const T* xr = x0 + (size_t)(16 * r + e / (NT * 16)) * K;
        const int nn = n0 + e % (NT * 16);
        return wave_dot(K, [&](int k) { return Elt<T>::to_f32(xr[k]); },
                        [&](int k) { return Op::value(w, 0, nn, k, N, K, 0); }, nan);
      });
      if (mine) y[(size_t)row * N + n] = Elt<T>::from_f32(sum);
    }
    if (r + 1 < R) __syncthreads();
  }
}

// Many outputs: the waves of a workgroup take NT tiles each and walk K together, the
// activations of a step in LDS for all of them (each wave by itself would read four to
// sixteen times the codes' bytes from L2).  Codes, scales and zero points come through a
// ring of the wave's own, NB - 1 steps ahead, the activations with them.
// 24 rows of 4096 inputs to 50257 outputs: 41 us, floor 16 (115 MB at 7.2 TB/s).  The copies
// alone take 28; then some 95 vector instructions and 16 matrix instructions a tile and step, on
// SIMDs of which the fullest have 4 waves where 3.1 would be even.  Two tiles a wave 44 us; 4 waves
// a workgroup 57, with two tiles 46; the next step's operands read ahead into registers 53 (150
// registers, a workgroup less on a CU) or 113 (128 of them, spilled).
constexpr int QL_WW = 8;

template <class Op, int R, int NT, int NB>
__global__ __launch_bounds__(64 * QL_WW) void q4_wide_kernel(const typename Op::elt* __restrict__ x, RowWeights w,
                                                             int rows, int N, int K,
                                                             typename Op::elt* __restrict__ y) {
  typedef typename Op::elt T;
  static_assert(sizeof(T) == 2, "bf16 activations");
  constexpr int RUN = 32, SB = Op::NG * RUN;            // a tile's scales of a step, then its zero points
  constexpr int SZ = SB + (Op::ZP ? Op::NG * 16 : 0);
  constexpr int XP = R < 2 ? 1 : R / 2;                 // copies of activations of a wave
  constexpr int TILE = 1024 + 256, MINE = NT * TILE, XB = 4096 * R;
  static_assert(SZ <= 256, "one copy");
  constexpr int PER = 2 * NT + XP;
  extern __shared__ char ql_ring[];                     // [NB][XB], then [waves][NB][MINE]
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, col = lane & 15;
  const int nt = ceil_div(N, TILE_N), r0 = blockIdx.y * (16 * R), steps = ceil_div(K, Q4_K);
  const int tile0 = (near_tile(blockIdx.x, gridDim.x) * QL_WW + wave) * NT;
  const T* const x0 = x + (size_t)r0 * K;
  char* const mine = ql_ring + NB * XB + wave * (NB * MINE);

  // copy c of a step's activations: rows 16 (c / 4) + 8 (c % 2) .., inputs 64 (c / 2 % 2) ..
  uint32_t xoff[XP];
#pragma unroll
  for (int i = 0; i < XP; ++i) {
    const int c = (wave + QL_WW * i) % (4 * R);
    xoff[i] = (uint32_t)min(16 * (c >> 2) + copy_row(c & 1), rows - 1 - r0) * K * 2u;
  }
  // what the next request copies
  const char *q[NT], *sz[NT];
  uint32_t sz_step = 0;
#pragma unroll
  for (int t = 0; t < NT; ++t) {  // tiles behind the last repeat it
    const typename Op::Src src = Op::tile(w, 0, min(tile0 + t, nt - 1) * TILE_N, N, K);
    q[t] = reinterpret_cast<const char*>(src.q);
    const int b = 4 * lane % SZ, o = b < SB ? b : b - SB;  // lanes behind the last copy some again
    const uint32_t run = b < SB ? RUN : 16, pitch = src.Np * (b < SB ? 2u : 1u);
    sz_step = Op::NG * pitch;
    sz[t] = (b < SB ? reinterpret_cast<const char*>(src.s) : reinterpret_cast<const char*>(src.z)) +
            (size_t)(o / run * pitch + o % run);
  }
  int rs = 0;
  auto request = [&](int slot) {
    char* to = mine + slot * MINE;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      copy_rows<2>(q[t], 16 * lane, to + t * TILE);
      __builtin_amdgcn_global_load_lds((gbl_ptr_t)sz[t], (lds_ptr_t)(to + t * TILE + 1024), 4, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < XP; ++i) {
      const int c = (wave + QL_WW * i) % (4 * R);
      // inputs behind K: any of the row's, taken out below
      const uint32_t k = min(rs * 256u + (c >> 1 & 1) * 128u + copy_byte(c & 1), 2u * K - 16u);
      copy_rows<0>(x0, xoff[i] + k, ql_ring + slot * XB + (c >> 2) * 4096 + (c >> 1 & 1) * 2048 + (c & 1) * 1024);
    }
    if (rs + 1 < steps) {  // else the last step again
      ++rs;
#pragma unroll
      for (int t = 0; t < NT; ++t) q[t] += 1024, sz[t] += sz_step;
    }
  };
  f32x4_t acc[NT][R];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < R; ++r) acc[t][r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int i = 0; i < NB - 1; ++i) request(i);
  int slot = 0;
#pragma unroll 1
  for (int s = 0; s < steps; ++s) {
    vm_wait<PER * (NB - 2)>();
    compiler_fence();
    __builtin_amdgcn_s_barrier();  // everyone's copies of this step; everyone has read the last one's
    compiler_fence();
    request(slot == 0 ? NB - 1 : slot - 1);
    const char* const from = mine + slot * MINE;
    typename Op::W v[NT];
    typename Op::X xv[R];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      v[t].q = *reinterpret_cast<const u32x4_t*>(from + t * TILE + 16 * lane);
#pragma unroll
      for (int g = 0; g < Op::NG; ++g) {
        v[t].s[g] = *reinterpret_cast<const T*>(from + t * TILE + 1024 + g * RUN + 2 * col);
        if (Op::ZP) v[t].z[g] = *reinterpret_cast<const uint8_t*>(from + t * TILE + 1024 + SB + g * 16 + col);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        xv[r].v[0][i] = *reinterpret_cast<const u32x4_t*>(ql_ring + slot * XB + r * 4096 + (i >> 1) * 2048 +
                                                          lds_off(col, (lane >> 4) + 4 * (i & 1)));
    lgkm_wait0();
    compiler_fence();
    if (s == steps - 1 && K % Q4_K) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (s * Q4_K + 32 * i + 8 * (lane >> 4) >= K) {
#pragma unroll
          for (int r = 0; r < R; ++r) xv[r].v[0][i] = u32x4_t{0, 0, 0, 0};
        }
    }
    Op::template step<4>(acc, v, xv);
    slot = slot + 1 == NB ? 0 : slot + 1;
  }
  vm_wait<0>();  // no copy into LDS outlives the workgroup
  compiler_fence();
  // a wave's results through its own part of the ring: value i of a lane at 64 i
  float* const out = reinterpret_cast<float*>(mine);
  static_assert(NT * R * 1024 <= NB * MINE, "the results fit the ring");
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      settle(acc[t][r]);
#pragma unroll
      for (int i = 0; i < 4; ++i) out[((t * R + r) * 4 + i) * 64 + lane] = acc[t][r][i];
    }
  lgkm_wait0();
  compiler_fence();
#pragma unroll 1
  for (int e = 0; e < NT * R * 4; ++e) {
    const int n = (tile0 + e / (4 * R)) * TILE_N + col, rb = r0 + 16 * (e / 4 % R) + e % 4, row = rb + 4 * (lane >> 4);
    float v = out[e * 64 + lane];
    const bool good = row < rows && n < N;
    redo_not_finite(v, good, row, [&](int l, bool& nan) {
      const T* xr = x + (size_t)(rb + 4 * (l >> 4)) * K;
      const int nn = n - col + (l & 15);
      return wave_dot(K, [&](int k) { return Elt<T>::to_f32(xr[k]); },
                        [&](int k) { return Op::value(w, 0, nn, k, N, K, 0); }, nan);
    });
    if (good) y[(size_t)row * N + n] = Elt<T>::from_f32(v);
  }
}

// -------------------------------------------------------------------- launches

#define MOE_Q4_GROUP(CALL, G)               \
  do {                                      \
    if (zeros) CALL(G, true); else CALL(G, false); \
  } while (0)
#define MOE_Q4_ALL(CALL)                        \
  do {                                          \
    if (s.group == 32) MOE_Q4_GROUP(CALL, 32);  \
    else if (s.group == 64) MOE_Q4_GROUP(CALL, 64); \
    else MOE_Q4_GROUP(CALL, 128);               \
  } while (0)

template <typename T>
static void pack_t(const Q4Shape& s, const void* w, void* codes, void* scales, void* zeros, hipStream_t st) {
  const int kt = ceil_div(s.K, Q4_K), nt = ceil_div(s.N, TILE_N);
#define MOE_CALL(GR_, ZP_)                                                                                          \
  hipLaunchKernelGGL((q4_pack_kernel<T, GR_, ZP_>), dim3((uint32_t)ceil_div(kt, QP_T) * nt, min(s.G, 65535)), dim3(256), 0, st, (const T*)w, s.G, s.N, s.K, \
                     kt, nt, (uint32_t*)codes, (T*)scales, (uint8_t*)zeros)
  MOE_Q4_ALL(MOE_CALL);
#undef MOE_CALL
}
template <typename T>
static void tile_t(const Q4Shape& s, const void* c_rm, const void* s_rm, const void* z_rm, void* codes, void* scales,
                   void* zeros, hipStream_t st) {
  const int kt = ceil_div(s.K, Q4_K), nt = ceil_div(s.N, TILE_N);
#define MOE_CALL(GR_, ZP_)                                                                                          \
  hipLaunchKernelGGL((q4_tile_kernel<T, GR_, ZP_>), dim3((uint32_t)ceil_div(kt, QP_T) * nt, min(s.G, 65535)), dim3(256), 0, st, (const uint8_t*)c_rm, \
                     (const T*)s_rm, (const uint8_t*)z_rm, s.G, s.N, s.K, kt, nt, (uint32_t*)codes, (T*)scales,      \
                     (uint8_t*)zeros)
  MOE_Q4_ALL(MOE_CALL);
#undef MOE_CALL
}
template <typename T>
static void unpack_t(const Q4Shape& s, const void* codes, const void* scales, const void* zeros, void* w,
                     hipStream_t st) {
  const int kt = ceil_div(s.K, Q4_K), nt = ceil_div(s.N, TILE_N);
#define MOE_CALL(GR_, ZP_)                                                                                          \
  hipLaunchKernelGGL((q4_unpack_kernel<T, GR_, ZP_>), dim3((uint32_t)ceil_div(kt, QP_T) * nt, min(s.G, 65535)), dim3(256), 0, st,              \
                     (const uint32_t*)codes, (const T*)scales, (const uint8_t*)zeros, s.G, s.N, s.K, kt, nt, (T*)w)
  MOE_Q4_ALL(MOE_CALL);
#undef MOE_CALL
}
template <class Op, int R, int NT, int U, int NW>
static void linear_as(const Q4Shape& s, int rows, const void* x, const RowWeights& w, void* y, hipStream_t st) {
  typedef typename Op::elt T;
  hipLaunchKernelGGL((q4_linear_kernel<Op, R, NT, U, NW>), dim3(ceil_div(s.N, NT * TILE_N), ceil_div(rows, 16 * R)),
                     dim3(64 * NW), 0, st, (const T*)x, w, rows, s.N, s.K, (T*)y);
}
template <class Op, int R, int NT, int NB>
static void wide_as(const Q4Shape& s, int rows, const void* x, const RowWeights& w, void* y, hipStream_t st) {
  typedef typename Op::elt T;
  constexpr int LDS = NB * (4096 * R + QL_WW * NT * 1280);
  hipLaunchKernelGGL((q4_wide_kernel<Op, R, NT, NB>), dim3(ceil_div(s.N, QL_WW * NT * TILE_N), ceil_div(rows, 16 * R)),
                     dim3(64 * QL_WW), LDS, st, (const T*)x, w, rows, s.N, s.K, (T*)y);
}
// Tiles of a workgroup by the number of tiles: one where that already leaves a CU more than
// one workgroup, more where their common activations count (a workgroup of eight waves fills
// a CU's registers), and past that the kernel that shares them.  Measured at 4096 inputs,
// groups of 64 with zero points, both sides of each border in us:
//   16 rows, 512 tiles: 1 tile 12.0, 2 11.5 (one row: 7.8, 11.1); 1536: 2 tiles 22.2, shared 20.1
//   (one row: 17.1, 20.3); 2048: 29.8, 21.4
//   32 rows, 256 tiles: 1 tile 12.0, 2 12.4; 512: 22.2, 13.4; 1024: 2 tiles 21.7, 4 17.7, shared
//   24.2; 1536: 4 tiles 30.2, shared 25.2
//   64 rows, 256 tiles: 1 tile 19.3, 2 24.2; 512: 33.8, 25.1, shared 36.7; 768: 2 tiles 45.8, 37.1
//   4 float32 rows, 256 tiles: 1 tile 12.8, 2 14.1; 512: 22.9, 15.2, 4 tiles 21.2; 768: 26.5, 21.5
// At other lengths of a row the borders lie elsewhere, by what a workgroup has to do (us):
//   1024 inputs: one row, 512 tiles: 1 tile 4.9, 2 3.3; 1536: 2 tiles 6.9, shared 7.1; 32 rows, 256
//   tiles: 4.6, 5.2; 512: 6.9, 5.3; 1024: 2 tiles 7.7, 4 7.2, shared 9.1; 64 rows, 256: 7.1, 8.3; 640:
//   2 tiles 15.3, shared 13.3; 4 float32 rows, 256: 6.4, 4.9; 640: 2 tiles 8.5, 4 6.6
//   14336 inputs: one row, 512 tiles: 20.8, 25.9; 1024: 39.7, 34.6; 1536: 2 tiles 56.9, shared 56.7;
//   32 rows, 256: 29.9, 32.2; 512: 56.5, 32.8; 1024: 62.1, 4 tiles 41.7, shared 72.8; 1536: 4 tiles
//   78.5, 73.2; 64 rows, 256: 56, 70; 512: 108, 74; 640: 2 tiles 144, shared 115; 4 float32 rows,
//   256: 33.5, 38.6; 512: 65.8, 39.5; 640: 75.6, 61.3
template <class Op>
static void linear_op(const Q4Shape& s, int rows, const void* x, const RowWeights& w, void* y, hipStream_t st) {
  const int nt = ceil_div(s.N, TILE_N);
  if constexpr (Op::PLANES == 1) {
    if (rows <= 16) {
      if (nt <= 512) linear_as<Op, 1, 1, 2, 16>(s, rows, x, w, y, st);
      else if (nt <= 1536) linear_as<Op, 1, 2, 2, 8>(s, rows, x, w, y, st);
      else wide_as<Op, 1, 1, 4>(s, rows, x, w, y, st);
    } else if (rows <= 32) {
      if (nt <= 256) linear_as<Op, 2, 1, 1, 8>(s, rows, x, w, y, st);
      else if (nt <= 512) linear_as<Op, 2, 2, 1, 8>(s, rows, x, w, y, st);
      else if (nt <= 1024) linear_as<Op, 2, 4, 1, 8>(s, rows, x, w, y, st);
      else wide_as<Op, 2, 1, 4>(s, rows, x, w, y, st);
    } else {
      if (nt <= 256) linear_as<Op, 4, 1, 1, 8>(s, rows, x, w, y, st);
      else if (nt <= 512) linear_as<Op, 4, 2, 1, 8>(s, rows, x, w, y, st);
      else wide_as<Op, 4, 1, 4>(s, rows, x, w, y, st);
    }
  } else {
    if (nt <= 256) linear_as<Op, 1, 1, 1, 16>(s, rows, x, w, y, st);
    else if (nt <= 512) linear_as<Op, 1, 2, 1, 8>(s, rows, x, w, y, st);
    else linear_as<Op, 1, 4, 1, 8>(s, rows, x, w, y, st);
  }
}
template <typename T>
static void linear_t(const Q4Shape& s, int rows, const void* x, const void* codes, const void* scales,
                     const void* zeros, void* y, hipStream_t st) {
  const RowWeights w{codes, scales, static_cast<const uint8_t*>(zeros)};
#define MOE_CALL(GR_, ZP_) linear_op<Q4Op<T, GR_, ZP_>>(s, rows, x, w, y, st)
  MOE_Q4_ALL(MOE_CALL);
#undef MOE_CALL
}

hipError_t launch_q4_pack(const Q4Shape& s, const void* w, void* codes, void* scales, void* zeros, hipStream_t st) {
  if (s.G == 0) return hipSuccess;
  if (s.dtype == DT_BF16) pack_t<bf16_t>(s, w, codes, scales, zeros, st);
  else pack_t<float>(s, w, codes, scales, zeros, st);
  return hipGetLastError();
}
hipError_t launch_q4_tile(const Q4Shape& s, const void* c_rm, const void* s_rm, const void* z_rm, void* codes,
                          void* scales, void* zeros, hipStream_t st) {
  if (s.G == 0) return hipSuccess;
  if (s.dtype == DT_BF16) tile_t<bf16_t>(s, c_rm, s_rm, z_rm, codes, scales, zeros, st);
  else tile_t<float>(s, c_rm, s_rm, z_rm, codes, scales, zeros, st);
  return hipGetLastError();
}
hipError_t launch_q4_unpack(const Q4Shape& s, const void* codes, const void* scales, const void* zeros, void* w,
                            hipStream_t st) {
  if (s.G == 0) return hipSuccess;
  if (s.dtype == DT_BF16) unpack_t<bf16_t>(s, codes, scales, zeros, w, st);
  else unpack_t<float>(s, codes, scales, zeros, w, st);
  return hipGetLastError();
}
hipError_t launch_q4_linear(const Q4Shape& s, int rows, const void* x, const void* codes, const void* scales,
                            const void* zeros, void* y, hipStream_t st) {
  if (rows == 0) return hipSuccess;
  if (s.dtype == DT_BF16) linear_t<bf16_t>(s, rows, x, codes, scales, zeros, y, st);
  else linear_t<float>(s, rows, x, codes, scales, zeros, y, st);
  return hipGetLastError();
}

}  // namespace moe
