// Low-rank adapters of many requests beside a projection: row r of a batch
// belongs to a token, the token to an adapter a (none if its id is outside
// [0, L)), and, behind the router, the row to an expert g:
//   out[r] = y[r] + scale[a] * B[a][g] (A[a][g] x[r])
// with v = A x summed in float32 over the whole K and never rounded to the
// element type: in bf16 the second product takes v as the sum of two bf16 values
// (v and its remainder: 16 bits of v survive, so its error, 2^-17, stays far
// below the rounding of the output, 2^-9), which fill the K lanes of the same
// matrix instruction that a rank of 16 would leave half empty.
//
// Both kernels take windows of 16 rows in the order of the batch, the rows of
// one matrix instruction.  A window's distinct (adapter, expert) pairs are run
// one after another, each keeping the rows that are its own (a row's result
// never meets another adapter's numbers, whatever they are), so that no sorting
// and no work table is needed: rows of one request follow each other in prefill
// and rows of one expert behind the router, where a window holds one or two pairs.
#include "common.h"
#include "launch.h"

namespace moe {

namespace {

constexpr int AW = 16;      // rows of a window
constexpr int MAX_G = 1024;

// What lane l of a wave knows of row r = 16 * window + l % 16.
struct AdaptRow {
  int a, g;      // adapter (-1: none) and expert
  long long x;   // row of x
  bool live;     // the row exists
};

// `off`: G + 1 offsets in LDS (G > 1 or given), already staged.
__device__ __forceinline__ AdaptRow adapt_row(const AdaptArgs& p, int r, const int32_t* off) {
  AdaptRow o{-1, 0, 0, false};
  const int count = p.expert_off ? min(off[p.G], p.rows) : p.rows;
  if (r >= count) return o;
  o.live = true;
  const int tok = p.row_tok ? p.row_tok[r] : r;
  int xr = r;
  if (p.x_rows) xr = p.x_rows[r];
  o.x = xr;
  if (tok < 0 || tok >= p.T || xr < 0 || xr >= p.x_count) return o;
  const int a = p.ids[tok];
  if (a < 0 || a >= p.L) return o;
  if (p.expert_off) {  // the last g with off[g] <= r
    int lo = 0, hi = p.G;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (off[mid] <= r) lo = mid;
      else hi = mid;
    }
    o.g = lo;
  }
  o.a = a;
  return o;
}

__device__ __forceinline__ void stage_offsets(const AdaptArgs& p, int32_t* off) {
  if (!p.expert_off) return;
  for (int i = threadIdx.x; i <= p.G; i += blockDim.x) off[i] = p.expert_off[i];
  __syncthreads();
}

__device__ __forceinline__ int adapt_rank(const AdaptArgs& p, int a) {
  const int r = p.ranks ? p.ranks[a] : p.R;
  return r < 0 ? 0 : (r > p.R ? p.R : r);
}

template <typename T>
__device__ __forceinline__ f32x4_t mma16(const u32x4_t& a, const u32x4_t& b, f32x4_t c) {
  if constexpr (sizeof(T) == 2) {
    return Mfma<bf16_t>::step(a, b, c);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = mfma_f32_4(__uint_as_float(a[i]), __uint_as_float(b[i]), c);
    return c;
  }
}

}  // namespace

// The distinct (adapter, expert) pairs of a window, as seen by every lane of a wave:
// f(rows, a, g, rank, mine) for each z-th of Z of them, in the order of their first
// rows.  `rank`: the lane's row's adapter's.
template <class F>
__device__ __forceinline__ void for_pairs(const AdaptRow& row, int rank, int z, int Z, F f) {
  uint32_t todo = (uint32_t)__ballot(row.a >= 0) & 0xffffu;
  for (int i = 0; todo; ++i) {
    const int first = __builtin_ctz(todo);
    const int a = __builtin_amdgcn_readlane(row.a, first), g = __builtin_amdgcn_readlane(row.g, first);
    const bool mine = row.a == a && row.g == g;
    const uint32_t rows = (uint32_t)__ballot(mine) & 0xffffu;
    todo &= ~rows;
    if (i % Z == z) f(rows, a, g, __builtin_amdgcn_readlane(rank, first), mine);
  }
}

// v[r][:] = scale A[a][g] x[r], partial over slice blockIdx.y of K: part[s][r][R],
// 0 behind the adapter's rank.
// The workgroup's four waves take quarters of the slice and are added in wave
// order.  A lane's 16 bytes of x row l % 16 and of A row l % 16 hold the same K.
// blockIdx.z takes every Z-th pair of the window: where windows are few (decode)
// and hold many adapters, their latencies pass side by side.
template <typename T, int RT>
__global__ __launch_bounds__(256) void adapt_shrink_kernel(AdaptArgs p, float* __restrict__ part) {
  constexpr int LE = 16 / (int)sizeof(T);
  constexpr int KS = 4 * LE;  // K of one step (four lane groups)
  __shared__ int32_t off[MAX_G + 1];
  __shared__ float red[4][AW][16 * RT + 1], scale[AW];
  stage_offsets(p, off);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, lg = lane >> 4;
  const AdaptRow row = adapt_row(p, (int)blockIdx.x * AW + l16, off);
  const int steps = (p.K + KS - 1) / KS, nq = gridDim.y * 4, q = blockIdx.y * 4 + wave;
  const int s0 = (int)((long long)steps * q / nq), s1 = (int)((long long)steps * (q + 1) / nq);
  f32x4_t acc[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const T* const xr = (const T*)p.x + (size_t)row.x * p.K;
  uint32_t done = 0;  // rows that this workgroup computes
  const int my_rank = row.a >= 0 ? adapt_rank(p, row.a) : 0;
  const float my_scale = row.a >= 0 && p.scales ? p.scales[row.a] : 1.0f;
  for_pairs(row, my_rank, blockIdx.z, gridDim.z, [&](uint32_t rows, int a, int g, int rank, bool mine) {
    done |= rows;
    const T* const am = (const T*)p.a + ((size_t)a * p.G + g) * (size_t)p.R * p.K;
    f32x4_t t[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) t[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    constexpr int U = RT <= 2 ? 8 : (RT <= 4 ? 4 : 2);  // steps in flight
    for (int s = s0; s < s1; s += U) {
      u32x4_t xv[U], av[U][RT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = (s + u) * KS + lg * LE;
        const bool in = s + u < s1 && k < p.K;
        xv[u] = u32x4_t{0u, 0u, 0u, 0u};
        if (in && mine) xv[u] = *reinterpret_cast<const u32x4_t*>(xr + k);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          av[u][i] = u32x4_t{0u, 0u, 0u, 0u};
          if (in && 16 * i + l16 < rank)
            av[u][i] = *reinterpret_cast<const u32x4_t*>(am + (size_t)(16 * i + l16) * p.K + k);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < RT; ++i) t[i] = mma16<T>(xv[u], av[u][i], t[i]);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if ((rows >> (4 * lg + r)) & 1u) acc[i][r] = t[i][r];
  });
  if (!done) return;  // the same for the four waves
  if (threadIdx.x < AW) scale[threadIdx.x] = my_scale;
  // acc[i][r] is row 4 * lg + r, rank 16 * i + l16
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave][4 * lg + r][16 * i + l16] = acc[i][r];
  __syncthreads();
  float* const out = part + ((size_t)blockIdx.y * p.rows + (size_t)blockIdx.x * AW) * p.R;
  for (int i = threadIdx.x; i < AW * p.R; i += 256) {
    const int r = i / p.R, c = i % p.R;
    if ((done >> r) & 1u) out[i] = scale[r] * ((red[0][r][c] + red[1][r][c]) + (red[2][r][c] + red[3][r][c]));
  }
}

// out[r] = y[r] + B v: a wave takes up to 4 chunks of 64 columns of a window, for
// every Z-th of its pairs.  The matrix instruction's rows are the columns of y:
// row i of tile j is column 32 (j / 2) + 8 (i / 4) + 4 (j % 2) + i % 4 of the
// chunk, so that a lane ends with runs of 8 columns of one row and four lanes with
// 64 contiguous bytes of it (bf16).  A fragment of B holds 4 * LE ranks (lane
// group lg: LE of them); bf16 multiplies it with v and with its remainder.  A wave
// has little to compute and much to wait for: all its rows of y are requested
// first, and B of the next DEPTH (pair, chunk) items while one is multiplied.
template <typename T, int NF>
__global__ __launch_bounds__(256) void adapt_expand_kernel(AdaptArgs p, const float* __restrict__ part, int S,
                                                           int chunks) {
  constexpr int LE = 16 / (int)sizeof(T);
  constexpr bool BF = sizeof(T) == 2;
  constexpr int CM = 4;                                    // chunks of 64 columns at most
  constexpr int YV = BF ? 2 : 4;                           // 16-byte pieces of a lane's 16 columns
  constexpr int DEPTH = NF == 1 ? 4 : (NF == 2 ? 2 : 1);   // items of B in registers
  __shared__ int32_t off[MAX_G + 1];
  stage_offsets(p, off);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4;
  const int r = (int)blockIdx.x * AW + l16;
  const int n_beg = ((int)blockIdx.y * 4 + wave) * chunks * 64;
  if (n_beg >= p.N) return;
  const bool inplace = p.y == p.out;
  // this lane's ranks: LE from (4 f + lg) LE on, f < NF; parts of rows without an
  // adapter were not written: they are read and left out
  float v[NF][LE];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int i = 0; i < LE; ++i) v[f][i] = 0.f;
  if (r < p.rows) {
    for (int s = 0; s < S; ++s) {
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const int c = (4 * f + lg) * LE;
        if (c < p.R) {
          const float4* src = reinterpret_cast<const float4*>(part + ((size_t)s * p.rows + r) * p.R + c);
#pragma unroll
          for (int i = 0; i < LE / 4; ++i) {
            const float4 q = src[i];
            v[f][4 * i] += q.x;
            v[f][4 * i + 1] += q.y;
            v[f][4 * i + 2] += q.z;
            v[f][4 * i + 3] += q.w;
          }
        }
      }
    }
  }
  const AdaptRow row = adapt_row(p, r, off);
  const int my_rank = row.a >= 0 ? adapt_rank(p, row.a) : 0;
  // the wave's pairs, one in each of the first lanes
  int pa = 0, pg = 0, prank = 0, np = 0;
  bool served = false;
  for_pairs(row, my_rank, blockIdx.z, gridDim.z, [&](uint32_t, int a, int g, int rank, bool mine) {
    if (lane == np) {
      pa = a;
      pg = g;
      prank = rank;
    }
    served |= mine;
    ++np;
  });
  // rows without an adapter are copied
  const bool copied = blockIdx.z == 0 && !inplace && row.live && row.a < 0;

  const T* const yr = (const T*)p.y + (size_t)r * p.N;
  T* const outr = (T*)p.out + (size_t)r * p.N;
  // column of piece i of a lane's share of chunk c
  auto col = [&](int c, int i) {
    return n_beg + 64 * c + (BF ? 32 * i + 8 * lg : 32 * (i >> 1) + 8 * lg + 4 * (i & 1));
  };
  u32x4_t yv[CM][YV];
#pragma unroll
  for (int c = 0; c < CM; ++c)
#pragma unroll
    for (int i = 0; i < YV; ++i) {
      const int n = col(c, i);
      yv[c][i] = u32x4_t{0u, 0u, 0u, 0u};
      if (c < chunks && (served || copied) && n < p.N) yv[c][i] = *reinterpret_cast<const u32x4_t*>(yr + n);
    }

  u32x4_t vf[BF ? 2 : 1][NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
#pragma unroll
    for (int i = 0; i < LE; ++i) v[f][i] = row.a >= 0 ? v[f][i] : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (BF) {
        const bf16_t h0 = f32_to_bf16(v[f][2 * i]), h1 = f32_to_bf16(v[f][2 * i + 1]);
        vf[0][f][i] = (uint32_t)h0 | ((uint32_t)h1 << 16);
        vf[BF ? 1 : 0][f][i] = (uint32_t)f32_to_bf16(v[f][2 * i] - bf16_to_f32(h0)) |
                               ((uint32_t)f32_to_bf16(v[f][2 * i + 1] - bf16_to_f32(h1)) << 16);
      } else {
        vf[0][f][i] = __float_as_uint(v[f][i]);
      }
    }
  }

  u32x4_t bv[DEPTH][4][NF];
  auto load_b = [&](u32x4_t (&b)[4][NF], int pair, int c) {
    const int rank = __builtin_amdgcn_readlane(prank, pair);
    const T* const bm = (const T*)p.b + ((size_t)__builtin_amdgcn_readlane(pa, pair) * p.G +
                                         __builtin_amdgcn_readlane(pg, pair)) * (size_t)p.N * p.R;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n_beg + 64 * c + 32 * (j >> 1) + 8 * (l16 >> 2) + 4 * (j & 1) + (l16 & 3);
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const int ch = (4 * f + lg) * LE;
        b[j][f] = u32x4_t{0u, 0u, 0u, 0u};
        if (ch < rank && n < p.N) b[j][f] = *reinterpret_cast<const u32x4_t*>(bm + (size_t)n * p.R + ch);
      }
    }
  };
  // chunk by chunk (its rows of y are registers), the pairs of each in turn
  const int items = np * chunks;
#pragma unroll
  for (int d = 0; d < DEPTH; ++d)
    if (d < items) load_b(bv[d], d % np, d / np);
#pragma unroll
  for (int c = 0; c < CM; ++c) {
    if (c >= chunks) break;
    f32x4_t acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int pair = 0; pair < np; ++pair) {
      const int it = c * np + pair, rank = __builtin_amdgcn_readlane(prank, pair);
      const bool mine = row.a == __builtin_amdgcn_readlane(pa, pair) && row.g == __builtin_amdgcn_readlane(pg, pair);
      auto step = [&](u32x4_t (&b)[4][NF]) {
        f32x4_t t[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          t[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int f = 0; f < NF; ++f) {
            const int left = rank - (4 * f + lg) * LE;  // ranks of the piece that exist
            u32x4_t w = b[j][f];
            if (left > 0 && left < LE) {  // what lies behind the rank may be anything
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if constexpr (BF) w[i] &= (2 * i < left ? 0xffffu : 0u) | (2 * i + 1 < left ? 0xffff0000u : 0u);
                else w[i] = i < left ? w[i] : 0u;
              }
            }
            t[j] = mma16<T>(w, vf[0][f], t[j]);
            if constexpr (BF) t[j] = mma16<T>(w, vf[1][f], t[j]);
          }
        }
        if (it + DEPTH < items) load_b(b, (it + DEPTH) % np, (it + DEPTH) / np);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (mine) acc[j] = t[j];
      };
      // the item's slot, as a compile-time index
#pragma unroll
      for (int d = 0; d < DEPTH; ++d)
        if (it % DEPTH == d) step(bv[d]);
    }
    // acc[j][e]: column 32 (j / 2) + 8 lg + 4 (j % 2) + e of row l16
#pragma unroll
    for (int i = 0; i < YV; ++i) {
      const int n = col(c, i);
      u32x4_t o;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if constexpr (BF) {
          const f32x4_t& q = acc[2 * i + (w >> 1)];
          o[w] = (uint32_t)f32_to_bf16(__uint_as_float(yv[c][i][w] << 16) + q[2 * (w & 1)]) |
                 ((uint32_t)f32_to_bf16(__uint_as_float(yv[c][i][w] & 0xffff0000u) + q[2 * (w & 1) + 1]) << 16);
        } else {
          o[w] = __float_as_uint(__uint_as_float(yv[c][i][w]) + acc[i][w]);
        }
      }
      if (copied) o = yv[c][i];
      if ((served || copied) && n < p.N) *reinterpret_cast<u32x4_t*>(outr + n) = o;
    }
  }
}

// Shares of a window's pairs: 1 where the windows fill the chip, more where they
// are few.
static int pair_shares(int waves) { return max(1, min(4, 4096 / max(1, waves))); }

int adapt_splits(int rows, int K, int elt) {
  const int windows = max(1, (rows + AW - 1) / AW);
  const int steps = (K * elt + 63) / 64;
  return max(1, min(min(8, (1024 + windows - 1) / windows), steps / 16));
}

template <typename T>
static void launch_adapt_t(const AdaptArgs& p, float* part, int S, hipStream_t st) {
  const int windows = (p.rows + AW - 1) / AW;
  const int n64 = (p.N + 63) / 64;
  const int chunks = max(1, min(4, (int)((long long)windows * n64 / 4096)));
  const int pieces = (n64 + 4 * chunks - 1) / (4 * chunks);
  const dim3 gs(windows, S, pair_shares(4 * windows * S)), ge(windows, pieces, pair_shares(4 * windows * pieces));
#define MOE_ADAPT(RT, NF)                                                                                      \
  do {                                                                                                         \
    hipLaunchKernelGGL((adapt_shrink_kernel<T, RT>), gs, dim3(256), 0, st, p, part);                           \
    hipLaunchKernelGGL((adapt_expand_kernel<T, NF>), ge, dim3(256), 0, st, p, (const float*)part, S, chunks);  \
  } while (0)
  const int rt = (p.R + 15) / 16;
  constexpr bool BF = sizeof(T) == 2;
  if (rt == 1) MOE_ADAPT(1, 1);
  else if (rt == 2) MOE_ADAPT(2, BF ? 1 : 2);
  else if (rt <= 4) MOE_ADAPT(4, BF ? 2 : 4);
  else MOE_ADAPT(8, BF ? 4 : 8);
#undef MOE_ADAPT
}

hipError_t launch_adapt(int dtype, const AdaptArgs& p, float* part, int S, hipStream_t st) {
  if (p.rows == 0) return hipSuccess;
  if (dtype == DT_BF16) launch_adapt_t<bf16_t>(p, part, S, st);
  else launch_adapt_t<float>(p, part, S, st);
  return hipGetLastError();
}

}  // namespace moe
