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

// v[r][:] = A[a][g] x[r], partial over slice blockIdx.y of K: part[s][r][R].
// The workgroup's four waves take quarters of the slice and are added in wave
// order.  A lane's 16 bytes of x row l % 16 and of A row l % 16 hold the same K.
template <typename T, int RT>
__global__ __launch_bounds__(256) void adapt_shrink_kernel(AdaptArgs p, float* __restrict__ part) {
  constexpr int LE = 16 / (int)sizeof(T);
  constexpr int KS = 4 * LE;  // K of one step (four lane groups)
  __shared__ int32_t off[MAX_G + 1];
  __shared__ float red[4][AW][16 * RT];
  stage_offsets(p, off);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, lg = lane >> 4;
  const AdaptRow row = adapt_row(p, (int)blockIdx.x * AW + l16, off);
  const int steps = (p.K + KS - 1) / KS, nq = gridDim.y * 4, q = blockIdx.y * 4 + wave;
  const int s0 = (int)((long long)steps * q / nq), s1 = (int)((long long)steps * (q + 1) / nq);
  f32x4_t acc[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const T* const xr = (const T*)p.x + (size_t)row.x * p.K;
  uint32_t todo = (uint32_t)__ballot(row.a >= 0) & 0xffffu;
  const bool any = todo != 0;
  while (todo) {
    const int first = __builtin_ctz(todo);
    const int a = __shfl(row.a, first, 64), g = __shfl(row.g, first, 64);
    const bool mine = row.a == a && row.g == g;
    const uint32_t rows = (uint32_t)__ballot(mine);
    todo &= ~rows;
    const int rank = adapt_rank(p, a);
    const T* const am = (const T*)p.a + ((size_t)a * p.G + g) * (size_t)p.R * p.K;
    f32x4_t t[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) t[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    constexpr int U = RT <= 2 ? 4 : 2;
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
  }
  if (!any) return;  // no adapter in the window (the same for the four waves): never read
  // acc[i][r] is row 4 * lg + r, rank 16 * i + l16
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave][4 * lg + r][16 * i + l16] = acc[i][r];
  __syncthreads();
  float* const out = part + ((size_t)blockIdx.y * p.rows + (size_t)blockIdx.x * AW) * p.R;
  const int left = min(AW, p.rows - (int)blockIdx.x * AW);
  for (int i = threadIdx.x; i < left * p.R; i += 256) {
    const int r = i / p.R, c = i % p.R;
    out[i] = (red[0][r][c] + red[1][r][c]) + (red[2][r][c] + red[3][r][c]);
  }
}

// out[r] = y[r] + scale * B v: each wave takes 64 columns at a time of a window.
// The matrix instruction's rows are the columns of y: row i of tile j is column
// 16 * (i / 4) + 4 * j + i % 4 of the 64, so that a lane ends with 16 columns of
// one row in a run and a row's 64 columns are one contiguous piece.
template <typename T, int RT>
__global__ __launch_bounds__(256) void adapt_expand_kernel(AdaptArgs p, const float* __restrict__ part, int S,
                                                           int cols) {
  constexpr int LE = 16 / (int)sizeof(T);       // ranks of a lane's chunk
  constexpr bool BF = sizeof(T) == 2;
  constexpr int STEPS = RT;                     // bf16: 2 R / 32; float: R / 16
  constexpr int YV = 16 / LE;                   // 16-byte pieces of a lane's 16 columns
  __shared__ int32_t off[MAX_G + 1];
  stage_offsets(p, off);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, lg = lane >> 4;
  const int r = (int)blockIdx.x * AW + l16;
  const AdaptRow row = adapt_row(p, r, off);
  const bool inplace = p.y == p.out;
  const uint32_t all = (uint32_t)__ballot(row.a >= 0) & 0xffffu;
  const int n_beg = ((int)blockIdx.y * 4 + wave) * cols, n_end = min(p.N, n_beg + cols);
  if (n_beg >= p.N) return;
  if (inplace && !all) return;

  // this lane's chunks of v: step st, chunk 4 * st + lg
  const int nchunk = p.R / LE;
  u32x4_t vf[STEPS];
  int bch[STEPS];  // the chunk of B's row that goes with it, -1: none
#pragma unroll
  for (int st = 0; st < STEPS; ++st) {
    const int c = 4 * st + lg;
    const bool lo = BF && c >= nchunk;
    const int rc = lo ? c - nchunk : c;
    bch[st] = rc < nchunk ? rc : -1;
    vf[st] = u32x4_t{0u, 0u, 0u, 0u};
    if (bch[st] < 0 || row.a < 0) continue;
    const int rank = adapt_rank(p, row.a);
    const float scale = p.scales ? p.scales[row.a] : 1.0f;
    float v[LE];
#pragma unroll
    for (int i = 0; i < LE; ++i) v[i] = 0.f;
    for (int s = 0; s < S; ++s) {
      const float* src = part + ((size_t)s * p.rows + r) * p.R + rc * LE;
#pragma unroll
      for (int i = 0; i < LE; ++i) v[i] += src[i];
    }
#pragma unroll
    for (int i = 0; i < LE; ++i) v[i] = rc * LE + i < rank ? v[i] * scale : 0.f;
    if constexpr (BF) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t h[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bf16_t hi = f32_to_bf16(v[2 * i + e]);
          h[e] = lo ? f32_to_bf16(v[2 * i + e] - bf16_to_f32(hi)) : hi;
        }
        vf[st][i] = h[0] | (h[1] << 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) vf[st][i] = __float_as_uint(v[i]);
    }
  }

  const T* const yr = (const T*)p.y + (size_t)r * p.N;
  T* const outr = (T*)p.out + (size_t)r * p.N;
  for (int n0 = n_beg; n0 < n_end; n0 += 64) {
    u32x4_t yv[YV];
#pragma unroll
    for (int i = 0; i < YV; ++i) {
      const int n = n0 + 16 * lg + i * LE;
      yv[i] = u32x4_t{0u, 0u, 0u, 0u};
      if (row.live && n < p.N) yv[i] = *reinterpret_cast<const u32x4_t*>(yr + n);
    }
    f32x4_t acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    uint32_t todo = all;
    while (todo) {
      const int first = __builtin_ctz(todo);
      const int a = __shfl(row.a, first, 64), g = __shfl(row.g, first, 64);
      const bool mine = row.a == a && row.g == g;
      todo &= ~(uint32_t)__ballot(mine);
      const int rank = adapt_rank(p, a);
      const T* const bm = (const T*)p.b + ((size_t)a * p.G + g) * (size_t)p.N * p.R;
      f32x4_t t[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) t[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int st = 0; st < STEPS; ++st) {
        const int left = bch[st] < 0 ? 0 : rank - bch[st] * LE;  // ranks of the chunk that exist
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = n0 + 16 * (l16 >> 2) + 4 * j + (l16 & 3);
          u32x4_t bv = {0u, 0u, 0u, 0u};
          if (left > 0 && n < p.N) bv = *reinterpret_cast<const u32x4_t*>(bm + (size_t)n * p.R + bch[st] * LE);
          if (left < LE) {  // what lies behind the rank may be anything
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if constexpr (BF) bv[i] &= (2 * i < left ? 0xffffu : 0u) | (2 * i + 1 < left ? 0xffff0000u : 0u);
              else bv[i] = i < left ? bv[i] : 0u;
            }
          }
          t[j] = mma16<T>(bv, vf[st], t[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (mine) acc[j] = t[j];
    }
    // acc[j][e]: column n0 + 16 * lg + 4 * j + e of row l16
    const bool write = row.live && !(inplace && row.a < 0);
#pragma unroll
    for (int i = 0; i < YV; ++i) {
      const int n = n0 + 16 * lg + i * LE;
      if (!write || n >= p.N) continue;
      u32x4_t o = yv[i];
      if (row.a >= 0) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          if constexpr (BF) {
            const int c = i * LE + 2 * w;
            o[w] = (uint32_t)f32_to_bf16(__uint_as_float(yv[i][w] << 16) + acc[c >> 2][c & 3]) |
                   ((uint32_t)f32_to_bf16(__uint_as_float(yv[i][w] & 0xffff0000u) + acc[(c + 1) >> 2][(c + 1) & 3]) << 16);
          } else {
            const int c = i * LE + w;
            o[w] = __float_as_uint(__uint_as_float(yv[i][w]) + acc[c >> 2][c & 3]);
          }
        }
      }
      *reinterpret_cast<u32x4_t*>(outr + n) = o;
    }
  }
}

int adapt_splits(int rows, int K, int elt) {
  const int windows = max(1, (rows + AW - 1) / AW);
  const int steps = (K * elt + 63) / 64;
  return max(1, min(min(8, (512 + windows - 1) / windows), steps / 16));
}

template <typename T>
static void launch_adapt_t(const AdaptArgs& p, float* part, int S, hipStream_t st) {
  const int windows = (p.rows + AW - 1) / AW;
  const int pieces = max(1, min((p.N + 255) / 256, (2048 + windows - 1) / windows));
  const int cols = ((p.N + pieces * 4 - 1) / (pieces * 4) + 63) / 64 * 64;
  const dim3 ge(windows, (p.N + 4 * cols - 1) / (4 * cols));
#define MOE_ADAPT(RT)                                                                                          \
  do {                                                                                                         \
    hipLaunchKernelGGL((adapt_shrink_kernel<T, RT>), dim3(windows, S), dim3(256), 0, st, p, part);             \
    hipLaunchKernelGGL((adapt_expand_kernel<T, RT>), ge, dim3(256), 0, st, p, (const float*)part, S, cols);    \
  } while (0)
  const int rt = (p.R + 15) / 16;
  if (rt == 1) MOE_ADAPT(1);
  else if (rt == 2) MOE_ADAPT(2);
  else if (rt <= 4) MOE_ADAPT(4);
  else MOE_ADAPT(8);
#undef MOE_ADAPT
}

hipError_t launch_adapt(int dtype, const AdaptArgs& p, float* part, int S, hipStream_t st) {
  if (p.rows == 0) return hipSuccess;
  if (dtype == DT_BF16) launch_adapt_t<bf16_t>(p, part, S, st);
  else launch_adapt_t<float>(p, part, S, st);
  return hipGetLastError();
}

}  // namespace moe
