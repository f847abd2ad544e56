// Low-rank adapters of many requests beside a projection: row r of a batch
// belongs to a token, the token to an adapter a (none if its id is outside
// [0, L)), and, behind the router, the row to an expert g:
//   out[r] = y[r] + scale[a] * B[a][g] (A[a][g] x[r])
// with v = scale * A x summed in float32 over the whole K and never rounded to the
// element type: in bf16 the second product takes v as the sum of two bf16 values
// (v and its remainder: 16 bits of v survive, so its error, 2^-17, stays far
// below the rounding of the output, 2^-9).
//
// Both kernels take windows of 16 rows in the order of the batch, the rows of
// one matrix instruction.  A window's distinct (adapter, expert) pairs are run
// one after another, each keeping the rows that are its own (a row's result
// never meets another adapter's numbers, whatever they are), so that no sorting
// and no work table is needed: rows of one request follow each other in prefill
// and rows of one expert behind the router, where a window holds one or two pairs.
//
// Bound by memory in prefill (4,096 rows, 2,048 -> 7,168, rank 32, 8 adapters: 15 us
// for the first product, 37 us for the second, which reads and writes 117 MB, a copy
// in the same shape taking 30), by latency in decode (128 rows, 32 adapters: 8.5 +
// 11 us; 1,150 permuted rows of 128 experts, 4 adapters: 10 + 17 us).  Where windows of
// a large batch hold many pairs it is bound by their products (4,096 rows of 32 mixed
// adapters, rank 16: 157 us; 32,768 permuted rows of 128 experts, 8 mixed adapters, 768
// -> 2,048: 248 us).  Ranks above 64 spill in the first product (up to 199 registers):
// rank 128 takes 103 us for 128 rows, 173 for 4,096 rows of 8 adapters (rank 64: 40 and
// 67).  float32: 30 us for 128 rows, 93 for 4,096 (2,048 -> 7,168, rank 16 and 32).
#include "common.h"
#include "launch.h"

namespace moe {

namespace {

constexpr int AW = 16;      // rows of a window
constexpr int MAX_G = 1024;

// What a lane knows of one row.
struct AdaptRow {
  int a, g, rank;  // adapter (-1: none), expert, rank
  float scale;
  int x;           // row of x
  bool live;       // the row exists
};

// `off`: G + 1 offsets in LDS (if there are groups), already staged.  Every load
// has an address in range and none waits behind a branch.
__device__ __forceinline__ AdaptRow adapt_row(const AdaptArgs& p, int r, const int32_t* off) {
  AdaptRow o{-1, 0, 0, 1.0f, 0, false};
  const int rc = min(r, p.rows - 1);
  const int tok = p.row_tok ? p.row_tok[rc] : rc;
  const int xr = p.x_rows ? p.x_rows[rc] : rc;
  o.live = r < (p.expert_off ? min(off[p.G], p.rows) : p.rows);
  if (p.T == 0) return o;
  const int a = p.ids[min(max(tok, 0), p.T - 1)];
  const int ac = min(max(a, 0), p.L - 1);
  const int rank = p.ranks ? p.ranks[ac] : p.R;
  const float scale = p.scales ? p.scales[ac] : 1.0f;
  if (!o.live || tok < 0 || tok >= p.T || xr < 0 || xr >= p.x_count || a != ac) return o;
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
  o.x = xr;
  o.rank = min(max(rank, 0), p.R);
  o.scale = scale;
  return o;
}

__device__ __forceinline__ void stage_offsets(const AdaptArgs& p, int32_t* off) {
  if (!p.expert_off) return;
  for (int i = threadIdx.x; i <= p.G; i += blockDim.x) off[i] = p.expert_off[i];
  __syncthreads();
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

// The distinct (adapter, expert) pairs of a window, of which lane l holds row
// l % 16 (a < 0: none): f(rows, first) for each z-th of Z of them, in the order of
// their first rows.
template <class F>
__device__ __forceinline__ void for_pairs(int a, int g, int z, int Z, F f) {
  uint32_t todo = (uint32_t)__ballot(a >= 0) & 0xffffu;
  for (int i = 0; todo; ++i) {
    const int first = __builtin_ctz(todo);
    const uint32_t rows = todo & (uint32_t)__ballot(a == __builtin_amdgcn_readlane(a, first) &&
                                                    g == __builtin_amdgcn_readlane(g, first));
    todo &= ~rows;
    if (i % Z == z) f(rows, first);
  }
}

}  // namespace

// v[r][:] = scale A[a][g] x[r], 0 behind the adapter's rank: float [rows][R], or in
// bf16 two arrays [rows][R], v rounded and its remainder rounded.  The workgroup's
// waves take equal parts of K and are added in wave order, so that a batch of one
// window is as parallel as its K is long.  A lane's 16 bytes of x row l % 16 and of
// A row l % 16 hold the same K.  blockIdx.y takes every Z-th pair of the window:
// where windows are few (decode) and hold many adapters, their latencies pass side
// by side.
template <typename T, int RT>
__global__ __launch_bounds__(1024) void adapt_shrink_kernel(AdaptArgs p, void* __restrict__ vout) {
  constexpr int LE = 16 / (int)sizeof(T);
  constexpr int KS = 4 * LE;  // K of one step (four lane groups)
  constexpr int LD = 16 * RT + 1;
  __shared__ int32_t off[MAX_G + 1];
  __shared__ float scale[AW];
  __shared__ int32_t ranks[AW];
  extern __shared__ float red[];  // [waves][AW][LD]
  stage_offsets(p, off);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), nw = blockDim.x >> 6;
  const int l16 = lane & 15, lg = lane >> 4;
  const int r = (int)blockIdx.x * AW + l16;
  const int steps = (p.K + KS - 1) / KS;
  const int s0 = steps * wave / nw, s1 = steps * (wave + 1) / nw;
  constexpr int U = RT <= 2 ? 4 : 2;  // steps in flight
  // x of the first steps, before anything is known of its adapter: every row's
  const int xr = p.x_rows ? min(max(p.x_rows[min(r, p.rows - 1)], 0), p.x_count - 1) : min(r, p.rows - 1);
  const T* const xb = (const T*)p.x + (size_t)xr * p.K;
  auto load_x = [&](u32x4_t (&x)[U], int s) {
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = *reinterpret_cast<const u32x4_t*>(xb + min((s + u) * KS + lg * LE, p.K - LE));
  };
  u32x4_t xv[U], av[U][RT];
  if (p.x_count > 0) load_x(xv, s0);
  const AdaptRow row = adapt_row(p, r, off);
  // the workgroup's pairs, one in each of the first lanes
  int pa = 0, pg = 0, np = 0;
  uint32_t prows = 0, done = 0;
  for_pairs(row.a, row.g, blockIdx.y, gridDim.y, [&](uint32_t rows, int first) {
    const int a = __builtin_amdgcn_readlane(row.a, first), g = __builtin_amdgcn_readlane(row.g, first);
    if (lane == np) {
      pa = a;
      pg = g;
      prows = rows;
    }
    done |= rows;
    ++np;
  });
  auto load_a = [&](u32x4_t (&m)[U][RT], int pair, int s) {
    const T* const am = (const T*)p.a + ((size_t)__builtin_amdgcn_readlane(pa, pair) * p.G +
                                         __builtin_amdgcn_readlane(pg, pair)) * (size_t)p.R * p.K;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = min((s + u) * KS + lg * LE, p.K - LE);
#pragma unroll
      for (int i = 0; i < RT; ++i)
        m[u][i] = *reinterpret_cast<const u32x4_t*>(am + (uint32_t)(min(16 * i + l16, p.R - 1) * p.K + k));
    }
  };
  f32x4_t acc[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (np) load_a(av, 0, s0);
  for (int s = s0; np && s < s1; s += U) {
    const bool more = s + U < s1;
    u32x4_t xn[U];
#pragma unroll
    for (int u = 0; u < U; ++u) xn[u] = xv[u];
    if (more) load_x(xn, s + U);
    // steps behind the wave's part, and K behind the end: zeros on both sides
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + u >= s1 || (s + u) * KS + lg * LE >= p.K) xv[u] = u32x4_t{0u, 0u, 0u, 0u};
    for (int q = 0; q < np; ++q) {
      u32x4_t an[U][RT];  // A of the next pair, or of the first one's next steps
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < RT; ++i) an[u][i] = av[u][i];
      if (q + 1 < np || more) load_a(an, q + 1 < np ? q + 1 : 0, q + 1 < np ? s : s + U);
      const uint32_t rows = (uint32_t)__builtin_amdgcn_readlane((int)prows, q);
      f32x4_t t[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) t[i] = acc[i];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool out = s + u >= s1 || (s + u) * KS + lg * LE >= p.K;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          u32x4_t m = av[u][i];
          if (out) m = u32x4_t{0u, 0u, 0u, 0u};
          t[i] = mma16<T>(xv[u], m, t[i]);
        }
      }
      // a row's sum takes its own pair's product only
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if ((rows >> (4 * lg + j)) & 1u) acc[i][j] = t[i][j];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < RT; ++i) av[u][i] = an[u][i];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) xv[u] = xn[u];
  }
  if (!done) return;  // the same for all waves
  if (threadIdx.x < AW) {
    scale[threadIdx.x] = row.scale;
    ranks[threadIdx.x] = row.rank;
  }
  // acc[i][r] is row 4 * lg + r, rank 16 * i + l16
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) red[(wave * AW + 4 * lg + r) * LD + 16 * i + l16] = acc[i][r];
  __syncthreads();
  for (int i = threadIdx.x; i < AW * p.R; i += blockDim.x) {
    const int r = i / p.R, c = i - r * p.R;
    if (!((done >> r) & 1u)) continue;
    float v = red[r * LD + c];
    for (int w = 1; w < nw; ++w) v += red[(w * AW + r) * LD + c];
    v = c < ranks[r] ? v * scale[r] : 0.f;  // A behind the rank may be anything
    const size_t at = (size_t)blockIdx.x * AW * p.R + i;
    if constexpr (sizeof(T) == 2) {
      // a finite v behind bf16's largest value keeps it and leaves the rest to the
      // remainder; an infinity has none (inf - inf is no number)
      const bool finite = fabsf(v) < INFINITY;
      const bf16_t hi = f32_to_bf16(finite ? fminf(fmaxf(v, -0x1.fep127f), 0x1.fep127f) : v);
      ((bf16_t*)vout)[at] = hi;
      ((bf16_t*)vout)[(size_t)p.rows * p.R + at] = finite ? f32_to_bf16(v - bf16_to_f32(hi)) : (bf16_t)0;
    } else {
      ((float*)vout)[at] = v;
    }
  }
}

// out[r] = y[r] + B v: a wave takes 64 columns of up to 8 windows, B of the pair at
// hand in registers.  The matrix instruction's rows are the columns of y: in bf16
// row i of tile j is column 32 (j / 2) + 8 (i / 4) + 4 (j % 2) + i % 4 of the 64, so
// that a lane ends with runs of 8 columns of one row.  A fragment of B holds 4 * LE ranks (lane group lg: LE of
// them); bf16 multiplies it with v and with its remainder.
//
// A wave has little to compute and much to wait for: what it needs of its rows is
// read once, y and v of the next D windows are in flight while one is multiplied,
// from addresses that depend on nothing (so that the waits count loads instead of
// draining them).  B of a pair is loaded when it changes.
//
// Waves a SIMD: as many as the registers of a form allow without spilling (NF = 2 is
// held to three, which it misses by six registers of its own accord).
//
// AHEAD: B of a window's next pair is requested while one is multiplied; taken where
// the waves are few, which is where windows hold many pairs, up to the rank whose
// fragments fit the registers (128 rows, 32 adapters: 21.2 -> 20.0 us a call with two
// shares of a window's pairs; 1,150 permuted rows, 128 x 4 adapters: 27.5 -> 26.8).
template <typename T, int NF, bool AHEAD>
__global__ __launch_bounds__(256, NF == 1 && !AHEAD ? 4 : (NF == 2 && !AHEAD ? 3 : (NF <= 4 ? 2 : 1))) void adapt_expand_kernel(AdaptArgs p, const T* __restrict__ vin, int wpw) {
  constexpr int LE = 16 / (int)sizeof(T);
  constexpr bool BF = sizeof(T) == 2;
  constexpr int YV = BF ? 2 : 4;                  // 16-byte pieces of a lane's 16 columns
  constexpr int NV = BF ? 2 : 1;                  // v and its remainder
  constexpr int D = 2;
  __shared__ int32_t off[MAX_G + 1];
  stage_offsets(p, off);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4;
  const int windows = (p.rows + AW - 1) / AW;
  const int n0 = ((int)blockIdx.x * 4 + wave) * 64;
  const int w0 = blockIdx.y * wpw, w1 = min(w0 + wpw, windows);
  if (n0 >= p.N) return;
  const bool inplace = p.y == p.out;
  const int nchunk = p.R / LE;

  // the lane's pieces of y: row ar[i] of the window from column cc[i] on, and its
  // ranks (those that do not exist: the last ones)
  int ar[YV], cc[YV], cv[NF];
#pragma unroll
  for (int i = 0; i < YV; ++i) {
    ar[i] = BF ? (l16 & 7) + 8 * i : l16;
    cc[i] = n0 + (BF ? 32 * (l16 >> 3) + 8 * lg : 16 * i + 4 * lg);
  }
#pragma unroll
  for (int f = 0; f < NF; ++f) cv[f] = min(4 * f + lg, nchunk - 1) * LE;
  u32x4_t yv[D][YV], vf[D][NV][NF];
  auto load_window = [&](u32x4_t (&y)[YV], u32x4_t (&v)[NV][NF], int w) {
    const int wc = min(w, windows - 1), last = p.rows - 1 - wc * AW, rl = min(l16, last);
    const T* const yb = (const T*)p.y + (size_t)wc * AW * p.N;
    const T* const vb = vin + (size_t)wc * AW * p.R;
#pragma unroll
    for (int i = 0; i < YV; ++i)
      y[i] = *reinterpret_cast<const u32x4_t*>(yb + (uint32_t)(min(ar[i], last) * p.N + min(cc[i], p.N - LE)));
#pragma unroll
    for (int e = 0; e < NV; ++e)
#pragma unroll
      for (int f = 0; f < NF; ++f)
        v[e][f] = *reinterpret_cast<const u32x4_t*>(vb + (size_t)e * p.rows * p.R + (uint32_t)(rl * p.R + cv[f]));
  };
#pragma unroll
  for (int d = 0; d < D; ++d) load_window(yv[d], vf[d], w0 + d);
  // the wave's rows, two a lane: row 16 w0 + lane and 64 further
  int ra[2], rg[2], rr[2], rlive = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const AdaptRow row = adapt_row(p, w0 * AW + 64 * h + lane, off);
    ra[h] = row.a;
    rg[h] = row.g;
    rr[h] = row.rank;
    rlive |= row.live ? 1 << h : 0;
  }

  auto load_b = [&](u32x4_t (&b)[4][NF], int a, int g) {
    const T* const bm = (const T*)p.b + ((size_t)a * p.G + g) * (size_t)p.N * p.R;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = BF ? 32 * (j >> 1) + 8 * (l16 >> 2) + 4 * (j & 1) + (l16 & 3) : 16 * j + l16;
      const int n = min(n0 + i, p.N - 1);
#pragma unroll
      for (int f = 0; f < NF; ++f) b[j][f] = *reinterpret_cast<const u32x4_t*>(bm + (uint32_t)(n * p.R + cv[f]));
    }
  };
  // t = B v of one pair; what lies behind its rank may be anything and is not used
  auto product = [&](const u32x4_t (&b)[4][NF], const u32x4_t (&v)[NV][NF], int rank, f32x4_t (&t)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      t[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const int left = rank - (4 * f + lg) * LE;  // ranks of the piece that exist
        u32x4_t w = b[j][f];
        if (left < LE) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (BF) w[i] &= (2 * i < left ? 0xffffu : 0u) | (2 * i + 1 < left ? 0xffff0000u : 0u);
            else w[i] = i < left ? w[i] : 0u;
          }
        }
#pragma unroll
        for (int e = 0; e < NV; ++e) t[j] = mma16<T>(w, v[e][f], t[j]);
      }
    }
  };
  u32x4_t bv[4][NF];
  int ba = -1, bg = -1;  // the pair in bv
  auto window = [&](const u32x4_t (&y)[YV], u32x4_t (&v)[NV][NF], int w) {
    const int i = (w - w0) * AW, h = i >> 6, src = (i & 63) + l16;
    const int a = __shfl(h ? ra[1] : ra[0], src, 64), g = __shfl(h ? rg[1] : rg[0], src, 64);
    const int rank = __shfl(h ? rr[1] : rr[0], src, 64);
    const bool live = (__shfl(rlive, src, 64) >> h) & 1;
    // v of rows without an adapter was not written
#pragma unroll
    for (int e = 0; e < NV; ++e)
#pragma unroll
      for (int f = 0; f < NF; ++f)
        if (a < 0 || (4 * f + lg) * LE >= p.R) v[e][f] = u32x4_t{0u, 0u, 0u, 0u};
    f32x4_t acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    uint32_t served = 0;
    auto multiply = [&](uint32_t rows, int first) {
      f32x4_t t[4];
      product(bv, v, __builtin_amdgcn_readlane(rank, first), t);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if ((rows >> l16) & 1u) acc[j] = t[j];
    };
    if constexpr (AHEAD) {
      // the pairs, one in each of the first lanes
      int firsts = 0, n = 0;
      uint32_t prows = 0;
      for_pairs(a, g, blockIdx.z, gridDim.z, [&](uint32_t rows, int first) {
        if (lane == n) {
          firsts = first;
          prows = rows;
        }
        served |= rows;
        ++n;
      });
      u32x4_t bn[4][NF];
      auto load_pair = [&](u32x4_t (&to)[4][NF], int q) {
        const int first = __builtin_amdgcn_readlane(firsts, q);
        load_b(to, __builtin_amdgcn_readlane(a, first), __builtin_amdgcn_readlane(g, first));
      };
      if (n) load_pair(bv, 0);
      for (int q = 0; q < n; ++q) {
        load_pair(bn, min(q + 1, n - 1));
        multiply((uint32_t)__builtin_amdgcn_readlane((int)prows, q), __builtin_amdgcn_readlane(firsts, q));
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int f = 0; f < NF; ++f) bv[j][f] = bn[j][f];
      }
    } else {
      for_pairs(a, g, blockIdx.z, gridDim.z, [&](uint32_t rows, int first) {
        const int pa = __builtin_amdgcn_readlane(a, first), pg = __builtin_amdgcn_readlane(g, first);
        if (pa != ba || pg != bg) load_b(bv, pa, pg);
        ba = pa;
        bg = pg;
        multiply(rows, first);
        served |= rows;
      });
    }
    // rows without an adapter are copied
    if (blockIdx.z == 0 && !inplace) served |= (uint32_t)__ballot(live && a < 0) & 0xffffu;
    if (!served) return;
    // an infinity in B meets v's value and its remainder, which may be 0 or of the other
    // sign: rows with a sum that is not finite are left to the end (where it is cheapest
    // in registers: 4,096 rows, 2,048 -> 7,168: 52.7 -> 53.1 us a call with it)
    uint32_t odd = 0;
    if constexpr (BF) {
      float zero = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) zero = fmaf(acc[j][e], 0.f, zero);
      const uint64_t b = __ballot(zero != zero);
      odd = (uint32_t)(b | (b >> 16) | (b >> 32) | (b >> 48)) & 0xffffu;
      served &= ~odd;
    }
    // acc[j][e]: column n0 + (bf16: 32 (j / 2) + 8 lg + 4 (j % 2), float: 16 j + 4 lg) + e of row l16
    u32x4_t o[YV];
    if constexpr (BF) {
      // to whole 128-byte lines: lanes l16 and l16 ^ 8 have half a line each of two
      // rows and swap one, so that a load or store covers 8 rows x 128 bytes
      auto swap = [&](const u32x4_t& lo, const u32x4_t& hi, u32x4_t& a0, u32x4_t& a1) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t send = l16 < 8 ? hi[q] : lo[q];
          const uint32_t got = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)send, 0x128, 0xf, 0xf, false);  // row_ror 8
          a0[q] = l16 < 8 ? lo[q] : got;
          a1[q] = l16 < 8 ? got : hi[q];
        }
      };
      u32x4_t m[2], t[2];
      swap(y[0], y[1], m[0], m[1]);
#pragma unroll
      for (int i2 = 0; i2 < 2; ++i2)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4_t& c = acc[2 * i2 + (q >> 1)];
          t[i2][q] = a < 0 ? m[i2][q]
                           : (uint32_t)f32_to_bf16(__uint_as_float(m[i2][q] << 16) + c[2 * (q & 1)]) |
                                 ((uint32_t)f32_to_bf16(__uint_as_float(m[i2][q] & 0xffff0000u) + c[2 * (q & 1) + 1]) << 16);
        }
      swap(t[0], t[1], o[0], o[1]);
    } else {
#pragma unroll
      for (int i2 = 0; i2 < YV; ++i2)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          o[i2][q] = a < 0 ? y[i2][q] : __float_as_uint(__uint_as_float(y[i2][q]) + acc[i2][q]);
    }
    T* const ob = (T*)p.out + (size_t)w * AW * p.N;
#pragma unroll
    for (int i2 = 0; i2 < YV; ++i2)
      if (((served >> ar[i2]) & 1u) && cc[i2] < p.N) *reinterpret_cast<u32x4_t*>(ob + (uint32_t)(ar[i2] * p.N + cc[i2])) = o[i2];
    // ... and summed from value and remainder together, a lane a column of the row
    if constexpr (BF) {
      for (; odd; odd &= odd - 1) {
        const int r = __builtin_ctz(odd), n = n0 + lane, rk = __builtin_amdgcn_readlane(rank, r);
        if (n >= p.N) continue;
        const T* const bm = (const T*)p.b + (((size_t)__builtin_amdgcn_readlane(a, r) * p.G +
                                              __builtin_amdgcn_readlane(g, r)) * p.N + n) * (size_t)p.R;
        const T* const vr = vin + ((size_t)w * AW + r) * p.R;
        float s = 0.f;
#pragma unroll 1
        for (int k = 0; k < rk; ++k)
          s = fmaf(bf16_to_f32(vr[k]) + bf16_to_f32(vr[(size_t)p.rows * p.R + k]), bf16_to_f32(bm[k]), s);
        const size_t at = ((size_t)w * AW + r) * p.N + n;
        ((T*)p.out)[at] = f32_to_bf16(bf16_to_f32(((const T*)p.y)[at]) + s);
      }
    }
  };
  for (int w = w0; w < w1; w += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (w + d < w1) window(yv[d], vf[d], w + d);
      load_window(yv[d], vf[d], w + d + D);
    }
  }
}

template <typename T>
static void launch_adapt_t(const AdaptArgs& p, void* v, hipStream_t st) {
  const int windows = (p.rows + AW - 1) / AW;
  const int cols = (p.N + 255) / 256;  // workgroups across the columns
  // windows of a wave: one while the waves are few, up to 8
  const int wpw = max(1, min(8, (int)((long long)windows * cols * 4 / 4096)));
  const int splits = (windows + wpw - 1) / wpw;
  // shares of a window's pairs: 1 where the windows fill the chip, 2 where they are
  // few (128 rows of 32 adapters, the one shape measured, us a call: 21.9 with 1, 20.0
  // with 2, 20.7 with 3, 21.6 with 4)
  const int ze = max(1, min(2, 4096 / (cols * 4 * splits)));
  const bool ahead = wpw == 1;
  const int rt = (p.R + 15) / 16, rtp = rt <= 2 ? rt : (rt <= 4 ? 4 : 8);
  const int steps = (p.K * (int)sizeof(T) + 63) / 64;
  const int nw = max(1, min(rtp <= 2 ? 16 : 32 / rtp, steps / 4));
  const int zs = max(1, min(16, 2048 / (windows * nw)));
  const size_t lds = (size_t)nw * AW * (16 * rtp + 1) * sizeof(float);
#define MOE_ADAPT(RT, NF)                                                                                       \
  do {                                                                                                          \
    hipLaunchKernelGGL((adapt_shrink_kernel<T, RT>), dim3(windows, zs), dim3(64 * nw), lds, st, p, v);          \
    if (ahead)                                                                                                  \
      hipLaunchKernelGGL((adapt_expand_kernel<T, NF, ((NF) <= 2)>), dim3(cols, splits, ze), dim3(256), 0, st, p,  \
                         (const T*)v, wpw);                                                                     \
    else                                                                                                        \
      hipLaunchKernelGGL((adapt_expand_kernel<T, NF, false>), dim3(cols, splits, ze), dim3(256), 0, st, p,      \
                         (const T*)v, wpw);                                                                     \
  } while (0)
  constexpr bool BF = sizeof(T) == 2;
  if (rt == 1) MOE_ADAPT(1, 1);
  else if (rt == 2) MOE_ADAPT(2, BF ? 1 : 2);
  else if (rt <= 4) MOE_ADAPT(4, BF ? 2 : 4);
  else MOE_ADAPT(8, BF ? 4 : 8);
#undef MOE_ADAPT
}

hipError_t launch_adapt(int dtype, const AdaptArgs& p, void* v, hipStream_t st) {
  if (p.rows == 0) return hipSuccess;
  if (dtype == DT_BF16) launch_adapt_t<bf16_t>(p, v, st);
  else launch_adapt_t<float>(p, v, st);
  return hipGetLastError();
}

}  // namespace moe
