// The whole layer for a few tokens (at most 16): moe_forward_few, moe_experts_few.
//
// With so few tokens the time is that of the chosen experts' weights and of the
// launches, so nothing is permuted: every chosen expert's weight tile is multiplied
// with all tokens at once (one 16-column matrix instruction, rowtile.h) and only the
// tokens that chose it are kept.
//
//   logits   float64 partial logits (route_grouped.hip)
//   select   one workgroup: per token the top k_t and their weights (select.h), then
//            the list of the experts that some token chose, ascending, with the mask
//            of its tokens, their weights and its first intermediate row
//   gate/up  H[row][i] = w_t * SiLU(x_t . Wg_i) * (x_t . Wu_i), one row for each
//            (expert, token) of the list and one per token for the always-on expert
//   down     out[t] = sum over the list of H . Wd: one workgroup owns 16 outputs of
//            all tokens and sums over every expert, so there is no combine
//
// The routing weight is applied to H in float32 before its one rounding to the
// element type, so that the down products of all experts share their accumulators.
#include "common.h"
#include "launch.h"
#include "rowtile.h"
#include "select.h"

namespace moe {

constexpr int FEW_NW = 8;                 // waves of a workgroup, each a share of K
constexpr int FEW_NT = 64 * FEW_NW;
constexpr int FEW_SEL_NT = 1024;          // one wave per token

// The list as the kernels read it (device memory).
struct FewList {
  int32_t* head;    // [0] experts of the list, [1] rows
  int32_t* expert;  // [cap]
  int32_t* mask;    // [cap] tokens, bit t
  int32_t* row;     // [cap] first row of H
  float* w;         // [T][E] weights, where a mask has its bit
};

// The list of the experts that some token chose, from mask[e] in LDS.
template <int NT>
__device__ void few_list(const uint32_t* mask, int E, const FewList& L, int32_t* stats, int32_t* wsum) {
  const int tid = threadIdx.x, per = (E + NT - 1) / NT;
  int act = 0, rows = 0;
  for (int j = 0; j < per; ++j) {
    const int e = tid * per + j;
    const uint32_t m = e < E ? mask[e] : 0;
    act += m != 0;
    rows += __popc(m);
  }
  const int ia = block_scan_incl<NT>(act, wsum), ir = block_scan_incl<NT>(rows, wsum);
  int at = ia - act, row = ir - rows;
  for (int j = 0; j < per; ++j) {
    const int e = tid * per + j;
    if (e >= E) break;
    const uint32_t m = mask[e];
    if (stats) stats[e] = __popc(m);
    if (!m) continue;
    L.expert[at] = e;
    L.mask[at] = (int32_t)m;
    L.row[at] = row;
    ++at;
    row += __popc(m);
  }
  if (tid == NT - 1) {
    L.head[0] = ia;
    L.head[1] = ir;
    if (stats) {
      stats[E] = ia;
      stats[E + 1] = ir;
    }
  }
}

// KPL logits a lane (E <= 64 * KPL).
template <int KPL>
__global__ __launch_bounds__(FEW_SEL_NT) void few_select_kernel(const double* __restrict__ part, int S,
                                                                const float* __restrict__ bias,
                                                                const int32_t* __restrict__ tok_off, int T, int E,
                                                                int k_max, float scale, FewList L, int32_t* stats) {
  extern __shared__ uint64_t few_smem[];
  __shared__ int32_t wsum[FEW_SEL_NT / 64];
  const int tid = threadIdx.x, t = tid >> 6, lane = tid & 63;
  uint32_t* mask = reinterpret_cast<uint32_t*>(few_smem);
  uint64_t* scratch = few_smem + (E + 1) / 2 + (size_t)t * (k_max + 1);
  float* wts = reinterpret_cast<float*>(few_smem + (E + 1) / 2 + (size_t)T * (k_max + 1)) + t * k_max;
  for (int e = tid; e < E; e += FEW_SEL_NT) mask[e] = 0;
  __syncthreads();
  if (t < T) {
    const int kt = tok_off[t + 1] - tok_off[t];
    uint32_t key[KPL];
#pragma unroll
    for (int s = 0; s < KPL; ++s) {
      const int e = lane + 64 * s;
      key[s] = 0;
      if (e < E) {
        double l = 0.0;
#pragma unroll 1
        for (int q = 0; q < S; ++q) l += part[((size_t)q * T + t) * E + e];
        if (bias) l += (double)bias[e];
        key[s] = logit_key((float)l);
      }
    }
    if (kt > 0) {
      int pos[KPL];
#pragma unroll
      for (int s = 0; s < KPL; ++s) pos[s] = -1;
      wave_topk_softmax_emit<KPL>(key, kt, scale, [&](int j, int s) { pos[s] = j; }, wts, scratch);
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
      for (int s = 0; s < KPL; ++s)
        if (pos[s] >= 0) {
          const int e = lane + 64 * s;
          L.w[t * E + e] = wts[pos[s]];
          atomicOr(&mask[e], 1u << t);
        }
    }
  }
  __syncthreads();
  few_list<FEW_SEL_NT>(mask, E, L, stats, wsum);
}

// The list from given routes.  An expert that a token names twice counts once with
// both weights; ids outside [0, E) are skipped; offsets outside the arrays are cut.
__global__ __launch_bounds__(FEW_SEL_NT) void few_routes_kernel(const int32_t* __restrict__ tok_off,
                                                                const int32_t* __restrict__ ids,
                                                                const float* __restrict__ w, int T, int E, int k_max,
                                                                FewList L) {
  extern __shared__ uint64_t few_smem[];
  __shared__ int32_t wsum[FEW_SEL_NT / 64];
  const int tid = threadIdx.x, t = tid >> 6, lane = tid & 63;
  uint32_t* mask = reinterpret_cast<uint32_t*>(few_smem);
  for (int e = tid; e < E; e += FEW_SEL_NT) mask[e] = 0;
  __syncthreads();
  if (t < T) {
    const int cap = T * k_max;
    const int beg = min(max(tok_off[t], 0), cap), n = min(min(max(tok_off[t + 1], beg), cap) - beg, k_max);
    const int id = lane < n ? ids[beg + lane] : -1;
    const float mine = lane < n ? w[beg + lane] : 0.f;
    bool first = id >= 0 && id < E;
    float sum = 0.f;
    for (int j = 0; j < n; ++j) {  // k_max <= 64: one entry a lane
      const int other = __shfl(id, j, 64);
      const float wj = __shfl(mine, j, 64);
      if (other == id) {
        sum += wj;
        if (j < lane) first = false;
      }
    }
    if (first) {
      L.w[t * E + id] = sum;
      atomicOr(&mask[id], 1u << t);
    }
  }
  __syncthreads();
  few_list<FEW_SEL_NT>(mask, E, L, nullptr, wsum);
}

// What the FFN kernels take.
struct FewFfn {
  int T, d, E, I, Is, blocked;
  const void* x;
  RowWeights w[6];  // gate, up, down, and the always-on expert's
  FewList L;
  void* h;          // rows of width max(I, Is), in planes
  size_t plane;     // elements of a plane
  int hw;           // width of an intermediate row
  void* out;
};

// Sum of the waves' accumulators of one tile, by one wave.
__device__ __forceinline__ f32x4_t few_sum(const f32x4_t* red) {
  const int lane = threadIdx.x & 63;
  f32x4_t v = red[lane];
#pragma unroll
  for (int w = 1; w < FEW_NW; ++w) v += red[w * 64 + lane];
  return v;
}

// Gate and up: a workgroup takes 16 intermediate columns of one expert at a time, its
// waves a share of d each, whose activations stay in registers from tile to tile when
// XS steps a wave cover d.
template <class Op, int XS, int NB>
__global__ __launch_bounds__(FEW_NT) void few_gateup_kernel(FewFfn p) {
  __shared__ f32x4_t red[2][2][FEW_NW * 64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int col = lane & 15;
  typedef typename Op::elt T;
  static_assert((2 * XS) % NB == 0, "the ring repeats with the tiles");
  const int n_list = p.L.head[0], n_rows = p.L.head[1];
  const int ci = p.I / TILE_N, cs = p.Is / TILE_N;
  const int n_items = n_list * ci + cs;
  const int steps = p.d / Op::KS;
  const int chunks = ceil_div(steps, FEW_NW * XS);
  const T* xrow = static_cast<const T*>(p.x) + (size_t)(col < p.T ? col : 0) * p.d;

  struct Tiles { typename Op::Src a[2]; };
  auto tiles_of = [&](int item) {
    const bool sh = item >= n_list * ci;
    const int idx = sh ? 0 : item / ci, n0 = (sh ? item - n_list * ci : item % ci) * TILE_N;
    const int mat = sh ? 0 : p.L.expert[idx], N = sh ? p.Is : p.I;
    Tiles t;
#pragma unroll
    for (int h = 0; h < 2; ++h) t.a[h] = Op::tile(p.w[h + (sh ? 3 : 0)], mat, n0, N, p.d, p.blocked);
    return t;
  };

  int item = blockIdx.x;
  if (item >= n_items) return;
  typename Op::X x[XS];
  int par = 0;
  for (; item < n_items; item += gridDim.x, par ^= 1) {
    const Tiles cur = tiles_of(item);
    f32x4_t acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    for (int c = 0; c < chunks; ++c) {
      const int c0 = (int)((long long)steps * c / chunks), c1 = (int)((long long)steps * (c + 1) / chunks);
      const int beg = c0 + (c1 - c0) * wave / FEW_NW, n = c0 + (c1 - c0) * (wave + 1) / FEW_NW - beg;
      if (chunks > 1 || item == (int)blockIdx.x) {
#pragma unroll
        for (int s = 0; s < XS; ++s) {
          x[s] = Op::load_x(xrow, min(beg + s, steps - 1));
          if (col >= p.T) Op::clear(x[s]);
          Op::finish_x(x[s]);
        }
      }
      typename Op::W ring[NB];
      auto step_of = [&](int f) { return min(beg + f % XS, steps - 1); };
#pragma unroll
      for (int f = 0; f < NB; ++f) ring[f] = Op::load(cur.a[f / XS], step_of(f));
#pragma unroll
      for (int f = 0; f < 2 * XS; ++f) {
        if (f % XS < n) Op::mma(acc[f / XS], ring[f % NB], x[f % XS]);
        if (f + NB < 2 * XS) ring[f % NB] = Op::load(cur.a[(f + NB) / XS], step_of(f + NB));
      }
    }
    red[par][0][wave * 64 + lane] = acc[0];
    red[par][1][wave * 64 + lane] = acc[1];
    __syncthreads();
    if (wave == 0) {
      f32x4_t g = few_sum(red[par][0]), u = few_sum(red[par][1]);
      const bool sh = item >= n_list * ci;
      const int idx = sh ? 0 : item / ci, n0 = (sh ? item - n_list * ci : item % ci) * TILE_N;
      const uint32_t m = sh ? (1u << p.T) - 1u : (uint32_t)p.L.mask[idx];
      if constexpr (Op::Q4) {
        auto again = [&](const RowWeights& w) {
          return [&, mat = sh ? 0 : p.L.expert[idx]](int r, int c) {
            const T* xr = static_cast<const T*>(p.x) + (size_t)c * p.d;
            return wave_dot(p.d, [&](int k) {
              return Elt<T>::to_f32(xr[k]) * Op::value(w, mat, n0 + r, k, sh ? p.Is : p.I, p.d, p.blocked);
            });
          };
        };
        redo_not_finite(g, (m >> col) & 1, again(p.w[sh ? 3 : 0]));
        redo_not_finite(u, (m >> col) & 1, again(p.w[sh ? 4 : 1]));
      }
      if ((m >> col) & 1) {
        const int row = (sh ? n_rows : p.L.row[idx]) + __popc(m & ((1u << col) - 1u));
        const float w = sh ? 1.f : p.L.w[col * p.E + p.L.expert[idx]];
        f32x4_t v;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = w * (silu(g[r]) * u[r]);
        Op::store_h(static_cast<typename Op::hid*>(p.h) + (size_t)row * p.hw + n0 + 4 * (lane >> 4), p.plane, v);
      }
    }
  }
}

// Down: a workgroup owns 16 outputs of every token; its waves share the steps of all
// the experts' intermediate columns, laid end to end.
template <class Op, int NB>
__global__ __launch_bounds__(FEW_NT) void few_down_kernel(FewFfn p) {
  __shared__ f32x4_t red[FEW_NW * 64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int col = lane & 15;
  const int n_list = p.L.head[0], n_rows = p.L.head[1];
  const int spe = p.I / Op::KS, routed = n_list * spe, steps = routed + p.Is / Op::KS;
  const int beg = (int)((long long)steps * wave / FEW_NW), n = (int)((long long)steps * (wave + 1) / FEW_NW) - beg;
  const int n0 = blockIdx.x * TILE_N;
  const typename Op::hid* h = static_cast<const typename Op::hid*>(p.h);

  // where the next requested step lies
  int idx, st;
  bool ok;
  typename Op::Src src;
  const typename Op::hid* hrow;
  auto seek = [&]() {
    const bool sh = idx >= n_list;
    const uint32_t m = sh ? (1u << p.T) - 1u : (uint32_t)p.L.mask[idx];
    ok = (m >> col) & 1;
    src = Op::tile(p.w[sh ? 5 : 2], sh ? 0 : p.L.expert[idx], n0, p.d, sh ? p.Is : p.I, p.blocked);
    hrow = h + (size_t)((sh ? n_rows : p.L.row[idx]) + (ok ? __popc(m & ((1u << col) - 1u)) : 0)) * p.hw;
  };
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  if (n > 0) {
    idx = beg < routed ? beg / spe : n_list;
    st = beg < routed ? beg % spe : beg - routed;
    seek();
    typename Op::W ring[NB];
    typename Op::X xr[NB];
    bool live[NB];
    int at = 0;
    auto next = [&]() {
      if (at + 1 < n) {
        ++at;
        ++st;
        if (idx < n_list && st == spe) {
          ++idx;
          st = 0;
          seek();
        }
      }
    };
#pragma unroll
    for (int f = 0; f < NB; ++f) {
      ring[f] = Op::load(src, st);
      xr[f] = Op::load_h(hrow, p.plane, st);
      live[f] = ok;
      next();
    }
    for (int s0 = 0; s0 < n; s0 += NB) {
#pragma unroll
      for (int f = 0; f < NB; ++f) {
        if (s0 + f < n) {
          typename Op::X x = xr[f];
          if (!live[f]) Op::clear(x);
          Op::finish_x(x);
          Op::mma(acc, ring[f], x);
        }
        ring[f] = Op::load(src, st);
        xr[f] = Op::load_h(hrow, p.plane, st);
        live[f] = ok;
        next();
      }
    }
  }
  red[wave * 64 + lane] = acc;
  __syncthreads();
  if (wave == 0) {
    f32x4_t v = few_sum(red);
    redo_not_finite(v, col < p.T, [&](int r, int c) {
      float s = 0.f;
      for (int i = 0; i <= n_list; ++i) {
        const bool sh = i == n_list;
        const uint32_t m = sh ? (p.Is ? (1u << p.T) - 1u : 0u) : (uint32_t)p.L.mask[i];
        if (!((m >> c) & 1)) continue;
        const typename Op::hid* hr = h + (size_t)((sh ? n_rows : p.L.row[i]) + __popc(m & ((1u << c) - 1u))) * p.hw;
        const int mat = sh ? 0 : p.L.expert[i], K = sh ? p.Is : p.I;
        s += wave_dot(K, [&](int k) {
          return Op::h_value(hr, p.plane, k) * Op::value(p.w[sh ? 5 : 2], mat, n0 + r, k, p.d, K, p.blocked);
        });
      }
      return s;
    });
    if (col < p.T) store_row4(static_cast<typename Op::elt*>(p.out) + (size_t)col * p.d + n0 + 4 * (lane >> 4), v);
  }
}

// -------------------------------------------------------------------- launches

// LDS of the selection: the masks, and each token's scratch and weights.
static size_t few_sel_lds(int T, int E, int k_max) {
  return (size_t)((E + 1) / 2) * 8 + (size_t)T * (k_max + 1) * 8 + (size_t)T * k_max * 4;
}

template <class Op, int XS, int NB, int NBD>
static hipError_t few_ffn(const FewFfn& p, int cap_items, hipStream_t st) {
  const int grid = min(256, cap_items);
  if (grid > 0) hipLaunchKernelGGL((few_gateup_kernel<Op, XS, NB>), dim3(grid), dim3(FEW_NT), 0, st, p);
  hipLaunchKernelGGL((few_down_kernel<Op, NBD>), dim3(p.d / TILE_N), dim3(FEW_NT), 0, st, p);
  return hipGetLastError();
}

// Activation steps that stay in a wave's registers: the fewest that hold its share of d.
template <class Op, int A, int NA, int B, int NB_, int C, int NC, int NBD>
static hipError_t few_ffn_xs(const FewFfn& p, int cap_items, hipStream_t st) {
  const int need = ceil_div(p.d / Op::KS, FEW_NW);
  if (need <= A) return few_ffn<Op, A, NA, NBD>(p, cap_items, st);
  if (need <= B) return few_ffn<Op, B, NB_, NBD>(p, cap_items, st);
  return few_ffn<Op, C, NC, NBD>(p, cap_items, st);
}

template <typename T>
static hipError_t few_ffn_type(const FewFfn& p, int group, int zeros, int cap, hipStream_t st) {
  if (group == 0) return few_ffn_xs<DenseOp<T>, 4, 8, 8, 8, 14, 7, 4>(p, cap, st);
#define MOE_FEW_Q4(G, Z)                                                                      \
  do {                                                                                        \
    if constexpr (sizeof(T) == 2) return few_ffn_xs<Q4Op<T, G, Z>, 2, 4, 4, 8, 7, 7, 4>(p, cap, st); \
    else return few_ffn<Q4Op<T, G, Z>, 2, 4, 2>(p, cap, st);                                  \
  } while (0)
#define MOE_FEW_G(G) do { if (zeros) MOE_FEW_Q4(G, true); else MOE_FEW_Q4(G, false); } while (0)
  if (group == 32) MOE_FEW_G(32);
  if (group == 64) MOE_FEW_G(64);
  MOE_FEW_G(128);
#undef MOE_FEW_G
#undef MOE_FEW_Q4
}

size_t few_h_bytes(int dtype, int q4, int T, int k_max, int I, int Is) {
  const size_t rows = (size_t)T * k_max + (Is ? T : 0);
  return rows * max(I, Is) * (dtype == DT_BF16 ? 2 : (q4 ? 6 : 4));
}

hipError_t launch_few(const FewLaunch& a, hipStream_t st) {
  if (a.T == 0 && !a.w_router) return hipSuccess;
  FewFfn p;
  p.T = a.T, p.d = a.d, p.E = a.E, p.I = a.I, p.Is = a.Is, p.blocked = a.blocked;
  p.x = a.x;
  for (int i = 0; i < 6; ++i) p.w[i] = RowWeights{a.w[i], a.scales[i], static_cast<const uint8_t*>(a.zeros[i])};
  p.L = FewList{a.head, a.expert, a.mask, a.row, a.wt};
  p.h = a.h;
  p.hw = max(a.I, a.Is);
  p.plane = ((size_t)a.T * a.k_max + (a.Is ? a.T : 0)) * p.hw;
  p.out = a.out;
  const size_t lds = few_sel_lds(a.T, a.E, a.k_max);
  hipError_t e;
  if (a.w_router) {
    e = launch_logits_f64(a.dtype, a.x, a.w_router, a.k, a.T, a.d, a.E, a.k_max, a.pol, a.S, a.part, a.tok_off,
                          a.status, st);
    if (e != hipSuccess) return e;
#define MOE_FEW_SELECT(KPL)                                                                                        \
  hipLaunchKernelGGL(few_select_kernel<KPL>, dim3(1), dim3(FEW_SEL_NT), lds, st, a.part, a.S, a.bias, a.tok_off, a.T, \
                     a.E, a.k_max, a.scale, p.L, a.stats)
    if (a.E <= 64) MOE_FEW_SELECT(1);
    else if (a.E <= 128) MOE_FEW_SELECT(2);
    else if (a.E <= 256) MOE_FEW_SELECT(4);
    else if (a.E <= 512) MOE_FEW_SELECT(8);
    else MOE_FEW_SELECT(16);
#undef MOE_FEW_SELECT
  } else {
    hipLaunchKernelGGL(few_routes_kernel, dim3(1), dim3(FEW_SEL_NT), lds, st, a.in_off, a.in_ids, a.in_w, a.T, a.E,
                       a.k_max, p.L);
  }
  e = hipGetLastError();
  if (e != hipSuccess || a.T == 0) return e;  // no tokens: the counts and the status only
  const int cap = min(a.E, a.T * a.k_max) * (a.I / TILE_N) + a.Is / TILE_N;
  return a.dtype == DT_BF16 ? few_ffn_type<bf16_t>(p, a.group, a.zeros[0] != nullptr, cap, st)
                            : few_ffn_type<float>(p, a.group, a.zeros[0] != nullptr, cap, st);
}

}  // namespace moe
