// The whole layer for a few tokens (at most 16): moe_forward_few, moe_experts_few.
//
// With so few tokens the time is that of the chosen experts' weights and of the
// launches, so nothing is permuted: every chosen expert's weight tile is multiplied
// with all tokens at once (one 16-column matrix instruction, rowtile.h) and only the
// tokens that chose it are kept.  Three launches (float32 with 4-bit weights: few_split_kernel
// before gate/up, four):
//
//   logits   float64 partial logits (given routes: none)
//   gate/up  every workgroup: per token the top k_t and their weights, then the list of
//            the experts that some token chose, ascending, all in LDS; then
//            H[row][i] = w * SiLU(x_t . Wg_i) * (x_t . Wu_i), with row and w those of the
//            token's choice of the expert (row t k_max + j for its j-th) and a row per
//            token for the always-on expert
//   down     out[t] = sum over the list of H . Wd: one workgroup owns 8 to 32 outputs of
//            all tokens and sums over every expert, so there is no combine
//
// The routing weight is applied to H in float32 before its one rounding to the
// element type, so that the down products of all experts share their accumulators.  (bf16: the
// matrix instruction takes no more, and moe_ffn rounds there too.  Against float64 the layer is
// off by 0.0023 of its norm, with H in float32 by 0.0017, of which the outputs' own rounding is
// most.)
//
// Measured (us; logits, gate/up, down; floor: weights at 7.2 TB/s of reads):
//   1 token, 128 experts of 768 x 2048, 8 of them: 4.4 + 15.6 + 7.5, floor 10.5 (latency)
//   4 tokens, 256 experts of 2048 x 7168, budgets 4 and 8, an always-on expert: 6 + 207 .. 265 +
//     112 .. 142 for 23 and 30 experts, 6.8 and 6.3 TB/s, floors 294 and 379
//   16 tokens, 256 experts of 384 x 2048, budgets 0 to 32: 4.9 + 66 .. 82 + 35 .. 44 for 99 and 132
//     experts, floors 65 and 87
//   codes in groups of 64 with zero points, 8 tokens, 256 experts of 2048 x 7168: 6 + 170 .. 190
//     + 69 .. 77 for 50 and 55 experts (190 .. 231 + 77 .. 85 in another run), floors 171 and 187
// Three launches: one launch with a ticket a phase took 57 us for the one token and 410 for the
// four, for its fences empty the caches and its workgroup fills a CU.
//
// The code is kept short on purpose: a launch begins with a cold instruction cache (a down
// kernel unrolled over a ring of 8 steps took 16 us for one token where 4 took 11).  Loops are
// rolled unless their loads must be in flight together.
#include "common.h"
#include "launch.h"
#include "rowtile.h"
#include "select.h"

namespace moe {

constexpr int FEW_T = MOE_FEW_MAX_T;
constexpr int FEW_S = 8;                  // slices of the partial logits, at most
// Slices that the logits are summed in: 4 for up to 2048 inputs (every gate/up workgroup
// reads them all), else 8 (twice the workgroups for the products).  Whole layers with experts of
// 128, us with 4 and with 8, bf16:
//   inputs                      1024          2048          4096          7168
//   16 tokens, 256 experts   23.6, 25.4    27.2, 28.2    35.2, 36.0    53.1, 53.0
//   16 tokens, 8 experts     15.1, 15.2    16.4, 15.5    22.3, 21.0    31.7, 29.7
//   1 token, 256 experts     13.1, 13.2    14.2, 13.7    15.9, 15.0    27.6, 25.5
//   1 token, 600 experts     15.1, 15.5    16.1, 16.5    18.2, 18.5    29.7, 30.1
// float32 likewise (16 tokens, 256 experts: 36.8, 37.7 at 2048; 84.3, 82.9 at 7168).
__host__ __device__ __forceinline__ int few_slices(int d) { return d <= 2048 ? 4 : 8; }

// What the launches take.
struct FewArgs {
  int T, d, E, I, Is, k_max, blocked;
  int stride;               // workgroups of the gate/up launch
  int hw;                   // width of a row of H: max(I, Is)
  int zero_row;             // rows: T k_max choices, T of the always-on expert, one of zeros
  // routing: partial logits, or given routes (part null)
  BudgetPolicy pol;
  float scale;
  const double* part;
  const float* bias;
  const int32_t* k;
  const int32_t *off, *ids;
  const float* wts;
  int32_t *stats, *status;
  int32_t* n_list;          // the list for the down launch: its length,
  int32_t* expert;          // the experts,
  uint32_t* rows;           // and their tokens' rows [.][16] (16 bits each)
  const void* x;
  void* h;                  // in planes
  size_t plane;             // elements of a plane
  const void* xh;           // 4-bit weights: x, as H is kept
  size_t xplane;
  void* out;
  RowWeights w[6];          // gate, up, down, and the always-on expert's
};
// a or b, by value: a reference to either would put both into memory.
__device__ __forceinline__ RowWeights pick(bool first, RowWeights a, RowWeights b) {
  return RowWeights{first ? a.w : b.w, first ? a.scales : b.scales, first ? a.zeros : b.zeros};
}

// The list of chosen experts, in LDS.
struct FewList {
  // while it is made (in the place of what the products need later)
  uint32_t* keys;   // [T][E]
  uint32_t* mask;   // [E] tokens of an expert, bit t
  uint32_t* all;    // [E][8] as rows, of every expert
  // what stays
  int32_t* expert;  // [min(E, T k_max)] ascending
  uint32_t* rows;   // [min(E, T k_max)][8] rows of H of its tokens, 16 bits each; zero_row: none
  float* w;         // [T k_max] weight of a choice
};
__host__ __device__ __forceinline__ int few_scratch_words(int T, int E) { return ((T + 9) * E + 3) & ~3; }
__host__ __device__ __forceinline__ int few_kept_words(int T, int E, int k_max) {
  return 9 * min(E, T * k_max) + T * k_max;
}
// The list lies behind what else the launch keeps in LDS (`used` bytes) and the scratch,
// which overlap.
__device__ __forceinline__ FewList few_carve(char* lds, int used, const FewArgs& p) {
  const int T = p.T, E = p.E, k_max = p.k_max;
  uint32_t* const scratch = reinterpret_cast<uint32_t*>(lds);
  uint32_t* const kept = scratch + max(used / 4, few_scratch_words(T, E));
  const int cap = min(E, T * k_max);
  FewList L;
  L.keys = scratch;
  L.mask = scratch + T * E;
  L.all = L.mask + E;
  L.expert = reinterpret_cast<int32_t*>(kept);
  L.rows = kept + cap;
  L.w = reinterpret_cast<float*>(kept + 9 * cap);
  return L;
}
__device__ __forceinline__ int few_row(const FewList& L, int idx, int t) {
  return reinterpret_cast<const uint16_t*>(L.rows)[idx * FEW_T + t];
}

// Largest of one value per lane, in every lane: row shifts, then the rows' last lanes
// passed on, which leaves the maximum in lane 63.  For whole waves only: a lane that a
// condition has switched off (the right side of && and || too) neither gives its value nor
// passes on the others', and lane 63 is read whether it is on or not.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#define MOE_DPP_MAX(ctrl, rows) \
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xf, false))
  MOE_DPP_MAX(0x111, 0xf);  // row_shr:1, 2, 4, 8
  MOE_DPP_MAX(0x112, 0xf);
  MOE_DPP_MAX(0x114, 0xf);
  MOE_DPP_MAX(0x118, 0xf);
  MOE_DPP_MAX(0x142, 0xa);  // row_bcast:15, 31
  MOE_DPP_MAX(0x143, 0xc);
#undef MOE_DPP_MAX
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// A token's choice from its keys, by one wave: the largest key kt times, ties to the lowest
// expert (select.h's keys and order; its radix search takes fewer steps from some 20 experts
// a token on, but many times the code).  Lane j ends with the j-th choice (kt <= 64) and its
// logit.
// Up to 256 experts: every lane sorts its four keys once, so that a round is the largest of
// the lanes' first keys (some 150 cycles; with four keys to look at in each round, 500).
__device__ __forceinline__ void few_choose256(const uint32_t* keys, int E, int kt, int& mine, float& logit) {
  const int lane = threadIdx.x & 63;
  uint32_t k[4];
  int e[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    e[s] = lane + 64 * s;
    k[s] = e[s] < E ? keys[e[s]] : 0;  // 0: none
  }
  // equal keys keep their order
  auto order = [&](int a, int b) {
    const bool swap = k[b] > k[a];
    const uint32_t ka = k[a];
    const int ea = e[a];
    k[a] = swap ? k[b] : ka;
    e[a] = swap ? e[b] : ea;
    k[b] = swap ? ka : k[b];
    e[b] = swap ? ea : e[b];
  };
  order(0, 1), order(1, 2), order(2, 3), order(0, 1), order(1, 2), order(0, 1);
#pragma unroll 1
  for (int j = 0; j < kt; ++j) {
    const uint32_t m = wave_max_u32(k[0]);
    const bool top = k[0] == m;
    uint64_t has = __ballot(top);
    if (has & (has - 1)) {  // several lanes: the lowest expert
      const uint32_t low = ~wave_max_u32(top ? ~(uint32_t)e[0] : 0u);
      has = __ballot(top && (uint32_t)e[0] == low);
    }
    const int l = __builtin_ctzll(has), pick = __builtin_amdgcn_readlane(e[0], l);
    mine = lane == j ? pick : mine;
    logit = lane == j ? key_logit(m) : logit;
    const bool own = lane == l;
#pragma unroll
    for (int s = 0; s < 3; ++s) {
      k[s] = own ? k[s + 1] : k[s];
      e[s] = own ? e[s + 1] : e[s];
    }
    k[3] = own ? 0 : k[3];
  }
}
// Up to 1024.
__device__ __forceinline__ void few_choose1024(const uint32_t* keys, int E, int kt, int& mine, float& logit) {
  const int lane = threadIdx.x & 63;
  uint32_t key[16];
#pragma unroll
  for (int s = 0; s < 16; ++s) key[s] = lane + 64 * s < E ? keys[lane + 64 * s] : 0;  // 0: none, or chosen
#pragma unroll 1
  for (int j = 0; j < kt; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int s = 1; s < 16; ++s) m = max(m, key[s]);
    m = wave_max_u32(m);
    int e = 0;
#pragma unroll
    for (int s = 15; s >= 0; --s) {
      const uint64_t has = __ballot(key[s] == m);
      e = has ? 64 * s + __builtin_ctzll(has) : e;
    }
#pragma unroll
    for (int s = 0; s < 16; ++s) key[s] = e == lane + 64 * s ? 0 : key[s];
    mine = lane == j ? e : mine;
    logit = lane == j ? key_logit(m) : logit;
  }
}

// The list, by a whole workgroup; every workgroup builds the same one, and the first
// stores it for the down launch.  Returns the number of experts.
template <int NT>
__device__ __forceinline__ int few_list(const FewArgs& p, const FewList& L) {
  constexpr int NW = NT / 64;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const bool first = blockIdx.x == 0;
  const uint32_t none = (uint32_t)p.zero_row * 0x10001u;
  int v = 0;
  if (p.part) {
    v = lane < p.T ? p.k[lane] : 0;
    const int n = p.T * p.E, slices = few_slices(p.d);
#pragma unroll 1
    for (int i = tid; i < n; i += 2 * NT) {  // two values in flight
      double part[2][FEW_S];
      float b[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int iu = min(i + u * NT, n - 1);
#pragma unroll
        for (int q = 0; q < FEW_S; ++q) part[u][q] = q < 4 || slices > 4 ? p.part[(size_t)q * n + iu] : 0.0;
        b[u] = p.bias ? p.bias[(uint32_t)iu % (uint32_t)p.E] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        double l = 0.0;
#pragma unroll
        for (int q = 0; q < FEW_S; ++q) l += part[u][q];
        if (p.bias) l += (double)b[u];
        if (i + u * NT < n) L.keys[i + u * NT] = max(logit_key((float)l), 1u);
      }
    }
  }
#pragma unroll 1
  for (int i = tid; i < 9 * p.E; i += NT) L.mask[i] = i < p.E ? 0 : none;  // and the rows behind them
  __syncthreads();
  int exec = 0;
  if (p.part) {
    const bool ok = budget_valid(v, p.k_max);
    const int kb = p.pol.policy == K_BATCH_MAX ? (int)wave_max_u32(ok ? (uint32_t)v : 0u) : 0;
    exec = lane < p.T ? budget_exec(v, p.k_max, p.pol, kb) : 0;
    const bool bad = __ballot(!ok) != 0;
    if (first && p.status && tid == 0) p.status[0] = bad ? MOE_DEV_BAD_K_BIT : 0;
  }
  // Where waves have two tokens and budgets can differ by much, the token with the i-th largest
  // goes with the one with the i-th least (16 tokens of 256 experts with budgets of 0, 8, 16, 32
  // by turns, two of 32 on a wave without: gate/up 85.8 -> 81.7 us; the ranks take 0.7).
  int rank = lane < p.T ? lane : 64;
  if (p.T > NW && p.k_max > 8) {
    rank = lane < p.T ? 0 : 64;
#pragma unroll 1
    for (int t = 0; t < p.T; ++t) {
      const int other = __builtin_amdgcn_readlane(exec, t);
      rank += other > exec || (other == exec && t < lane) ? 1 : 0;
    }
  }
#pragma unroll 1
  for (int i = 0; i < p.T; i += NW) {
    const uint64_t turn = __ballot(rank == (i & NW ? i + NW - 1 - wave : i + wave));
    if (!turn) continue;
    const int t = __builtin_ctzll(turn);
    int e = -1;
    float w = 0.f;
    if (p.part) {
      const int kt = __builtin_amdgcn_readlane(exec, t);
      if (p.E <= 256) few_choose256(L.keys + t * p.E, p.E, kt, e, w);
      else few_choose1024(L.keys + t * p.E, p.E, kt, e, w);
      const float ex = e >= 0 ? expf(w - __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(w)))) : 0.f;
      float sum = ex;
#pragma unroll 1
      for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, 64);
      w = ex * (p.scale / sum);
    } else {
      // Given routes (k_max <= 64: one entry a lane).  An expert that the token names twice
      // counts once with both weights; ids outside [0, E) are skipped; offsets outside the
      // arrays are cut.
      const int cap = p.T * p.k_max;
      const int beg = min(max(p.off[t], 0), cap), n = min(min(max(p.off[t + 1], beg), cap) - beg, p.k_max);
      const int id = lane < n ? p.ids[beg + lane] : -1;
      const float mine = lane < n ? p.wts[beg + lane] : 0.f;
      e = id >= 0 && id < p.E ? id : -1;
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        const bool same = __shfl(id, j, 64) == id;
        const float wj = __shfl(mine, j, 64);
        w += same ? wj : 0.f;
        if (same && j < lane) e = -1;
      }
    }
    if ((uint32_t)e < (uint32_t)p.E) {  // the tables have E rows
      L.w[t * p.k_max + lane] = w;
      reinterpret_cast<uint16_t*>(L.all)[e * FEW_T + t] = (uint16_t)(t * p.k_max + lane);
      atomicOr(&L.mask[e], 1u << t);
    }
  }
  __syncthreads();
  // a wave lists the experts of every NW-th chunk of 64, and counts what lies before them
  // itself
  int base = 0, rows = 0;
#pragma unroll 1
  for (int c = 0; 64 * c < p.E; ++c) {
    const int e = 64 * c + lane;
    const uint32_t m = e < p.E ? L.mask[e] : 0;
    const uint64_t act = __ballot(m != 0);
    if (c % NW == wave && m) {
      const int at = base + __popcll(act & ((1ull << lane) - 1ull));
      L.expert[at] = e;
      if (first) p.expert[at] = e;
    }
    if (first && wave == 0 && p.stats) {
      if (e < p.E) p.stats[e] = __popc(m);
      rows += __popc(m);
    }
    base += __popcll(act);
  }
  if (first && wave == 0) {
    if (lane == 0) p.n_list[0] = base;
    if (p.stats) {
#pragma unroll 1
      for (int o = 32; o >= 1; o >>= 1) rows += __shfl_xor(rows, o, 64);
      if (lane == 0) {
        p.stats[p.E] = base;
        p.stats[p.E + 1] = rows;
      }
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int i = tid; i < base * 8; i += NT) {
    const uint32_t r = L.all[L.expert[i >> 3] * 8 + (i & 7)];
    L.rows[i] = r;
    if (first) p.rows[i] = r;
  }
  __syncthreads();
  return base;
}

// The waves' accumulators of a tile in LDS, [waves][64 lanes][4]; the sum of output n (of
// 16) for token t, in wave order.
template <int NW>
__device__ __forceinline__ float few_sum(const f32x4_t* red, int n, int t) {
  const float* r = reinterpret_cast<const float*>(red) + ((n >> 2) * 16 + t) * 4 + (n & 3);
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) v += r[w * 256];
  return v;
}

// Rows of zeros for the tokens without a part in an expert.
template <class Op, int NT>
__device__ __forceinline__ void few_zero_row(const FewArgs& p) {
  typename Op::hid* const h = static_cast<typename Op::hid*>(p.h);
#pragma unroll 1
  for (int q = 0; q < Op::PLANES; ++q)
#pragma unroll 1
    for (int i = threadIdx.x; i < p.hw; i += NT) h[q * p.plane + (size_t)p.zero_row * p.hw + i] = 0;
}

// H of column n of a row.
template <class Op>
__device__ __forceinline__ void few_store_h(const FewArgs& p, const FewList& L, bool sh, int n, float g, float u,
                                            int row) {
  const float rw = sh ? 1.f : L.w[row];
  Op::store_h(static_cast<typename Op::hid*>(p.h) + (size_t)row * p.hw + n, p.plane, rw * (silu(g) * u));
}

// ---- element weights ----
// A wave streams its share of K through a ring of its own in LDS: copies of whole 128-byte
// lines straight from memory, past the caches (weights are read once), NB steps of 16 rows
// x 128 bytes ahead and on into the workgroup's next item, the activations of a step beside
// its weights.  So the loop is short, needs no barrier, and its loads may carry the
// non-temporal hint, which would fetch lines twice that two register loads take by halves
// (reads of 2 GiB: 7.2 TB/s with it, 6.4 without).  Bound by memory: gate/up of 30 experts
// reads 6.8 TB/s; a ring in registers, two or four steps deep, 37 and 41 us for the one token
// (now 27 in all) and 362 .. 400 for the four (now 365).
constexpr int FEW_RW = 8;                 // waves of a workgroup
constexpr int FEW_RT = 64 * FEW_RW;

__device__ __forceinline__ void few_barrier() {
  lgkm_wait0();
  compiler_fence();
  __builtin_amdgcn_s_barrier();
  compiler_fence();
}

// A step's operand from LDS.
template <typename T>
__device__ __forceinline__ typename DenseOp<T>::W few_frag(const char* tile) {
  const int lane = threadIdx.x & 63;
  typename DenseOp<T>::W w;
#pragma unroll
  for (int i = 0; i < 2; ++i) w.v[i] = *reinterpret_cast<const u32x4_t*>(tile + lds_off(lane & 15, (lane >> 4) + 4 * i));
  return w;
}

// Gate and up: a workgroup takes every p.stride-th item, 8 intermediate columns of one expert:
// a tile of 8 gate rows and the same 8 up rows.  (16 columns, two tiles, leave one token's 384
// items on 256 workgroups: 15.7 us for the last one where 11.1 did the first.)  XQ: copies of
// the activations, 1 for up to 8 tokens.
template <typename T, int NB, int XQ>
__global__ __launch_bounds__(FEW_RT) void few_gateup_dense_kernel(FewArgs p) {
  typedef DenseOp<T> Op;
  constexpr int SLOT = 2048 + 1024 * XQ, PER = 2 + XQ;
  extern __shared__ char few_ring[];  // the rings and the waves' sums (the list's scratch before), the list
  const RowWeights wg = p.w[0], wu = p.w[1], sg = p.w[3], su = p.w[4];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  f32x4_t* const red = reinterpret_cast<f32x4_t*>(few_ring + FEW_RW * NB * SLOT);
  const FewList L = few_carve(few_ring, FEW_RW * NB * SLOT + FEW_RT * 16, p);
  const int n_list = few_list<FEW_RT>(p, L);
  if (blockIdx.x == 0) few_zero_row<Op, FEW_RT>(p);
  const int ci = p.I / 8, routed = n_list * ci;
  const int n_items = routed + p.Is / 8;
  const int steps = p.d / Op::KS, kstr = w_kstep<T>(p.blocked) * (int)sizeof(T);
  const int beg = steps * wave / FEW_RW, end = steps * (wave + 1) / FEW_RW;
  const int pitch = (p.blocked ? Op::KS : p.d) * (int)sizeof(T);
  // a lane's place in the copies: tile rows 0..7 of gate, 8..15 (rows 0..7 of up)
  const uint32_t row0 = (uint32_t)copy_row(0) * pitch;
  const uint32_t goff = row0 + copy_byte(0), uoff = row0 + copy_byte(1);
  uint32_t xoff[XQ];
#pragma unroll
  for (int q = 0; q < XQ; ++q)  // rows behind the last token repeat it; their sums are not used
    xoff[q] = (uint32_t)min(copy_row(q), p.T - 1) * p.d * (uint32_t)sizeof(T) + copy_byte(q);
  char* const ring = few_ring + wave * NB * SLOT;

  // requests: a step of the item `want`; behind the last item its last step again
  int want = blockIdx.x, rs = beg;
  const char *rg = nullptr, *ru = nullptr;
  auto seek = [&]() {
    const bool sh = want >= routed;
    const int idx = sh ? 0 : (int)((uint32_t)want / (uint32_t)ci);
    const int n0 = (sh ? want - routed : want - idx * ci) * 8, N = sh ? p.Is : p.I;
    const int mat = sh ? 0 : __builtin_amdgcn_readfirstlane(L.expert[idx]);
    const size_t o = ((size_t)mat * N * p.d + Op::corner(n0, p.d, p.blocked)) * sizeof(T);
    rg = static_cast<const char*>(sh ? sg.w : wg.w) + o;
    ru = static_cast<const char*>(sh ? su.w : wu.w) + o;
  };
  auto request = [&](int slot) {
    char* const to = ring + slot * SLOT;
    const size_t o = (size_t)rs * kstr;
    copy_rows<2>(rg + o, goff, to);
    copy_rows<2>(ru + o, uoff, to + 1024);
#pragma unroll
    for (int q = 0; q < XQ; ++q) copy_rows<0>(static_cast<const char*>(p.x) + rs * 128, xoff[q], to + 2048 + 1024 * q);
    if (rs + 1 < end) {
      ++rs;
    } else if (want + p.stride < n_items) {
      want += p.stride;
      rs = beg;
      seek();
    }
  };
  const bool live = beg < end && want < n_items;
  if (live) {
    seek();
#pragma unroll 1
    for (int i = 0; i < NB; ++i) request(i);
  }
  int slot = 0;
#pragma unroll 1
  for (int item = blockIdx.x; item < n_items; item += p.stride) {
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int s = beg; s < end; ++s) {
      vm_wait<PER * (NB - 1)>();
      compiler_fence();
      const char* const from = ring + slot * SLOT;
      const typename Op::W w = few_frag<T>(from), xw = few_frag<T>(from + 2048);
      lgkm_wait0();  // read before the slot is filled again
      compiler_fence();
      request(slot);
      slot = slot + 1 == NB ? 0 : slot + 1;
      Op::mma(acc, w, typename Op::X{{xw.v[0], xw.v[1]}});
    }
    settle(acc);
    red[wave * 64 + lane] = acc;
    few_barrier();
    if (wave < 2) {
      const bool sh = item >= routed;
      const int idx = sh ? 0 : (int)((uint32_t)item / (uint32_t)ci);
      const int n0 = (sh ? item - routed : item - idx * ci) * 8;
      const int j = tid & 7, t = tid >> 3;
      const float g = few_sum<FEW_RW>(red, j, t), u = few_sum<FEW_RW>(red, j + 8, t);
      const int row = sh ? p.T * p.k_max + t : few_row(L, idx, t);
      if (t < p.T && row != p.zero_row) few_store_h<Op>(p, L, sh, n0 + j, g, u, row);
    }
    few_barrier();
  }
  vm_wait<0>();  // no copy into LDS outlives the workgroup
}

// The list that the gate/up launch stored, into LDS: experts, and their tokens' rows.
template <int NT>
__device__ __forceinline__ int few_load_list(const FewArgs& p, uint32_t* to) {
  const int cap = min(p.E, p.T * p.k_max);
#pragma unroll 1
  for (int i = threadIdx.x; i < 9 * cap; i += NT)  // what lies behind the list is not used
    to[i] = i < cap ? (uint32_t)p.expert[i] : p.rows[i - cap];
  return __builtin_amdgcn_readfirstlane(p.n_list[0]);
}

// An output that is not finite, from its own token's products alone.
template <class Op>
__device__ __forceinline__ float few_down_again(const FewArgs& p, const int32_t* l_expert, const uint16_t* row_of,
                                                int n_list, int n, int t, bool& nan) {
  float sum = 0.f;
#pragma unroll 1
  for (int i = 0; i <= n_list; ++i) {
    const bool sh = i == n_list;
    if (sh && !p.Is) break;
    const int row = sh ? p.T * p.k_max + t : row_of[i * FEW_T + t];
    if (row == p.zero_row) continue;
    const int mat = sh ? 0 : l_expert[i], K = sh ? p.Is : p.I;
    const typename Op::hid* const hr = static_cast<const typename Op::hid*>(p.h) + (size_t)row * p.hw;
    sum += wave_dot(K, [&](int k) { return Op::h_value(hr, p.plane, k); },
                    [&](int k) { return Op::value(pick(sh, p.w[5], p.w[2]), mat, n, k, p.d, K, p.blocked); }, nan);
    if (nan) break;
  }
  return sum;
}

// Down: a workgroup owns some outputs of every token; its waves share the steps of all the
// experts' intermediate columns, laid end to end.  Tokens without a part in an expert read
// the row of zeros.
// PAIR (up to 8 tokens): a tile is 8 outputs at two steps, rows 8 .. 15 and columns 8 .. 15
// those of the second, and what a step's rows have with the other's columns is not used.  Of
// 2048 outputs that gives 256 workgroups where tiles of 16 leave half of the GPU idle.
// Otherwise 16 outputs, a step at a time.
template <typename T, int NB, bool PAIR>
__global__ __launch_bounds__(FEW_RT) void few_down_dense_kernel(FewArgs p) {
  typedef DenseOp<T> Op;
  constexpr int SLOT = 4096, PER = 4, ROWS = PAIR ? 8 : 16, H = PAIR ? 1 : 2;
  extern __shared__ char few_ring[];  // the rings, the waves' sums, the list
  const RowWeights wr = p.w[2], ws = p.w[5];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int n0 = blockIdx.x * ROWS;
  f32x4_t* const red = reinterpret_cast<f32x4_t*>(few_ring + FEW_RW * NB * SLOT);
  const int32_t* const l_expert = reinterpret_cast<const int32_t*>(red + FEW_RT);
  const uint16_t* const row_of = reinterpret_cast<const uint16_t*>(l_expert + min(p.E, p.T * p.k_max));
  const int n_list = few_load_list<FEW_RT>(p, reinterpret_cast<uint32_t*>(red + FEW_RT));
  __syncthreads();
  const int spe = p.I / Op::KS, routed = n_list * spe, steps = routed + p.Is / Op::KS;
  const int beg = steps * wave / FEW_RW, end = steps * (wave + 1) / FEW_RW;
  const int rounds = PAIR ? (end - beg + 1) / 2 : end - beg;
  const int kstr = w_kstep<T>(p.blocked) * (int)sizeof(T);
  char* const ring = few_ring + wave * NB * SLOT;

  // requests: step st of expert idx of the list (behind it: the always-on expert); behind the
  // wave's end its last step again, in a pair with rows of zeros
  int idx = beg < routed ? (int)((uint32_t)beg / (uint32_t)spe) : n_list, st = beg - min(idx * spe, routed), left = end - beg;
  const char* rw = nullptr;
  uint32_t woff = 0, hoff[H];
  uint32_t wjump = 0;  // from a tile's row to the one 8 further
  const uint32_t zero = (uint32_t)p.zero_row * p.hw * (uint32_t)sizeof(T);
  auto seek = [&]() {
    const bool sh = idx >= n_list;
    const int K = sh ? p.Is : p.I;
    const int mat = sh ? 0 : __builtin_amdgcn_readfirstlane(l_expert[idx]);
    rw = static_cast<const char*>(sh ? ws.w : wr.w) +
         ((size_t)mat * p.d * K + Op::corner(n0, K, p.blocked)) * sizeof(T);
    const int pitch = (p.blocked ? Op::KS : K) * (int)sizeof(T);
    woff = (uint32_t)copy_row(0) * pitch;
    wjump = 8u * pitch;
#pragma unroll
    for (int q = 0; q < H; ++q) {
      const int t = copy_row(q);
      const int row = sh ? (t < p.T ? p.T * p.k_max + t : p.zero_row) : row_of[idx * FEW_T + t];
      hoff[q] = (uint32_t)row * p.hw * (uint32_t)sizeof(T);
    }
  };
  auto advance = [&]() {
    --left;
    if (left > 0) {
      ++st;
      if (idx < n_list && st == spe) {
        ++idx;
        st = 0;
        seek();
      }
    }
  };
  auto request = [&](int slot) {
    char* const to = ring + slot * SLOT;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const char* const h = static_cast<const char*>(p.h) + st * 128;
      const uint32_t b = copy_byte(q);
      copy_rows<2>(rw + (size_t)st * kstr + (PAIR ? 0u : q * wjump), woff + b, to + 1024 * q);
      copy_rows<0>(h, (PAIR && left <= 0 ? zero : hoff[PAIR ? 0 : q]) + b, to + 2048 + 1024 * q);
      if (PAIR || q == 1) advance();
    }
  };
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  if (beg < end) {
    seek();
#pragma unroll 1
    for (int i = 0; i < NB; ++i) request(i);
    int slot = 0;
#pragma unroll 1
    for (int s = 0; s < rounds; ++s) {
      vm_wait<PER * (NB - 1)>();
      compiler_fence();
      const char* const from = ring + slot * SLOT;
      const typename Op::W w = few_frag<T>(from), xw = few_frag<T>(from + 2048);
      lgkm_wait0();
      compiler_fence();
      request(slot);
      slot = slot + 1 == NB ? 0 : slot + 1;
      Op::mma(acc, w, typename Op::X{{xw.v[0], xw.v[1]}});
    }
    vm_wait<0>();  // no copy into LDS outlives the workgroup
  }
  settle(acc);
  red[wave * 64 + lane] = acc;
  __syncthreads();
  if (wave < (PAIR ? 1 : 4)) {
    const int j = tid % ROWS, t = tid / ROWS;
    float v = few_sum<FEW_RW>(red, j, t);
    if (PAIR) v += few_sum<FEW_RW>(red, j + 8, t + 8);
    redo_not_finite(v, t < p.T, t, [&](int l, bool& nan) {
      const int i = wave * 64 + l;
      return few_down_again<Op>(p, l_expert, row_of, n_list, n0 + i % ROWS, i / ROWS, nan);
    });
    if (t < p.T) static_cast<T*>(p.out)[(size_t)t * p.d + n0 + j] = Elt<T>::from_f32(v);
  }
}

// ---- 4-bit weights ----
// As with element weights, a wave streams its share of K through a ring in LDS: at each step
// NT tiles' codes (1 KB each in a row), their scales and zero points, and the activations,
// which the tiles share.  With every load in registers and none ahead (all 16 waves waiting
// at the end of each item) the 8 tokens took 284 .. 306 + 150 .. 164 us.  What bounds gate/up
// now is the copies: 157 .. 172 of 170 .. 190 us without any product; of each 4.35 KB of a step
// 2 are codes (without the activations 131, without the scales, 32 bytes of a line at a time,
// 129).  Down reads 5.6 TB/s.
// Float32 activations are read as the three bf16 parts that few_split_kernel leaves in the
// workspace (2.3 us): taken apart beside each tile they were most of 57 us of a gate/up launch
// that takes 15 now (5 tokens, 61 experts of 640 x 1152, latency).
// XQ 1: up to 8 tokens lie in rows 0, 1, 4, 5, .. of the 16, and a lane scales two results
// where it has four of 16 tokens (the vector instructions are as long as the copies).
template <class Op, int NT, int XQ, int WAVES>
struct FewQ {
  typedef typename Op::elt T;
  typedef typename Op::hid H;
  static constexpr int RT = XQ == 1 ? 2 : 4;              // results of a lane
  static constexpr int RUN = 16 * (int)sizeof(T);         // a tile's scales of one group
  // a tile's scales of a step, then its zero points
  static constexpr int SB = Op::NG * RUN, ZB = Op::ZP ? Op::NG * 16 : 0, SZ = NT * (SB + ZB), SC = (SZ + 255) / 256;
  static constexpr int X0 = NT * 1024, S0 = X0 + 2048 * XQ * Op::PLANES, SLOT = S0 + 256 * SC;
  // Waves: 8 for gate/up, whose items all of them end together (16: 210 us where 8 took 197, 256
  // experts, 8 tokens), 16 for down (8 tokens, 2048 outputs: 51 us of both launches with 16, 54
  // with 8) where two slots of each fit.
  static constexpr bool FITS = 2 * WAVES * SLOT + NT * WAVES * 64 * RT * 4 + 4096 <= 160 * 1024;
  static constexpr int NW = FITS ? WAVES : 8;
  static constexpr int SW = Op::PLANES * XQ > 3 ? 4 : NW;  // waves that stream: 16 float32 tokens' slots fit 4
  static constexpr int RING = SW * SLOT, SUMS = NT * SW * 64 * RT * 4;  // bytes: one slot of each, their sums
  static constexpr int PER = NT + 2 * XQ * Op::PLANES + SC;

  // where the next step's operands come from
  const char* q[NT];
  const char* sz[SC];           // of a lane
  uint32_t sz_step[SC];
  const H* x;

  __device__ __forceinline__ void seek(const typename Op::Src (&t)[NT], const H* xs, int step) {
    const uint32_t lane = threadIdx.x & 63, Np = t[0].Np;
#pragma unroll
    for (int i = 0; i < NT; ++i) q[i] = reinterpret_cast<const char*>(t[i].q) + (size_t)step * 1024;
#pragma unroll
    for (int c = 0; c < SC; ++c) {  // lanes behind the last copy some again
      const uint32_t b = (256 * c + 4 * lane) % SZ, in = b % (SB + ZB);
      const bool one = NT == 1 || b < SB + ZB, z = ZB && in >= SB;
      const uintptr_t sa = (uintptr_t)t[0].s, sb = (uintptr_t)t[NT - 1].s, za = (uintptr_t)t[0].z, zb = (uintptr_t)t[NT - 1].z;
      const uintptr_t at_s = one ? sa : sb, at_z = one ? za : zb;
      const char* const from = reinterpret_cast<const char*>(z ? at_z : at_s);
      const uint32_t run = z ? 16u : (uint32_t)RUN, o = z ? in - SB : in, pitch = Np * (z ? 1u : (uint32_t)sizeof(T));
      sz_step[c] = Op::NG * pitch;
      sz[c] = from + (o / run * pitch + o % run) + (size_t)step * sz_step[c];
    }
    x = xs + step * Op::KS;
  }
  // Requests a step and goes on to the next one.  Activations: a lane's rows start off[] bytes
  // behind x, planes `plane` elements apart.
  __device__ __forceinline__ void request(char* to, size_t plane, const uint32_t (&off)[XQ], bool on) {
#pragma unroll
    for (int i = 0; i < NT; ++i) copy_rows<2>(q[i], (threadIdx.x & 63) * 16, to + 1024 * i);
#pragma unroll
    for (int c = 0; c < SC; ++c)
      __builtin_amdgcn_global_load_lds((gbl_ptr_t)sz[c], (lds_ptr_t)(to + S0 + 256 * c), 4, 0, 0);
#pragma unroll
    for (int p = 0; p < Op::PLANES; ++p)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < XQ; ++c)
          copy_rows<0>(x + p * plane + 64 * h, off[c], to + X0 + 1024 * ((p * 2 + h) * XQ + c));
    if (on) {
#pragma unroll
      for (int i = 0; i < NT; ++i) q[i] += 1024;
#pragma unroll
      for (int c = 0; c < SC; ++c) sz[c] += sz_step[c];
      x += Op::KS;
    }
  }
  __device__ __forceinline__ static void load(const char* from, typename Op::W (&w)[NT], typename Op::X& x) {
    const int lane = threadIdx.x & 63, n = lane & 15, row = XQ == 1 ? (n >> 2) * 2 + (n & 1) : n;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      w[i].q = *reinterpret_cast<const u32x4_t*>(from + 1024 * i + 16 * lane);
#pragma unroll
      for (int g = 0; g < Op::NG; ++g) {
        w[i].s[g] = *reinterpret_cast<const T*>(from + S0 + i * (SB + ZB) + g * RUN + n * (int)sizeof(T));
        if (Op::ZP) w[i].z[g] = *reinterpret_cast<const uint8_t*>(from + S0 + i * (SB + ZB) + SB + g * 16 + n);
      }
    }
#pragma unroll
    for (int p = 0; p < Op::PLANES; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x.v[p][i] = *reinterpret_cast<const u32x4_t*>(from + X0 + 1024 * XQ * (p * 2 + i / 2) +
                                                      lds_off(row, (lane >> 4) + 4 * (i & 1)));
  }
  // The waves' results of tile i in LDS, and their sum for output n of token t, in wave order.
  __device__ __forceinline__ static void keep(float* red, int i, f32x4_t acc) {
    if (SW < NW && threadIdx.x >= SW * 64) return;
#pragma unroll
    for (int r = 0; r < RT; ++r) red[(i * SW * 64 + threadIdx.x) * RT + r] = acc[r];
  }
  __device__ __forceinline__ static float sum(const float* red, int i, int n, int t) {
    const float* const r = red + (i * SW * 64 + t / RT * 16 + n) * RT + t % RT;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < SW; ++w) v += r[w * 64 * RT];
    return v;
  }
};

template <class Op, int NB, int XQ>
__global__ __launch_bounds__((64 * FewQ<Op, 2, XQ, 8>::NW)) void few_gateup_q4_kernel(FewArgs p) {
  typedef FewQ<Op, 2, XQ, 8> Q;
  typedef typename Op::elt T;
  typedef typename Op::hid H;
  extern __shared__ char few_ring[];  // the rings and the waves' sums (the list's scratch before), the list
  const RowWeights wg = p.w[0], wu = p.w[1], sg = p.w[3], su = p.w[4];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  float* const red = reinterpret_cast<float*>(few_ring + NB * Q::RING);
  const FewList L = few_carve(few_ring, NB * Q::RING + 2 * Q::SUMS, p);
  const int n_list = few_list<64 * Q::NW>(p, L);
  if (blockIdx.x == 0) few_zero_row<Op, 64 * Q::NW>(p);
  const int ci = p.I / TILE_N, routed = n_list * ci;
  const int n_items = routed + p.Is / TILE_N, first = near_tile(blockIdx.x, p.stride);
  const int steps = p.d / Op::KS;
  const int beg = wave < Q::SW ? steps * wave / Q::SW : 0, end = wave < Q::SW ? steps * (wave + 1) / Q::SW : 0;
  uint32_t xoff[XQ];
#pragma unroll
  for (int c = 0; c < XQ; ++c)  // rows behind the last token repeat it; their sums are not used
    xoff[c] = (uint32_t)min(copy_row(c), p.T - 1) * p.d * (uint32_t)sizeof(H) + copy_byte(c);
  char* const ring = few_ring + wave * NB * Q::SLOT;

  // requests: a step of the item `want`; behind the last item its last step again
  Q rq;
  int want = first, rs = beg;
  auto seek = [&]() {
    const bool sh = want >= routed;
    const int idx = sh ? 0 : (int)((uint32_t)want / (uint32_t)ci);
    const int n0 = (sh ? want - routed : want - idx * ci) * TILE_N, N = sh ? p.Is : p.I;
    const int mat = sh ? 0 : __builtin_amdgcn_readfirstlane(L.expert[idx]);
    rq.seek({Op::tile(pick(sh, sg, wg), mat, n0, N, p.d), Op::tile(pick(sh, su, wu), mat, n0, N, p.d)},
            static_cast<const H*>(p.xh), beg);
  };
  auto request = [&](int slot) {
    const bool on = rs + 1 < end;
    rq.request(ring + slot * Q::SLOT, p.xplane, xoff, on);
    if (on) {
      ++rs;
    } else if (want + p.stride < n_items) {
      want += p.stride;
      rs = beg;
      seek();
    }
  };
  if (beg < end && want < n_items) {
    seek();
#pragma unroll 1
    for (int i = 0; i < NB; ++i) request(i);
  }
  int slot = 0, turn = 0;
#pragma unroll 1
  for (int item = first; item < n_items; item += p.stride) {
    f32x4_t acc[2][1] = {{{0.f, 0.f, 0.f, 0.f}}, {{0.f, 0.f, 0.f, 0.f}}};
#pragma unroll 1
    for (int s = beg; s < end; ++s) {
      vm_wait<Q::PER * (NB - 1)>();
      compiler_fence();
      typename Op::W w[2];
      typename Op::X x[1];
      Q::load(ring + slot * Q::SLOT, w, x[0]);
      lgkm_wait0();  // read before the slot is filled again
      compiler_fence();
      request(slot);
      slot = slot + 1 == NB ? 0 : slot + 1;
      Op::template step<Q::RT>(acc, w, x);
    }
    settle(acc[0][0]);
    settle(acc[1][0]);
    // sums of one item and the next by turns: the waves that add them up (others each time) are
    // past the next barrier before their half is written again
    float* const part = red + (turn & 1) * (Q::SUMS / 4);
    Q::keep(part, 0, acc[0][0]);
    Q::keep(part, 1, acc[1][0]);
    few_barrier();
    const int adds = (wave + 2 * XQ * turn++) % Q::NW;
    if (adds < 2 * XQ) {
      const bool sh = item >= routed;
      const int idx = sh ? 0 : (int)((uint32_t)item / (uint32_t)ci);
      const int n0 = (sh ? item - routed : item - idx * ci) * TILE_N, N = sh ? p.Is : p.I;
      const int mat = sh ? 0 : __builtin_amdgcn_readfirstlane(L.expert[idx]);
      const int lane = tid & 63, j = lane & 15, t = 4 * adds + (lane >> 4);
      float g = Q::sum(part, 0, j, t), u = Q::sum(part, 1, j, t);
      const int row = sh ? p.T * p.k_max + t : few_row(L, idx, t);
      const bool mine = t < p.T && row != p.zero_row;
      auto again = [&](RowWeights rw, float& val) {
        redo_not_finite(val, mine, t, [&](int l, bool& nan) {
          const T* xr = static_cast<const T*>(p.x) + (size_t)(4 * adds + (l >> 4)) * p.d;
          const int nn = n0 + (l & 15);
          return wave_dot(p.d, [&](int k) { return Elt<T>::to_f32(xr[k]); },
                          [&](int k) { return Op::value(rw, mat, nn, k, N, p.d, 0); }, nan);
        });
      };
      again(pick(sh, sg, wg), g);
      again(pick(sh, su, wu), u);
      if (mine) few_store_h<Op>(p, L, sh, n0 + j, g, u, row);
    }
  }
  vm_wait<0>();  // no copy into LDS outlives the workgroup
}

// Down: NT tiles of 16 outputs for every token, otherwise as with element weights.
template <class Op, int NB, int XQ, int NT>
__global__ __launch_bounds__((64 * FewQ<Op, NT, XQ, 16>::NW)) void few_down_q4_kernel(FewArgs p) {
  typedef FewQ<Op, NT, XQ, 16> Q;
  typedef typename Op::hid H;
  extern __shared__ char few_ring[];  // the rings, the waves' sums, the list
  const RowWeights wr = p.w[2], ws = p.w[5];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = near_tile(blockIdx.x, gridDim.x) * (NT * TILE_N);
  float* const red = reinterpret_cast<float*>(few_ring + NB * Q::RING);
  int32_t* const list = reinterpret_cast<int32_t*>(red + Q::SUMS / 4);
  const int32_t* const l_expert = list;
  const uint16_t* const row_of = reinterpret_cast<const uint16_t*>(list + min(p.E, p.T * p.k_max));
  const int n_list = few_load_list<64 * Q::NW>(p, reinterpret_cast<uint32_t*>(list));
  __syncthreads();
  const int spe = p.I / Op::KS, routed = n_list * spe, steps = routed + p.Is / Op::KS;
  const int beg = wave < Q::SW ? steps * wave / Q::SW : 0, end = wave < Q::SW ? steps * (wave + 1) / Q::SW : 0;
  char* const ring = few_ring + wave * NB * Q::SLOT;

  // requests: step st of expert idx of the list (behind it: the always-on expert); behind the
  // wave's end its last step again
  int idx = beg < routed ? (int)((uint32_t)beg / (uint32_t)spe) : n_list, st = beg - min(idx * spe, routed), left = end - beg;
  Q rq;
  uint32_t hoff[XQ];
  auto seek = [&]() {
    const bool sh = idx >= n_list;
    const int mat = sh ? 0 : __builtin_amdgcn_readfirstlane(l_expert[idx]);
    typename Op::Src t[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) t[i] = Op::tile(pick(sh, ws, wr), mat, n0 + i * TILE_N, p.d, sh ? p.Is : p.I);
    rq.seek(t, static_cast<const H*>(p.h), st);
#pragma unroll
    for (int c = 0; c < XQ; ++c) {
      const int tok = copy_row(c);
      const int row = sh ? (tok < p.T ? p.T * p.k_max + tok : p.zero_row) : row_of[idx * FEW_T + tok];
      hoff[c] = (uint32_t)row * p.hw * (uint32_t)sizeof(H) + copy_byte(c);
    }
  };
  auto request = [&](int slot) {
    const bool on = left > 1;
    rq.request(ring + slot * Q::SLOT, p.plane, hoff, on);
    --left;
    if (on) {
      ++st;
      if (idx < n_list && st == spe) {
        ++idx;
        st = 0;
        seek();
      }
    }
  };
  f32x4_t acc[NT][1];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i][0] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (beg < end) {
    seek();
#pragma unroll 1
    for (int i = 0; i < NB; ++i) request(i);
    int slot = 0;
#pragma unroll 1
    for (int s = beg; s < end; ++s) {
      vm_wait<Q::PER * (NB - 1)>();
      compiler_fence();
      typename Op::W w[NT];
      typename Op::X x[1];
      Q::load(ring + slot * Q::SLOT, w, x[0]);
      lgkm_wait0();
      compiler_fence();
      request(slot);
      slot = slot + 1 == NB ? 0 : slot + 1;
      Op::template step<Q::RT>(acc, w, x);
    }
    vm_wait<0>();  // no copy into LDS outlives the workgroup
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    settle(acc[i][0]);
    Q::keep(red, i, acc[i][0]);
  }
  __syncthreads();
  if (wave < 2 * XQ * NT) {
    const int j = tid % (NT * 16), t = tid / (NT * 16);
    float v = Q::sum(red, j >> 4, j & 15, t);
    redo_not_finite(v, t < p.T, t, [&](int l, bool& nan) {
      const int i = wave * 64 + l;
      return few_down_again<Op>(p, l_expert, row_of, n_list, n0 + i % (NT * 16), i / (NT * 16), nan);
    });
    if (t < p.T) static_cast<typename Op::elt*>(p.out)[(size_t)t * p.d + n0 + j] = Elt<typename Op::elt>::from_f32(v);
  }
}

// The three bf16 parts of float32 activations (2.3 us, a launch's latency).
__global__ __launch_bounds__(256) void few_split_kernel(const float* __restrict__ x, int n, bf16_t* __restrict__ to) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  uint32_t a, b, c;
  split3(x[i], a, b, c);
  to[i] = (bf16_t)(a >> 16);
  to[n + i] = (bf16_t)(b >> 16);
  to[2 * n + i] = (bf16_t)(c >> 16);
}

// Partial logits part[slices][T][E] in float64 on the f64 matrix instruction: a workgroup
// takes 16 experts and a slice of d for all tokens, its 8 waves a share each, added in
// wave order; 2.4 us (8 experts, 256 inputs) to 6.3 (256, 7168), latency.  (Lane l supplies the values of row l % 16 from LE (l / 16) on of a step,
// value i of every lane in instruction i.)
constexpr int FEW_LW = 8;
typedef double f64x4_t __attribute__((ext_vector_type(4)));

template <typename T>
__global__ __launch_bounds__(64 * FEW_LW) void few_logits_kernel(const T* __restrict__ x, const T* __restrict__ w,
                                                                 int T_, int d, int E, double* __restrict__ part) {
  constexpr int LE = 16 / (int)sizeof(T), KS = 4 * LE;
  __shared__ f64x4_t red[FEW_LW * 64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int l16 = lane & 15, lg = lane >> 4;
  const int e0 = blockIdx.x * 16, steps = d / KS, nq = gridDim.y * FEW_LW, q = blockIdx.y * FEW_LW + wave;
  const int s0 = steps * q / nq, s1 = steps * (q + 1) / nq;
  const T* wr = w + (size_t)min(e0 + l16, E - 1) * d + lg * LE;
  const T* xr = x + (size_t)min(l16, T_ - 1) * d + lg * LE;
  f64x4_t acc = {0.0, 0.0, 0.0, 0.0};
  for (int s = s0; s < s1; ++s) {
    const u32x4_t wv = *reinterpret_cast<const u32x4_t*>(wr + (size_t)s * KS);
    const u32x4_t xv = *reinterpret_cast<const u32x4_t*>(xr + (size_t)s * KS);
#pragma unroll
    for (int i = 0; i < LE; ++i) {
      double a, b;
      if constexpr (sizeof(T) == 2) {
        a = (double)__uint_as_float((i & 1) ? wv[i / 2] & 0xffff0000u : wv[i / 2] << 16);
        b = (double)__uint_as_float((i & 1) ? xv[i / 2] & 0xffff0000u : xv[i / 2] << 16);
      } else {
        a = (double)__uint_as_float(wv[i]);
        b = (double)__uint_as_float(xv[i]);
      }
      acc = __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, acc, 0, 0, 0);
    }
  }
  settle(acc);
  red[wave * 64 + lane] = acc;
  __syncthreads();
  // acc[i]: expert 4 i + lg, token l16; a thread sums one value
  if (threadIdx.x < 256) {
    const int src = threadIdx.x & 63, i = threadIdx.x >> 6;
    const int e = e0 + 4 * i + (src >> 4), t = src & 15;
    double s = 0.0;
#pragma unroll
    for (int v = 0; v < FEW_LW; ++v) s += red[v * 64 + src][i];
    if (t < T_ && e < E) part[((size_t)blockIdx.y * T_ + t) * E + e] = s;
  }
}

// No tokens: no counts, a status of 0.
__global__ void few_none_kernel(int32_t* stats, int n, int32_t* status) {
  for (int i = threadIdx.x; i < n && stats; i += blockDim.x) stats[i] = 0;
  if (threadIdx.x == 0 && status) status[0] = 0;
}

// -------------------------------------------------------------------- launches

template <class K>
static hipError_t few_launch(K kernel, int grid, int threads, size_t lds, const FewArgs& p, hipStream_t st) {
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(threads), lds, st, p);
  return hipGetLastError();
}

// Ring depths: as many steps as 160 KB of LDS hold beside the list (5 with one copy of
// activations, 4 with two, one less where the list is long).
constexpr int FEW_LDS = 160 * 1024;

template <typename T, bool PAIR>
static hipError_t few_dense_down(const FewArgs& p, int more, hipStream_t st) {
  constexpr int SLOTS = FEW_RW * 4096;
  const int tiles = p.d / (PAIR ? 8 : 16);
  return 4 * SLOTS + more <= FEW_LDS
             ? few_launch(few_down_dense_kernel<T, 4, PAIR>, tiles, FEW_RT, 4 * SLOTS + more, p, st)
             : few_launch(few_down_dense_kernel<T, 3, PAIR>, tiles, FEW_RT, 3 * SLOTS + more, p, st);
}

template <typename T, int NB, int XQ>
static hipError_t few_dense(FewArgs p, hipStream_t st) {
  constexpr int RING = FEW_RW * NB * (2048 + 1024 * XQ), LESS = FEW_RW * (NB - 1) * (2048 + 1024 * XQ);
  p.stride = min(256, min(p.E, p.T * p.k_max) * (p.I / 8) + p.Is / 8);
  const int scratch = few_scratch_words(p.T, p.E) * 4, sums = FEW_RT * 16;
  const int kept = few_kept_words(p.T, p.E, p.k_max) * 4, list = 36 * min(p.E, p.T * p.k_max);
  const int up = max(RING + sums, scratch) + kept;
  const hipError_t e =
      up <= FEW_LDS ? few_launch(few_gateup_dense_kernel<T, NB, XQ>, p.stride, FEW_RT, up, p, st)
                    : few_launch(few_gateup_dense_kernel<T, NB - 1, XQ>, p.stride, FEW_RT,
                                 max(LESS + sums, scratch) + kept, p, st);
  if (e != hipSuccess) return e;
  // Pairs for up to 8 tokens, unless tiles of 16 fill the CUs evenly.  gate/up and down of 4 bf16
  // tokens, 32 experts of 1024, 4 of them a token, us in tiles of 16 and in pairs:
  //   2048 outputs (128 tiles) 39.3, 35.3   4096 (256) 53.6, 55.9   8192 (512) 99, 104
  //   4224 (264) 66.8, 64.8                 6144 (384) 84.5, 83.7   8320 (520) 108.9, 109.1
  // Where tiles of 16 leave few CUs idle without filling them pairs cost up to 6%: 3968 (248) 53.5,
  // 56.1; 7168 (448) 95.6, 101.5; of 64 experts of 2048 at 7168 341.9, 340.4, of one token 113.5,
  // 116.3.  float32: 2048 69, 61; 4096 106, 106; 6144 163, 157; 7168 186, 190; 8192 231, 227.
  return XQ == 1 && p.d / 16 % 256 ? few_dense_down<T, true>(p, sums + list, st) : few_dense_down<T, false>(p, sums + list, st);
}

// Steps of a ring: 160 KB less the sums and 4 KB for a list.
constexpr int few_depth(int ring, int sums, int most) {
  const int deep = (FEW_LDS - 4096 - sums) / ring;
  return deep < 1 ? 1 : deep < most ? deep : most;
}

template <class Op, int XQ, int NT>
static hipError_t few_q4_down(const FewArgs& p, int list, hipStream_t st) {
  typedef FewQ<Op, NT, XQ, 16> Q;
  constexpr int SUMS = Q::SUMS, NB = few_depth(Q::RING, SUMS, 5), LESS = NB > 1 ? NB - 1 : 1;
  const int lds = NB * Q::RING + SUMS + list, tiles = p.d / (NT * TILE_N);
  return lds <= FEW_LDS ? few_launch(few_down_q4_kernel<Op, NB, XQ, NT>, tiles, 64 * Q::NW, lds, p, st)
                        : few_launch(few_down_q4_kernel<Op, LESS, XQ, NT>, tiles, 64 * Q::NW,
                                     LESS * Q::RING + SUMS + list, p, st);
}

template <class Op, int XQ>
static hipError_t few_q4_as(FewArgs p, hipStream_t st) {
  if (Op::PLANES == 1) {
    p.xh = p.x;
  } else {
    const int n = p.T * p.d;
    bf16_t* const to = static_cast<bf16_t*>(p.h) + Op::PLANES * p.plane;
    p.xh = to, p.xplane = n;
    hipLaunchKernelGGL(few_split_kernel, dim3(ceil_div(n, 256)), dim3(256), 0, st, (const float*)p.x, n, to);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int kept = few_kept_words(p.T, p.E, p.k_max) * 4, list = 36 * min(p.E, p.T * p.k_max);
  p.stride = min(256, min(p.E, p.T * p.k_max) * (p.I / TILE_N) + p.Is / TILE_N);
  // ring depths: as many steps as 160 KB of LDS hold, one less where the list is long
  typedef FewQ<Op, 2, XQ, 8> Q;
  constexpr int SUMS = 2 * Q::SUMS, NB = few_depth(Q::RING, SUMS, 4), LESS = NB > 1 ? NB - 1 : 1;
  const int scratch = few_scratch_words(p.T, p.E) * 4;
  const int up = max(NB * Q::RING + SUMS, scratch) + kept;
  hipError_t e;
  if (up <= FEW_LDS) e = few_launch(few_gateup_q4_kernel<Op, NB, XQ>, p.stride, 64 * Q::NW, up, p, st);
  else e = few_launch(few_gateup_q4_kernel<Op, LESS, XQ>, p.stride, 64 * Q::NW, max(LESS * Q::RING + SUMS, scratch) + kept, p, st);
  if (e != hipSuccess) return e;
  // Two tiles of outputs share their activations where more than 256 tiles are there for 256
  // CUs (8 tokens, 32 experts of 1024, gate/up with it, us with one and with two: 4096 outputs
  // 42, 45; 4224 51, 46; 7168 69, 63; 12288 99, 97; one token 15.6, 17.0; 19.0, 17.0; 21.6, 19.6;
  // 31.9, 28.8; 16 tokens 61, 65; 76, 66; 100, 89; 153, 145).
  return p.d > 256 * TILE_N ? few_q4_down<Op, XQ, 2>(p, list, st) : few_q4_down<Op, XQ, 1>(p, list, st);
}

template <class Op>
static hipError_t few_q4(const FewArgs& p, hipStream_t st) {
  return p.T <= 8 ? few_q4_as<Op, 1>(p, st) : few_q4_as<Op, 2>(p, st);
}

template <typename T>
static hipError_t few_ffn(const FewArgs& p, int group, int zeros, hipStream_t st) {
  if (group == 0) return p.T <= 8 ? few_dense<T, 5, 1>(p, st) : few_dense<T, 4, 2>(p, st);
  if (group == 32) return zeros ? few_q4<Q4Op<T, 32, true>>(p, st) : few_q4<Q4Op<T, 32, false>>(p, st);
  if (group == 64) return zeros ? few_q4<Q4Op<T, 64, true>>(p, st) : few_q4<Q4Op<T, 64, false>>(p, st);
  return zeros ? few_q4<Q4Op<T, 128, true>>(p, st) : few_q4<Q4Op<T, 128, false>>(p, st);
}

size_t few_part_count(int T, int E) { return (size_t)FEW_S * T * E; }
size_t few_h_bytes(int dtype, int T, int d, int k_max, int I, int Is) {
  const size_t rows = (size_t)T * k_max + T + 1;  // choices, the always-on expert's, zeros
  // float32 with 4-bit weights: three planes, and x in three planes behind them
  return dtype == DT_BF16 ? rows * max(I, Is) * 2 : (rows * max(I, Is) + (size_t)T * d) * 6;
}

hipError_t launch_few(const FewLaunch& a, hipStream_t st) {
  if (a.T == 0) {
    if (a.stats || a.status)
      hipLaunchKernelGGL(few_none_kernel, dim3(1), dim3(256), 0, st, a.stats, a.E + 2, a.status);
    return hipGetLastError();
  }
  FewArgs p{};
  p.T = a.T, p.d = a.d, p.E = a.E, p.I = a.I, p.Is = a.Is, p.k_max = a.k_max, p.blocked = a.blocked;
  p.x = a.x;
  for (int i = 0; i < 6; ++i) p.w[i] = RowWeights{a.w[i], a.scales[i], static_cast<const uint8_t*>(a.zeros[i])};
  p.off = a.in_off, p.ids = a.in_ids, p.wts = a.in_w;
  p.stats = a.stats, p.status = a.status;
  p.n_list = a.n_list, p.expert = a.expert, p.rows = a.rows;
  p.h = a.h;
  p.hw = max(a.I, a.Is);
  p.zero_row = a.T * a.k_max + a.T;
  p.plane = ((size_t)p.zero_row + 1) * p.hw;
  p.out = a.out;
  if (a.w_router) {
    p.part = a.part, p.bias = a.bias, p.k = a.k, p.pol = a.pol, p.scale = a.scale;
    const dim3 grid(ceil_div(a.E, 16), few_slices(a.d));
    if (a.dtype == DT_BF16)
      hipLaunchKernelGGL(few_logits_kernel<bf16_t>, grid, dim3(64 * FEW_LW), 0, st, (const bf16_t*)a.x,
                         (const bf16_t*)a.w_router, a.T, a.d, a.E, a.part);
    else
      hipLaunchKernelGGL(few_logits_kernel<float>, grid, dim3(64 * FEW_LW), 0, st, (const float*)a.x,
                         (const float*)a.w_router, a.T, a.d, a.E, a.part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return a.dtype == DT_BF16 ? few_ffn<bf16_t>(p, a.group, a.zeros[0] != nullptr, st)
                            : few_ffn<float>(p, a.group, a.zeros[0] != nullptr, st);
}

}  // namespace moe
