// Few activation rows against streamed weights: operands of 16-row weight tiles.
//
// A wave multiplies a tile of 16 weight rows with up to 16 activation rows by
// 16x16 matrix instructions; lane l supplies row l % 16 of either side, and the
// result holds rows 4 * (l / 16) + r of the first side and column l % 16, a row of the
// second.  Element weights are the first side.  4-bit weights are the second, so that a
// lane's results share one scale and one zero point.  With few rows the weights' bytes are
// the time, so an operand's `W` is what one lane loads of a tile for one step of K, `X`
// the matching activations:
//
//   DenseOp<bf16>   64 of K: two 16-byte loads, 2 instructions
//   DenseOp<float>  32 of K: two 16-byte loads, 8 instructions
//   Q4Op            128 of K: one 16-byte load of codes and the groups' scales
//
// 4-bit weights.  W[n][k] = s (q - z) with one scale s (and zero point z) for a
// row's group of GROUP inputs.  A code becomes the bf16 value 16 + q without
// arithmetic: bf16 numbers from 16 to 32 are 1/8 apart, so 0x4180 + 8 q is 16 + q.
// The matrix instruction sums x (16 + q) over a group, exact products in float32,
// and the group ends with  acc += s (sum - (16 + z) sum x),  sum x from the same
// instruction with ones for weights.  (The usual base 128 would lose two to
// three more bits to the difference.)  Two mask-and-or operations and shifts for two codes,
// where a conversion of each would cost four.
// What that leaves: an error of some roundings of s sum |x| (32 + q + z), the size of what is
// summed and subtracted again.  For codes all over their range that is 5 (z = 0) to 12 times
// (z = 8) the result's own sum |x| |q - z|, two to four bits; where all lie next to their zero
// point it is more.
// float32 activations are cut into three bf16 parts of 8 bits each, which hold all
// 24 bits (of values below 2^-110 the last ones lie under bf16's least: an error of 1e-6 at
// 2^-114, 2e-5 at 2^-118), and run as three instructions: the float32 matrix instruction
// takes four times the time of all three.
//
// Matrix instructions run whatever the lanes' mask says, so a condition around one has to
// be scalar (the same for the wave, and known to the compiler to be).
//
// Order of the codes: 1 KB per 16 rows x 128 inputs, lane l's 16 bytes at 16 l:
// row l % 16, word i (of 4) inputs 32 i + 8 (l / 16) + 0..7, input 2 j in bits 4 j
// and input 2 j + 1 in bits 16 + 4 j, which the masks above take apart in place.
// A wave reads a whole tile step as 1 KB in a row.
#pragma once

#include "common.h"

namespace moe {

constexpr int TILE_N = 16;
constexpr int Q4_K = 128;                         // inputs of a code tile
constexpr uint32_t BF16_ONES = 0x3f803f80u;       // two bf16 ones

// A weight matrix stack as a kernel takes it: row-major, blocked, or codes.
struct RowWeights {
  const void* w;       // elements, or codes
  const void* scales;  // ELT [groups][Np]
  const uint8_t* zeros;  // [groups][Np], null: 8
};

__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// A load at `bytes` of a lane from what its wave has in common (a scalar base and a 32-bit
// offset: one vector register where a pointer takes two for each load in flight).
template <typename V>
__device__ __forceinline__ V at(const void* base, uint32_t bytes, int ahead = 0) {
  return *reinterpret_cast<const V*>(static_cast<const char*>(base) + bytes + ahead);
}

// One 1 KB copy into LDS: eight rows of 128 bytes, lane l to 16 l.
template <int AUX>
__device__ __forceinline__ void copy_rows(const void* base, uint32_t lane_off, char* lds) {
  __builtin_amdgcn_global_load_lds((gbl_ptr_t)(static_cast<const char*>(base) + lane_off), (lds_ptr_t)lds, 16, 0, AUX);
}
// Row (0..7) and byte of a lane in copy q of a 16-row tile, its chunks swizzled as lds_off
// reads them.
__device__ __forceinline__ int copy_row(int q) { return 8 * q + ((int)(threadIdx.x & 63) >> 3); }
__device__ __forceinline__ uint32_t copy_byte(int q) { return 16 * ((threadIdx.x & 7) ^ lds_swz(copy_row(q))); }

// Tiles side by side share their scales' 128-byte lines, so the workgroups of one XCD (every
// eighth) take neighbours: the tile of workgroup b of n.
__device__ __forceinline__ int near_tile(int b, int n) { return n & 7 ? b : (b & 7) * (n >> 3) + (b >> 3); }

// Three bf16 parts of a float32 that add up to it (each cut off after 8 bits); a
// value that is not finite stays whole in the first.
__device__ __forceinline__ void split3(float f, uint32_t& a, uint32_t& b, uint32_t& c) {
  const uint32_t u = __float_as_uint(f);
  const bool fin = (u & 0x7f800000u) != 0x7f800000u;
  a = fin ? u & 0xffff0000u : (u | ((u & 0x007fffffu) ? 0x00400000u : 0u)) & 0xffff0000u;
  const float r = fin ? f - __uint_as_float(a) : 0.f;
  b = __float_as_uint(r) & 0xffff0000u;
  c = __float_as_uint(r - __uint_as_float(b)) & 0xffff0000u;
}

template <typename T>
struct DenseOp {
  typedef T elt;
  typedef T hid;                                  // element of the intermediate rows
  static constexpr int KS = 128 / sizeof(T);      // of K per step
  static constexpr int PLANES = 1;
  struct W { u32x4_t v[2]; };
  struct X { u32x4_t v[2]; };
  // w_offset of row n0's first element; a block's rows are KS elements long.
  __device__ __forceinline__ static size_t corner(int n0, int K, int blocked) {
    return blocked ? (size_t)(n0 & ~63) * K + (n0 & 63) * KS : (size_t)n0 * K;
  }
  __device__ __forceinline__ static void mma(f32x4_t& acc, const W& w, const X& x) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (sizeof(T) == 2) {
        acc = Mfma<bf16_t>::step(w.v[i], x.v[i], acc);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) acc = mfma_f32_4(__uint_as_float(w.v[i][j]), __uint_as_float(x.v[i][j]), acc);
      }
    }
  }
  // One element, and one of an intermediate row.
  __device__ __forceinline__ static float value(const RowWeights& m, int mat, int n, int k, int N, int K, int blocked) {
    return Elt<T>::to_f32(static_cast<const T*>(m.w)[(size_t)mat * N * K + w_offset<T>(n, k, K, blocked)]);
  }
  __device__ __forceinline__ static float h_value(const hid* row, size_t, int k) { return Elt<T>::to_f32(row[k]); }
  // An intermediate value (one rounding to the element type, as moe_ffn keeps H).
  __device__ __forceinline__ static void store_h(hid* p, size_t, float v) { *p = Elt<T>::from_f32(v); }
};

template <typename T, int GROUP, bool ZEROS>
struct Q4Op {
  typedef T elt;
  typedef bf16_t hid;                             // float32: three planes of it
  static constexpr int KS = Q4_K;
  static constexpr int PLANES = sizeof(T) == 2 ? 1 : 3;
  static constexpr bool ZP = ZEROS;
  static constexpr int NG = Q4_K / GROUP;         // groups of a step
  static constexpr int PER = 4 / NG;              // instructions of a group
  struct W {
    u32x4_t q;
    T s[NG];                                      // of row lane % 16
    uint8_t z[ZEROS ? NG : 1];
  };
  struct X { u32x4_t v[PLANES][4]; };
  struct Src { const u32x4_t* q; const T* s; const uint8_t* z; int Np; };

  __device__ __forceinline__ static Src tile(const RowWeights& m, int mat, int n0, int N, int K) {
    const int kt = ceil_div(K, Q4_K), nt = ceil_div(N, TILE_N), Np = nt * TILE_N;
    const size_t g = (size_t)mat * kt * NG * Np + n0;
    return Src{static_cast<const u32x4_t*>(m.w) + ((size_t)mat * nt + n0 / TILE_N) * kt * 64,
               static_cast<const T*>(m.scales) + g, ZEROS ? m.zeros + g : nullptr, Np};
  }
  // Codes are read once: past the caches.
  __device__ __forceinline__ static W load(const Src& s, int step) {
    W w;
    const uint32_t lane = threadIdx.x & 63, row = lane & 15;
    w.q = __builtin_nontemporal_load(s.q + (size_t)step * 64 + lane);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const size_t o = (size_t)(step * NG + g) * s.Np;
      w.s[g] = at<T>(s.s + o, row * (uint32_t)sizeof(T));
      if constexpr (ZEROS) w.z[g] = at<uint8_t>(s.z + o, row);
    }
    return w;
  }
  __device__ __forceinline__ static void set3(X& x, int i, const f32x4_t& a, const f32x4_t& b) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t l[3], h[3];
      split3(j < 2 ? a[2 * j] : b[2 * j - 4], l[0], l[1], l[2]);
      split3(j < 2 ? a[2 * j + 1] : b[2 * j - 3], h[0], h[1], h[2]);
#pragma unroll
      for (int p = 0; p < PLANES; ++p) x.v[p][i][j] = (l[p] >> 16) | h[p];
    }
  }
  // Activations of a step: the lane's row starts `row` bytes behind base.  Inputs from K on
  // read as zero (K a multiple of 8).
  __device__ __forceinline__ static X load_x(const T* base, uint32_t row, int step, int K) {
    X x;
    const uint32_t o = row + 8 * sizeof(T) * ((threadIdx.x & 63) >> 4);
    const int k0 = step * KS + 8 * ((threadIdx.x & 63) >> 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = k0 + 32 * i < K;
      const T* p = base + step * KS + 32 * i;
      const uint32_t off = in ? o : 0;
      if (!in) p = base;
      if constexpr (sizeof(T) == 2) {
        const u32x4_t v = at<u32x4_t>(p, off);
        x.v[0][i] = in ? v : u32x4_t{0, 0, 0, 0};
      } else {
        f32x4_t a = at<f32x4_t>(p, off), b = at<f32x4_t>(p, off, 16);
        if (!in) a = b = f32x4_t{0.f, 0.f, 0.f, 0.f};
        set3(x, i, a, b);
      }
    }
    return x;
  }
  // A word's eight codes as bf16 values 16 + q.  (`base` as a value the compiler does not know
  // makes mask and or one instruction: of two constants it can hold one.)
  __device__ __forceinline__ static u32x4_t widen(uint32_t q) {
    uint32_t base = 0x41804180u;
    asm("" : "+v"(base));
    return u32x4_t{((q << 3) & 0x00780078u) | base, ((q >> 1) & 0x00780078u) | base,
                   ((q >> 5) & 0x00780078u) | base, ((q >> 9) & 0x00780078u) | base};
  }
  // A step of NT tiles and R blocks of 16 activation rows, the first RT of a lane's four
  // results of each.  The tiles' products run side by side (one waits for the one before it
  // in its sum), and a group is scaled behind the next one's.
  template <int RT, int NT, int R>
  __device__ __forceinline__ static void step(f32x4_t (&acc)[NT][R], const W (&w)[NT], const X (&x)[R]) {
    const u32x4_t one = {BF16_ONES, BF16_ONES, BF16_ONES, BF16_ONES};
    f32x4_t a[2][NT][R], sum[2][R];
    auto scale = [&](int g) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float s = Elt<T>::to_f32(w[t].s[g]), z = ZEROS ? 16.f + (float)w[t].z[g] : 24.f;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int i = 0; i < RT; ++i)
            acc[t][r][i] = fmaf(s, fmaf(-z, sum[g & 1][r][i], a[g & 1][t][r][i]), acc[t][r][i]);
      }
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int g = i / PER, o = g & 1;
      if (i % PER == 0) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          sum[o][r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int t = 0; t < NT; ++t) a[o][t][r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
      }
      u32x4_t b[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) b[t] = widen(w[t].q[i]);
#pragma unroll
      for (int p = PLANES - 1; p >= 0; --p)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          sum[o][r] = Mfma<bf16_t>::step(x[r].v[p][i], one, sum[o][r]);
#pragma unroll
          for (int t = 0; t < NT; ++t) a[o][t][r] = Mfma<bf16_t>::step(x[r].v[p][i], b[t], a[o][t][r]);
        }
      if (i % PER == PER - 1 && g > 0) scale(g - 1);
    }
    scale(NG - 1);
  }
  __device__ __forceinline__ static float value(const RowWeights& m, int mat, int n, int k, int N, int K, int) {
    const int kt = ceil_div(K, Q4_K), nt = ceil_div(N, TILE_N), c = k % Q4_K;
    const uint32_t* w = static_cast<const uint32_t*>(m.w) + (((size_t)mat * nt + n / TILE_N) * kt + k / Q4_K) * 256;
    const uint32_t q = w[((c / 8 % 4) * 16 + n % TILE_N) * 4 + c / 32] >> (4 * (c % 8 / 2) + 16 * (c & 1));
    const size_t g = ((size_t)mat * kt * NG + k / GROUP) * (nt * TILE_N) + n;
    return Elt<T>::to_f32(static_cast<const T*>(m.scales)[g]) * (float)((int)(q & 15u) - (ZEROS ? (int)m.zeros[g] : 8));
  }
  __device__ __forceinline__ static float h_value(const hid* row, size_t plane, int k) {
    float v = 0.f;
#pragma unroll
    for (int p = PLANES - 1; p >= 0; --p) v += bf16_to_f32(row[p * plane + k]);
    return v;
  }
  __device__ __forceinline__ static void store_h(hid* p, size_t plane, float v) {
    if constexpr (PLANES == 1) {
      *p = Elt<T>::from_f32(v);
    } else {
      uint32_t a, b, c;
      split3(v, a, b, c);
      p[0] = (hid)(a >> 16);
      p[plane] = (hid)(b >> 16);
      p[2 * plane] = (hid)(c >> 16);
    }
  }
};

// Wait states between the last matrix instruction of a loop and the first use of its result
// behind the loop: a block that is entered from the loop's end and from elsewhere came out
// without them (a store to LDS right behind the branch took one of the four values before it
// was there).  19 are the most that the longest instruction asks for.
template <typename V>
__device__ __forceinline__ void settle(V& acc) { asm volatile("s_nop 15\n\ts_nop 3" : "+v"(acc)); }

// ---- sums that are not finite ----
// A matrix instruction multiplies every column with every row: an infinity or NaN among
// the weights turns the zeros of tokens that have no part in them into NaN, and the
// codes' difference turns an infinite activation into one.  An output that is not finite
// is therefore summed again from its own products alone, by a whole wave.
__device__ __forceinline__ bool not_finite(float v) { return !(fabsf(v) < INFINITY); }

// Sum over k < K of x(k) w(k), the same in every lane; nan: an x among them is no number.
template <class FX, class FW>
__device__ __forceinline__ float wave_dot(int K, FX x, FW w, bool& nan) {
  float s = 0.f;
  bool bad = false;
#pragma unroll 4
  for (int k = threadIdx.x & 63; k < K; k += 64) {
    const float v = x(k);
    bad |= v != v;
    s += v * w(k);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
  nan |= __ballot(bad) != 0;
  return s;
}

// Replaces a lane's value that is not finite (where `mine`) by f(lane, nan).  `row` is the
// lane's row of activations: where one of them is no number (nan), so are all of the row's
// outputs, and the wave is done with them (4 tokens, 256 experts, one of the tokens with a
// NaN: the layer took 4.1 ms when each output was summed again).
template <class F>
__device__ __forceinline__ void redo_not_finite(float& v, bool mine, int row, F f) {
  uint64_t todo = __ballot(mine && not_finite(v));
#pragma unroll 1
  while (todo) {
    const int l = __builtin_ctzll(todo);
    bool nan = false;
    const float s = f(l, nan);
    const bool same = nan ? row == __builtin_amdgcn_readlane(row, l) : (int)(threadIdx.x & 63) == l;
    if (same && (todo >> (threadIdx.x & 63) & 1)) v = nan ? __uint_as_float(0x7fc00000u) : s;
    todo &= ~__ballot(same);
  }
}

}  // namespace moe
