// Norms before and after a block, fused with the block's gate, its residual
// scale and (moe_combine_norm) with the weighted combine:
//   y  = the block's output, or sum_j w_j Y[inv_perm_j] (+ Y_shared) in float32
//   p  = post ? norm(y) : y
//   r  = resid + alpha * gate * p          -> resid_out
//   x  = norm(r)                           -> x_out
//   norm(v) = (v - mean) * rsqrt(mean((v - mean)^2) + eps) * (w_offset + w) + b
// with mean = 0 for the RMS norm.  One workgroup per row, the row in registers
// from the first load to the last store: y, resid and each operand vector are
// read once, r and x written once, nothing is rounded between (the second norm
// takes r before its rounding to the element type).  All statistics are
// float32; the layer norm centres before it squares, so its variance does not
// cancel.
//
// Bound by memory where there are rows enough: 8,192 x 2,048 bf16 with both norms,
// four rows of traffic a token, 29 us (4.6 TB/s; a copy of 2 GiB reaches 4.9), the
// combine of 4,096 x 7,168 with k in {4, 8} 114 us (5.1 TB/s).  Few rows are bound
// by latency: one row of 7,168 4.6 us, 128 rows behind their combine 10 us (offsets,
// rows, two reductions, one after the other).  CH chunks a thread: as few as make a
// row of up to 1,024 chunks at most 512 threads, a wider one at most 1,024 (one wave
// with four chunks of 2,048 columns took 94 us where one chunk a thread takes 29, its
// loads waiting for one another).  Eight and sixteen chunks (rows of more than 32,768
// bf16, 16,384 float32) do not fit the registers of 1,024 threads and spill: 512 rows
// of 65,536 bf16 213 us, a quarter of the copy's rate.
#include "common.h"
#include "launch.h"

#include <type_traits>

namespace moe {

namespace {

// LE elements of T starting at p, as floats (16 bytes).
template <typename T>
__device__ __forceinline__ void unpack16(const u32x4_t& v, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      f[2 * i] = __uint_as_float(v[i] << 16);
      f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    } else {
      f[i] = __uint_as_float(v[i]);
    }
  }
}
template <typename T>
__device__ __forceinline__ u32x4_t pack16(const float* f) {
  u32x4_t o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) o[i] = (uint32_t)f32_to_bf16(f[2 * i]) | ((uint32_t)f32_to_bf16(f[2 * i + 1]) << 16);
    else o[i] = __float_as_uint(f[i]);
  }
  return o;
}

// Sum of one float per thread over the workgroup: a butterfly in each wave,
// then the wave sums in ascending order (every thread adds them the same way).
__device__ __forceinline__ float block_sum(float v, float* red) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, nw = blockDim.x >> 6;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  if (nw == 1) return v;
  if (lane == 0) red[w] = v;
  __syncthreads();
  float s = red[0];
  for (int i = 1; i < nw; ++i) s += red[i];
  __syncthreads();
  return s;
}

}  // namespace

// A thread owns CH chunks of LE = 16 / sizeof(T) elements.  VEC: chunk q is the
// 16-byte chunk tid + blockDim * q of the row (d a multiple of LE, so that every
// row starts on 16 bytes); otherwise element i of chunk q is element tid +
// blockDim * (LE q + i), so that odd widths still read whole lines.
template <typename T, int CH, bool VEC>
struct RowIo {
  static constexpr int LE = 16 / (int)sizeof(T);
  // One operand's chunks as they were read; elements that are not there are 0.
  struct Part {
    u32x4_t v[CH];
    __device__ __forceinline__ float get(int q, int i) const {
      if constexpr (sizeof(T) == 2) return __uint_as_float(i & 1 ? v[q][i >> 1] & 0xffff0000u : v[q][i >> 1] << 16);
      else return __uint_as_float(v[q][i]);
    }
  };
  int d;
  __device__ __forceinline__ int at(int q, int i) const {
    return VEC ? (int)(threadIdx.x + blockDim.x * q) * LE + i : (int)(threadIdx.x + blockDim.x * (LE * q + i));
  }
  __device__ __forceinline__ bool has(int q, int i) const { return at(q, VEC ? 0 : i) < d; }
  template <bool NT = false>
  __device__ __forceinline__ void read(const void* base, size_t first, Part& f) const {
    const T* const p = (const T*)base + first;
#pragma unroll
    for (int q = 0; q < CH; ++q) {
      f.v[q] = u32x4_t{0u, 0u, 0u, 0u};
      if constexpr (VEC) {
        const u32x4_t* const c = reinterpret_cast<const u32x4_t*>(p + at(q, 0));
        if (has(q, 0)) f.v[q] = NT ? __builtin_nontemporal_load(c) : *c;
      } else {
#pragma unroll
        for (int i = 0; i < LE; ++i)
          if (has(q, i)) {
            if constexpr (sizeof(T) == 2) f.v[q][i >> 1] |= (uint32_t)p[at(q, i)] << (16 * (i & 1));
            else f.v[q][i] = __float_as_uint(p[at(q, i)]);
          }
      }
    }
  }
  // Non-temporal: the row's next reader is another kernel (8,192 x 2,048 bf16,
  // four rows of traffic a token: 33 -> 27 us for the norm alone).  With the kernel
  // that reads x behind it, us a pair, cached against non-temporal: the router at
  // 1 x 7168 22.2 / 22.3, 8,192 x 2,048 93.9 / 96.4, 4,096 x 7168 158.8 / 157.5; the
  // experts' gate/up at 1 x 7168 43.6 / 43.6, 8,192 x 2,048 500 / 499, 4,096 x 7168
  // 386 / 350.
  __device__ __forceinline__ void write(void* base, size_t first, const float (&f)[CH][LE]) const {
    T* const p = (T*)base + first;
#pragma unroll
    for (int q = 0; q < CH; ++q) {
      if constexpr (VEC) {
        if (has(q, 0)) __builtin_nontemporal_store(pack16<T>(f[q]), reinterpret_cast<u32x4_t*>(p + at(q, 0)));
      } else {
#pragma unroll
        for (int i = 0; i < LE; ++i)
          if (has(q, i)) p[at(q, i)] = Elt<T>::from_f32(f[q][i]);
      }
    }
  }
  // v = norm(v)
  __device__ __forceinline__ void norm(float (&v)[CH][LE], const NormRow& n, bool has_w, const Part& w, bool has_b,
                                       const Part& b, float* red) const {
    if (n.layer) {
      float s = 0.f;
#pragma unroll
      for (int q = 0; q < CH; ++q)
#pragma unroll
        for (int i = 0; i < LE; ++i) s += v[q][i];
      const float mean = block_sum(s, red) / (float)d;
#pragma unroll
      for (int q = 0; q < CH; ++q)
#pragma unroll
        for (int i = 0; i < LE; ++i) v[q][i] = has(q, i) ? v[q][i] - mean : 0.f;
    }
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < CH; ++q)
#pragma unroll
      for (int i = 0; i < LE; ++i) s = fmaf(v[q][i], v[q][i], s);
    const float rs = 1.0f / sqrtf(block_sum(s, red) / (float)d + n.eps);
#pragma unroll
    for (int q = 0; q < CH; ++q)
#pragma unroll
      for (int i = 0; i < LE; ++i) {
        float o = v[q][i] * rs;
        if (has_w) o *= n.w_offset + w.get(q, i);
        if (has_b) o += b.get(q, i);
        v[q][i] = o;
      }
  }
};

// The row's operands.  EARLY (short rows, where there are registers for it): all of
// them are requested at once, before anything is known of y, so that their
// latencies pass together; otherwise each before its use.
template <typename T, int CH, bool VEC, bool EARLY_>
struct RowParts {
  static constexpr bool EARLY = EARLY_;
  typename RowIo<T, CH, VEC>::Part resid, post_w, post_b, gate, pre_w, pre_b;
  template <bool NT>
  __device__ __forceinline__ void early(const RowIo<T, CH, VEC>& io, const NormRow& n, size_t row) {
    if (n.resid) io.template read<NT>(n.resid, row, resid);
    if constexpr (EARLY) {
      if (n.has_y && n.post && n.post_w) io.read(n.post_w, 0, post_w);
      if (n.has_y && n.post && n.post_b) io.read(n.post_b, 0, post_b);
      if (n.gate_mode >= MOE_GATE_CHANNEL && n.gate_mode != MOE_GATE_TOKEN)
        io.read(n.gate, n.gate_mode == MOE_GATE_FULL ? row : 0, gate);
      if (n.x_out && n.pre_w) io.read(n.pre_w, 0, pre_w);
      if (n.x_out && n.pre_b) io.read(n.pre_b, 0, pre_b);
    }
  }
};

// The chain behind y (v in: y, float32).  resid, y and the outputs may be the
// same buffers: a thread writes only elements that it alone has read before.
template <typename T, int CH, bool VEC, bool EARLY>
__device__ __forceinline__ void norm_chain(float (&v)[CH][16 / sizeof(T)], const RowIo<T, CH, VEC>& io,
                                           const NormRow& n, RowParts<T, CH, VEC, EARLY>& o, int t, float* red) {
  constexpr int LE = 16 / (int)sizeof(T);
  const size_t row = (size_t)t * io.d;
  if (n.has_y) {
    if (n.post) {
      if (!EARLY && n.post_w) io.read(n.post_w, 0, o.post_w);
      if (!EARLY && n.post_b) io.read(n.post_b, 0, o.post_b);
      io.norm(v, n, n.post_w != nullptr, o.post_w, n.post_b != nullptr, o.post_b, red);
    }
    if (n.gate_mode == MOE_GATE_TOKEN) {
      const float g = Elt<T>::to_f32(((const T*)n.gate)[t]);
#pragma unroll
      for (int q = 0; q < CH; ++q)
#pragma unroll
        for (int i = 0; i < LE; ++i) v[q][i] *= g;
    } else if (n.gate_mode != MOE_GATE_NONE) {
      if (!EARLY) io.read(n.gate, n.gate_mode == MOE_GATE_FULL ? row : 0, o.gate);
#pragma unroll
      for (int q = 0; q < CH; ++q)
#pragma unroll
        for (int i = 0; i < LE; ++i) v[q][i] *= o.gate.get(q, i);
    }
#pragma unroll
    for (int q = 0; q < CH; ++q)
#pragma unroll
      for (int i = 0; i < LE; ++i) v[q][i] = n.resid ? fmaf(n.alpha, v[q][i], o.resid.get(q, i)) : n.alpha * v[q][i];
  } else {
#pragma unroll
    for (int q = 0; q < CH; ++q)
#pragma unroll
      for (int i = 0; i < LE; ++i) v[q][i] = o.resid.get(q, i);
  }
  if (n.resid_out) io.write(n.resid_out, row, v);
  if (n.x_out) {
    // elements past the row do not count: they are 0 here
    if (!EARLY && n.pre_w) io.read(n.pre_w, 0, o.pre_w);
    if (!EARLY && n.pre_b) io.read(n.pre_b, 0, o.pre_b);
    io.norm(v, n, n.pre_w != nullptr, o.pre_w, n.pre_b != nullptr, o.pre_b, red);
    io.write(n.x_out, row, v);
  }
}

template <typename T, int CH, bool VEC>
__global__ __launch_bounds__(CH <= 2 ? 512 : 1024) void norm_kernel(const T* y, NormRow n) {
  constexpr int LE = 16 / (int)sizeof(T);
  __shared__ float red[16];
  const RowIo<T, CH, VEC> io{n.d};
  const int t = blockIdx.x;
  float v[CH][LE];
  typename RowIo<T, CH, VEC>::Part yp;
  RowParts<T, CH, VEC, (CH <= 2)> o;
  if (n.has_y) io.read(y, (size_t)t * n.d, yp);
  o.template early<false>(io, n, (size_t)t * n.d);
#pragma unroll
  for (int q = 0; q < CH; ++q)
#pragma unroll
    for (int i = 0; i < LE; ++i) v[q][i] = n.has_y ? yp.get(q, i) : 0.f;
  norm_chain(v, io, n, o, t, red);
}

// The combine of combine.hip (same order of the same fused multiply-adds),
// kept in float32 and followed by the chain above.  The rows of CBN
// assignments are requested together.
template <typename T, int CH, int CBN>
__global__ __launch_bounds__(CH <= 2 ? 512 : 1024) void combine_norm_kernel(const T* __restrict__ yp, const T* __restrict__ ysh,
                                                            const int32_t* __restrict__ tok_off,
                                                            const float* __restrict__ wts,
                                                            const int32_t* __restrict__ inv_perm, int cap, NormRow n) {
  constexpr int LE = 16 / (int)sizeof(T);
  __shared__ float red[16];
  const RowIo<T, CH, true> io{n.d};
  const int t = blockIdx.x;
  const int a0 = max(tok_off[t], 0), a1 = min(tok_off[t + 1], cap);
  // resid is read past the caches like the rows of Y; with y_shared read so as well
  // the call is slower (4,096 x 7,168, k in {4, 8}: 114 against 119 us)
  RowParts<T, CH, true, CH == 1> o;
  o.template early<true>(io, n, (size_t)t * n.d);
  float v[CH][LE];
#pragma unroll
  for (int q = 0; q < CH; ++q)
#pragma unroll
    for (int i = 0; i < LE; ++i) v[q][i] = 0.f;
  for (int b = a0; b < a1; b += CBN) {
    u32x4_t r[CBN][CH];
    float w[CBN];
    int p[CBN];
#pragma unroll
    for (int j = 0; j < CBN; ++j) {
      p[j] = inv_perm[min(b + j, a1 - 1)];
      w[j] = wts[min(b + j, a1 - 1)];
      if (b + j >= a1 || p[j] >= cap) p[j] = -1;
    }
#pragma unroll
    for (int j = 0; j < CBN; ++j)
#pragma unroll
      for (int q = 0; q < CH; ++q) {
        r[j][q] = u32x4_t{0u, 0u, 0u, 0u};
        if (p[j] >= 0 && io.has(q, 0))
          r[j][q] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(yp + (size_t)p[j] * n.d + io.at(q, 0)));
      }
#pragma unroll
    for (int j = 0; j < CBN; ++j) {
      if (p[j] < 0) continue;
#pragma unroll
      for (int q = 0; q < CH; ++q) {
        float f[LE];
        unpack16<T>(r[j][q], f);
#pragma unroll
        for (int i = 0; i < LE; ++i) v[q][i] = fmaf(w[j], f[i], v[q][i]);
      }
    }
  }
  if (ysh) {
    typename RowIo<T, CH, true>::Part sh;
    io.read(ysh, (size_t)t * n.d, sh);
#pragma unroll
    for (int q = 0; q < CH; ++q)
#pragma unroll
      for (int i = 0; i < LE; ++i) v[q][i] += sh.get(q, i);
  }
  norm_chain(v, io, n, o, t, red);
}

// A launch holds less than 2^32 threads (and the runtime does not refuse more): at
// most ROWS rows of up to 1,024 threads each.  Larger batches take several launches,
// the operands moved on (with the row in a second grid dimension instead, the widest
// rows spill more and take a fifth longer).
constexpr int ROWS = 1 << 21;
template <typename T>
static T* past(T* p, size_t elements, size_t size) {
  using C = std::conditional_t<std::is_const_v<T>, const char, char>;
  return p ? (T*)((C*)p + elements * size) : nullptr;
}
static NormRow past_rows(NormRow n, int t0, size_t size) {
  const size_t e = (size_t)t0 * n.d;
  n.resid = past(n.resid, e, size);
  n.resid_out = past(n.resid_out, e, size);
  n.x_out = past(n.x_out, e, size);
  if (n.gate_mode == MOE_GATE_TOKEN) n.gate = past(n.gate, t0, size);
  if (n.gate_mode == MOE_GATE_FULL) n.gate = past(n.gate, e, size);
  return n;
}

// Threads of a row: enough for CH chunks each, in whole waves.
static int row_threads(int nch, int ch) { return ((nch + ch - 1) / ch + 63) / 64 * 64; }

template <typename T>
static void launch_norm_t(const T* y, const NormRow& n, int T_, hipStream_t st) {
  constexpr int LE = 16 / (int)sizeof(T);
  const int nch = (n.d + LE - 1) / LE;
  const bool vec = n.d % LE == 0;
#define MOE_NORM(CH)                                                                                              \
  do {                                                                                                            \
    if (vec) hipLaunchKernelGGL((norm_kernel<T, CH, true>), dim3(T_), dim3(row_threads(nch, CH)), 0, st, y, n);   \
    else hipLaunchKernelGGL((norm_kernel<T, CH, false>), dim3(T_), dim3(row_threads(nch, CH)), 0, st, y, n);      \
  } while (0)
  if (nch <= 512) MOE_NORM(1);
  else if (nch <= 1024) MOE_NORM(2);
  else if (nch <= 4096) MOE_NORM(4);
  else if (nch <= 8192) MOE_NORM(8);
  else MOE_NORM(16);
#undef MOE_NORM
}

hipError_t launch_norm(int dtype, const void* y, const NormRow& n, int T, hipStream_t st) {
  const size_t size = dtype == DT_BF16 ? 2 : 4;
  for (int t0 = 0; t0 < T; t0 += min(ROWS, T - t0)) {
    const NormRow r = past_rows(n, t0, size);
    const void* const yr = past(y, (size_t)t0 * n.d, size);
    if (dtype == DT_BF16) launch_norm_t<bf16_t>((const bf16_t*)yr, r, min(ROWS, T - t0), st);
    else launch_norm_t<float>((const float*)yr, r, min(ROWS, T - t0), st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T>
static void launch_combine_norm_t(const T* yp, const T* ysh, const int32_t* tok_off, const float* wts,
                                  const int32_t* inv_perm, int cap, const NormRow& n, int T_, hipStream_t st) {
  constexpr int LE = 16 / (int)sizeof(T);
  const int nch = n.d / LE;
#define MOE_CNORM(CH, CBN)                                                                                          \
  hipLaunchKernelGGL((combine_norm_kernel<T, CH, CBN>), dim3(T_), dim3(row_threads(nch, CH)), 0, st, yp, ysh, tok_off, \
                     wts, inv_perm, cap, n)
  if (nch <= 512) MOE_CNORM(1, 8);
  else if (nch <= 1024) MOE_CNORM(2, 8);
  else if (nch <= 4096) MOE_CNORM(4, 4);
  else if (nch <= 8192) MOE_CNORM(8, 2);
  else MOE_CNORM(16, 1);
#undef MOE_CNORM
}

hipError_t launch_combine_norm(int dtype, const void* yp, const void* ysh, const int32_t* tok_off, const float* wts,
                               const int32_t* inv_perm, int cap, const NormRow& n, int T, hipStream_t st) {
  const size_t size = dtype == DT_BF16 ? 2 : 4;
  for (int t0 = 0; t0 < T; t0 += min(ROWS, T - t0)) {
    const NormRow r = past_rows(n, t0, size);
    const void* const yr = past(ysh, (size_t)t0 * n.d, size);
    const int rows = min(ROWS, T - t0);
    if (dtype == DT_BF16)
      launch_combine_norm_t<bf16_t>((const bf16_t*)yp, (const bf16_t*)yr, tok_off + t0, wts, inv_perm, cap, r, rows, st);
    else
      launch_combine_norm_t<float>((const float*)yp, (const float*)yr, tok_off + t0, wts, inv_perm, cap, r, rows, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
