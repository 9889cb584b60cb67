// RMS norm with the residual's addition and an 8-bit output with one scale
// per row (E4M3 or INT8), for the layers of a block that run on 8-bit
// operands.
//
//   h = round(x + residual)                  (the residual stream, 16 bits or fp32)
//   t = h w                                  (fp32; exact for 16-bit h and w)
//   rstd = 1 / sqrt(mean(h^2) + eps)         (1 without the norm)
//   s = max|t| rstd / top,   q = rn(t top / max|t|),   top = 448 or 127
//
// The normalised row is t rstd, so dividing it by its scale cancels rstd: the
// codes need the row's maximum only and do not depend on the order in which
// the squares are summed.  Both statistics come from one pass over the row,
// which stays in registers between the pass and the conversion.
//
// Bound by memory: x and the residual are read once, h, the codes and the
// scales written once.  The two statistics of a row cross the warps of its
// CTA through shared memory behind a single barrier.  Three kernels:
//   rms8_kernel       one CTA per row: the row goes straight into registers
//   rms8_flat_kernel  the same for packed rows whose length is no multiple of
//                     16 bytes: x, residual, h and codes are cut at the 16-byte
//                     boundaries of the whole matrix and not of the row, which
//                     all of them share; a row's first and last piece are
//                     partial, and the weight is shifted into place
//   rms8_ring_kernel  many 16-byte aligned rows: persistent CTAs whose next
//                     rows are always on their way into a ring in shared
//                     memory (bulk copies), so that loads do not pause while
//                     a row is reduced and converted
//
// Measured (B200): bf16 4608 x 3072 with residual and weight 19.9 us (99 MB,
// 5.0 TB/s; with a weight row for every row 25.7), 16896 x 12288 without either
// 101 us (623 MB, 6.2 TB/s), fp32 4608 x 3072 33.6 us (184 MB, 5.5 TB/s), one
// row of 4096 2.2 us, packed rows of 5000 x 6001 with residual and weight 61 us
// (210 MB, 3.4 TB/s).
#pragma once

#include <cuda_fp8.h>

#include <type_traits>

#include "kg_common.cuh"

namespace svdq {

enum : int { DT_BF16 = 0, DT_FP16 = 1, DT_FP32 = 2, DT_E4M3 = 3, DT_INT8 = 4 };

template <int DT> struct ElemOf { using type = uint16_t; };
template <> struct ElemOf<DT_FP32> { using type = float; };

template <int DT>
__device__ __forceinline__ float to_f32(typename ElemOf<DT>::type v) {
  if constexpr (DT == DT_BF16) return __uint_as_float(static_cast<uint32_t>(v) << 16);
  else if constexpr (DT == DT_FP16) return __half2float(__ushort_as_half(v));
  else return v;
}
template <int DT>
__device__ __forceinline__ typename ElemOf<DT>::type from_f32(float v) {
  if constexpr (DT == DT_BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  else if constexpr (DT == DT_FP16) return __half_as_ushort(__float2half_rn(v));
  else return v;
}

// VEC consecutive elements in one access of 16, 8, 4 bytes or one element.
template <int DT, int VEC>
struct Pack {
  using E = typename ElemOf<DT>::type;
  static constexpr int BYTES = VEC * sizeof(E);
  using V = std::conditional_t<BYTES == 16, uint4, std::conditional_t<BYTES == 8, uint2, std::conditional_t<BYTES == 4 && VEC == 2, uint32_t, E>>>;
  union {
    V q;
    E e[VEC];
  };
  __device__ __forceinline__ void load(const E* p) { q = __ldcs(reinterpret_cast<const V*>(p)); }
  __device__ __forceinline__ void load_cached(const E* p) { q = __ldg(reinterpret_cast<const V*>(p)); }
  __device__ __forceinline__ void store(E* p) const { *reinterpret_cast<V*>(p) = q; }
};

// Elements 2i and 2i + 1 as a pair of fp32, and back.
template <int DT, int VEC>
__device__ __forceinline__ uint64_t get2(const Pack<DT, VEC>& a, int i) {
  if constexpr (DT == DT_FP32) {
    return f2_pack(a.e[2 * i], a.e[2 * i + 1]);
  } else {
    const uint32_t u = reinterpret_cast<const uint32_t*>(a.e)[i];
    if constexpr (DT == DT_BF16) return f2_pack(bf16lo(u), bf16hi(u));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
    return f2_pack(f.x, f.y);
  }
}
template <int DT, int VEC>
__device__ __forceinline__ void set2(Pack<DT, VEC>& a, int i, uint64_t v) {
  if constexpr (DT == DT_FP32) {
    a.e[2 * i] = f2_lo(v);
    a.e[2 * i + 1] = f2_hi(v);
  } else if constexpr (DT == DT_BF16) {
    reinterpret_cast<uint32_t*>(a.e)[i] = pack_bf16x2(f2_lo(v), f2_hi(v));
  } else {
    const __half2 h = __floats2half2_rn(f2_lo(v), f2_hi(v));
    reinterpret_cast<uint32_t*>(a.e)[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
}
// a <- round(a + b)
template <int DT, int VEC>
__device__ __forceinline__ void add_to(Pack<DT, VEC>& a, const Pack<DT, VEC>& b) {
  if constexpr (VEC == 1) {
    a.e[0] = from_f32<DT>(to_f32<DT>(a.e[0]) + to_f32<DT>(b.e[0]));
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) set2(a, i, f2_add(get2(a, i), get2(b, i)));
  }
}
// The larger of m, |a| and |b|; NaN if any is.
__device__ __forceinline__ float max_abs(float m, float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

struct RmsParams {
  const void* x;
  const void* res;      // or null
  void* h;              // or null
  const void* w;        // or null
  uint8_t* codes;
  float* scales;
  int64_t ldx, ldr, ldh, ldw, ldc;  // elements
  int64_t w_rows;       // rows of x that share a row of w (0: all)
  float inv_K;
  int K;
  int norm, int8;
  float eps;
};

// Below this the reciprocal top / max|t| would overflow fp32: the row becomes
// zero codes with a zero scale.
constexpr float kRmsTiny = 3.0092655e-36f;  // 2^-118
// The squares of a row with values above about 2^60 may overflow fp32: such
// rows (only those) are summed again scaled by 2^-80.
constexpr float kRmsDown = 8.2718061e-25f;  // 2^-80

// Block-wide sum, in a fixed order; every thread gets it.
__device__ __forceinline__ float block_sum(float v, float* red, int nw) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (nw > 1) {
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < nw ? red[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return v;
}

// The row's statistics, joined over the CTA in a fixed order; the barrier
// also ends the warps' reads of the row.  Neither is negative, so their bits
// are ordered like their values, NaN above infinity.  Every thread gets the
// maximum and whether the sum may be too large for fp32; the sum itself is
// only joined where it is used, in the first warp.
struct RmsStats {
  uint64_t ss = 0;   // two partial sums of squares
  float top = 0.f;   // max |t|
};
struct RmsJoined {
  uint32_t top;
  float ss;          // first warp
  bool large;        // a warp's sum is 2^123 or more: with 32 of them the total may overflow
};
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ RmsJoined rms8_join(const RmsParams& p, const RmsStats& st, float* red_s, uint32_t* red_m, int nw) {
  constexpr uint32_t kLarge = (123u + 127u) << 23;
  RmsJoined j;
  j.top = __reduce_max_sync(0xffffffffu, __float_as_uint(st.top));
  j.ss = p.norm ? warp_sum(f2_lo(st.ss) + f2_hi(st.ss)) : 0.f;
  j.large = __float_as_uint(j.ss) >= kLarge;
  if (nw > 1) {
    const int l = threadIdx.x & 31;
    if (l == 0) {
      red_s[threadIdx.x >> 5] = j.ss;
      red_m[threadIdx.x >> 5] = j.top;
    }
    __syncthreads();
    j.top = __reduce_max_sync(0xffffffffu, l < nw ? red_m[l] : 0u);
    if (p.norm) {
      const float v = l < nw ? red_s[l] : 0.f;
      j.large = __reduce_max_sync(0xffffffffu, __float_as_uint(v)) >= kLarge;
      if (threadIdx.x < 32) j.ss = warp_sum(v);
    }
  } else {
    __syncwarp();
  }
  return j;
}

// t of elements 2i, 2i + 1 (VEC = 1: of the element, with 0).
template <int DT, int VEC, bool HW>
__device__ __forceinline__ uint64_t rms8_t(const Pack<DT, VEC>& a, const Pack<DT, VEC>& g, int i) {
  if constexpr (VEC == 1) {
    const float v = to_f32<DT>(a.e[0]);
    return f2_pack(HW ? v * to_f32<DT>(g.e[0]) : v, 0.f);
  } else {
    const uint64_t v = get2(a, i);
    return HW ? f2_mul(v, get2(g, i)) : v;
  }
}
template <int DT, int VEC, bool HW>
__device__ __forceinline__ void rms8_stats(const RmsParams& p, const Pack<DT, VEC>& a, const Pack<DT, VEC>& g, RmsStats& st) {
  if (p.norm) {
    if constexpr (VEC == 1) {
      const uint64_t v = f2_pack(to_f32<DT>(a.e[0]), 0.f);
      st.ss = f2_fma(v, v, st.ss);
    } else {
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) {
        const uint64_t v = get2(a, i);
        st.ss = f2_fma(v, v, st.ss);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < (VEC + 1) / 2; ++i) {
    const uint64_t t = rms8_t<DT, VEC, HW>(a, g, i);
    st.top = max_abs(st.top, f2_lo(t), f2_hi(t));
  }
}

template <int DT, int VEC>
__device__ __forceinline__ float rms8_squares_down(const Pack<DT, VEC>& a, float s) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const float v = to_f32<DT>(a.e[i]) * kRmsDown;
    s = fmaf(v, v, s);
  }
  return s;
}

// The factor from t to the codes; thread 0 writes the row's scale.  `again`:
// the row's squares summed scaled by kRmsDown (called by the whole CTA or not
// at all).
template <class F>
__device__ __forceinline__ float rms8_scale(const RmsParams& p, int64_t row, const RmsJoined& j, F again) {
  const float amax = __uint_as_float(j.top);
  const bool finite = j.top < 0x7F800000u;
  const bool live = finite && amax >= kRmsTiny;
  const float lim = p.int8 ? 127.f : 448.f;
  float s2 = 0.f;
  const bool down = finite && j.large;
  if (down) s2 = again();
  if (threadIdx.x == 0) {
    float rstd = 1.f;
    if (p.norm) rstd = down ? kRmsDown / sqrtf(s2 * p.inv_K) : 1.f / sqrtf(fmaf(j.ss, p.inv_K, p.eps));
    p.scales[row] = live ? __fdiv_rn(amax * rstd, lim) : finite ? 0.f : __uint_as_float(0x7FC00000u);
  }
  return live ? __fdiv_rn(lim, amax) : 0.f;
}

template <int DT, int VEC, bool HW, bool I8>
__device__ __forceinline__ void rms8_codes(const Pack<DT, VEC>& a, const Pack<DT, VEC>& g, float inv,
                                           uint8_t* out) {
  const uint64_t inv2 = f2_pack(inv, inv);
  uint32_t q[(VEC + 3) / 4] = {};
#pragma unroll
  for (int i = 0; i < (VEC + 1) / 2; ++i) {
    const uint64_t z = f2_mul(rms8_t<DT, VEC, HW>(a, g, i), inv2);
    uint32_t two;
    if constexpr (I8)  // at most 127 (1 + 2^-23): rounds to at most 127
      two = (static_cast<uint32_t>(__float2int_rn(f2_lo(z))) & 0xFFu) | (static_cast<uint32_t>(__float2int_rn(f2_hi(z))) & 0xFFu) << 8;
    else
      two = __nv_cvt_float2_to_fp8x2(make_float2(f2_lo(z), f2_hi(z)), __NV_SATFINITE, __NV_E4M3);
    q[i / 2] |= two << (16 * (i % 2));
  }
  if constexpr (VEC == 8) *reinterpret_cast<uint2*>(out) = make_uint2(q[0], q[1]);
  else if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(out) = q[0];
  else out[0] = static_cast<uint8_t>(q[0]);
}

// CH chunks of VEC elements per thread; HW: with a weight; I8: INT8 codes.
template <int DT, int VEC, int CH, bool HW, bool I8>
__global__ void __launch_bounds__(1024, 1) rms8_kernel(const RmsParams p) {
  using E = typename ElemOf<DT>::type;
  __shared__ float red_s[32];
  __shared__ uint32_t red_m[32];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = blockIdx.x;
  const int nt = blockDim.x;
  const int nw = nt >> 5;
  const E* x = static_cast<const E*>(p.x) + row * p.ldx;
  const E* r = static_cast<const E*>(p.res) + row * p.ldr;
  E* h = static_cast<E*>(p.h) + row * p.ldh;
  const E* w = static_cast<const E*>(p.w) + (HW && p.w_rows ? row / p.w_rows * p.ldw : 0);
  uint8_t* codes = p.codes + row * p.ldc;

  // The row stays packed in registers; t is formed twice (for the maximum and
  // for the codes) rather than kept, which leaves room for twice the threads.
  Pack<DT, VEC> a[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = (c * nt + static_cast<int>(threadIdx.x)) * VEC;
    if (k < p.K) a[c].load(x + k);
  }
  if (p.res) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int k = (c * nt + static_cast<int>(threadIdx.x)) * VEC;
      if (k < p.K) {
        Pack<DT, VEC> b;
        b.load(r + k);
        add_to(a[c], b);
        if (p.h) a[c].store(h + k);
      }
    }
  } else if (p.h) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int k = (c * nt + static_cast<int>(threadIdx.x)) * VEC;
      if (k < p.K) a[c].store(h + k);
    }
  }
  RmsStats st;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = (c * nt + static_cast<int>(threadIdx.x)) * VEC;
    if (k < p.K) {
      Pack<DT, VEC> g;
      if (HW) g.load_cached(w + k);
      rms8_stats<DT, VEC, HW>(p, a[c], g, st);
    }
  }
  const RmsJoined j = rms8_join(p, st, red_s, red_m, nw);
  const float inv = rms8_scale(p, row, j, [&] {
    float s2 = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int k = (c * nt + static_cast<int>(threadIdx.x)) * VEC;
      if (k < p.K) s2 = rms8_squares_down<DT, VEC>(a[c], s2);
    }
    return block_sum(s2, red_s, nw);
  });
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = (c * nt + static_cast<int>(threadIdx.x)) * VEC;
    if (k >= p.K) continue;
    Pack<DT, VEC> g;
    if (HW) g.load_cached(w + k);
    rms8_codes<DT, VEC, HW, I8>(a[c], g, inv, codes + k);
  }
}

// ------------------------------------------- packed rows of any length
// VEC elements from index `at` of a row of K (others give 0).
template <int DT, int VEC>
__device__ __forceinline__ void load_within(Pack<DT, VEC>& v, const typename ElemOf<DT>::type* row, int at, int K) {
  if (at >= 0 && at + VEC <= K) {
    v.load_cached(row + at);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v.e[i] = at + i >= 0 && at + i < K ? __ldg(row + at + i) : typename ElemOf<DT>::type(0);
  }
}

// Weights k .. k + VEC - 1 of an aligned row, where k + phase is a multiple of
// VEC: two aligned pieces, shifted by the same amount in the whole CTA.
template <int DT, int VEC>
__device__ __forceinline__ void load_shifted(Pack<DT, VEC>& g, const typename ElemOf<DT>::type* w, int k, int phase, int K) {
  Pack<DT, VEC> lo, hi;
  load_within<DT, VEC>(lo, w, k + phase - VEC, K);
  load_within<DT, VEC>(hi, w, k + phase, K);
  uint32_t t[8] = {lo.q.x, lo.q.y, lo.q.z, lo.q.w, hi.q.x, hi.q.y, hi.q.z, hi.q.w};
  const int s = VEC - phase;                       // 1 .. VEC elements
  const int words = DT == DT_FP32 ? s : s / 2;     // 0 .. 4
  if (words & 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = t[i + 4];
  }
  if (words & 2) {
#pragma unroll
    for (int i = 0; i < 6; ++i) t[i] = t[i + 2];
  }
  if (words & 1) {
#pragma unroll
    for (int i = 0; i < 7; ++i) t[i] = t[i + 1];
  }
  if (DT != DT_FP32 && (s & 1)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = __byte_perm(t[i], t[i + 1], 0x5432);
  }
  g.q = make_uint4(t[0], t[1], t[2], t[3]);
}

// A piece at element k of a row; its elements outside the row are 0.
template <int DT, int VEC>
__device__ __forceinline__ void load_piece(Pack<DT, VEC>& v, const typename ElemOf<DT>::type* row, int k, int K) {
  using E = typename ElemOf<DT>::type;
  if (k >= 0 && k + VEC <= K) {
    v.load(row + k);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v.e[i] = k + i >= 0 && k + i < K ? row[k + i] : E(0);
  }
}

template <int DT, int CH, bool HW, bool I8>
__global__ void __launch_bounds__(512, 1) rms8_flat_kernel(const RmsParams p) {
  using E = typename ElemOf<DT>::type;
  constexpr int VEC = 16 / sizeof(E);
  __shared__ float red_s[32];
  __shared__ uint32_t red_m[32];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = blockIdx.x;
  const int nt = blockDim.x;
  const int nw = nt >> 5;
  const E* x = static_cast<const E*>(p.x) + row * p.ldx;
  const E* r = static_cast<const E*>(p.res) + row * p.ldr;
  E* h = static_cast<E*>(p.h) + row * p.ldh;
  const E* w = static_cast<const E*>(p.w) + (HW && p.w_rows ? row / p.w_rows * p.ldw : 0);
  uint8_t* codes = p.codes + row * p.ldc;
  const int phase = static_cast<int>(row * p.ldx & (VEC - 1));  // the row starts this far into a piece
  auto first = [&](int c) { return (c * nt + static_cast<int>(threadIdx.x)) * VEC - phase; };  // element of piece c

  Pack<DT, VEC> a[CH], g[HW ? CH : 1];  // shifting the weight costs more than keeping it
#pragma unroll
  for (int c = 0; c < CH; ++c)
    if (first(c) < p.K) load_piece(a[c], x, first(c), p.K);
  if (p.res) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (first(c) < p.K) {
        Pack<DT, VEC> b;
        load_piece(b, r, first(c), p.K);
        add_to(a[c], b);
      }
    }
  }
  RmsStats st;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = first(c);
    if (k < p.K) {
      if (p.h) {
        if (k >= 0 && k + VEC <= p.K) {
          a[c].store(h + k);
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i)
            if (k + i >= 0 && k + i < p.K) h[k + i] = a[c].e[i];
        }
      }
      if (HW) load_shifted<DT, VEC>(g[HW ? c : 0], w, k, phase, p.K);
      rms8_stats<DT, VEC, HW>(p, a[c], g[HW ? c : 0], st);
    }
  }
  const RmsJoined j = rms8_join(p, st, red_s, red_m, nw);
  const float inv = rms8_scale(p, row, j, [&] {
    float s2 = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (first(c) < p.K) s2 = rms8_squares_down<DT, VEC>(a[c], s2);
    return block_sum(s2, red_s, nw);
  });
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = first(c);
    if (k >= p.K) continue;
    if (k >= 0 && k + VEC <= p.K) {
      rms8_codes<DT, VEC, HW, I8>(a[c], g[HW ? c : 0], inv, codes + k);
    } else {
      __align__(8) uint8_t q[VEC];
      rms8_codes<DT, VEC, HW, I8>(a[c], g[HW ? c : 0], inv, q);
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (k + i >= 0 && k + i < p.K) codes[k + i] = q[i];
    }
  }
}

// ------------------------------------------------------------- the ring form
// Wait site of the first bounded wait that expired in a call without an error
// word of its own; svdq_ops_device_error_site reads and clears it.
__device__ int g_ops_err;

struct RmsRing {
  int64_t M;
  int slots;       // rows of the ring
  int row_bytes;   // K elements
  uint64_t timeout_ns;
  int skip_row;    // test hook: the row whose copies are left out (-1: none)
};

// In place of a warp's maximum of |t|: the warp has given the row up.  Above
// every maximum, NaN included.
constexpr uint32_t kRmsGivenUp = 0xFFFFFFFFu;

// Shared memory: slots x (x row, residual row), then the barriers.
template <int DT, int CH, bool HW, bool I8>
__global__ void __launch_bounds__(512, 2) rms8_ring_kernel(const RmsParams p, const RmsRing g) {
  using E = typename ElemOf<DT>::type;
  constexpr int VEC = 16 / sizeof(E);
  constexpr int SLOTS = 8;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t bars[SLOTS];
  __shared__ float red_s[2][32];
  __shared__ uint32_t red_m[2][32];
  __shared__ int abort_flag;
  const int nt = blockDim.x, nw = nt >> 5;
  const uint32_t bar0 = smem_u32(bars);
  const Guard guard{&g_ops_err, &abort_flag, g.timeout_ns};
  const uint32_t slot_bytes = g.row_bytes * (p.res ? 2u : 1u);
  if (threadIdx.x == 0) {
    for (int i = 0; i < g.slots; ++i) mbar_init(bar0 + 8 * i, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  auto issue = [&](int64_t row, int slot) {  // thread 0
    const uint32_t dst = smem_u32(ring) + slot * slot_bytes;
    mbar_expect_tx(bar0 + 8 * slot, slot_bytes);
    if (row == g.skip_row) return;
    bulk_load(dst, static_cast<const E*>(p.x) + row * p.ldx, g.row_bytes, bar0 + 8 * slot);
    if (p.res) bulk_load(dst + g.row_bytes, static_cast<const E*>(p.res) + row * p.ldr, g.row_bytes, bar0 + 8 * slot);
  };
  if (threadIdx.x == 0)
    for (int i = 0; i < g.slots; ++i) {
      const int64_t row = blockIdx.x + static_cast<int64_t>(i) * gridDim.x;
      if (row < g.M) issue(row, i);
    }
  Pack<DT, VEC> w[CH];   // the weight row in use
  int64_t w_end = 0;     // the first row that it does not serve
  int slot = 0;
  uint32_t ph = 0;
  int it = 0;
  int64_t row = blockIdx.x;
  for (; row < g.M; row += gridDim.x, it ^= 1) {
    if (HW && row >= w_end) {
      const int64_t w_row = p.w_rows ? row / p.w_rows : 0;
      w_end = p.w_rows ? (w_row + 1) * p.w_rows : g.M;
      const E* src = static_cast<const E*>(p.w) + w_row * p.ldw;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int k = (c * nt + static_cast<int>(threadIdx.x)) * VEC;
        if (k < p.K) w[c].load_cached(src + k);
      }
    }
    // a warp with an expired wait says so at the join's barrier: the CTA goes on or gives up as one
    if (!__all_sync(0xffffffffu, wait_bounded(bar0 + 8 * slot, ph, guard, 0x321))) {
      if (nw > 1) {
        if ((threadIdx.x & 31) == 0) red_m[it][threadIdx.x >> 5] = kRmsGivenUp;
        __syncthreads();
      }
      break;
    }
    const uint8_t* sx = ring + slot * slot_bytes;
    Pack<DT, VEC> a[CH];
    RmsStats st;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int k = (c * nt + static_cast<int>(threadIdx.x)) * VEC;
      if (k < p.K) {
        a[c].q = *reinterpret_cast<const uint4*>(sx + k * sizeof(E));
        if (p.res) {
          Pack<DT, VEC> b;
          b.q = *reinterpret_cast<const uint4*>(sx + g.row_bytes + k * sizeof(E));
          add_to(a[c], b);
        }
        if (p.h) a[c].store(static_cast<E*>(p.h) + row * p.ldh + k);
        rms8_stats<DT, VEC, HW>(p, a[c], w[c], st);
      }
    }
    const RmsJoined j = rms8_join(p, st, red_s[it], red_m[it], nw);
    if (j.top == kRmsGivenUp) break;
    // every thread has read the slot (the join's barrier): the next row in
    if (threadIdx.x == 0) {
      const int64_t next = row + static_cast<int64_t>(g.slots) * gridDim.x;
      if (next < g.M) issue(next, slot);
    }
    const float inv = rms8_scale(p, row, j, [&] {
      float s2 = 0.f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int k = (c * nt + static_cast<int>(threadIdx.x)) * VEC;
        if (k < p.K) s2 = rms8_squares_down<DT, VEC>(a[c], s2);
      }
      return block_sum(s2, red_s[it], nw);
    });
  #pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int k = (c * nt + static_cast<int>(threadIdx.x)) * VEC;
      if (k < p.K) rms8_codes<DT, VEC, HW, I8>(a[c], w[c], inv, p.codes + row * p.ldc + k);
    }
    if (++slot == g.slots) { slot = 0; ph ^= 1; }
  }
  if (row < g.M && threadIdx.x == 0) {  // given up: the rows left say so, copies on their way land before the CTA leaves
    for (int64_t left = row; left < g.M; left += gridDim.x) p.scales[left] = __uint_as_float(0x7FC00000u);
    drain_loads(bar0, (1u << g.slots) - 1, ph ? (1u << g.slots) - (1u << slot) : (1u << slot) - 1, g.slots, g.timeout_ns);
  }
}

}  // namespace svdq
