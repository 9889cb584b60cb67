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
// scales written once.  A CTA owns one row; its two statistics cross the
// warps through shared memory behind a single barrier, and the CTAs that
// share an SM hide each other's barriers and loads.
#pragma once

#include <cuda_fp8.h>

#include "ptx.cuh"

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

// VEC consecutive elements: 16 bytes at once, or one element.
template <int DT, int VEC>
struct Pack {
  using E = typename ElemOf<DT>::type;
  union {
    uint4 q;
    E e[VEC];
  };
  __device__ __forceinline__ void load(const E* p) {
    if constexpr (VEC * sizeof(E) == 16) q = __ldcs(reinterpret_cast<const uint4*>(p));
    else e[0] = __ldcs(p);
  }
  __device__ __forceinline__ void load_cached(const E* p) {
    if constexpr (VEC * sizeof(E) == 16) q = __ldg(reinterpret_cast<const uint4*>(p));
    else e[0] = __ldg(p);
  }
  __device__ __forceinline__ void store(E* p) const {
    if constexpr (VEC * sizeof(E) == 16) *reinterpret_cast<uint4*>(p) = q;
    else p[0] = e[0];
  }
};

struct RmsParams {
  const void* x;
  const void* res;      // or null
  void* h;              // or null
  const void* w;        // or null
  uint8_t* codes;
  float* scales;
  int64_t ldx, ldr, ldh, ldw, ldc;  // elements
  int64_t w_rows;       // rows of x that share a row of w
  int K;
  int norm, int8;
  float eps;
};

// Below this the reciprocal top / max|t| would overflow fp32: the row becomes
// zero codes with a zero scale.
constexpr float kRmsTiny = 3.0092655e-36f;  // 2^-118
// The squares of a row with values above about 2^63 overflow fp32: such rows
// (only those) are summed again scaled by 2^-80.
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

// CH chunks of VEC elements per thread.
template <int DT, int VEC, int CH>
__global__ void __launch_bounds__(1024) rms8_kernel(const RmsParams p) {
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
  const E* w = static_cast<const E*>(p.w) + (p.w ? row / p.w_rows * p.ldw : 0);
  uint8_t* codes = p.codes + row * p.ldc;

  float t[CH * VEC];
  Pack<DT, VEC> a[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = (c * nt + static_cast<int>(threadIdx.x)) * VEC;
    if (k < p.K) a[c].load(x + k);
#pragma unroll
    for (int i = 0; i < VEC; ++i) t[c * VEC + i] = 0.f;
  }
  if (p.res) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int k = (c * nt + static_cast<int>(threadIdx.x)) * VEC;
      if (k < p.K) {
        Pack<DT, VEC> b;
        b.load(r + k);
#pragma unroll
        for (int i = 0; i < VEC; ++i) a[c].e[i] = from_f32<DT>(to_f32<DT>(a[c].e[i]) + to_f32<DT>(b.e[i]));
      }
    }
  }
  float ss = 0.f;
  uint32_t top = 0;  // |t| as bits: ordered like the values, NaN above infinity
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = (c * nt + static_cast<int>(threadIdx.x)) * VEC;
    if (k < p.K) {
      if (p.h) a[c].store(h + k);
      Pack<DT, VEC> g;
      if (p.w) g.load_cached(w + k);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float v = to_f32<DT>(a[c].e[i]);
        ss = fmaf(v, v, ss);
        const float tv = p.w ? v * to_f32<DT>(g.e[i]) : v;
        t[c * VEC + i] = tv;
        top = max(top, __float_as_uint(tv) & 0x7FFFFFFFu);
      }
    }
  }
  top = __reduce_max_sync(0xffffffffu, top);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (nw > 1) {
    if ((threadIdx.x & 31) == 0) {
      red_s[threadIdx.x >> 5] = ss;
      red_m[threadIdx.x >> 5] = top;
    }
    __syncthreads();
    const int l = threadIdx.x & 31;
    top = __reduce_max_sync(0xffffffffu, l < nw ? red_m[l] : 0u);
    ss = l < nw ? red_s[l] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  }
  const float amax = __uint_as_float(top);
  const bool finite = top < 0x7F800000u;
  float rstd = 1.f;
  if (p.norm) {
    rstd = 1.f / sqrtf(ss / static_cast<float>(p.K) + p.eps);
    if (finite && !(ss < INFINITY)) {  // the same for the whole CTA
      float s2 = 0.f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int k = (c * nt + static_cast<int>(threadIdx.x)) * VEC;
        if (k < p.K) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const float v = to_f32<DT>(a[c].e[i]) * kRmsDown;
            s2 = fmaf(v, v, s2);
          }
        }
      }
      s2 = block_sum(s2, red_s, nw);
      rstd = kRmsDown / sqrtf(s2 / static_cast<float>(p.K));
    }
  }
  const float lim = p.int8 ? 127.f : 448.f;
  const bool live = amax >= kRmsTiny;
  const float inv = live && finite ? __fdiv_rn(lim, amax) : 0.f;
  if (threadIdx.x == 0)
    p.scales[row] = finite ? (live ? __fdiv_rn(amax * rstd, lim) : 0.f) : __uint_as_float(0x7FC00000u);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = (c * nt + static_cast<int>(threadIdx.x)) * VEC;
    if (k >= p.K) continue;
    uint32_t q[(VEC + 3) / 4] = {};
    if (p.int8) {
#pragma unroll
      for (int i = 0; i < VEC; ++i)  // |t inv| <= 127 (1 + 2^-23): rounds to at most 127
        q[i / 4] |= (static_cast<uint32_t>(__float2int_rn(t[c * VEC + i] * inv)) & 0xFFu) << (8 * (i % 4));
    } else if constexpr (VEC == 1) {
      q[0] = __nv_cvt_float_to_fp8(t[c] * inv, __NV_SATFINITE, __NV_E4M3);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; i += 2)
        q[i / 4] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
                        make_float2(t[c * VEC + i] * inv, t[c * VEC + i + 1] * inv), __NV_SATFINITE, __NV_E4M3))
                    << (8 * (i % 4));
    }
    if constexpr (VEC == 8) *reinterpret_cast<uint2*>(codes + k) = make_uint2(q[0], q[1]);
    else if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(codes + k) = q[0];
    else codes[k] = static_cast<uint8_t>(q[0]);
  }
}

}  // namespace svdq
