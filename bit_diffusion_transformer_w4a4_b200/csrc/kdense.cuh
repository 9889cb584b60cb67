// Dense linear layer with a fused epilogue, for the layers of a block that
// stay at 16 or 8 bits:
//
//   Y = residual + gate * act(s_a s_w (A W^T) + bias)
//
// A [M x K] activations, W [N x K] weights (both K-major), one operand type:
// bf16, fp16, E4M3 or INT8; fp32 accumulation (int32 for INT8); Y, bias, gate
// and residual bf16 or fp16.
//
// The tensor cores compute the transposed tile: the MMA's M side is 128
// features (256 over a pair of SMs), its N side the tokens.  An accumulator
// lane is then one feature, so the bias and the weight scale are one register
// per thread, a warp's loads and stores of a token's row cover 32 consecutive
// features for any alignment and row stride, and a call with few tokens pads
// them to 16 and not to 128.
//
// All operand types go through one pipeline that counts in bytes: a k-block is
// 128 bytes of a row (64 16-bit or 128 8-bit elements) in the 128-byte
// swizzle, and one MMA consumes 32 bytes.  The tensor maps zero-fill rows
// beyond M and N and elements beyond K.
//
// Measured (B200, back to back): bf16 4608 x 3072 -> 3072 with bias, gate and
// residual 77 us (1.13 PFLOP/s), E4M3 4608 x 3072 -> 12288 with GELU 163 us
// (2.14), INT8 16896 x 12288 -> 3072 496 us (2.57); on different boxes 75 to
// 78, 158 to 169 and 484 to 518.  All three draw 984 to 993 of the 1000 W, at
// 1462, 1342 and 1290 MHz; the tensor pipe is busy 72 and 74 % of the cycles in
// the first two, L2 41 and 42 %.  2 x 3072 -> 18432 streams its weights at
// 5.3 TB/s (21 us).  A gate row per token, read element by element, costs the
// first call 31 us (77 -> 108).
#pragma once

#include "kg_common.cuh"
#include "krms8.cuh"

namespace svdq {

enum : int { DK_F16 = 0, DK_E4M3 = 1, DK_INT8 = 2 };       // operand kinds
enum : int { DENSE_NONE = 0, DENSE_GELU = 1, DENSE_SILU = 2 };
// How Y is stored and the residual loaded, by their alignment: 2 bytes at a
// time (any), 4 bytes after an exchange between lanes (N and the row distances
// even), or as tiles through shared memory and tensor maps (16-byte aligned
// rows; pair kernel only).
enum : int { STORE_PLAIN = 0, STORE_PAIRED = 1 };  // the tiled form is a kernel of its own

struct DenseParams {
  uint16_t* y;
  const uint16_t* bias;   // [N] or null
  const uint16_t* gate;   // [ceil(M / gate_rows) x N] or null
  const uint16_t* res;    // [M x N] or null
  const float* sa;        // [M] or null
  const float* sw;        // [N] or null
  int64_t ldy, ldr, ldg;  // elements
  int gate_rows;
  int M, N;
  int kblk;               // 128-byte k-blocks
  int num_f, num_t;       // feature and token tiles
  int split;              // CTAs (pairs) that share a tile's K range
  int act;
  int store;              // form of the stores and residual loads (below)
  int* err;               // or null
  uint64_t timeout_ns;
  int stuck;              // test hook: the first CTA's first stage waits for an arrival that never comes
};

__host__ __device__ constexpr uint32_t idesc_dense(int kind, int out, int M, int N) {
  // D format f32 / s32; operand format bf16 (1) or fp16 (0), E4M3 (0), S8 (1)
  const uint32_t d = kind == DK_INT8 ? 2u : 1u;
  const uint32_t f = kind == DK_INT8 ? 1u : kind == DK_E4M3 ? 0u : out == DT_BF16 ? 1u : 0u;
  return (d << 4) | (f << 7) | (f << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

#define SVDQ_DENSE_MMA(GROUP, KIND)                                                             \
  asm volatile(                                                                                 \
      "{\n\t.reg .pred p;\n\t"                                                                  \
      "setp.ne.b32 p, %4, 0;\n\t"                                                               \
      "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, p;\n\t}" ::"r"(d),     \
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)                                               \
      : "memory")

template <int KIND, bool PAIR>
__device__ __forceinline__ void dense_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (PAIR) {
    if constexpr (KIND == DK_F16) SVDQ_DENSE_MMA("2", "f16");
    else if constexpr (KIND == DK_E4M3) SVDQ_DENSE_MMA("2", "f8f6f4");
    else SVDQ_DENSE_MMA("2", "i8");
  } else {
    if constexpr (KIND == DK_F16) SVDQ_DENSE_MMA("1", "f16");
    else if constexpr (KIND == DK_E4M3) SVDQ_DENSE_MMA("1", "f8f6f4");
    else SVDQ_DENSE_MMA("1", "i8");
  }
}
#undef SVDQ_DENSE_MMA

// ------------------------------------------------------------------ epilogue
// What a lane keeps of its feature n for a whole tile.
struct DenseLane {
  bool on;          // n < N
  float sw, bias;
  float gate;       // of gate row g, which serves the tokens before gate_end
  int g, gate_end;
};

template <int OUT>
__device__ __forceinline__ DenseLane dense_lane(const DenseParams& p, int n, int m0) {
  DenseLane l;
  l.on = n < p.N;
  l.sw = l.on && p.sw ? __ldg(p.sw + n) : 1.f;
  l.bias = l.on && p.bias ? to_f32<OUT>(__ldg(p.bias + n)) : 0.f;
  l.gate = 0.f;
  l.g = l.gate_end = 0;
  if (p.gate && m0 < p.M) {
    l.g = m0 / p.gate_rows;
    l.gate_end = (l.g + 1) * p.gate_rows;
    if (l.on) l.gate = to_f32<OUT>(__ldg(p.gate + static_cast<int64_t>(l.g) * p.ldg + n));
  }
  return l;
}

// SiLU of two values: x / (1 + 2^(-x log2 e)), with the same approximate
// exponential and reciprocal as the GELU.
__device__ __forceinline__ uint64_t silu2(uint64_t x) {
  const uint64_t a = f2_mul(x, f2_pack(-1.44269504089f, -1.44269504089f));
  float e0, e1, r0, r1;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(f2_lo(a)));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(f2_hi(a)));
  const uint64_t d = f2_add(f2_pack(e0, e1), f2_pack(1.0f, 1.0f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(f2_lo(d)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(f2_hi(d)));
  return f2_mul(x, f2_pack(r0, r1));
}

// gate * act(s_a s_w acc + bias) of NC accumulator columns (tokens m0 ..) of
// feature n, in pairs of tokens.  sa: the tokens' scales (8-bit kinds; 8-byte
// aligned), or null.
template <int KIND, int OUT, int NC>
__device__ __forceinline__ void dense_math(const DenseParams& p, DenseLane& l, int m0, int n, const uint32_t* acc,
                                           const float* sa, uint64_t* x) {
#pragma unroll
  for (int i = 0; i < NC / 2; ++i)
    x[i] = KIND == DK_INT8 ? f2_pack(static_cast<float>(static_cast<int>(acc[2 * i])),
                                     static_cast<float>(static_cast<int>(acc[2 * i + 1])))
                           : f2_pack(__uint_as_float(acc[2 * i]), __uint_as_float(acc[2 * i + 1]));
  const uint64_t b2 = f2_pack(l.bias, l.bias);
  if constexpr (KIND != DK_F16) {
    const uint64_t w2 = f2_pack(l.sw, l.sw);
    if (sa) {
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) x[i] = f2_mul(x[i], *reinterpret_cast<const uint64_t*>(sa + 2 * i));
    }
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) x[i] = f2_fma(x[i], w2, b2);
  } else {
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) x[i] = f2_add(x[i], b2);
  }
  if (p.act == DENSE_GELU) {
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) x[i] = gelu_tanh2(x[i]);
  } else if (p.act == DENSE_SILU) {
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) x[i] = silu2(x[i]);
  }
  if (p.gate) {
    if (m0 + NC <= l.gate_end || p.M <= l.gate_end) {  // one gate row for all
      const uint64_t g2 = f2_pack(l.gate, l.gate);
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) x[i] = f2_mul(x[i], g2);
    } else {
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        if (m0 + j >= l.gate_end && m0 + j < p.M) {
          ++l.g;
          l.gate_end += p.gate_rows;
          if (l.on) l.gate = to_f32<OUT>(__ldg(p.gate + static_cast<int64_t>(l.g) * p.ldg + n));
        }
        x[j / 2] = j % 2 ? f2_pack(f2_lo(x[j / 2]), f2_hi(x[j / 2]) * l.gate)
                         : f2_pack(f2_lo(x[j / 2]) * l.gate, f2_hi(x[j / 2]));
      }
    }
  }
}

// Stores.  In the plain form a lane owns its feature's column of Y: 2 bytes a
// store, 64 contiguous bytes a warp, any alignment.  In the paired form
// lanes 2i and 2i + 1 first exchange values, so that the even lane holds both
// features for token j and the odd one both for token j + 1: half the loads
// and stores, and half the registers of a prefetched residual.
//
// dense_residual: the residual of NC tokens m0 .. in the form that
// dense_store takes, one 32-bit word per token pair (paired) or per token.
template <int OUT, int NC, bool PAIRED>
__device__ __forceinline__ void dense_residual(const DenseParams& p, const DenseLane& l, int m0, int n, uint32_t* r) {
  if constexpr (PAIRED) {
    const int odd = n & 1;
    const uint16_t* src = p.res + static_cast<int64_t>(m0 + odd) * p.ldr + (n - odd);
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) {
      r[i] = l.on && m0 + odd + 2 * i < p.M ? *reinterpret_cast<const uint32_t*>(src) : 0u;
      src += 2 * p.ldr;
    }
  } else {
    const uint16_t* src = p.res + static_cast<int64_t>(m0) * p.ldr + n;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      r[j] = l.on && m0 + j < p.M ? *src : 0u;
      src += p.ldr;
    }
  }
}

template <int OUT>
__device__ __forceinline__ uint32_t pack_out(float lo, float hi) {
  if constexpr (OUT == DT_BF16) return pack_bf16x2(lo, hi);
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int OUT, int NC, bool PAIRED>
__device__ __forceinline__ void dense_store(const DenseParams& p, const DenseLane& l, int m0, int n, const uint64_t* x,
                                            const uint32_t* r) {
  if constexpr (PAIRED) {
    const int odd = n & 1;
    uint16_t* dst = p.y + static_cast<int64_t>(m0 + odd) * p.ldy + (n - odd);
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) {
      const float lo = f2_lo(x[i]), hi = f2_hi(x[i]);
      const float got = __shfl_xor_sync(0xffffffffu, odd ? lo : hi, 1);
      float a = odd ? got : lo, b = odd ? hi : got;
      if (p.res) {
        a += to_f32<OUT>(static_cast<uint16_t>(r[i]));
        b += to_f32<OUT>(static_cast<uint16_t>(r[i] >> 16));
      }
      if (l.on && m0 + odd + 2 * i < p.M) *reinterpret_cast<uint32_t*>(dst) = pack_out<OUT>(a, b);
      dst += 2 * p.ldy;
    }
  } else {
    uint16_t* dst = p.y + static_cast<int64_t>(m0) * p.ldy + n;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      float v = j % 2 ? f2_hi(x[j / 2]) : f2_lo(x[j / 2]);
      if (p.res) v += to_f32<OUT>(static_cast<uint16_t>(r[j]));
      if (l.on && m0 + j < p.M) *dst = from_f32<OUT>(v);
      dst += p.ldy;
    }
  }
}

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// Sets the abort flag (at `flag` of each CTA's shared memory) of all CTAs of
// the cluster.  A thread that has given up calls it before a cluster barrier,
// behind which the cluster's CTAs then agree.
__device__ __forceinline__ void raise_in_cluster(uint32_t flag, int ctas) {
  for (int r = 0; r < ctas; ++r) st_cluster_u32(mapa_shared(flag, r), 1);
}
// The sums over `split` CTAs (ranks step o + first) of a feature's NC
// consecutive tokens at `addr` of each one's [token][128 features] partial
// tile, in rank order: they do not depend on timing.
template <int KIND, int NC>
__device__ __forceinline__ void dense_join(uint32_t addr, int split, int step, int first, uint32_t* v) {
  constexpr int G = NC == 2 ? 8 : 2;  // CTAs whose sums are fetched at a time
#pragma unroll
  for (int j = 0; j < NC; ++j) v[j] = 0;
#pragma unroll 1
  for (int o0 = 0; o0 < split; o0 += G) {
    uint32_t w[G][NC];
#pragma unroll
    for (int o = 0; o < G; ++o) {
      const uint32_t at = mapa_shared(addr, step * min(o0 + o, split - 1) + first);
#pragma unroll
      for (int j = 0; j < NC; ++j) w[o][j] = o0 + o < split ? ld_cluster_u32(at + j * 512) : 0u;
    }
#pragma unroll
    for (int o = 0; o < G; ++o)
#pragma unroll
      for (int j = 0; j < NC; ++j)
        v[j] = KIND == DK_INT8 ? v[j] + w[o][j] : __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(w[o][j]));
  }
}

// ------------------------------------------------ pairs of SMs, large calls
// A cluster of two CTAs owns 256 features x BN tokens: rank r loads weight
// rows [128 r, 128 r + 128) and token rows [BN/2 r, BN/2 r + BN/2) of the
// tile, the leader issues the pair's MMAs (M = 256), and each SM accumulates
// its 128 features x BN tokens.  Persistent over tiles; two accumulators in
// tensor memory, so the epilogue of one tile runs under the MMAs of the next.
// Warps: 0 TMA, 1 MMA and tensor memory, 2-3 idle, 4-19 epilogue: each of the
// 16 takes 32 features x 64 tokens.  In the tiled form two warps (64 features,
// a full line of Y) have a box of 8 KB in shared memory: the residual arrives
// in it by a tensor load while the tile is being summed, the accumulator is
// read in the matrix-fragment layout, stmatrix transposes the rounded result
// into the box in place, and a tensor store takes it from there: an eighth of
// an instruction per element where lane exchanges and 4-byte stores take about
// five (bf16 4608 x 3072 -> 3072 with residual 75 us; 3074 features, one tile
// row more and 4-byte stores, 88; 3073, 2-byte stores, 95).
constexpr int DP_THREADS = 640;
constexpr int DP_EPI_WARPS = 16;

struct DensePairSmem {
  static constexpr int BN = 256;
  static constexpr int W_BYTES = 128 * 128;
  static constexpr int A_BYTES = BN / 2 * 128;
  static constexpr int STAGE = W_BYTES + A_BYTES;
  static constexpr int STAGES = 5;
  static constexpr uint32_t TX = 2 * STAGE;
  static constexpr int OUT_OFF = STAGES * STAGE;            // [8 pairs of warps][64 tokens][64 features], 128-byte swizzle
  static constexpr int OUT_BYTES = 64 * 64 * 2;
  static constexpr int BAR_OFF = OUT_OFF + DP_EPI_WARPS / 2 * OUT_BYTES;
  static constexpr int TOTAL = BAR_OFF + 512 + 1024;
  static_assert(TOTAL <= 232448, "shared memory per CTA");
};

// Tiles in bands of kDenseBand token tiles, features outermost inside a band:
// the tiles that run at one time share few weight and token blocks.
constexpr int kDenseBand = 8;
__device__ __forceinline__ void dense_tile(const DenseParams& p, int tile, int& ft, int& tt) {
  const int band = tile / (kDenseBand * p.num_f);
  const int in = tile - band * kDenseBand * p.num_f;
  const int wide = min(kDenseBand, p.num_t - band * kDenseBand);
  ft = in / wide;
  tt = band * kDenseBand + in - ft * wide;
}

// The tiled epilogue of one warp: 32 features from n0, 64 tokens from m0.
// Thread t works on features n0 + t / 4 + 8 f (f = 0 .. 3) and tokens
// m0 + 8 k + 2 (t % 4) and + 1 (k = 0 .. 7).
template <int KIND, int OUT>
struct DenseTileOut {
  float bias[4], sw[4], gate[4];
  uint64_t sa[8];  // scales of its token pairs
  bool one_gate;   // all its tokens share a gate row (else the row is looked up per element)

  // What does not depend on the accumulator, loaded while it is being summed.
  __device__ __forceinline__ void prepare(const DenseParams& p, int n0, int m0, int lane) {
    const bool gated = p.gate && m0 < p.M;  // tokens beyond M have no gate row
    const int g0 = gated ? m0 / p.gate_rows : 0;
    one_gate = gated && min(m0 + 64, p.M) <= (g0 + 1) * p.gate_rows;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const int n = n0 + 8 * f + (lane >> 2);
      const bool on = n < p.N;
      bias[f] = on && p.bias ? to_f32<OUT>(__ldg(p.bias + n)) : 0.f;
      sw[f] = KIND != DK_F16 && on && p.sw ? __ldg(p.sw + n) : 1.f;
      gate[f] = on && one_gate ? to_f32<OUT>(__ldg(p.gate + static_cast<int64_t>(g0) * p.ldg + n)) : 0.f;
    }
    if (KIND != DK_F16) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int m = m0 + 8 * k + 2 * (lane & 3);
        sa[k] = p.sa ? f2_pack(m < p.M ? __ldg(p.sa + m) : 0.f, m + 1 < p.M ? __ldg(p.sa + m + 1) : 0.f) : f2_pack(1.f, 1.f);
      }
    }
  }

  // box: the warps' shared memory, holding the residual if there is one; q: the
  // warp's half of its features is q % 2.
  // `done` is called when the accumulator has been read.
  template <class F>
  __device__ __forceinline__ void run(const DenseParams& p, uint32_t taddr, uint32_t box, int q, int n0, int m0, int lane, F done) const {
    // lane 8 i + j of a matrix access: token j of column block i / 2, feature block i % 2
    const int mtok = ((lane >> 4) << 3) + (lane & 7), mfeat = (lane >> 3) & 1;
    uint32_t v[2][16];
    tmem_ld_16x256b_x4(taddr, v[0]);
#pragma unroll
    for (int c = 0; c < 4; ++c) {  // 16 features x 32 tokens; the next chunk is read under this one
      const int half = c / 2;
      tmem_ld_wait();
      if (c < 3)
        tmem_ld_16x256b_x4(taddr + (static_cast<uint32_t>(16 * ((c + 1) / 2)) << 16) + 32 * ((c + 1) % 2), v[(c + 1) % 2]);
      else
        done();
#pragma unroll
      for (int kk = 0; kk < 4; kk += 2) {
        const int k0 = 4 * (c % 2) + kk;
        uint64_t x[4];  // (block k0, feature a), (k0, b), (k0 + 1, a), (k0 + 1, b): a pair of tokens each
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int f = 2 * half + i % 2;
          const uint32_t lo = v[c % 2][4 * kk + 2 * i], hi = v[c % 2][4 * kk + 2 * i + 1];
          x[i] = KIND == DK_INT8 ? f2_pack(static_cast<float>(static_cast<int>(lo)), static_cast<float>(static_cast<int>(hi)))
                                 : f2_pack(__uint_as_float(lo), __uint_as_float(hi));
          const uint64_t b2 = f2_pack(bias[f], bias[f]);
          if constexpr (KIND != DK_F16) x[i] = f2_fma(f2_mul(x[i], sa[k0 + i / 2]), f2_pack(sw[f], sw[f]), b2);
          else x[i] = f2_add(x[i], b2);
        }
        if (p.act == DENSE_GELU) {
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = gelu_tanh2(x[i]);
        } else if (p.act == DENSE_SILU) {
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = silu2(x[i]);
        }
        if (p.gate) {
          if (one_gate) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = f2_mul(x[i], f2_pack(gate[2 * half + i % 2], gate[2 * half + i % 2]));
          } else {
#pragma unroll 1
            for (int j = 0; j < 2; ++j) {  // the pairs' first and second tokens
              float g[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int n = n0 + 8 * (2 * half + i % 2) + (lane >> 2), m = m0 + 8 * (k0 + i / 2) + 2 * (lane & 3) + j;
                g[i] = n < p.N && m < p.M ? to_f32<OUT>(__ldg(p.gate + static_cast<int64_t>(m / p.gate_rows) * p.ldg + n)) : 0.f;
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) x[i] = f2_mul(x[i], j ? f2_pack(1.f, g[i]) : f2_pack(g[i], 1.f));
            }
          }
        }
        const uint32_t at = box + swz_off(8 * k0 + mtok, 4 * (q & 1) + 2 * half + mfeat, 128);
        if (p.res) {
          uint32_t r[4];
          ldmatrix_x4_trans(at, r);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[i] = f2_add(x[i], f2_pack(to_f32<OUT>(static_cast<uint16_t>(r[i])), to_f32<OUT>(static_cast<uint16_t>(r[i] >> 16))));
        }
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack_out<OUT>(f2_lo(x[i]), f2_hi(x[i]));
        stmatrix_x4_trans(at, o[0], o[1], o[2], o[3]);
      }
    }
  }
};

// TILED: the tiled form; else p.store says which.  p.split > 1 (not TILED):
// a cluster of p.split pairs shares the K range of one tile, and the sums meet
// in distributed shared memory as in the single-SM kernel.
template <int KIND, int OUT, bool TILED>
__global__ void __launch_bounds__(DP_THREADS, 1)
    dense_pair_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a,
                      const __grid_constant__ CUtensorMap tm_y, const __grid_constant__ CUtensorMap tm_r,
                      const __grid_constant__ DenseParams p) {
  using S = DensePairSmem;
  constexpr int BN = S::BN;
  constexpr int NST = S::STAGES;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::BAR_OFF);
  const uint32_t bar_full = smem_u32(bars);
  const uint32_t bar_empty = smem_u32(bars + NST);
  const uint32_t bar_acc_full = smem_u32(bars + 2 * NST);       // two
  const uint32_t bar_acc_empty = smem_u32(bars + 2 * NST + 2);  // two, the leader's count
  const uint32_t bar_drain = smem_u32(bars + 2 * NST + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * NST + 5);
  const uint32_t bar_res = smem_u32(bars + 2 * NST + 6);        // one per pair of epilogue warps
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // the stages that this CTA has loaded and the parities of their last loads
  volatile uint32_t* loads = reinterpret_cast<volatile uint32_t*>(bars + 2 * NST + 6 + DP_EPI_WARPS / 2);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int split = TILED ? 1 : p.split;
  const uint32_t crank = cluster_ctarank();
  const uint32_t rank = crank & 1, lead = crank & ~1u;  // rank in the pair; the pair's leader
  const int pr = static_cast<int>(crank >> 1);          // this pair's slice of K
  const int cid = static_cast<int>(blockIdx.x) / (2 * split);
  const int nclu = static_cast<int>(gridDim.x) / (2 * split);
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.kblk) * pr / split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.kblk) * (pr + 1) / split);
  const uint16_t both = static_cast<uint16_t>(0x3u << lead);
  const Guard guard{p.err ? p.err : &g_ops_err, abort_flag, p.timeout_ns};
  const int num_tiles = p.num_f * p.num_t;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(bar_full + 8 * s, 1 + (p.stuck && s + blockIdx.x == 0));
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_acc_full + 8 * i, 1);
      mbar_init(bar_acc_empty + 8 * i, 2 * DP_EPI_WARPS);
    }
    mbar_init(bar_drain, 1);
    for (int i = 0; i < DP_EPI_WARPS / 2; ++i) mbar_init(bar_res + 8 * i, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();  // barriers of both CTAs initialised, tensor memory allocated
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();  // operands and outputs may belong to the previous kernel of the stream
  griddep_launch_dependents();

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_w);
      tma_prefetch_desc(&tm_a);
      const uint32_t full0 = mapa_shared(bar_full, lead);  // the leader's full barriers
      int s = 0;
      uint32_t ph = 0, issued = 0, issued_par = 0;
      bool ok = true;
      for (int tile = cid; tile < num_tiles && ok; tile += nclu) {
        int ft, tt;
        dense_tile(p, tile, ft, tt);
        const int wrow = ft * 256 + static_cast<int>(rank) * 128;
        const int arow = tt * BN + static_cast<int>(rank) * (BN / 2);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!(ok = wait_bounded(bar_empty + 8 * s, ph ^ 1, guard, 0x301))) break;
          const uint32_t st = sbase + s * S::STAGE;
          if (rank == 0) mbar_expect_tx(bar_full + 8 * s, S::TX);
          // whole boxes always: what lies beyond N, M or K is zero-filled
          const int kc = kb * (KIND == DK_F16 ? 64 : 128);
          tma_load_2d_pair(st, &tm_w, full0 + 8 * s, kc, wrow);
          tma_load_2d_pair(st + S::W_BYTES, &tm_a, full0 + 8 * s, kc, arow);
          issued |= 1u << s;
          issued_par = (issued_par & ~(1u << s)) | (ph << s);
          if (++s == NST) { s = 0; ph ^= 1; }
        }
      }
      loads[0] = issued;
      loads[1] = issued_par;
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      constexpr uint32_t id = idesc_dense(KIND, OUT, 256, BN);
      const uint64_t dW0 = smem_desc(sbase, 16, 1024, SWZ_128B);
      const uint64_t dA0 = smem_desc(sbase + S::W_BYTES, 16, 1024, SWZ_128B);
      constexpr uint64_t kStage = S::STAGE >> 4;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = cid, j = 0; tile < num_tiles && ok; tile += nclu, ++j) {
        const int ac = j & 1;
        const uint32_t d = tmem + ac * 256;
        if (j > 1 && !(ok = wait_bounded_cl(bar_acc_empty + 8 * ac, ((j >> 1) - 1) & 1, guard, 0x302))) break;
        tc_fence_after();
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!(ok = wait_bounded(bar_full + 8 * s, ph, guard, 0x303))) break;
          tc_fence_after();
          const uint64_t so = kStage * s;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dense_mma<KIND, true>(d, dW0 + so + 2 * i, dA0 + so + 2 * i, id, (kb != kb0) | (i != 0));
          tc_commit_pair(bar_empty + 8 * s, both);
          if (++s == NST) { s = 0; ph ^= 1; }
        }
        if (!ok) break;
        tc_commit_pair(bar_acc_full + 8 * ac, both);
      }
      // every MMA of the pair has completed before either CTA frees tensor memory
      tc_commit_pair(bar_drain, static_cast<uint16_t>(1u << lead));
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(bar_drain, 0) && global_timer_ns() - t0 < p.timeout_ns) {
      }
    }
  } else if (warp >= 4) {
    const int e = warp - 4;
    constexpr int CW = BN / 4;           // tokens of this warp
    const int q = warp & 3;              // tensor-memory lane group of this warp
    const int c0 = (e >> 2) * CW;
    const uint32_t acc_empty0 = mapa_shared(bar_acc_empty, lead);
    const int b = (e >> 2) * 2 + (q >> 1);  // the box shared with the other warp of its 64 features
    const uint32_t box = sbase + S::OUT_OFF + b * S::OUT_BYTES;
    const uint32_t res_full = bar_res + 8 * b;
    const bool first = (q & 1) == 0 && lane == 0;  // issues the box's tensor copies
    uint32_t res_ph = 0;
    bool res_on = false;                 // a residual load is in flight
    for (int tile = cid, j = 0; tile < num_tiles; tile += nclu, ++j) {
      int ft, tt;
      dense_tile(p, tile, ft, tt);
      const int ac = j & 1;
      const int n0 = ft * 256 + static_cast<int>(rank) * 128 + q * 32;
      const int m0 = tt * BN + c0;
      const uint32_t ta = tmem + (static_cast<uint32_t>(q * 32) << 16) + ac * 256 + c0;
      auto acc_read = [&] {  // this warp has read its part of the accumulator
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty0 + 8 * ac);
      };
      if constexpr (TILED) {
        const int nb = n0 - 32 * (q & 1);  // the box's first feature
        const bool on = nb < p.N && m0 < p.M;
        if (first) bulk_wait_read();       // the previous tile has left the box
        if (p.res && on && first) {
          mbar_expect_tx(res_full, S::OUT_BYTES);
          tma_load_2d(box, &tm_r, res_full, nb, m0);
        }
        res_on = p.res && on;
        DenseTileOut<KIND, OUT> out;
        out.prepare(p, n0, m0, lane);
        bool ok = wait_bounded(bar_acc_full + 8 * ac, (j >> 1) & 1, guard, 0x304, 64);
        if (ok && res_on) {
          ok = wait_bounded(res_full, res_ph, guard, 0x305);
          if (ok) res_ph ^= 1;
          res_on = !ok;
        }
        // both warps of a box go on or give up together; the box is free
        if (!named_barrier_all(1 + b, 64, ok)) break;
        tc_fence_after();
        if (on) {
          out.run(p, ta, box, q, n0, m0, lane, acc_read);
          fence_proxy_async_smem();
          named_barrier(1 + b, 64);        // both warps have written
          if (first) {
            tma_store_2d(&tm_y, box, nb, m0);
            bulk_commit();
          }
        } else {
          acc_read();
        }
        continue;
      }
      if (split > 1) {  // one tile per cluster: the partial sums take the stages' place
        if (!__all_sync(0xffffffffu, wait_bounded(bar_acc_full, 0, guard, 0x304, 64))) break;
        tc_fence_after();
        uint32_t* part = reinterpret_cast<uint32_t*>(smem);
#pragma unroll 1
        for (int c = 0; c < CW; c += 32) {
          uint32_t v[32];
          tmem_ld_x32(ta + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) part[(c0 + c + i) * 128 + q * 32 + lane] = v[i];
        }
        acc_read();
        break;
      }
      const int n = n0 + lane;
      DenseLane l = dense_lane<OUT>(p, n, m0);
      // the boxes hold the warps' token scales
      float* sa = reinterpret_cast<float*>(smem + S::OUT_OFF) + e * CW;
      if (KIND != DK_F16 && p.sa) {
        __syncwarp();  // the previous tile's scales have been read
        for (int i = lane; i < CW; i += 32) sa[i] = m0 + i < p.M ? __ldg(p.sa + m0 + i) : 0.f;
        __syncwarp();
      }
      const float* sc = KIND != DK_F16 && p.sa ? sa : nullptr;
      if (p.store == STORE_PAIRED) {
        uint32_t r[CW / 2];
        if (p.res) dense_residual<OUT, CW, true>(p, l, m0, n, r);
        if (!__all_sync(0xffffffffu, wait_bounded(bar_acc_full + 8 * ac, (j >> 1) & 1, guard, 0x304, 64))) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < CW; c += 16) {
          uint32_t v[16];
          uint64_t x[8];
          tmem_ld_x16(ta + c, v);
          tmem_ld_wait();
          if (c + 16 == CW) acc_read();
          dense_math<KIND, OUT, 16>(p, l, m0 + c, n, v, sc ? sc + c : nullptr, x);
          dense_store<OUT, 16, true>(p, l, m0 + c, n, x, r + c / 2);
        }
      } else {
        if (!__all_sync(0xffffffffu, wait_bounded(bar_acc_full + 8 * ac, (j >> 1) & 1, guard, 0x304, 64))) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < CW; c += 16) {
          uint32_t v[16], r[16];
          uint64_t x[8];
          tmem_ld_x16(ta + c, v);
          if (p.res) dense_residual<OUT, 16, false>(p, l, m0 + c, n, r);
          tmem_ld_wait();
          if (c + 16 == CW) acc_read();
          dense_math<KIND, OUT, 16>(p, l, m0 + c, n, v, sc ? sc + c : nullptr, x);
          dense_store<OUT, 16, false>(p, l, m0 + c, n, x, r);
        }
      }
    }
    if (first) {
      if (res_on) {  // given up with the residual on its way
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(res_full, res_ph) && global_timer_ns() - t0 < p.timeout_ns) {
        }
      }
      bulk_wait_all();  // the stores are done before the shared memory goes
    }
  }

  __syncwarp();
  if (*abort_flag) raise_in_cluster(smem_u32(const_cast<int*>(abort_flag)), 2 * split);
  if constexpr (!TILED) {
    if (split > 1) {
      __syncwarp();
      cluster_sync();  // every pair's partial sums are in place, or all know that some are not
      if (warp >= 4 && !*abort_flag) {
        const int e = warp - 4, q = warp & 3;
        int ft, tt;
        dense_tile(p, cid, ft, tt);
        const int f = q * 32 + lane, n = ft * 256 + static_cast<int>(rank) * 128 + f;
        const int cols = BN / split / 4;  // tokens of this warp: 32 or 16
        const int c0 = pr * (BN / split) + (e >> 2) * cols;
        const int m0 = tt * BN + c0;
        float* sa = reinterpret_cast<float*>(smem + S::OUT_OFF) + e * 64;
        if (KIND != DK_F16 && p.sa) {
          if (lane < cols) sa[lane] = m0 + lane < p.M ? __ldg(p.sa + m0 + lane) : 0.f;
          __syncwarp();
        }
        const float* sc = KIND != DK_F16 && p.sa ? sa : nullptr;
        DenseLane l = dense_lane<OUT>(p, n, m0);
#pragma unroll 1
        for (int c = 0; c < cols && m0 + c < p.M; c += 16) {
          uint32_t r[16], v[16];
          if (p.res) {
            if (p.store == STORE_PAIRED) dense_residual<OUT, 16, true>(p, l, m0 + c, n, r);
            else dense_residual<OUT, 16, false>(p, l, m0 + c, n, r);
          }
          dense_join<KIND, 16>(sbase + ((c0 + c) * 128 + f) * 4, split, 2, rank, v);
          uint64_t x[8];
          dense_math<KIND, OUT, 16>(p, l, m0 + c, n, v, sc ? sc + c : nullptr, x);
          if (p.store == STORE_PAIRED) dense_store<OUT, 16, true>(p, l, m0 + c, n, x, r);
          else dense_store<OUT, 16, false>(p, l, m0 + c, n, x, r);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // the pair's MMAs, loads and remote arrivals are all done
  // Given up (every CTA of the cluster knows): loads on their way land before a
  // CTA leaves.  The leader's barriers count those of both; a stage that only
  // the other CTA has loaded was loaded a wait's limit ago.  Passing that CTA's
  // stages on as well takes registers from the epilogue (INT8 16896 x 12288 ->
  // 3072 499 -> 505 us).
  if (*abort_flag) {
    if (threadIdx.x == 0 && rank == 0) drain_loads(bar_full, loads[0], loads[1], NST, p.timeout_ns);
    __syncwarp();
    cluster_sync();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// -------------------------------------------- single SMs, few tokens or tiles
// One CTA per (128 features x BN tokens, slice of K).  A cluster of `split`
// CTAs shares a tile's K range; their partial sums meet in distributed shared
// memory, each CTA adds up and stores its share of the tokens, in rank order,
// so the result does not depend on timing and needs no workspace.
// Warps: 0 TMA, 1 MMA and tensor memory, 2-5 epilogue.
constexpr int DS_THREADS = 192;

template <int BN>
struct DenseSoloSmem {
  static constexpr int W_BYTES = 128 * 128;
  static constexpr int A_BYTES = BN * 128;
  static constexpr int STAGE = W_BYTES + A_BYTES;
  static constexpr int STAGES = BN <= 32 ? 5 : BN == 64 ? 4 : 3;  // two CTAs fit an SM
  static constexpr int BAR_OFF = STAGES * STAGE;
  static constexpr int SA_OFF = BAR_OFF + 256;                    // [BN] token scales
  static constexpr int TOTAL = SA_OFF + BN * 4 + 1024;
  static_assert(128 * BN * 4 <= BAR_OFF, "the partial tile fits the stages");
  static_assert(2 * TOTAL <= 232448, "shared memory of two CTAs");
};

template <int KIND, int OUT, int BN>
__global__ void __launch_bounds__(DS_THREADS, 2)
    dense_solo_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a,
                      const __grid_constant__ DenseParams p) {
  using S = DenseSoloSmem<BN>;
  constexpr int NST = S::STAGES;
  constexpr int COLS = BN < 32 ? 32 : BN;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::BAR_OFF);
  const uint32_t bar_full = smem_u32(bars);
  const uint32_t bar_empty = smem_u32(bars + NST);
  const uint32_t bar_acc = smem_u32(bars + 2 * NST);
  const uint32_t bar_drain = smem_u32(bars + 2 * NST + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * NST + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // the stages that this CTA has loaded and the parities of their last loads
  volatile uint32_t* loads = reinterpret_cast<volatile uint32_t*>(bars + 2 * NST + 3);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int split = p.split;
  const int rank = static_cast<int>(blockIdx.x) % split;
  const int tile = static_cast<int>(blockIdx.x) / split;
  const int ft = tile % p.num_f, tt = tile / p.num_f;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.kblk) * rank / split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.kblk) * (rank + 1) / split);
  const Guard guard{p.err ? p.err : &g_ops_err, abort_flag, p.timeout_ns};

  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(bar_full + 8 * s, 1 + (p.stuck && s + blockIdx.x == 0));
      mbar_init(bar_empty + 8 * s, 1);
    }
    mbar_init(bar_acc, 1);
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_w);
      tma_prefetch_desc(&tm_a);
      int s = 0;
      uint32_t ph = 0, issued = 0, issued_par = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait_bounded(bar_empty + 8 * s, ph ^ 1, guard, 0x311)) break;
        const uint32_t st = sbase + s * S::STAGE;
        mbar_expect_tx(bar_full + 8 * s, S::STAGE);
        const int kc = kb * (KIND == DK_F16 ? 64 : 128);
        tma_load_2d(st, &tm_w, bar_full + 8 * s, kc, ft * 128);
        tma_load_2d(st + S::W_BYTES, &tm_a, bar_full + 8 * s, kc, tt * BN);
        issued |= 1u << s;
        issued_par = (issued_par & ~(1u << s)) | (ph << s);
        if (++s == NST) { s = 0; ph ^= 1; }
      }
      loads[0] = issued;
      loads[1] = issued_par;
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t id = idesc_dense(KIND, OUT, 128, BN);
      const uint64_t dW0 = smem_desc(sbase, 16, 1024, SWZ_128B);
      const uint64_t dA0 = smem_desc(sbase + S::W_BYTES, 16, 1024, SWZ_128B);
      constexpr uint64_t kStage = S::STAGE >> 4;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!(ok = wait_bounded(bar_full + 8 * s, ph, guard, 0x312))) break;
        tc_fence_after();
        const uint64_t so = kStage * s;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          dense_mma<KIND, false>(tmem, dW0 + so + 2 * i, dA0 + so + 2 * i, id, (kb != kb0) | (i != 0));
        tc_commit(bar_empty + 8 * s);
        if (++s == NST) { s = 0; ph ^= 1; }
      }
      if (ok) tc_commit(bar_acc);
      tc_commit(bar_drain);
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(bar_drain, 0) && global_timer_ns() - t0 < p.timeout_ns) {
      }
    }
  }
  const int q = warp & 3;
  const int f = q * 32 + lane;          // feature of the tile
  const int n = ft * 128 + f;
  const int m0 = tt * BN;
  const int valid = min(BN, p.M - m0);  // tokens of the tile
  bool ok = true;
  DenseLane l = {};
  float* sa = reinterpret_cast<float*>(smem + S::SA_OFF);
  const float* sc = KIND != DK_F16 && p.sa ? sa : nullptr;
  if (sc) {
    for (int i = threadIdx.x; i < BN; i += DS_THREADS) sa[i] = m0 + i < p.M ? __ldg(p.sa + m0 + i) : 0.f;
    __syncthreads();
  }
  if (warp >= 2) {
    l = dense_lane<OUT>(p, n, m0);
    ok = __all_sync(0xffffffffu, wait_bounded(bar_acc, 0, guard, 0x313, 32));
    tc_fence_after();
    const uint32_t ta = tmem + (static_cast<uint32_t>(q * 32) << 16);
    if (split == 1) {
      if (ok) {
#pragma unroll 1
        for (int c = 0; c < valid; c += 16) {
          uint32_t v[16], r[16];
          uint64_t x[8];
          tmem_ld_x16(ta + c, v);
          if (p.res) {
            if (p.store == STORE_PAIRED) dense_residual<OUT, 16, true>(p, l, m0 + c, n, r);
            else dense_residual<OUT, 16, false>(p, l, m0 + c, n, r);
          }
          tmem_ld_wait();
          dense_math<KIND, OUT, 16>(p, l, m0 + c, n, v, sc ? sc + c : nullptr, x);
          if (p.store == STORE_PAIRED) dense_store<OUT, 16, true>(p, l, m0 + c, n, x, r);
          else dense_store<OUT, 16, false>(p, l, m0 + c, n, x, r);
        }
      }
    } else if (ok) {
      // every stage has been consumed: the partial tile goes into their place
      uint32_t* part = reinterpret_cast<uint32_t*>(smem);
#pragma unroll 1
      for (int c = 0; c < valid; c += 16) {
        uint32_t v[16];
        tmem_ld_x16(ta + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(c + j) * 128 + f] = v[j];
      }
    }
  }
  __syncwarp();
  if (split > 1) {
    cluster_sync();  // all partial tiles are in place, or their CTAs' flags are up
    if (warp >= 2) {
      // asked under the first loads of the partial tiles
      const uint32_t lost = lane < split ? ld_cluster_u32(mapa_shared(smem_u32(const_cast<int*>(abort_flag)), lane)) : 0u;
      // this CTA's tokens: 16 at a time where there are as many, else two
      const int unit = valid >= 16 * split ? 16 : 2;
      const int per = unit * ((valid + unit * split - 1) / (unit * split));
      const int c1 = min(valid, (rank + 1) * per);
      if (p.gate) l = dense_lane<OUT>(p, n, m0 + rank * per);
      if (unit == 16) {
#pragma unroll 1
        for (int c = rank * per; c < c1; c += 16) {
          uint32_t v[16], r[16];
          uint64_t x[8];
          if (p.res) {
            if (p.store == STORE_PAIRED) dense_residual<OUT, 16, true>(p, l, m0 + c, n, r);
            else dense_residual<OUT, 16, false>(p, l, m0 + c, n, r);
          }
          dense_join<KIND, 16>(sbase + (c * 128 + f) * 4, split, 1, 0, v);
          if (__any_sync(0xffffffffu, lost)) break;
          dense_math<KIND, OUT, 16>(p, l, m0 + c, n, v, sc ? sc + c : nullptr, x);
          if (p.store == STORE_PAIRED) dense_store<OUT, 16, true>(p, l, m0 + c, n, x, r);
          else dense_store<OUT, 16, false>(p, l, m0 + c, n, x, r);
        }
      } else {
        for (int c = rank * per; c < c1; c += 2) {
          uint32_t v[2], r[2];
          uint64_t x[1];
          if (p.res) dense_residual<OUT, 2, false>(p, l, m0 + c, n, r);
          dense_join<KIND, 2>(sbase + (c * 128 + f) * 4, split, 1, 0, v);
          if (__any_sync(0xffffffffu, lost)) break;
          dense_math<KIND, OUT, 2>(p, l, m0 + c, n, v, sc ? sc + c : nullptr, x);
          dense_store<OUT, 2, false>(p, l, m0 + c, n, x, r);
        }
      }
    }
    cluster_sync();  // no CTA leaves while its partial tile may be read
  }
  tc_fence_before();
  __syncthreads();
  // given up: loads still on their way land before the CTA leaves
  if (threadIdx.x == 0 && *abort_flag) drain_loads(bar_full, loads[0], loads[1], NST, p.timeout_ns);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, COLS);
  }
}

}  // namespace svdq
