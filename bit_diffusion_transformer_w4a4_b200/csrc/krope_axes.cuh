// Rotary positions with several axes (text index, time, height, width, ...),
// applied to Q and K or written as a table of (cos, sin).
//
// Pair p of a head belongs to one axis and turns by angle(p) = pos[token,
// axis(p)] * f(p) radians:
//   (a, b) <- (a cos - b sin, a sin + b cos),
// with sin negated for the inverse rotation, which is also the gradient.
// Interleaved pairs are the elements (2p, 2p + 1), split halves (p, p + R/2);
// elements R .. D - 1 of a head pass through.
//
// Angles: an fp32 product of a far position and its frequency is off by whole
// radians, so the angle is formed in fp64 and in half turns (the plan holds
// f / pi), reduced by whole turns to [-1, 1], and only then goes through the
// fp32 sincospi.  A persistent CTA takes groups of a few tokens; the angles of
// its next group are computed into shared memory under the first loads of the
// present one, and every thread uses the (cos, sin) of its own elements for
// all heads of Q and K, so the fp64 work is paid per token and not per head.
//
// Bound by memory: every element is read once and written once, in pieces of
// 16, 8 or 4 bytes as the layout allows (else element by element).  Groups of
// four tokens and four CTAs an SM were the fastest of 2, 4, 8 and 3, 4, 5 on
// 4608 tokens of 48 heads of 128 (bf16, interleaved): 21.5 us, 5.3 TB/s; 32768
// tokens of 32 heads, split halves: 95 us, 5.6 TB/s.  Heads that only allow
// narrow pieces pay for it: 20000 tokens of 20 heads of 70 take 45 us
// interleaved (4 bytes) and 51 us in split halves (2 bytes), floor 17.
#pragma once

#include "krms8.cuh"

namespace svdq {

constexpr int ROPE_MAX_D = 256;
constexpr int ROPE_MAX_PAIRS = ROPE_MAX_D / 2;
constexpr int ROPE_THREADS = 256;
constexpr int ROPE_TOKENS = 4;   // tokens per group
constexpr int ROPE_CTAS = 4;     // resident CTAs per SM

struct RopePlan {
  double f[ROPE_MAX_PAIRS];      // half turns per unit of position
  uint8_t axis[ROPE_MAX_PAIRS];
  int D, pairs, interleaved;
};

struct RopePos {
  const void* p;
  int type;                      // 0 int32, 1 int64, 2 fp32
  int64_t sb, ss, sa;            // strides in elements (batch, token, axis)
};

struct RopeTensor {
  const void* x;
  void* out;
  int heads;
  int64_t xb, xs, xh, ob, os, oh;  // strides in elements (batch, token, head)
};

struct RopeParams {
  RopePlan plan;
  RopePos pos;
  RopeTensor t[2];
  uint32_t S, tokens, groups;    // tokens per sequence and in all, groups of ROPE_TOKENS
  float sign;                    // -1: inverse
  int pass;                      // elements beyond the rotated span are copied
};

__device__ __forceinline__ float2 rope_cos_sin(const RopePos& pos, int64_t b, int64_t s, int axis, double f) {
  const int64_t o = b * pos.sb + s * pos.ss + axis * pos.sa;
  double v;
  if (pos.type == 0) v = static_cast<double>(__ldg(static_cast<const int*>(pos.p) + o));
  else if (pos.type == 1) v = static_cast<double>(__ldg(static_cast<const long long*>(pos.p) + o));
  else v = static_cast<double>(__ldg(static_cast<const float*>(pos.p) + o));
  const double u = v * f;
  const float turn = static_cast<float>(u - 2.0 * rint(0.5 * u));
  float2 cs;
  sincospif(turn, &cs.y, &cs.x);
  return cs;
}

// VEC elements per piece: a rotating unit of the interleaved form is one piece
// (VEC / 2 pairs), of the split form two pieces (VEC pairs); the scalar unit
// is one pair in both.  Units beyond the rotating ones copy one piece.
template <int DT, int VEC, bool INTER>
__global__ void __launch_bounds__(ROPE_THREADS, ROPE_CTAS) rope_axes_kernel(const __grid_constant__ RopeParams p) {
  using E = typename ElemOf<DT>::type;
  constexpr bool TWO = !INTER || VEC == 1;                   // a unit's pairs span two pieces
  constexpr int NP = TWO ? VEC : VEC / 2;                    // pairs per rotating unit
  constexpr int BYTES = VEC * sizeof(E);
  constexpr int HB = TWO ? (BYTES >= 16 ? 2 : BYTES >= 8 ? 4 : 8) : (BYTES >= 16 ? 4 : BYTES >= 8 ? 8 : 16);  // heads in flight
  __shared__ __align__(16) float cosines[2][ROPE_TOKENS][ROPE_MAX_PAIRS], sines[2][ROPE_TOKENS][ROPE_MAX_PAIRS];
  __shared__ double freq[ROPE_MAX_PAIRS];
  __shared__ uint8_t axis[ROPE_MAX_PAIRS];
  const int pairs = p.plan.pairs;
  if (threadIdx.x < pairs) {  // lanes' own indexes into the parameters replay: once per CTA, not per angle
    freq[threadIdx.x] = p.plan.f[threadIdx.x];
    axis[threadIdx.x] = p.plan.axis[threadIdx.x];
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  auto tokens_of = [&](uint32_t group) {
    const uint32_t first = group * ROPE_TOKENS;
    return first < p.tokens ? static_cast<int>(min(static_cast<uint32_t>(ROPE_TOKENS), p.tokens - first)) : 0;
  };
  auto angles = [&](uint32_t group, int buf) {
    const int n = tokens_of(group);
    for (int i = threadIdx.x; i < n * pairs; i += ROPE_THREADS) {
      const int t = i / pairs, pr = i - t * pairs;
      const uint32_t tok = group * ROPE_TOKENS + t, b = tok / p.S;
      const float2 v = rope_cos_sin(p.pos, b, tok - b * p.S, axis[pr], freq[pr]);
      cosines[buf][t][pr] = v.x;
      sines[buf][t][pr] = v.y * p.sign;
    }
  };

  const int rot = pairs / NP;                                // rotating units
  const int units = rot + (p.pass ? (p.plan.D - 2 * pairs) / VEC : 0);
  const int lanes = ROPE_THREADS / units;
  const int u = threadIdx.x % units;
  const int lane = threadIdx.x / units;                      // >= lanes: helps with the angles only
  const bool turns = u < rot;
  const int step = INTER ? 1 : pairs;                        // from a pair's first element to its second
  const int off = !turns ? 2 * pairs + (u - rot) * VEC : INTER ? u * NP * 2 : u * NP;

  int buf = 0;
  angles(blockIdx.x, 0);
  __syncthreads();
  for (uint32_t group = blockIdx.x; group < p.groups; group += gridDim.x, buf ^= 1) {
    const int nt = tokens_of(group);
    // lanes share out the tokens first, then the heads of a token
    const int per = max(1, lanes / nt);                      // head lanes per token
    bool ahead = true;                                       // the next group's angles are still to do
    for (int t = lane < lanes ? lane / per : nt; t < nt; t += max(1, lanes / per)) {
      const uint32_t tok = group * ROPE_TOKENS + t, b = tok / p.S, s = tok - b * p.S;
      const int h0 = lane % per;
#pragma unroll 1
      for (int w = 0; w < 2; ++w) {                          // Q, K
        const RopeTensor& q = p.t[w];
        const E* x = static_cast<const E*>(q.x) + b * q.xb + s * q.xs + h0 * q.xh + off;
        E* o = static_cast<E*>(q.out) + b * q.ob + s * q.os + h0 * q.oh + off;
        const int64_t dx = per * q.xh, dy = per * q.oh;
#pragma unroll 1
        for (int left = q.heads - h0; left > 0; left -= per * HB) {
          // HB heads' loads go out before the first is used
          Pack<DT, VEC> va[HB], vb[TWO ? HB : 1];
#pragma unroll
          for (int j = 0; j < HB; ++j) {
            if (j * per < left) {
              va[j].load(x);
              if (TWO && turns) vb[TWO ? j : 0].load(x + step);
            }
            x += dx;
          }
          if (ahead) {  // under the first loads
            ahead = false;
            angles(group + gridDim.x, buf ^ 1);
          }
          const float* c = &cosines[buf][t][u * NP];
          const float* sn = &sines[buf][t][u * NP];
#pragma unroll
          for (int j = 0; j < HB; ++j) {
            if (j * per < left) {
              if (turns) {
                if constexpr (VEC == 1) {
                  const float a0 = to_f32<DT>(va[j].e[0]), b0 = to_f32<DT>(vb[j].e[0]);
                  va[j].e[0] = from_f32<DT>(a0 * c[0] - b0 * sn[0]);
                  vb[j].e[0] = from_f32<DT>(a0 * sn[0] + b0 * c[0]);
                } else if constexpr (INTER) {
#pragma unroll
                  for (int i = 0; i < NP; ++i) {
                    const uint64_t v = get2(va[j], i);
                    const float a0 = f2_lo(v), b0 = f2_hi(v);
                    set2(va[j], i, f2_pack(a0 * c[i] - b0 * sn[i], a0 * sn[i] + b0 * c[i]));
                  }
                } else {
#pragma unroll
                  for (int i = 0; i < NP / 2; ++i) {         // two pairs at a time
                    const uint64_t a2 = get2(va[j], i), b2 = get2(vb[j], i);
                    const uint64_t c2 = *reinterpret_cast<const uint64_t*>(c + 2 * i);
                    const uint64_t s2 = *reinterpret_cast<const uint64_t*>(sn + 2 * i);
                    const uint64_t n2 = s2 ^ 0x8000000080000000ull;
                    set2(va[j], i, f2_fma(b2, n2, f2_mul(a2, c2)));
                    set2(vb[j], i, f2_fma(b2, c2, f2_mul(a2, s2)));
                  }
                }
                if (TWO) vb[TWO ? j : 0].store(o + step);
              }
              va[j].store(o);
            }
            o += dy;
          }
        }
      }
    }
    if (ahead) angles(group + gridDim.x, buf ^ 1);
    __syncthreads();
  }
}

struct RopeTableParams {
  RopePlan plan;
  RopePos pos;
  int64_t S, tokens;
  float2* table;                 // [tokens][pairs]
};

// One thread per table entry.  Far from the memory's speed (4608 tokens of 64
// pairs 5.8 us, 16896 18.0 us: 0.4 us and 1.4 us of stores): the lanes' own
// indexes into the parameters replay, and every entry pays two 64-bit
// divisions, the fp64 reduction and the sincospi.
__global__ void __launch_bounds__(ROPE_THREADS) rope_table_kernel(const __grid_constant__ RopeTableParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * ROPE_THREADS + threadIdx.x;
  const int64_t tok = i / p.plan.pairs;
  if (tok >= p.tokens) return;
  const int pr = static_cast<int>(i - tok * p.plan.pairs);
  p.table[i] = rope_cos_sin(p.pos, tok / p.S, tok % p.S, p.plan.axis[pr], p.plan.f[pr]);
}

}  // namespace svdq
