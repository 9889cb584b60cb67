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
// fp32 sincospi.  One CTA computes the angles of its few tokens once into
// shared memory; every thread keeps the (cos, sin) of its own elements in
// registers while it walks over the heads of Q and K, so the fp64 work is paid
// per token and not per head.
//
// Bound by memory: every element is read once and written once, in 16-byte
// pieces where the layout allows (else one pair per thread).
#pragma once

#include "krms8.cuh"

namespace svdq {

constexpr int ROPE_MAX_D = 256;
constexpr int ROPE_MAX_PAIRS = ROPE_MAX_D / 2;
constexpr int ROPE_THREADS = 256;
constexpr int ROPE_TOKENS = 4;   // tokens per CTA

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
  int64_t S, tokens;             // tokens per sequence and in all
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
__global__ void __launch_bounds__(ROPE_THREADS, 4) rope_axes_kernel(const __grid_constant__ RopeParams p) {
  using E = typename ElemOf<DT>::type;
  constexpr bool TWO = !INTER || VEC == 1;                   // a unit's pairs span two pieces
  constexpr int NP = TWO ? VEC : VEC / 2;                    // pairs per rotating unit
  constexpr int HB = TWO ? 2 : 4;
  __shared__ float2 cs[ROPE_TOKENS][ROPE_MAX_PAIRS];
  __shared__ double freq[ROPE_MAX_PAIRS];
  __shared__ uint8_t axis[ROPE_MAX_PAIRS];
  if (threadIdx.x < p.plan.pairs) {  // lanes' own indexes into the parameters replay: once per pair, not per angle
    freq[threadIdx.x] = p.plan.f[threadIdx.x];
    axis[threadIdx.x] = p.plan.axis[threadIdx.x];
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  const int pairs = p.plan.pairs;
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * ROPE_TOKENS;
  const int nt = static_cast<int>(min(static_cast<int64_t>(ROPE_TOKENS), p.tokens - tok0));
  for (int i = threadIdx.x; i < nt * pairs; i += ROPE_THREADS) {
    const int t = i / pairs, pr = i - t * pairs;
    const int64_t tok = tok0 + t;
    float2 v = rope_cos_sin(p.pos, tok / p.S, tok % p.S, axis[pr], freq[pr]);
    v.y *= p.sign;
    cs[t][pr] = v;
  }
  __syncthreads();

  const int rot = pairs / NP;                                // rotating units
  const int units = rot + (p.pass ? (p.plan.D - 2 * pairs) / VEC : 0);
  const int lanes = ROPE_THREADS / units;
  const int u = threadIdx.x % units;
  const int lane = threadIdx.x / units;
  if (lane >= lanes) return;
  // lanes share out the tokens first, then the heads of a token
  const int per = max(1, lanes / nt);                        // head lanes per token
  const int H0 = p.t[0].heads, heads = H0 + p.t[1].heads;
  const bool turns = u < rot;
  const int step = INTER ? 1 : pairs;                        // from a pair's first element to its second
  const int off = !turns ? 2 * pairs + (u - rot) * VEC : INTER ? u * NP * 2 : u * NP;
  for (int t = lane / per; t < nt; t += max(1, lanes / per)) {
    const int64_t tok = tok0 + t, b = tok / p.S, s = tok % p.S;
    const E* x0 = static_cast<const E*>(p.t[0].x) + b * p.t[0].xb + s * p.t[0].xs + off;
    const E* x1 = static_cast<const E*>(p.t[1].x) + b * p.t[1].xb + s * p.t[1].xs + off;
    E* o0 = static_cast<E*>(p.t[0].out) + b * p.t[0].ob + s * p.t[0].os + off;
    E* o1 = static_cast<E*>(p.t[1].out) + b * p.t[1].ob + s * p.t[1].os + off;
    float2 c[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) c[i] = turns ? cs[t][u * NP + i] : make_float2(1.f, 0.f);
    for (int h0 = lane % per; h0 < heads; h0 += per * HB) {
      // HB heads' loads go out before the first is used
      Pack<DT, VEC> va[HB], vb[TWO ? HB : 1];
#pragma unroll
      for (int j = 0; j < HB; ++j) {
        const int hh = h0 + j * per;
        if (hh < heads) {
          const E* x = hh < H0 ? x0 + hh * p.t[0].xh : x1 + (hh - H0) * p.t[1].xh;
          va[j].load(x);
          if (TWO && turns) vb[TWO ? j : 0].load(x + step);
        }
      }
#pragma unroll
      for (int j = 0; j < HB; ++j) {
        const int hh = h0 + j * per;
        if (hh < heads) {
          E* o = hh < H0 ? o0 + hh * p.t[0].oh : o1 + (hh - H0) * p.t[1].oh;
          if (turns) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
              E& ea = TWO ? va[j].e[i] : va[j].e[(2 * i) % VEC];
              E& eb = TWO ? vb[TWO ? j : 0].e[i] : va[j].e[(2 * i + 1) % VEC];
              const float a0 = to_f32<DT>(ea), b0 = to_f32<DT>(eb);
              ea = from_f32<DT>(a0 * c[i].x - b0 * c[i].y);
              eb = from_f32<DT>(a0 * c[i].y + b0 * c[i].x);
            }
            if (TWO) vb[TWO ? j : 0].store(o + step);
          }
          va[j].store(o);
        }
      }
    }
  }
}

struct RopeTableParams {
  RopePlan plan;
  RopePos pos;
  int64_t S, tokens;
  float2* table;                 // [tokens][pairs]
};

// One thread per table entry; bound by the 8-byte stores.
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
