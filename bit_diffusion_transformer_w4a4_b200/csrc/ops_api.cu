// Host side of the operators around the 4-bit layers: the dense linear with a
// fused epilogue, the RMS norm with an 8-bit output and rotary positions with
// several axes.  Argument validation, variant choice and launches; the C
// declarations and their documentation live in include/svdq.h.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <type_traits>
#include <utility>

#include "host_common.cuh"
#include "kdense.cuh"
#include "krms8.cuh"
#include "krope_axes.cuh"

using namespace svdq;

struct svdq_rope {
  RopePlan plan;
  int axes;
};

namespace {

struct DeviceInfo {
  int dev = 0, sms = 0;
};

// check_device() of the current device, asked once per device ordinal.
svdq_status device_info(DeviceInfo* d) {
  static std::atomic<int> known[64];  // SM count of a usable device
  int dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64) {
    if (const int sms = known[dev].load(std::memory_order_acquire); sms > 0) {
      d->dev = dev;
      d->sms = sms;
      return SVDQ_OK;
    }
  } else {
    cudaGetLastError();
  }
  if (svdq_status s = check_device(&d->dev, &d->sms); s != SVDQ_OK) return s;
  if (d->dev < 64) known[d->dev].store(d->sms, std::memory_order_release);
  return SVDQ_OK;
}

// svdq_ops_debug_set_fault of this thread.
struct OpsDebug {
  uint32_t mask = 0;
  uint64_t timeout_ns = kDefaultTimeoutNs;
};
thread_local OpsDebug ops_debug;
constexpr uint32_t kFaultDense = 1, kFaultNorm = 2;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int dtype_size(int t) { return t == SVDQ_FP32 ? 4 : t == SVDQ_BF16 || t == SVDQ_FP16 ? 2 : 1; }

// `rows` rows of `width` bytes, `ld` bytes apart.
struct Region {
  const void* p;
  int64_t rows, width, ld;
  uintptr_t lo() const { return reinterpret_cast<uintptr_t>(p); }
  uintptr_t hi() const { return lo() + static_cast<uintptr_t>((rows - 1) * ld + width); }
};

// Whether two regions share bytes.  Column ranges of one buffer (the same row
// distance) that do not meet are apart although their spans interleave.
bool overlap(const Region& a, const Region& b) {
  if (!a.p || !b.p || a.rows < 1 || b.rows < 1) return false;
  if (a.hi() <= b.lo() || b.hi() <= a.lo()) return false;
  if (a.ld == b.ld && a.ld > 0) {
    const Region& l = a.lo() <= b.lo() ? a : b;
    const Region& h = a.lo() <= b.lo() ? b : a;
    const int64_t o = static_cast<int64_t>((h.lo() - l.lo()) % static_cast<uintptr_t>(a.ld));
    if (l.width <= o && o + h.width <= a.ld) return false;
  }
  return true;
}
bool same(const Region& a, const Region& b) { return a.p == b.p && (a.ld == b.ld || a.rows == 1); }

// ------------------------------------------------------------------ RMS norm
constexpr int kRmsSlots = 2;               // rows of a CTA of the ring form
constexpr int kRmsRingMax = 220 * 1024;    // its shared memory

// call(has weight, INT8) as constants
template <class F>
svdq_status rms_kinds(const RmsParams& p, F call) {
  using std::false_type;
  using std::true_type;
  if (p.w) return p.int8 ? call(true_type{}, true_type{}) : call(true_type{}, false_type{});
  return p.int8 ? call(false_type{}, true_type{}) : call(false_type{}, false_type{});
}

template <int DT, int VEC, int CH>
svdq_status launch_rms_t(const RmsParams& p, int64_t M, int nt, cudaStream_t st) {
  LaunchCfg lc(dim3(static_cast<unsigned>(M)), dim3(nt), 0, st);
  return rms_kinds(p, [&](auto hw, auto i8) -> svdq_status {
    SVDQ_TRY(cudaLaunchKernelEx(&lc.cfg, rms8_kernel<DT, VEC, CH, hw.value, i8.value>, p));
    return SVDQ_OK;
  });
}

template <int DT, int VEC>
svdq_status launch_rms_v(const RmsParams& p, int64_t M, int sms, cudaStream_t st) {
  const int64_t pieces = cdiv(p.K, VEC);
  // pieces a thread: one where a few rows have the device to themselves
  // (latency), else two to four, for loads in flight and fewer warps to join
  const int64_t want = M <= 2 * sms ? 1 : pieces <= 256 ? 2 : 4;
  const int64_t ch = std::max(want, cdiv(pieces, 1024));
  auto threads = [&](int c) { return static_cast<int>(cdiv(cdiv(pieces, c), 32) * 32); };
  if (ch <= 1) return launch_rms_t<DT, VEC, 1>(p, M, threads(1), st);
  if (ch <= 2) return launch_rms_t<DT, VEC, 2>(p, M, threads(2), st);
  if (ch <= 4) return launch_rms_t<DT, VEC, 4>(p, M, threads(4), st);
  if constexpr (VEC <= 4) {
    if (ch <= 8) return launch_rms_t<DT, VEC, 8>(p, M, threads(8), st);
  }
  if constexpr (VEC == 1) {
    if (ch <= 32) return launch_rms_t<DT, VEC, 32>(p, M, threads(32), st);
  }
  return SVDQ_ERR_SHAPE;
}

// Packed rows of any length (see rms8_flat_kernel).
template <int DT, int CH>
svdq_status launch_rms_flat_t(const RmsParams& p, int64_t M, int nt, cudaStream_t st) {
  LaunchCfg lc(dim3(static_cast<unsigned>(M)), dim3(nt), 0, st);
  return rms_kinds(p, [&](auto hw, auto i8) -> svdq_status {
    SVDQ_TRY(cudaLaunchKernelEx(&lc.cfg, rms8_flat_kernel<DT, CH, hw.value, i8.value>, p));
    return SVDQ_OK;
  });
}

template <int DT>
svdq_status launch_rms_flat(const RmsParams& p, int64_t M, int sms, cudaStream_t st) {
  constexpr int V = DT == DT_FP32 ? 4 : 8;
  const int64_t pieces = cdiv(p.K + V - 1, V);  // a row may start inside one
  // pieces a thread: two (8000 x 4001 fp32 85 us, 97 with four; bf16 16000 x 301
  // 22.8, 27.3 with one; 8000 x 2047 36.7, 40.9 with one), but one
  //   where a few rows have the device to themselves (296 x 2047 bf16 3.4 us, 3.9
  //   with two; the other way 296 x 4001, 4.6 and 4.3), and
  //   for 65 to 128 pieces, which two a thread spread over two warps of 33 to 64
  //   threads (16000 x 701 33.5 us, 42.9 with two; 2000 x 851 7.0, 7.9; the other
  //   way from about 97 pieces on with many rows: 16000 x 901 40.2 and 36.1)
  const int64_t want = M <= 2 * sms || (pieces > 64 && pieces <= 128) ? 1 : 2;
  const int64_t ch = std::max(want, cdiv(pieces, 512));
  auto threads = [&](int c) { return static_cast<int>(cdiv(cdiv(pieces, c), 32) * 32); };
  if (ch <= 1) return launch_rms_flat_t<DT, 1>(p, M, threads(1), st);
  if (ch <= 2) return launch_rms_flat_t<DT, 2>(p, M, threads(2), st);
  if (ch <= 4) return launch_rms_flat_t<DT, 4>(p, M, threads(4), st);
  if (ch <= 8) return launch_rms_flat_t<DT, 8>(p, M, threads(8), st);
  return launch_rms_v<DT, 1>(p, M, sms, st);
}

// Many aligned rows (see rms8_ring_kernel).
template <int DT, int CH, bool HW, bool I8>
svdq_status launch_rms_ring_k(const RmsParams& p, int64_t M, int sms, int nt, cudaStream_t st) {
  const int row_bytes = p.K * (DT == DT_FP32 ? 4 : 2);
  const int slot = row_bytes * (p.res ? 2 : 1);
  if (svdq_status s = ensure_smem<rms8_ring_kernel<DT, CH, HW, I8>>(kRmsRingMax); s != SVDQ_OK) return s;
  static std::atomic<int> known{0};  // registers per thread: the same on every device
  int regs = known.load(std::memory_order_relaxed);
  if (regs == 0) {
    cudaFuncAttributes fa;
    SVDQ_TRY(cudaFuncGetAttributes(&fa, rms8_ring_kernel<DT, CH, HW, I8>));
    known.store(regs = std::max(16, fa.numRegs), std::memory_order_relaxed);
  }
  // as many persistent CTAs as are resident at once: by shared memory, by
  // registers (granted per warp in steps of 8 a thread), by threads.  More
  // slots a CTA instead of more CTAs was slower (16896 x 12288: 102 us with two
  // slots, 109 with four)
  const int smem = kRmsSlots * slot;
  const int by_regs = 65536 / (static_cast<int>(cdiv(regs, 8) * 8) * nt);
  const int per_sm = std::max(1, std::min({(227 * 1024) / (smem + 2048), by_regs, 2048 / nt, 32}));
  RmsRing g{M, kRmsSlots, row_bytes, ops_debug.timeout_ns, ops_debug.mask & kFaultNorm ? static_cast<int>(M / 3) : -1};
  LaunchCfg lc(dim3(static_cast<unsigned>(std::min<int64_t>(M, static_cast<int64_t>(sms) * per_sm))), dim3(nt), smem, st);
  SVDQ_TRY(cudaLaunchKernelEx(&lc.cfg, rms8_ring_kernel<DT, CH, HW, I8>, p, g));
  return SVDQ_OK;
}

template <int DT, int CH>
svdq_status launch_rms_ring_t(const RmsParams& p, int64_t M, int sms, int nt, cudaStream_t st) {
  return rms_kinds(p, [&](auto hw, auto i8) { return launch_rms_ring_k<DT, CH, hw.value, i8.value>(p, M, sms, nt, st); });
}

template <int DT>
svdq_status launch_rms_ring(const RmsParams& p, int64_t M, int sms, cudaStream_t st) {
  constexpr int V = DT == DT_FP32 ? 4 : 8;
  const int64_t pieces = p.K / V;
  auto threads = [&](int c) { return static_cast<int>(cdiv(cdiv(pieces, c), 32) * 32); };
  // 16-byte pieces a thread: one for short rows (16384 x 256: 8.0 us, 8.6 with
  // two), two where an SM has few rows and latency counts, else four, which
  // spread a row's fixed cost over fewer warps (4608 x 3072: 19.4 us, 20.2 with one)
  if (threads(1) <= 128) return launch_rms_ring_t<DT, 1>(p, M, sms, threads(1), st);
  if (M <= 4 * sms && threads(2) <= 512) return launch_rms_ring_t<DT, 2>(p, M, sms, threads(2), st);
  return launch_rms_ring_t<DT, 4>(p, M, sms, threads(4), st);
}

template <int DT>
svdq_status launch_rms(const RmsParams& p, int64_t M, int sms, cudaStream_t st) {
  constexpr int V = DT == DT_FP32 ? 4 : 8;
  const bool vec = p.K % V == 0 && aligned16(p.x) && p.ldx % V == 0 && (!p.res || (aligned16(p.res) && p.ldr % V == 0)) &&
                   (!p.h || (aligned16(p.h) && p.ldh % V == 0)) && (!p.w || (aligned16(p.w) && p.ldw % V == 0)) &&
                   aligned(p.codes, V) && p.ldc % V == 0;
  if (!vec) {
    // 5000 x 6001 bf16 with residual: 59 us in shared pieces, 232 element by element
    // (and 40 x 101 1.9 us element by element, 3.1 in pieces)
    const bool flat = p.K >= 32 * V && aligned16(p.x) && aligned16(p.res) && aligned16(p.h) && aligned16(p.w) &&
                      aligned(p.codes, V) && (!p.res || (p.ldr - p.ldx) % V == 0) && (!p.h || (p.ldh - p.ldx) % V == 0) &&
                      (p.ldc - p.ldx) % V == 0 && (!p.w_rows || p.ldw % V == 0);
    return flat ? launch_rms_flat<DT>(p, M, sms, st) : launch_rms_v<DT, 1>(p, M, sms, st);
  }
  const int64_t slot = static_cast<int64_t>(p.K) * (DT == DT_FP32 ? 4 : 2) * (p.res ? 2 : 1);
  // From more than one row an SM on, the ring (4608 x 3072 bf16 with residual:
  // 19.4 us, 22.6 direct; 300 x 3072: 2.9, 3.8 direct; 148 x 3072: 2.4, 2.2 direct)
  if (M > sms && kRmsSlots * slot <= kRmsRingMax && p.K / V <= 4 * 512) return launch_rms_ring<DT>(p, M, sms, st);
  return launch_rms_v<DT, V>(p, M, sms, st);
}

// --------------------------------------------------------------------- rotary
template <int DT, int VEC>
svdq_status launch_rope_v(const RopeParams& p, int sms, cudaStream_t st) {
  LaunchCfg lc(dim3(static_cast<unsigned>(std::min<int64_t>(p.groups, static_cast<int64_t>(sms) * ROPE_CTAS))),
               dim3(ROPE_THREADS), 0, st);
  SVDQ_TRY(p.plan.interleaved ? cudaLaunchKernelEx(&lc.cfg, rope_axes_kernel<DT, VEC, true>, p)
                              : cudaLaunchKernelEx(&lc.cfg, rope_axes_kernel<DT, VEC, false>, p));
  return SVDQ_OK;
}

template <int DT>
svdq_status launch_rope(const RopeParams& p, int sms, cudaStream_t st) {
  // the widest access that every piece of a head starts on (20000 tokens of 20
  // heads of 70, interleaved: 45 us in 4-byte pieces, 76 element by element)
  const int R = 2 * p.plan.pairs;
  const int es = DT == DT_FP32 ? 4 : 2;
  auto fits = [&](int v) {
    bool ok = (p.plan.interleaved ? R : R / 2) % v == 0 && (p.plan.D - R) % v == 0;
    for (const RopeTensor& t : p.t)
      ok = ok && (t.heads == 0 || (aligned(t.x, v * es) && aligned(t.out, v * es) && t.xb % v == 0 && t.xs % v == 0 &&
                                   t.xh % v == 0 && t.ob % v == 0 && t.os % v == 0 && t.oh % v == 0));
    return ok;
  };
  if constexpr (DT != DT_FP32) {
    if (fits(8)) return launch_rope_v<DT, 8>(p, sms, st);
  }
  if (fits(4)) return launch_rope_v<DT, 4>(p, sms, st);
  if (fits(2)) return launch_rope_v<DT, 2>(p, sms, st);
  return launch_rope_v<DT, 1>(p, sms, st);
}

// The bytes of a [B, S, H, D] tensor with strides: its dimensions by rising
// stride, n elements each, and as they come.
struct Nest {
  const void* p;
  int64_t n[3], st[3];  // bytes
  int64_t row;          // bytes of a head
  int64_t dn[3], dst[3];  // B, S, H (1 and 0 where all heads share one address)
  int64_t span(int dims) const {  // of the `dims` innermost dimensions
    int64_t w = row;
    for (int i = 0; i < dims; ++i) w += (n[i] - 1) * st[i];
    return w;
  }
};
Nest nest(const void* p, int64_t B, int64_t S, int64_t H, const int64_t* stride, int64_t D, int es) {
  Nest t{p, {1, 1, 1}, {0, 0, 0}, D * es, {1, 1, 1}, {0, 0, 0}};
  const int64_t n[3] = {B, S, H};
  int64_t order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int64_t a, int64_t b) {
    return std::make_pair(n[a] > 1, stride[a]) < std::make_pair(n[b] > 1, stride[b]);
  });
  for (int i = 0; i < 3; ++i) {
    t.n[i] = n[order[i]];
    t.st[i] = t.n[i] > 1 ? stride[order[i]] * es : 0;
    if (n[i] > 1 && stride[i] > 0) {
      t.dn[i] = n[i];
      t.dst[i] = stride[i] * es;
    }
  }
  return t;
}
// Whether no two heads of the tensor meet.
bool nests(const Nest& t) {
  for (int i = 0; i < 3; ++i)
    if (t.n[i] > 1 && t.st[i] < t.span(i)) return false;
  return true;
}
// Whether heads of two tensors meet whose dimensions have the same strides
// (those of one entry aside).  Of a dimension only the difference of the two
// indexes counts, and of that only the few values that bring what is inside
// the dimension within reach.  Other strides: true.
struct HeadsMeet {
  const Nest &a, &b;
  int64_t st[3];
  int order[3];  // dimensions by rising stride

  HeadsMeet(const Nest& a_, const Nest& b_) : a(a_), b(b_), order{0, 1, 2} {
    for (int i = 0; i < 3; ++i) st[i] = std::max(a.dst[i], b.dst[i]);
    std::sort(order, order + 3, [&](int x, int y) { return st[x] < st[y]; });
  }
  int64_t span(const Nest& t, int dims) const {
    int64_t w = t.row;
    for (int i = 0; i < dims; ++i) w += (t.dn[order[i]] - 1) * t.dst[order[i]];
    return w;
  }
  // delta: bytes from a's start to b's; dims: the dimensions left
  bool operator()(int64_t delta, int dims) const {
    if (delta >= span(a, dims) || -delta >= span(b, dims)) return false;
    if (dims == 0) return true;
    const int d = order[dims - 1];
    if (st[d] == 0) return (*this)(delta, dims - 1);
    if (a.dn[d] > 1 && b.dn[d] > 1 && a.dst[d] != b.dst[d]) return true;
    const int64_t in_a = span(a, dims - 1), in_b = span(b, dims - 1);
    // a's index less b's; the difference from a's entry to b's is delta - e st
    auto floor_div = [](int64_t x, int64_t y) { return x / y - (x % y < 0); };
    const int64_t lo = std::max(floor_div(delta - in_a, st[d]) + 1, 1 - b.dn[d]);
    const int64_t hi = std::min(floor_div(delta + in_b - 1, st[d]), a.dn[d] - 1);
    if (hi - lo >= 8) return true;  // heads of one tensor that overlap themselves
    for (int64_t e = lo; e <= hi; ++e)
      if ((*this)(delta - e * st[d], dims - 1)) return true;
    return false;
  }
};
// Whether two tensors are not known to be apart: neither by their spans, nor by
// the column ranges of their outermost dimension, nor (two outermost dimensions
// that form one) by those of the next, nor head by head.
bool may_meet(const Nest& a, const Nest& b) {
  if (!a.p || !b.p) return false;
  if (!overlap(Region{a.p, a.n[2], a.span(2), a.st[2]}, Region{b.p, b.n[2], b.span(2), b.st[2]})) return false;
  auto merges = [](const Nest& t) { return t.n[2] == 1 || t.st[2] == t.n[1] * t.st[1]; };
  if (merges(a) && merges(b) &&
      !overlap(Region{a.p, a.n[1] * a.n[2], a.span(1), a.st[1]}, Region{b.p, b.n[1] * b.n[2], b.span(1), b.st[1]}))
    return false;
  return HeadsMeet(a, b)(reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p), 3);
}

constexpr int64_t kRopeMaxTokens = 1ll << 31;
constexpr int64_t kRopeMaxSpan = 1ll << 44;  // elements of a dimension's extent

svdq_status rope_pos(const svdq_rope_positions* pos, int64_t B, int64_t S, int axes, RopePos* out, Nest* where) {
  if (!pos) return SVDQ_ERR_INVALID_ARG;
  if (pos->type != SVDQ_POS_INT32 && pos->type != SVDQ_POS_INT64 && pos->type != SVDQ_POS_FP32)
    return SVDQ_ERR_INVALID_ARG;
  if (!pos->p) return SVDQ_ERR_INVALID_ARG;
  if (!aligned(pos->p, pos->type == SVDQ_POS_INT64 ? 8 : 4)) return SVDQ_ERR_ALIGNMENT;
  const int64_t stride[3] = {pos->batch_stride, pos->token_stride, pos->axis_stride}, n[3] = {B, S, axes};
  for (int i = 0; i < 3; ++i)
    if (stride[i] < 0 || (n[i] > 1 && stride[i] > kRopeMaxSpan / n[i])) return SVDQ_ERR_SHAPE;
  *where = nest(pos->p, B, S, axes, stride, 1, pos->type == SVDQ_POS_INT64 ? 8 : 4);
  *out = RopePos{pos->p, static_cast<int>(pos->type), pos->batch_stride, pos->token_stride, pos->axis_stride};
  return SVDQ_OK;
}

// ---------------------------------------------------------------------- dense
// Clusters of two CTAs that fit on the device at once (cached per device,
// stored + 1).
template <int KIND, int OUT, bool TILED>
int dense_pair_clusters(const DeviceInfo& d) {
  static std::atomic<int> cache[64];
  if (d.dev < 0 || d.dev >= 64) return 0;
  if (const int known = cache[d.dev].load(std::memory_order_acquire); known > 0) return known - 1;
  constexpr int smem = DensePairSmem::TOTAL;
  if (ensure_smem<dense_pair_kernel<KIND, OUT, TILED>>(smem) != SVDQ_OK) return 0;
  LaunchCfg lc(dim3(2 * (d.sms / 2)), dim3(DP_THREADS), smem, nullptr, 2);
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, dense_pair_kernel<KIND, OUT, TILED>, &lc.cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;  // not cached: the next call asks again
  }
  cache[d.dev].store(n + 1, std::memory_order_release);
  return n;
}

struct DenseCall {
  const svdq_dense_desc* d;
  DeviceInfo dev;
  DenseParams p;
  cudaStream_t st;
  int64_t lda, ldw;  // bytes
  bool tiled;        // Y and the residual can go through tensor maps
};

// Maps of W and A with boxes of 128 bytes x rows.
template <int KIND, int OUT>
svdq_status dense_maps(const DenseCall& c, int wrows, int arows, CUtensorMap* tw, CUtensorMap* ta) {
  constexpr CUtensorMapDataType dt = KIND != DK_F16 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : OUT == DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  constexpr int es = KIND == DK_F16 ? 2 : 1;
  if (svdq_status s = make_tmap(tw, c.d->w, dt, es, c.d->K, c.d->N, 128 / es, wrows, CU_TENSOR_MAP_SWIZZLE_128B, c.ldw);
      s != SVDQ_OK)
    return s;
  return make_tmap(ta, c.d->a, dt, es, c.d->K, c.d->M, 128 / es, arows, CU_TENSOR_MAP_SWIZZLE_128B, c.lda);
}

template <int KIND, int OUT, bool TILED>
svdq_status launch_dense_pair(DenseCall& c, int split) {
  constexpr int BN = DensePairSmem::BN;
  constexpr int smem = DensePairSmem::TOTAL;
  const int clusters = dense_pair_clusters<KIND, OUT, TILED>(c.dev);
  if (clusters < 1) return SVDQ_ERR_CUDA;
  CUtensorMap tw, ta, ty, tr;
  if (svdq_status s = dense_maps<KIND, OUT>(c, 128, BN / 2, &tw, &ta); s != SVDQ_OK) return s;
  ty = tr = ta;  // not used unless the stores are tiled
  if constexpr (TILED) {
    constexpr CUtensorMapDataType dt = OUT == DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    if (svdq_status s = make_tmap(&ty, c.d->y, dt, 2, c.d->N, c.d->M, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B, 2 * c.d->ldy);
        s != SVDQ_OK)
      return s;
    if (c.d->residual)
      if (svdq_status s = make_tmap(&tr, c.d->residual, dt, 2, c.d->N, c.d->M, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B, 2 * c.d->ldr);
          s != SVDQ_OK)
        return s;
  }
  c.p.num_f = static_cast<int>(cdiv(c.p.N, 256));
  c.p.num_t = static_cast<int>(cdiv(c.p.M, BN));
  const int tiles = c.p.num_f * c.p.num_t;
  c.p.split = split;
  LaunchCfg lc(dim3(split > 1 ? 2 * split * tiles : 2 * std::min(tiles, clusters)), dim3(DP_THREADS), smem, c.st, 2 * split);
  SVDQ_TRY(cudaLaunchKernelEx(&lc.cfg, dense_pair_kernel<KIND, OUT, TILED>, tw, ta, ty, tr, c.p));
  return SVDQ_OK;
}

template <int KIND, int OUT, int BN>
svdq_status launch_dense_solo(DenseCall& c, int split) {
  constexpr int smem = DenseSoloSmem<BN>::TOTAL;
  if (svdq_status s = ensure_smem<dense_solo_kernel<KIND, OUT, BN>>(smem); s != SVDQ_OK) return s;
  CUtensorMap tw, ta;
  if (svdq_status s = dense_maps<KIND, OUT>(c, 128, BN, &tw, &ta); s != SVDQ_OK) return s;
  c.p.num_f = static_cast<int>(cdiv(c.p.N, 128));
  c.p.num_t = static_cast<int>(cdiv(c.p.M, BN));
  c.p.split = split;
  LaunchCfg lc(dim3(static_cast<unsigned>(split) * c.p.num_f * c.p.num_t), dim3(DS_THREADS), smem, c.st, split);
  SVDQ_TRY(cudaLaunchKernelEx(&lc.cfg, dense_solo_kernel<KIND, OUT, BN>, tw, ta, c.p));
  return SVDQ_OK;
}

// The variant of a call: tile size and K split, by the estimated time of each
// in microseconds.  The model is what bounds the kernels: a fixed part, and
// per wave of resident CTAs the K loop, whose block takes as long as the
// latency of its loads over the stages in flight or as the bytes of the CTAs
// that share an SM, whichever is more, plus the store of the tile; a split
// adds its join, and clusters of four and eight leave some SMs without a CTA.
// Its constants are fitted to 493 measured (M, N, K, type) with up to 19
// variants each: the choice is within 2 % of the fastest variant on average
// and within a third at worst.  What is lost by fixed choices: 512 x 2048 ->
// 3072 takes 12.9 us in 128 x 64 tiles, 15.7 on pairs; 4608 x 3072 -> 3072
// 61 on pairs, 80 in 128 x 128 tiles; 1 x 12288 -> 640 9.3 split in eight, 69
// whole; 512 x 6144 -> 3072 25 on pairs split in two, 35 whole.
struct DenseChoice {
  int pair;   // pairs of SMs
  int bn;     // tokens per tile
  int split;  // CTAs or pairs that share a tile's K range
};

DenseChoice dense_choose(int64_t M, int64_t N, int kblk, int sms) {
  const float scale = static_cast<float>(sms) / 148.f;  // of the capacities, measured on 148 SMs
  auto waves = [&](int64_t n, float cap) { return std::ceil(static_cast<float>(n) / std::max(1.f, cap * scale)); };
  DenseChoice best{1, 256, 1};
  float least = INFINITY;
  auto offer = [&](DenseChoice c, float t) {
    if (t < least) {
      least = t;
      best = c;
    }
  };
  const int64_t pairs = cdiv(N, 256) * cdiv(M, 256);
  for (int i = 0, s = 1; s <= 4; ++i, s *= 2) {
    if (s > 1 && 2 * s > kblk) break;
    constexpr float cap[3] = {74.f, 31.f, 15.f}, join[3] = {0.f, 1.4f, 2.9f};
    offer({1, 256, s}, 5.0f + join[i] + waves(pairs, cap[i]) * (static_cast<float>(kblk) / s * 0.32f + 1.25f));
  }
  for (int i = 0, bn = 16; bn <= 128; ++i, bn *= 2) {
    if (i > 0 && bn >= 2 * M) break;
    const int64_t tiles = cdiv(N, 128) * cdiv(M, bn);
    for (int j = 0, s = 1; s <= 8; ++j, s *= 2) {
      if (s > 1 && 2 * s > kblk) break;
      constexpr float latency[4] = {0.167f, 0.205f, 0.217f, 0.341f};  // a k-block, by bn
      constexpr float cap[4] = {246.f, 296.f, 140.f, 127.f}, join[4] = {0.f, 1.4f, 0.9f, 0.7f};
      const float here = std::min(static_cast<float>(tiles * s), cap[j] * scale) / sms;  // CTAs on an SM
      const float block = std::max(latency[i], here * (16384 + bn * 128) / 143000.f);
      offer({0, bn, s}, 4.6f + join[j] + waves(tiles * s, cap[j]) * (static_cast<float>(kblk) / s * block + 0.0106f * bn));
    }
  }
  return best;
}

template <int KIND, int OUT>
svdq_status launch_dense(DenseCall& c) {
  const DenseChoice v = dense_choose(c.p.M, c.p.N, c.p.kblk, c.dev.sms);
  if (v.pair) {
    return c.tiled && v.split == 1 ? launch_dense_pair<KIND, OUT, true>(c, 1) : launch_dense_pair<KIND, OUT, false>(c, v.split);
  }
  switch (v.bn) {
    case 16: return launch_dense_solo<KIND, OUT, 16>(c, v.split);
    case 32: return launch_dense_solo<KIND, OUT, 32>(c, v.split);
    case 64: return launch_dense_solo<KIND, OUT, 64>(c, v.split);
  }
  return launch_dense_solo<KIND, OUT, 128>(c, v.split);
}

}  // namespace

extern "C" {

svdq_status svdq_dense_forward(const svdq_dense_desc* desc, void* stream) {
  if (!desc) return SVDQ_ERR_INVALID_ARG;
  svdq_dense_desc own = *desc;
  const svdq_dense_desc* d = &own;
  const bool wide = d->in == SVDQ_BF16 || d->in == SVDQ_FP16;
  if (!wide && d->in != SVDQ_E4M3 && d->in != SVDQ_INT8) return SVDQ_ERR_INVALID_ARG;
  if (d->out != SVDQ_BF16 && d->out != SVDQ_FP16) return SVDQ_ERR_INVALID_ARG;
  if (wide && d->out != d->in) return SVDQ_ERR_INVALID_ARG;
  if (wide && (d->a_scale || d->w_scale)) return SVDQ_ERR_INVALID_ARG;
  if (d->act != SVDQ_ACT_NONE && d->act != SVDQ_ACT_GELU && d->act != SVDQ_ACT_SILU) return SVDQ_ERR_INVALID_ARG;
  const int64_t M = d->M, N = d->N, K = d->K;
  const int64_t es = wide ? 2 : 1;
  if (M < 0 || M > (1 << 24) || N < 1 || N > (1 << 24) || K < 1 || K > 65536) return SVDQ_ERR_SHAPE;
  if (cdiv(M, 16) * cdiv(N, 128) > (1 << 27)) return SVDQ_ERR_SHAPE;
  constexpr int64_t kLdMax = 1ll << 36;
  if ((d->residual && d->ldr < 0) || (d->gate && (d->gate_rows < 1 || d->ldg < 0))) return SVDQ_ERR_SHAPE;
  // the distance of a single row says nothing
  if (M <= 1) {
    own.lda = K;
    own.ldy = own.ldr = N;
  }
  if (N == 1) own.ldw = K;
  if (d->gate && d->gate_rows >= M) own.ldg = N;
  if ((M > 1 && (d->lda < K || d->ldy < N)) || (N > 1 && d->ldw < K)) return SVDQ_ERR_SHAPE;
  if (d->lda > kLdMax || d->ldw > kLdMax || d->ldy > kLdMax) return SVDQ_ERR_SHAPE;
  if ((d->residual && d->ldr > kLdMax) || (d->gate && d->ldg > kLdMax)) return SVDQ_ERR_SHAPE;
  if (M == 0) return SVDQ_OK;
  if (!d->a || !d->w || !d->y) return SVDQ_ERR_INVALID_ARG;
  // rows that are read through tensor maps start on 16-byte boundaries
  if (!aligned16(d->a) || !aligned16(d->w)) return SVDQ_ERR_ALIGNMENT;
  if ((M > 1 && d->lda * es % 16 != 0) || (N > 1 && d->ldw * es % 16 != 0)) return SVDQ_ERR_ALIGNMENT;
  if (!aligned(d->y, 2) || !aligned(d->bias, 2) || !aligned(d->gate, 2) || !aligned(d->residual, 2) ||
      !aligned(d->a_scale, 4) || !aligned(d->w_scale, 4) || !aligned(d->device_error, 4))
    return SVDQ_ERR_ALIGNMENT;
  const int64_t gates = d->gate ? (M - 1) / d->gate_rows + 1 : 0;
  const Region y{d->y, M, 2 * N, 2 * d->ldy};
  const Region r{d->residual, M, 2 * N, 2 * d->ldr};
  if (overlap(y, Region{d->a, M, K * es, d->lda * es}) || overlap(y, Region{d->w, N, K * es, d->ldw * es}) ||
      overlap(y, Region{d->bias, 1, 2 * N, 2 * N}) || overlap(y, Region{d->gate, gates, 2 * N, 2 * d->ldg}) ||
      overlap(y, Region{d->a_scale, 1, 4 * M, 4 * M}) || overlap(y, Region{d->w_scale, 1, 4 * N, 4 * N}) ||
      (overlap(y, r) && !same(y, r)))
    return SVDQ_ERR_INVALID_ARG;
  for (const Region& t : {y, Region{d->a, M, K * es, d->lda * es}, Region{d->w, N, K * es, d->ldw * es},
                          Region{d->bias, 1, 2 * N, 2 * N}, Region{d->gate, gates, 2 * N, 2 * d->ldg}, r,
                          Region{d->a_scale, 1, 4 * M, 4 * M}, Region{d->w_scale, 1, 4 * N, 4 * N}})
    if (overlap(t, Region{d->device_error, 1, 4, t.ld})) return SVDQ_ERR_INVALID_ARG;
  DenseCall c;
  c.d = d;
  if (svdq_status s = device_info(&c.dev); s != SVDQ_OK) return s;
  c.st = static_cast<cudaStream_t>(stream);
  const int64_t packed = cdiv(K * es, 16) * 16;  // row distance of a single row: any
  c.lda = M > 1 ? d->lda * es : packed;
  c.ldw = N > 1 ? d->ldw * es : packed;
  c.p = DenseParams{};
  c.p.y = static_cast<uint16_t*>(d->y);
  c.p.bias = static_cast<const uint16_t*>(d->bias);
  c.p.gate = static_cast<const uint16_t*>(d->gate);
  c.p.res = static_cast<const uint16_t*>(d->residual);
  c.p.sa = d->a_scale;
  c.p.sw = d->w_scale;
  c.p.ldy = d->ldy;
  c.p.ldr = d->ldr;
  c.p.ldg = d->ldg;
  c.p.gate_rows = static_cast<int>(std::min(d->gate ? d->gate_rows : M, M));
  c.p.M = static_cast<int>(M);
  c.p.N = static_cast<int>(N);
  c.p.kblk = static_cast<int>(cdiv(K * es, 128));
  c.p.act = static_cast<int>(d->act);
  auto rows_by = [&](int64_t n) {  // Y's and the residual's rows start on multiples of n elements
    return aligned(d->y, 2 * n) && (M == 1 || d->ldy % n == 0) &&
           (!d->residual || (aligned(d->residual, 2 * n) && (M == 1 || d->ldr % n == 0)));
  };
  c.p.store = N % 2 == 0 && rows_by(2) ? STORE_PAIRED : STORE_PLAIN;
  // a tensor store writes whole 16-byte pieces of a row, also across the end
  // that its map gives it: N itself a multiple of them too
  c.tiled = M > 1 && N % 8 == 0 && rows_by(8) && (!d->residual || d->ldr > 0);
  c.p.err = d->device_error;
  c.p.timeout_ns = ops_debug.timeout_ns;
  c.p.stuck = (ops_debug.mask & kFaultDense) != 0;
  const bool bf = d->out == SVDQ_BF16;
  if (wide) return bf ? launch_dense<DK_F16, DT_BF16>(c) : launch_dense<DK_F16, DT_FP16>(c);
  if (d->in == SVDQ_E4M3) return bf ? launch_dense<DK_E4M3, DT_BF16>(c) : launch_dense<DK_E4M3, DT_FP16>(c);
  return bf ? launch_dense<DK_INT8, DT_BF16>(c) : launch_dense<DK_INT8, DT_FP16>(c);
}

svdq_status svdq_rms_quantize8(const svdq_rms8_desc* desc, void* stream) {
  if (!desc) return SVDQ_ERR_INVALID_ARG;
  svdq_rms8_desc own = *desc;
  const svdq_rms8_desc* d = &own;
  if (d->in != SVDQ_BF16 && d->in != SVDQ_FP16 && d->in != SVDQ_FP32) return SVDQ_ERR_INVALID_ARG;
  if (d->out != SVDQ_E4M3 && d->out != SVDQ_INT8) return SVDQ_ERR_INVALID_ARG;
  if (d->norm != 0 && d->norm != 1) return SVDQ_ERR_INVALID_ARG;
  if (d->norm && !(d->eps > 0.0f && d->eps < 1.0f)) return SVDQ_ERR_INVALID_ARG;
  const int64_t M = d->M, K = d->K;
  if (M < 0 || M > INT32_MAX || K < 1 || K > 32768) return SVDQ_ERR_SHAPE;
  constexpr int64_t kLdMax = 1ll << 28;
  if (d->ldx < 0 || (d->residual && d->ldr < 0) || (d->weight && (d->weight_rows < 1 || d->ldw < 0))) return SVDQ_ERR_SHAPE;
  // the distance of a single row says nothing
  if (M <= 1) own.ldx = own.ldr = own.ldh = own.ldc = K;
  if (d->weight && d->weight_rows >= M) own.ldw = K;
  if (d->ldx > kLdMax || (d->residual && d->ldr > kLdMax)) return SVDQ_ERR_SHAPE;
  if (M > 1 && (d->ldc < K || (d->h && d->ldh < K))) return SVDQ_ERR_SHAPE;
  if (d->ldc > kLdMax || (d->h && d->ldh > kLdMax)) return SVDQ_ERR_SHAPE;
  if (d->weight && d->ldw > kLdMax) return SVDQ_ERR_SHAPE;
  if (M == 0) return SVDQ_OK;
  if (!d->x || !d->codes || !d->scales) return SVDQ_ERR_INVALID_ARG;
  const int es = dtype_size(d->in);
  if (!aligned(d->x, es) || !aligned(d->residual, es) || !aligned(d->h, es) || !aligned(d->weight, es) ||
      !aligned(d->scales, 4))
    return SVDQ_ERR_ALIGNMENT;
  const Region x{d->x, M, K * es, d->ldx * es}, r{d->residual, M, K * es, d->ldr * es};
  const Region h{d->h, M, K * es, d->ldh * es}, c{d->codes, M, K, d->ldc};
  const Region s{d->scales, 1, 4 * M, 4 * M};
  const Region w{d->weight, d->weight ? (M - 1) / d->weight_rows + 1 : 0, K * es, d->ldw * es};
  if ((overlap(h, x) && !same(h, x)) || (overlap(h, r) && !same(h, r)) || overlap(h, w) || overlap(h, c) ||
      overlap(h, s) || overlap(c, x) || overlap(c, r) || overlap(c, w) || overlap(c, s) || overlap(s, x) ||
      overlap(s, r) || overlap(s, w))
    return SVDQ_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (svdq_status e = device_info(&dev); e != SVDQ_OK) return e;
  RmsParams p{};
  p.x = d->x;
  p.res = d->residual;
  p.h = d->h;
  p.w = d->weight;
  p.codes = static_cast<uint8_t*>(d->codes);
  p.scales = d->scales;
  p.ldx = d->ldx;
  p.ldr = d->ldr;
  p.ldh = d->ldh;
  p.ldw = d->ldw;
  p.ldc = d->ldc;
  p.w_rows = d->weight && d->weight_rows < M ? d->weight_rows : 0;
  p.inv_K = 1.0f / static_cast<float>(K);
  p.K = static_cast<int>(K);
  p.norm = d->norm;
  p.int8 = d->out == SVDQ_INT8;
  p.eps = d->eps;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d->in == SVDQ_BF16) return launch_rms<DT_BF16>(p, M, dev.sms, st);
  if (d->in == SVDQ_FP16) return launch_rms<DT_FP16>(p, M, dev.sms, st);
  return launch_rms<DT_FP32>(p, M, dev.sms, st);
}

svdq_status svdq_ops_device_error_site(void* stream, int* site) {
  if (!site) return SVDQ_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (svdq_status s = device_info(&dev); s != SVDQ_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaStreamCaptureStatus capturing;
  SVDQ_TRY(cudaStreamIsCapturing(st, &capturing));
  if (capturing != cudaStreamCaptureStatusNone) return SVDQ_ERR_INVALID_ARG;
  int seen = 0;
  SVDQ_TRY(cudaMemcpyFromSymbolAsync(&seen, g_ops_err, sizeof(int), 0, cudaMemcpyDeviceToHost, st));
  SVDQ_TRY(cudaStreamSynchronize(st));
  if (seen) {
    const int none = 0;
    SVDQ_TRY(cudaMemcpyToSymbolAsync(g_ops_err, &none, sizeof(int), 0, cudaMemcpyHostToDevice, st));
    SVDQ_TRY(cudaStreamSynchronize(st));
  }
  *site = seen;
  return SVDQ_OK;
}

svdq_status svdq_ops_debug_dense_variant(int64_t M, int64_t N, int64_t K, svdq_dtype in, int sms, int* variant) {
  if (!variant || sms < 1) return SVDQ_ERR_INVALID_ARG;
  if (in != SVDQ_BF16 && in != SVDQ_FP16 && in != SVDQ_E4M3 && in != SVDQ_INT8) return SVDQ_ERR_INVALID_ARG;
  if (M < 1 || M > (1 << 24) || N < 1 || N > (1 << 24) || K < 1 || K > 65536) return SVDQ_ERR_SHAPE;
  const DenseChoice v = dense_choose(M, N, static_cast<int>(cdiv(K * dtype_size(in), 128)), sms);
  variant[0] = v.pair;
  variant[1] = v.bn;
  variant[2] = v.split;
  return SVDQ_OK;
}

svdq_status svdq_ops_debug_set_fault(uint32_t mask, uint32_t timeout_us) {
  if (mask & ~(kFaultDense | kFaultNorm)) return SVDQ_ERR_INVALID_ARG;
  ops_debug.mask = mask;
  ops_debug.timeout_ns = timeout_us ? std::max<uint64_t>(timeout_us, 1000) * 1000ull : kDefaultTimeoutNs;
  return SVDQ_OK;
}

svdq_status svdq_rope_load(const svdq_rope_desc* d, svdq_rope_t* out) {
  if (!d || !out) return SVDQ_ERR_INVALID_ARG;
  *out = nullptr;
  if (d->head_dim < 2 || d->head_dim > ROPE_MAX_D) return SVDQ_ERR_SHAPE;
  if (d->axes < 1 || d->axes > SVDQ_ROPE_MAX_AXES) return SVDQ_ERR_SHAPE;
  int64_t R = 0;
  for (int a = 0; a < d->axes; ++a) {
    if (d->axis_dim[a] < 2 || d->axis_dim[a] % 2 != 0 || d->axis_dim[a] > ROPE_MAX_D) return SVDQ_ERR_SHAPE;
    R += d->axis_dim[a];
  }
  if (R > d->head_dim) return SVDQ_ERR_SHAPE;
  if ((d->interleaved != 0 && d->interleaved != 1) || (d->shared != 0 && d->shared != 1)) return SVDQ_ERR_INVALID_ARG;
  for (int a = 0; a < (d->shared ? 1 : d->axes); ++a)
    if (!(d->theta[a] >= 1.0) || !(d->theta[a] <= 1e30)) return SVDQ_ERR_INVALID_ARG;
  svdq_rope* h = new (std::nothrow) svdq_rope();
  if (!h) return SVDQ_ERR_OOM;
  h->axes = d->axes;
  h->plan.D = static_cast<int>(d->head_dim);
  h->plan.pairs = static_cast<int>(R / 2);
  h->plan.interleaved = d->interleaved;
  int pr = 0;
  for (int a = 0; a < d->axes; ++a)
    for (int i = 0; i < d->axis_dim[a] / 2; ++i, ++pr) {
      const double e = d->shared ? 2.0 * pr / static_cast<double>(R) : 2.0 * i / static_cast<double>(d->axis_dim[a]);
      h->plan.f[pr] = std::pow(d->theta[d->shared ? 0 : a], -e) / 3.14159265358979323846;
      h->plan.axis[pr] = static_cast<uint8_t>(a);
    }
  *out = h;
  return SVDQ_OK;
}

svdq_status svdq_rope_free(svdq_rope_t h) {
  delete h;
  return SVDQ_OK;
}

svdq_status svdq_rope_apply(svdq_rope_t h, svdq_dtype dtype, int64_t B, int64_t S, const svdq_rope_positions* pos,
                            const svdq_rope_tensor* q, const svdq_rope_tensor* k, int inverse, void* stream) {
  if (!h || !q) return SVDQ_ERR_INVALID_ARG;
  if (dtype != SVDQ_BF16 && dtype != SVDQ_FP16 && dtype != SVDQ_FP32) return SVDQ_ERR_INVALID_ARG;
  if (inverse != 0 && inverse != 1) return SVDQ_ERR_INVALID_ARG;
  if (B < 0 || S < 0 || B > kRopeMaxTokens || S > kRopeMaxTokens || (B > 0 && S > kRopeMaxTokens / B)) return SVDQ_ERR_SHAPE;
  const int es = dtype_size(dtype);
  RopeParams p{};
  const svdq_rope_tensor* in[2] = {q, k};
  Nest from[2] = {}, to[2] = {};
  for (int i = 0; i < 2; ++i) {
    if (!in[i]) continue;
    const svdq_rope_tensor& t = *in[i];
    if (t.heads < 0 || t.heads > 65536) return SVDQ_ERR_SHAPE;
    for (int a = 0; a < 3; ++a) {
      const int64_t n = a == 0 ? B : a == 1 ? S : t.heads;
      if (t.stride[a] < 0 || t.out_stride[a] < 0) return SVDQ_ERR_SHAPE;
      if (n > 1 && (t.stride[a] > kRopeMaxSpan / n || t.out_stride[a] > kRopeMaxSpan / n)) return SVDQ_ERR_SHAPE;
    }
    if (t.heads == 0 || B == 0 || S == 0) continue;
    if (!t.x || !t.out) return SVDQ_ERR_INVALID_ARG;
    if (!aligned(t.x, es) || !aligned(t.out, es)) return SVDQ_ERR_ALIGNMENT;
    if (t.x == t.out)
      for (int a = 0; a < 3; ++a)
        if ((a == 0 ? B : a == 1 ? S : t.heads) > 1 && t.stride[a] != t.out_stride[a]) return SVDQ_ERR_INVALID_ARG;
    from[i] = nest(t.x, B, S, t.heads, t.stride, h->plan.D, es);
    to[i] = nest(t.out, B, S, t.heads, t.out_stride, h->plan.D, es);
    if (!nests(to[i])) return SVDQ_ERR_SHAPE;
    if (t.x != t.out && may_meet(from[i], to[i])) return SVDQ_ERR_INVALID_ARG;
    p.t[i] = RopeTensor{t.x, t.out, static_cast<int>(t.heads), t.stride[0], t.stride[1], t.stride[2],
                        t.out_stride[0], t.out_stride[1], t.out_stride[2]};
    if (t.x != t.out && h->plan.D > 2 * h->plan.pairs) p.pass = 1;
  }
  if (may_meet(to[0], to[1]) || may_meet(to[0], from[1]) || may_meet(from[0], to[1])) return SVDQ_ERR_INVALID_ARG;
  if (B == 0 || S == 0 || p.t[0].heads + p.t[1].heads == 0) return SVDQ_OK;
  Nest at;
  if (svdq_status s = rope_pos(pos, B, S, h->axes, &p.pos, &at); s != SVDQ_OK) return s;
  if (may_meet(at, to[0]) || may_meet(at, to[1])) return SVDQ_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (svdq_status s = device_info(&dev); s != SVDQ_OK) return s;
  p.plan = h->plan;
  p.S = static_cast<uint32_t>(S);
  p.tokens = static_cast<uint32_t>(B * S);
  p.groups = static_cast<uint32_t>(cdiv(B * S, ROPE_TOKENS));
  p.sign = inverse ? -1.f : 1.f;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == SVDQ_BF16) return launch_rope<DT_BF16>(p, dev.sms, st);
  if (dtype == SVDQ_FP16) return launch_rope<DT_FP16>(p, dev.sms, st);
  return launch_rope<DT_FP32>(p, dev.sms, st);
}

svdq_status svdq_rope_table(svdq_rope_t h, int64_t B, int64_t S, const svdq_rope_positions* pos, float* table,
                            void* stream) {
  if (!h) return SVDQ_ERR_INVALID_ARG;
  if (B < 0 || S < 0 || B > kRopeMaxTokens || S > kRopeMaxTokens || (B > 0 && S > kRopeMaxTokens / B)) return SVDQ_ERR_SHAPE;
  if (B == 0 || S == 0) return SVDQ_OK;
  if (!table) return SVDQ_ERR_INVALID_ARG;
  if (!aligned(table, 8)) return SVDQ_ERR_ALIGNMENT;
  RopeTableParams p{};
  Nest at;
  if (svdq_status s = rope_pos(pos, B, S, h->axes, &p.pos, &at); s != SVDQ_OK) return s;
  const int64_t bytes = B * S * h->plan.pairs * 8;
  if (overlap(Region{at.p, 1, at.span(3), 0}, Region{table, 1, bytes, 0})) return SVDQ_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (svdq_status s = device_info(&dev); s != SVDQ_OK) return s;
  p.plan = h->plan;
  p.S = S;
  p.tokens = B * S;
  p.table = reinterpret_cast<float2*>(table);
  const int64_t blocks = cdiv(p.tokens * p.plan.pairs, ROPE_THREADS);
  if (blocks > INT32_MAX) return SVDQ_ERR_SHAPE;
  LaunchCfg lc(dim3(static_cast<unsigned>(blocks)), dim3(ROPE_THREADS), 0, static_cast<cudaStream_t>(stream));
  SVDQ_TRY(cudaLaunchKernelEx(&lc.cfg, rope_table_kernel, p));
  return SVDQ_OK;
}

}  // extern "C"
