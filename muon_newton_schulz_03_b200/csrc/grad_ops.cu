// Operators on lists of gradients: the norm of all of them together, the
// clipped copy, and the AdamW update of the tensors that Muon does not take
// (embeddings, heads, norms, biases), which takes the clip multiplier in its
// own pass.
//
// All of them are bound by HBM (2 to 20 operations an element against 2 to
// 32 bytes), so each makes one pass over its tensors in 16-byte accesses. A
// launch covers a whole list: a block works on one unit, `unit` consecutive
// elements of one tensor, and finds its tensor by binary search over the
// units' prefix. The tables of pointers travel as kernel arguments (up to 32
// KB), not through device memory: nothing is uploaded, a captured graph
// holds its own copy, and calls on different streams share nothing. Longer
// lists take several launches.
//
// Sums are held in fp64 and added in a fixed order (unit partials, then one
// tree over them), so results repeat bit for bit.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace muon {

namespace {

constexpr int kThreads = 256;
constexpr int kFinishThreads = 1024;

// Waits for the kernel before this one on the stream (no effect in a normal
// launch), and lets the next one be scheduled while this one drains.
__device__ __forceinline__ void dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dep_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Tensor of a block: unit0[i] <= blk < unit0[i + 1]. Empty tensors have no units.
__device__ __forceinline__ int find_tensor(const int* unit0, int count, int blk) {
  int lo = 0, hi = count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (unit0[mid] <= blk) lo = mid; else hi = mid;
  }
  return lo;
}

// 16-bit and 32-bit element types: values of one 16-byte vector as floats.
template <int kType> struct Elem;
template <> struct Elem<GRAD_F32> {
  typedef float T;
  static constexpr int kVec = 4;
  static __device__ __forceinline__ float get(const void* p, long long i) { return static_cast<const float*>(p)[i]; }
  static __device__ __forceinline__ void unpack(const uint4& r, float* v) {
    v[0] = __uint_as_float(r.x); v[1] = __uint_as_float(r.y); v[2] = __uint_as_float(r.z); v[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ void put(void* p, long long i, float v) { static_cast<float*>(p)[i] = v; }
  static __device__ __forceinline__ uint4 pack(const float* v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};
template <> struct Elem<GRAD_BF16> {
  typedef __nv_bfloat16 T;
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float get(const void* p, long long i) {
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  }
  static __device__ __forceinline__ void unpack(const uint4& r, float* v) {
    const unsigned w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void put(void* p, long long i, float v) {
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  }
  static __device__ __forceinline__ uint4 pack(const float* v) {
    uint4 r;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&r);
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
    return r;
  }
};
template <> struct Elem<GRAD_F16> {
  typedef __half T;
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float get(const void* p, long long i) {
    return __half2float(static_cast<const __half*>(p)[i]);
  }
  static __device__ __forceinline__ void unpack(const uint4& r, float* v) {
    const __half2* h = reinterpret_cast<const __half2*>(&r);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = __half22float2(h[k]);
      v[2 * k] = f.x;
      v[2 * k + 1] = f.y;
    }
  }
  static __device__ __forceinline__ void put(void* p, long long i, float v) {
    static_cast<__half*>(p)[i] = __float2half_rn(v);
  }
  static __device__ __forceinline__ uint4 pack(const float* v) {
    uint4 r;
    __half2* h = reinterpret_cast<__half2*>(&r);
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = __floats2half2_rn(v[2 * k], v[2 * k + 1]);
    return r;
  }
};

// ---------------------------------------------------------------------------
// Norm
// ---------------------------------------------------------------------------

// What a block or a thread carries: a sum of squares in fp64, or the largest
// magnitude as the bits of |g| in fp32 (ordered like the values, NaN above
// infinity, so that a NaN anywhere is the result).
struct SumSq {
  double v;
  static __device__ __forceinline__ SumSq zero() { return SumSq{0.0}; }
  static __device__ __forceinline__ SumSq load(const SumSq* p) { return SumSq{__ldcg(&p->v)}; }
  template <int kType> __device__ __forceinline__ void add(const float* x) {
    if constexpr (kType == GRAD_F32) {
      // fp64 per element: an fp32 square can overflow or vanish.
#pragma unroll
      for (int k = 0; k < 4; ++k) v += (double)x[k] * (double)x[k];
    } else {
      // The products of 16-bit values are exact in fp32; eight of them are
      // added there (at most 7 roundings of 2^-24), unless the sum is so
      // large or small that a square may have left fp32's range.
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) s = fmaf(x[k], x[k], s);
      if (s > 1e-24f && s < 1e30f) {
        v += (double)s;
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v += (double)x[k] * (double)x[k];
      }
    }
  }
  __device__ __forceinline__ void add1(float x) { v += (double)x * (double)x; }
  __device__ __forceinline__ void join(const SumSq& o) { v += o.v; }
  __device__ __forceinline__ SumSq peer(int o) const {
    SumSq r;
    r.v = __shfl_xor_sync(0xffffffffu, v, o);
    return r;
  }
  __device__ __forceinline__ double norm() const { return sqrt(v); }
};
struct MaxAbs {
  unsigned long long v;   // as wide as SumSq: they share the partials' array
  static __device__ __forceinline__ MaxAbs zero() { return MaxAbs{0}; }
  static __device__ __forceinline__ MaxAbs load(const MaxAbs* p) { return MaxAbs{__ldcg(&p->v)}; }
  template <int kType> __device__ __forceinline__ void add(const float* x) {
#pragma unroll
    for (int k = 0; k < Elem<kType>::kVec; ++k) add1(x[k]);
  }
  __device__ __forceinline__ void add1(float x) {
    v = max((unsigned)v, __float_as_uint(x) & 0x7fffffffu);
  }
  __device__ __forceinline__ void join(const MaxAbs& o) { v = max((unsigned)v, (unsigned)o.v); }
  __device__ __forceinline__ MaxAbs peer(int o) const {
    MaxAbs r;
    r.v = __shfl_xor_sync(0xffffffffu, (unsigned)v, o);
    return r;
  }
  __device__ __forceinline__ double norm() const { return (double)__uint_as_float((unsigned)v); }
};

// Sum over the block, valid in thread 0.
template <class Acc, int kBlock>
__device__ __forceinline__ Acc block_join(Acc a) {
  __shared__ Acc red[kBlock / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a.join(a.peer(o));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[warp] = a;
  __syncthreads();
  Acc t = Acc::zero();
  if (warp == 0) {
    if (lane < kBlock / 32) t = red[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t.join(t.peer(o));
  }
  return t;
}

// Elements [e0, e1) of a tensor by kStride threads: scalars up to the first
// 16-byte boundary, then vectors, four in flight per thread, then the rest.
template <class Acc, int kType, int kStride>
__device__ __forceinline__ Acc unit_norm(const void* base, long long e0, long long e1, int tid) {
  typedef Elem<kType> E;
  typedef typename E::T T;
  Acc a = Acc::zero();
  const T* p = static_cast<const T*>(base) + e0;
  const long long n = e1 - e0;
  const int head = (int)min((long long)(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T)), n);
  const long long nv = (n - head) / E::kVec;
  const uint4* q = reinterpret_cast<const uint4*>(p + head);
  long long i = tid;
  for (; i + 3 * kStride < nv; i += 4 * kStride) {
    uint4 r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = q[i + k * kStride];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float x[E::kVec];
      E::unpack(r[k], x);
      a.template add<kType>(x);
    }
  }
  for (; i < nv; i += kStride) {
    float x[E::kVec];
    E::unpack(q[i], x);
    a.template add<kType>(x);
  }
  if (tid < head) a.add1(E::get(p, tid));
  const long long t = head + nv * E::kVec + tid;
  if (t < n) a.add1(E::get(p, t));
  return a;
}

template <class Acc, int kStride>
__device__ __forceinline__ Acc unit_norm(int type, const void* base, long long e0, long long e1, int tid) {
  switch (type) {
    case GRAD_F32: return unit_norm<Acc, GRAD_F32, kStride>(base, e0, e1, tid);
    case GRAD_BF16: return unit_norm<Acc, GRAD_BF16, kStride>(base, e0, e1, tid);
    default: return unit_norm<Acc, GRAD_F16, kStride>(base, e0, e1, tid);
  }
}

template <class Acc, int kCap>
__global__ void __launch_bounds__(kThreads) g1_norm(const __grid_constant__ GradTable<kCap> t, int unit,
                                                    Acc* __restrict__ partials) {
  const int blk = blockIdx.x;
  const int i = find_tensor(t.unit0, t.count, blk);
  const unsigned long long meta = t.meta[i];
  const long long e0 = (long long)(blk - t.unit0[i]) * unit;
  const long long e1 = min(e0 + unit, grad_numel(meta));
  dep_wait();
  dep_release();
  const Acc a = block_join<Acc, kThreads>(unit_norm<Acc, kThreads>(grad_src(meta), t.src[i], e0, e1, threadIdx.x));
  if (threadIdx.x == 0) partials[blk] = a;
}

// min(1, max_norm / (norm + 1e-6)); NaN stays NaN, no bound is 1.
__device__ __forceinline__ float clip_scale(double norm, float max_norm) {
  if (isinf(max_norm)) return 1.0f;
  const double c = (double)max_norm / (norm + 1e-6);
  return c >= 1.0 ? 1.0f : (float)c;
}

// All partials, by one block; valid in thread 0.
template <class Acc, int kBlock>
__device__ __forceinline__ Acc join_partials(const Acc* all, long long nunits) {
  Acc a = Acc::zero();
  long long i = threadIdx.x;
  for (; i + 7 * kBlock < nunits; i += 8 * kBlock) {
    Acc b[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) b[k] = Acc::load(all + i + k * kBlock);
#pragma unroll
    for (int k = 0; k < 8; ++k) a.join(b[k]);
  }
  for (; i < nunits; i += kBlock) a.join(Acc::load(all + i));
  return block_join<Acc, kBlock>(a);
}

// One tensor's norm from its units' partials, by one warp.
template <class Acc>
__device__ __forceinline__ void tensor_norm(const int* unit0, int i, const Acc* partials, float* per_tensor) {
  const int lane = threadIdx.x & 31;
  Acc a = Acc::zero();
  for (int u = unit0[i] + lane; u < unit0[i + 1]; u += 32) a.join(Acc::load(partials + u));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a.join(a.peer(o));
  if (lane == 0) per_tensor[i] = (float)a.norm();
}

// Block 0 (of the launch that has `out`): the norm of everything and its clip
// multiplier. Other blocks: a warp per tensor.
template <class Acc, int kCap>
__global__ void __launch_bounds__(kFinishThreads) g2_finish(const __grid_constant__ SpanTable<kCap> t,
                                                            const Acc* all, long long nunits, float max_norm,
                                                            float* __restrict__ out, const Acc* partials,
                                                            float* __restrict__ per_tensor) {
  dep_wait();
  dep_release();
  if (blockIdx.x == 0) {
    if (out == nullptr) return;
    const Acc a = join_partials<Acc, kFinishThreads>(all, nunits);
    if (threadIdx.x == 0) {
      const double norm = a.norm();
      out[0] = (float)norm;
      out[1] = clip_scale(norm, max_norm);
    }
    return;
  }
  const int i = (int)(blockIdx.x - 1) * (kFinishThreads / 32) + (int)(threadIdx.x >> 5);
  if (i < t.count) tensor_norm(t.unit0, i, partials, per_tensor);
}

// ---------------------------------------------------------------------------
// Clipped copy
// ---------------------------------------------------------------------------

// dst[e0..e1) = s * src, each rounded once to dst's type. `phase` elements
// bring both to a 16-byte boundary at every unit (units are multiples of 8);
// kNoPhase: no such number, so elements go one by one.
template <int kSrc, int kDst, int kStride>
__device__ __forceinline__ void unit_scale(const void* src, void* dst, long long e0, long long e1, int phase, float s,
                                           int tid) {
  typedef Elem<kSrc> S;
  typedef Elem<kDst> D;
  constexpr int kStep = 8;
  long long head = e1 - e0;
  if (phase != kNoPhase) {
    head = min((long long)phase, head);
    const long long nv = (e1 - e0 - head) / kStep;
    const uint4* in = reinterpret_cast<const uint4*>(static_cast<const typename S::T*>(src) + e0 + head);
    uint4* out = reinterpret_cast<uint4*>(static_cast<typename D::T*>(dst) + e0 + head);
    constexpr int kIn = kStep / S::kVec, kOut = kStep / D::kVec;
    for (long long i = tid; i < nv; i += kStride) {
      float x[kStep];
      uint4 r[kIn];
#pragma unroll
      for (int k = 0; k < kIn; ++k) r[k] = __ldcs(in + i * kIn + k);
#pragma unroll
      for (int k = 0; k < kIn; ++k) S::unpack(r[k], x + k * S::kVec);
#pragma unroll
      for (int k = 0; k < kStep; ++k) x[k] *= s;
#pragma unroll
      for (int k = 0; k < kOut; ++k) __stcs(out + i * kOut + k, D::pack(x + k * D::kVec));
    }
    for (long long e = e0 + head + nv * kStep + tid; e < e1; e += kStride) D::put(dst, e, S::get(src, e) * s);
  }
  for (long long e = e0 + tid; e < e0 + head; e += kStride) D::put(dst, e, S::get(src, e) * s);
}

template <int kSrc, int kStride>
__device__ __forceinline__ void unit_scale_to(unsigned long long meta, const void* src, void* dst, long long e0,
                                              long long e1, float s, int tid) {
  const int phase = grad_phase(meta);
  switch (grad_dst(meta)) {
    case GRAD_F32: unit_scale<kSrc, GRAD_F32, kStride>(src, dst, e0, e1, phase, s, tid); break;
    case GRAD_BF16: unit_scale<kSrc, GRAD_BF16, kStride>(src, dst, e0, e1, phase, s, tid); break;
    default: unit_scale<kSrc, GRAD_F16, kStride>(src, dst, e0, e1, phase, s, tid); break;
  }
}

template <int kStride>
__device__ __forceinline__ void unit_scale(unsigned long long meta, const void* src, void* dst, long long e0,
                                           long long e1, float s, int tid) {
  if (s == 1.0f && src == dst) return;   // in place and inside the bound: nothing changes
  switch (grad_src(meta)) {
    case GRAD_F32: unit_scale_to<GRAD_F32, kStride>(meta, src, dst, e0, e1, s, tid); break;
    case GRAD_BF16: unit_scale_to<GRAD_BF16, kStride>(meta, src, dst, e0, e1, s, tid); break;
    default: unit_scale_to<GRAD_F16, kStride>(meta, src, dst, e0, e1, s, tid); break;
  }
}

template <int kCap>
__global__ void __launch_bounds__(kThreads) g3_scale(const __grid_constant__ ScaleTable<kCap> t, int unit,
                                                     const float* __restrict__ scale) {
  // Last unit first: what the norm's pass read last is still in L2.
  const int blk = (int)(gridDim.x - 1 - blockIdx.x);
  const int i = find_tensor(t.unit0, t.count, blk);
  const unsigned long long meta = t.meta[i];
  const long long e0 = (long long)(blk - t.unit0[i]) * unit;
  const long long e1 = min(e0 + unit, grad_numel(meta));
  dep_wait();
  dep_release();
  unit_scale<kThreads>(meta, t.src[i], t.dst[i], e0, e1, __ldcg(scale), threadIdx.x);
}

// ---------------------------------------------------------------------------
// Small lists: norm, and clipped copy, in one kernel on one cluster
// ---------------------------------------------------------------------------

// A small list costs launches, not bytes: here the cluster's barrier takes the
// place of the second and third launch. A warp takes a unit of 1024 elements;
// the partials go through global memory (they stay in L2), and every block
// adds them all, in the same order, to have the multiplier.
constexpr int kSmallBlocks = 8;      // the largest portable cluster
constexpr int kSmallThreads = 1024;

template <class Acc, int kCap, bool kScale>
__global__ void __cluster_dims__(kSmallBlocks, 1, 1) __launch_bounds__(kSmallThreads)
    g5_small(const __grid_constant__ ScaleTable<kCap> t, float max_norm, float* __restrict__ out, Acc* partials,
             float* __restrict__ per_tensor) {
  __shared__ float shared_scale;
  const int lane = threadIdx.x & 31;
  const int warp = (int)(threadIdx.x >> 5) * kSmallBlocks + (int)blockIdx.x;   // over the cluster, blocks in turn
  constexpr int kWarps = kSmallBlocks * kSmallThreads / 32;
  const int nunits = t.unit0[t.count];
  dep_wait();
  dep_release();
  for (int u = warp; u < nunits; u += kWarps) {
    const int i = find_tensor(t.unit0, t.count, u);
    const unsigned long long meta = t.meta[i];
    const long long e0 = (long long)(u - t.unit0[i]) * kGradSmallUnit;
    const long long e1 = min(e0 + kGradSmallUnit, grad_numel(meta));
    Acc a = unit_norm<Acc, 32>(grad_src(meta), t.src[i], e0, e1, lane);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a.join(a.peer(o));
    if (lane == 0) partials[u] = a;
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (kScale || blockIdx.x == 0) {
    const Acc a = join_partials<Acc, kSmallThreads>(partials, nunits);
    if (threadIdx.x == 0) {
      const double norm = a.norm();
      shared_scale = clip_scale(norm, max_norm);
      if (blockIdx.x == 0) {
        out[0] = (float)norm;
        out[1] = shared_scale;
      }
    }
  }
  if (kScale) {
    __syncthreads();
    const float s = shared_scale;
    for (int u = warp; u < nunits; u += kWarps) {
      const int i = find_tensor(t.unit0, t.count, u);
      const unsigned long long meta = t.meta[i];
      const long long e0 = (long long)(u - t.unit0[i]) * kGradSmallUnit;
      const long long e1 = min(e0 + kGradSmallUnit, grad_numel(meta));
      unit_scale<32>(meta, t.src[i], t.dst[i], e0, e1, s, lane);
    }
  } else if (per_tensor != nullptr) {
    for (int i = warp; i < t.count; i += kWarps) tensor_norm(t.unit0, i, partials, per_tensor);
  }
}

// ---------------------------------------------------------------------------
// AdamW
// ---------------------------------------------------------------------------

struct AdamW {
  float decay, b1, omb1, b2, omb2, eps, step_size, rsqrt_bc2, gscale;
  __device__ __forceinline__ void operator()(float& p, float& m, float& v, float g) const {
    g *= gscale;
    m = fmaf(b1, m, omb1 * g);
    v = fmaf(b2, v, omb2 * (g * g));
    const float den = fmaf(sqrtf(v), rsqrt_bc2, eps);
    p = fmaf(p, decay, -step_size * (m / den));
  }
};

template <int kType>
__device__ __forceinline__ void unit_adamw(float* p, const void* g, float* m, float* v, long long e0, long long e1,
                                           int phase, const AdamW& f) {
  typedef Elem<kType> E;
  constexpr int kStep = 8;
  long long head = e1 - e0;
  if (phase != kNoPhase) {
    head = min((long long)phase, head);
    const long long b = e0 + head, nv = (e1 - b) / kStep;
    const uint4* gq = reinterpret_cast<const uint4*>(static_cast<const typename E::T*>(g) + b);
    float4* pq = reinterpret_cast<float4*>(p + b);
    float4* mq = reinterpret_cast<float4*>(m + b);
    float4* vq = reinterpret_cast<float4*>(v + b);
    constexpr int kIn = kStep / E::kVec;
    for (long long i = threadIdx.x; i < nv; i += kThreads) {
      uint4 r[kIn];
      float4 pv[2], mv[2], vv[2];
#pragma unroll
      for (int k = 0; k < kIn; ++k) r[k] = __ldcs(gq + i * kIn + k);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        pv[k] = __ldcs(pq + 2 * i + k);
        mv[k] = __ldcs(mq + 2 * i + k);
        vv[k] = __ldcs(vq + 2 * i + k);
      }
      float x[kStep];
#pragma unroll
      for (int k = 0; k < kIn; ++k) E::unpack(r[k], x + k * E::kVec);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        f(pv[k].x, mv[k].x, vv[k].x, x[4 * k]);
        f(pv[k].y, mv[k].y, vv[k].y, x[4 * k + 1]);
        f(pv[k].z, mv[k].z, vv[k].z, x[4 * k + 2]);
        f(pv[k].w, mv[k].w, vv[k].w, x[4 * k + 3]);
        __stcs(pq + 2 * i + k, pv[k]);
        __stcs(mq + 2 * i + k, mv[k]);
        __stcs(vq + 2 * i + k, vv[k]);
      }
    }
    for (long long e = b + nv * kStep + threadIdx.x; e < e1; e += kThreads) f(p[e], m[e], v[e], E::get(g, e));
  }
  for (long long e = e0 + threadIdx.x; e < e0 + head; e += kThreads) f(p[e], m[e], v[e], E::get(g, e));
}

template <int kCap>
__global__ void __launch_bounds__(kThreads) g4_adamw(const __grid_constant__ AdamTable<kCap> t, int unit,
                                                     const __grid_constant__ AdamArgs a) {
  const int blk = (int)(gridDim.x - 1 - blockIdx.x);   // as g3_scale: what was read last is still in L2
  const int i = find_tensor(t.unit0, t.count, blk);
  const unsigned long long meta = t.meta[i];
  const long long e0 = (long long)(blk - t.unit0[i]) * unit;
  const long long e1 = min(e0 + unit, grad_numel(meta));
  AdamW f{a.decay, a.b1, a.omb1, a.b2, a.omb2, a.eps, a.step_size, a.rsqrt_bc2, 1.0f};
  dep_wait();
  dep_release();
  if (a.grad_scale != nullptr) f.gscale = __ldcg(a.grad_scale);
  if (a.step != nullptr) {
    __shared__ float corr[2];
    if (threadIdx.x == 0) {
      const double k = (double)__ldcg(a.step);
      corr[0] = (float)(a.lr / (1.0 - pow(a.beta1, k)));
      corr[1] = (float)(1.0 / sqrt(1.0 - pow(a.beta2, k)));
    }
    __syncthreads();
    f.step_size = corr[0];
    f.rsqrt_bc2 = corr[1];
  }
  switch (grad_src(meta)) {
    case GRAD_F32: unit_adamw<GRAD_F32>(t.p[i], t.g[i], t.m[i], t.v[i], e0, e1, grad_phase(meta), f); break;
    case GRAD_BF16: unit_adamw<GRAD_BF16>(t.p[i], t.g[i], t.m[i], t.v[i], e0, e1, grad_phase(meta), f); break;
    default: unit_adamw<GRAD_F16>(t.p[i], t.g[i], t.m[i], t.v[i], e0, e1, grad_phase(meta), f); break;
  }
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------

// A launch that may be scheduled while the kernel before it drains (it waits
// for that kernel's end before its first access).
template <class... P, class... A>
cudaError_t launch_dep(void (*kernel)(P...), unsigned grid, unsigned block, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

int esize(int type) { return type == GRAD_F32 ? 4 : 2; }

// Elements (0 to 7) after which every pointer is on a 16-byte boundary, or
// kNoPhase; types[k] is pointer k's element type.
int common_phase(const void* const* ptr, const int* types, int n) {
  int h = 0;
  for (int k = 0; k < n; ++k) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(ptr[k]) / (uintptr_t)esize(types[k]);
    if (types[k] != GRAD_F32) h = (int)(-at & 7);
    else if (h < 4 && k == 0) h = (int)(-at & 3);
  }
  for (int k = 0; k < n; ++k)
    if ((reinterpret_cast<uintptr_t>(ptr[k]) + (uintptr_t)(h * esize(types[k]))) % 16) return kNoPhase;
  return h;
}

template <int kCap>
void fill(ScaleTable<kCap>& t, const GradItem* it, int n, int unit) {
  t.count = n;
  t.unit0[0] = 0;
  for (int i = 0; i < n; ++i) {
    t.src[i] = it[i].src;
    t.dst[i] = it[i].dst;
    const void* ptr[2] = {it[i].src, it[i].dst};
    const int types[2] = {it[i].stype, it[i].dtype};
    t.meta[i] = grad_meta(it[i].numel, it[i].stype, it[i].dtype, common_phase(ptr, types, 2));
    t.unit0[i + 1] = t.unit0[i] + grad_units(it[i].numel, unit);
  }
}

template <class Acc, int kCap>
cudaError_t norm_launch(const GradItem* it, int n, int unit, int units, double* partials, cudaStream_t st) {
  GradTable<kCap> t;
  t.count = n;
  t.unit0[0] = 0;
  for (int i = 0; i < n; ++i) {
    t.src[i] = it[i].src;
    t.meta[i] = grad_meta(it[i].numel, it[i].stype, it[i].dtype, kNoPhase);
    t.unit0[i + 1] = t.unit0[i] + grad_units(it[i].numel, unit);
  }
  return launch_dep(g1_norm<Acc, kCap>, (unsigned)units, kThreads, st, t, unit, reinterpret_cast<Acc*>(partials));
}

template <class Acc, int kCap>
cudaError_t finish_launch(const GradItem* it, int n, int unit, const double* all, long long nunits, float max_norm,
                          float* out, const double* partials, float* per_tensor, cudaStream_t st) {
  SpanTable<kCap> t;
  t.count = n;
  t.unit0[0] = 0;
  for (int i = 0; i < n; ++i) t.unit0[i + 1] = t.unit0[i] + grad_units(it[i].numel, unit);
  const unsigned grid = 1 + (unsigned)((n + kFinishThreads / 32 - 1) / (kFinishThreads / 32));
  return launch_dep(g2_finish<Acc, kCap>, grid, kFinishThreads, st, t, reinterpret_cast<const Acc*>(all), nunits,
                    max_norm, out, reinterpret_cast<const Acc*>(partials), per_tensor);
}

template <int kCap>
cudaError_t scale_launch(const GradItem* it, int n, int unit, int units, const float* scale, cudaStream_t st) {
  ScaleTable<kCap> t;
  fill(t, it, n, unit);
  return launch_dep(g3_scale<kCap>, (unsigned)units, kThreads, st, t, unit, scale);
}

template <class Acc, int kCap>
cudaError_t small_launch(const GradItem* it, int n, bool scale, float max_norm, float* out, float* per_tensor,
                         double* partials, cudaStream_t st) {
  ScaleTable<kCap> t;
  fill(t, it, n, kGradSmallUnit);
  return launch_dep(scale ? g5_small<Acc, kCap, true> : g5_small<Acc, kCap, false>, kSmallBlocks, kSmallThreads, st, t,
                    max_norm, out, reinterpret_cast<Acc*>(partials), per_tensor);
}

template <int kCap>
cudaError_t adamw_launch(const AdamItem* it, int n, int unit, int units, const AdamArgs& a, cudaStream_t st) {
  AdamTable<kCap> t;
  t.count = n;
  t.unit0[0] = 0;
  for (int i = 0; i < n; ++i) {
    t.p[i] = it[i].p;
    t.g[i] = it[i].g;
    t.m[i] = it[i].m;
    t.v[i] = it[i].v;
    const void* ptr[4] = {it[i].p, it[i].m, it[i].v, it[i].g};
    const int types[4] = {GRAD_F32, GRAD_F32, GRAD_F32, it[i].gtype};
    t.meta[i] = grad_meta(it[i].numel, it[i].gtype, GRAD_F32, common_phase(ptr, types, 4));
    t.unit0[i + 1] = t.unit0[i] + grad_units(it[i].numel, unit);
  }
  return launch_dep(g4_adamw<kCap>, (unsigned)units, kThreads, st, t, unit, a);
}

template <class Acc>
cudaError_t norm_for(const GradItem* it, int n, int unit, int units, double* partials, cudaStream_t st) {
  if (n <= kGradCapSmall) return norm_launch<Acc, kGradCapSmall>(it, n, unit, units, partials, st);
  if (n <= kGradCapMid) return norm_launch<Acc, kGradCapMid>(it, n, unit, units, partials, st);
  return norm_launch<Acc, kNormCap>(it, n, unit, units, partials, st);
}

template <class Acc>
cudaError_t finish_for(const GradItem* it, int n, int unit, const double* all, long long nunits, float max_norm,
                       float* out, const double* partials, float* per_tensor, cudaStream_t st) {
  if (!per_tensor) n = 0;
  if (n <= kGradCapSmall)
    return finish_launch<Acc, kGradCapSmall>(it, n, unit, all, nunits, max_norm, out, partials, per_tensor, st);
  return finish_launch<Acc, kNormCap>(it, n, unit, all, nunits, max_norm, out, partials, per_tensor, st);
}

template <class Acc>
cudaError_t small_for(const GradItem* it, int n, bool scale, float max_norm, float* out, float* per_tensor,
                      double* partials, cudaStream_t st) {
  if (n <= kGradCapSmall)
    return small_launch<Acc, kGradCapSmall>(it, n, scale, max_norm, out, per_tensor, partials, st);
  return small_launch<Acc, kGradCapMid>(it, n, scale, max_norm, out, per_tensor, partials, st);
}

}  // namespace

cudaError_t launch_grad_norm(const GradItem* it, int n, int unit, int units, int kind, double* partials,
                             cudaStream_t st) {
  return kind == GRAD_NORM_INF ? norm_for<MaxAbs>(it, n, unit, units, partials, st)
                               : norm_for<SumSq>(it, n, unit, units, partials, st);
}

cudaError_t launch_grad_finish(const GradItem* it, int n, int unit, int kind, const double* all, long long nunits,
                               float max_norm, float* out, const double* partials, float* per_tensor,
                               cudaStream_t st) {
  return kind == GRAD_NORM_INF
             ? finish_for<MaxAbs>(it, n, unit, all, nunits, max_norm, out, partials, per_tensor, st)
             : finish_for<SumSq>(it, n, unit, all, nunits, max_norm, out, partials, per_tensor, st);
}

cudaError_t launch_grad_small(const GradItem* it, int n, int kind, bool scale, float max_norm, float* out,
                              float* per_tensor, double* partials, cudaStream_t st) {
  return kind == GRAD_NORM_INF ? small_for<MaxAbs>(it, n, scale, max_norm, out, per_tensor, partials, st)
                               : small_for<SumSq>(it, n, scale, max_norm, out, per_tensor, partials, st);
}

cudaError_t launch_grad_scale(const GradItem* it, int n, int unit, int units, const float* scale, cudaStream_t st) {
  if (n <= kGradCapSmall) return scale_launch<kGradCapSmall>(it, n, unit, units, scale, st);
  if (n <= kGradCapMid) return scale_launch<kGradCapMid>(it, n, unit, units, scale, st);
  return scale_launch<kScaleCap>(it, n, unit, units, scale, st);
}

cudaError_t launch_adamw(const AdamItem* it, int n, int unit, int units, const AdamArgs& a, cudaStream_t st) {
  if (n <= kGradCapSmall) return adamw_launch<kGradCapSmall>(it, n, unit, units, a, st);
  if (n <= kGradCapMid) return adamw_launch<kGradCapMid>(it, n, unit, units, a, st);
  return adamw_launch<kAdamCap>(it, n, unit, units, a, st);
}

}  // namespace muon
