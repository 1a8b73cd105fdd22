// Operators on lists of gradients: the norm of all of them together, the
// clipped copy, and the AdamW update of the tensors that Muon does not take
// (embeddings, heads, norms, biases), which takes the clip multiplier in its
// own pass.
//
// All of them are bound by HBM (2 to 20 operations an element against 2 to
// 28 bytes), so each makes one pass over its tensors in 32-byte accesses. A
// launch covers a whole list: a block works on one unit, 2^unit consecutive
// elements of one tensor, and finds its tensor through a short index. The
// tables of pointers travel as kernel arguments (up to 32 KB), not through
// device memory: nothing is uploaded, a captured graph holds its own copy,
// and calls on different streams share nothing. Longer lists take several
// launches. Measured rates: norm 7.2 to 7.3 TB/s, clipped copy and AdamW 7.0
// (lists of 1 to 14 GB).
//
// Sums are held in fp64, but for sixteen squares of 16-bit values at a time,
// which are added in fp32 first (see SumSq::Part). The order is fixed (unit
// partials, then one tree over them), so results repeat bit for bit.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace muon {

namespace {

constexpr int kThreads = 256;
constexpr int kFinishThreads = 1024;
constexpr int kClusterBlocks = 8;   // the largest portable cluster

// Waits for the kernel before this one on the stream (no effect in a normal
// launch); lets the next one be scheduled while this one drains. Only kernels
// that another kernel of the same call follows let it. What follows a call's
// last kernel may be one of another library that reads parameters (weights, a
// multiplier) before it waits.
__device__ __forceinline__ void dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dep_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Tensor of a unit: unit0[i] <= u < unit0[i + 1]. Empty tensors have no units.
template <int kCap>
__device__ __forceinline__ int find_tensor(const UnitIndex<kCap>& x, int u) {
  const int k = u >> x.shift;
  int lo = x.tensor_of[k], hi = x.tensor_of[k + 1] + 1;   // a unit of bucket k is in [lo, hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (x.unit0[mid] <= u) lo = mid; else hi = mid;
  }
  return lo;
}

// What a thread moves at once: 32 bytes (one 256-bit access) or 16. Measured on B200, AdamW of 537 M elements: 2.02 ms with
// 32-byte accesses, 2.08 to 2.34 ms with 16-byte ones (lanes 32 bytes apart
// write half sectors; lanes 16 bytes apart need twice the instructions).
template <int kWords>
struct Words {
  unsigned x[kWords];
};
// `once`: the lines may leave L2 first, because nothing reads them again soon.
__device__ __forceinline__ Words<8> load_words(const Words<8>* p, bool once) {
  Words<8> r;
  if (once)
    asm volatile("ld.global.L2::evict_first.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r.x[0]), "=r"(r.x[1]), "=r"(r.x[2]), "=r"(r.x[3]), "=r"(r.x[4]), "=r"(r.x[5]), "=r"(r.x[6]),
                   "=r"(r.x[7])
                 : "l"(p)
                 : "memory");
  else
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r.x[0]), "=r"(r.x[1]), "=r"(r.x[2]), "=r"(r.x[3]), "=r"(r.x[4]), "=r"(r.x[5]), "=r"(r.x[6]),
                   "=r"(r.x[7])
                 : "l"(p)
                 : "memory");
  return r;
}
__device__ __forceinline__ Words<4> load_words(const Words<4>* p, bool once) {
  const uint4* q = reinterpret_cast<const uint4*>(p);
  const uint4 v = once ? __ldcs(q) : *q;
  return Words<4>{{v.x, v.y, v.z, v.w}};
}
__device__ __forceinline__ void store_words(Words<8>* p, const Words<8>& r, bool once) {
  if (once)
    asm volatile("st.global.L2::evict_first.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r.x[0]),
                 "r"(r.x[1]), "r"(r.x[2]), "r"(r.x[3]), "r"(r.x[4]), "r"(r.x[5]), "r"(r.x[6]), "r"(r.x[7])
                 : "memory");
  else
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r.x[0]), "r"(r.x[1]),
                 "r"(r.x[2]), "r"(r.x[3]), "r"(r.x[4]), "r"(r.x[5]), "r"(r.x[6]), "r"(r.x[7])
                 : "memory");
}
__device__ __forceinline__ void store_words(Words<4>* p, const Words<4>& r, bool once) {
  uint4* q = reinterpret_cast<uint4*>(p);
  const uint4 v = make_uint4(r.x[0], r.x[1], r.x[2], r.x[3]);
  if (once) __stcs(q, v); else *q = v;
}

// An element type: one element, and the values of a word.
template <int kType> struct Elem;
template <> struct Elem<GRAD_F32> {
  typedef float T;
  static constexpr int kPerWord = 1;
  static __device__ __forceinline__ float get(const void* p, long long i) { return static_cast<const float*>(p)[i]; }
  static __device__ __forceinline__ void put(void* p, long long i, float v) { static_cast<float*>(p)[i] = v; }
  static __device__ __forceinline__ void unpack(unsigned w, float* v) { v[0] = __uint_as_float(w); }
  static __device__ __forceinline__ unsigned pack(const float* v) { return __float_as_uint(v[0]); }
};
template <> struct Elem<GRAD_BF16> {
  typedef __nv_bfloat16 T;
  static constexpr int kPerWord = 2;
  static __device__ __forceinline__ float get(const void* p, long long i) {
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  }
  static __device__ __forceinline__ void put(void* p, long long i, float v) {
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  }
  static __device__ __forceinline__ void unpack(unsigned w, float* v) {
    v[0] = __uint_as_float(w << 16);
    v[1] = __uint_as_float(w & 0xffff0000u);
  }
  static __device__ __forceinline__ unsigned pack(const float* v) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[0], v[1]);
    return *reinterpret_cast<const unsigned*>(&h);
  }
};
template <> struct Elem<GRAD_F16> {
  typedef __half T;
  static constexpr int kPerWord = 2;
  static __device__ __forceinline__ float get(const void* p, long long i) {
    return __half2float(static_cast<const __half*>(p)[i]);
  }
  static __device__ __forceinline__ void put(void* p, long long i, float v) {
    static_cast<__half*>(p)[i] = __float2half_rn(v);
  }
  static __device__ __forceinline__ void unpack(unsigned w, float* v) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    v[0] = f.x;
    v[1] = f.y;
  }
  static __device__ __forceinline__ unsigned pack(const float* v) {
    const __half2 h = __floats2half2_rn(v[0], v[1]);
    return *reinterpret_cast<const unsigned*>(&h);
  }
};

// kN consecutive elements at p (on a boundary of their size) as floats, and back.
template <int kType, int kN>
__device__ __forceinline__ void load_floats(const void* p, float* v, bool once) {
  constexpr int kPer = Elem<kType>::kPerWord;
  const Words<kN / kPer> r = load_words(static_cast<const Words<kN / kPer>*>(p), once);
#pragma unroll
  for (int k = 0; k < kN / kPer; ++k) Elem<kType>::unpack(r.x[k], v + k * kPer);
}
template <int kType, int kN>
__device__ __forceinline__ void store_floats(void* p, const float* v, bool once) {
  constexpr int kPer = Elem<kType>::kPerWord;
  Words<kN / kPer> r;
#pragma unroll
  for (int k = 0; k < kN / kPer; ++k) r.x[k] = Elem<kType>::pack(v + k * kPer);
  store_words(static_cast<Words<kN / kPer>*>(p), r, once);
}

// ---------------------------------------------------------------------------
// Norm
// ---------------------------------------------------------------------------

// What a block carries: a sum of squares in fp64, or the largest magnitude as
// the bits of |g| in fp32 (ordered like the values, NaN above infinity, so
// that a NaN anywhere is the result). Both are 8 bytes: they share the array
// of partials. Part<kType> is a thread's share of a unit.
struct SumSq {
  double v;
  static __device__ __forceinline__ SumSq zero() { return SumSq{0.0}; }
  static __device__ __forceinline__ SumSq load(const SumSq* p) { return SumSq{__ldcg(&p->v)}; }
  __device__ __forceinline__ unsigned long long bits() const { return (unsigned long long)__double_as_longlong(v); }
  __device__ __forceinline__ void join(const SumSq& o) { v += o.v; }
  __device__ __forceinline__ SumSq peer(int o) const { return SumSq{__shfl_xor_sync(0xffffffffu, v, o)}; }
  __device__ __forceinline__ double norm() const { return sqrt(v); }

  template <int kType>
  struct Part {
    double v = 0.0;
    // 32 bytes. 16-bit values: their products are exact in fp32, where two
    // sums of eight are made, one instruction a value, and joined (at most 8
    // roundings of 2^-24); unless the sum is so large or small that a square
    // may have left fp32's range. The pass is bound by HBM, but a long list
    // of bf16 runs into the board's power limit, so instructions count: 3.5
    // GB took 557 us when each value was first made an fp32 one, at 1.5 GHz.
    __device__ __forceinline__ void add(const Words<8>& r) {
      if constexpr (kType != GRAD_F32) {
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          s0 = square_add(r.x[k], s0);
          s1 = square_add(r.x[k + 1], s1);
        }
        const float s = s0 + s1;
        if (s > 1e-24f && s < 1e30f) {
          v += (double)s;
          return;
        }
        unsigned any = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) any |= r.x[k];
        if ((any & 0x7fff7fffu) == 0) return;   // all zero
      }
      // fp64 per element: an fp32 square can overflow or vanish.
      constexpr int kPer = Elem<kType>::kPerWord;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float x[kPer];
        Elem<kType>::unpack(r.x[k], x);
#pragma unroll
        for (int j = 0; j < kPer; ++j) add1(x[j]);
      }
    }
    static __device__ __forceinline__ float square_add(unsigned w, float s) {
      const unsigned short lo = (unsigned short)w, hi = (unsigned short)(w >> 16);
      if constexpr (kType == GRAD_BF16) {
        asm("fma.rn.f32.bf16 %0, %1, %1, %0;" : "+f"(s) : "h"(lo));
        asm("fma.rn.f32.bf16 %0, %1, %1, %0;" : "+f"(s) : "h"(hi));
      } else {
        asm("fma.rn.f32.f16 %0, %1, %1, %0;" : "+f"(s) : "h"(lo));
        asm("fma.rn.f32.f16 %0, %1, %1, %0;" : "+f"(s) : "h"(hi));
      }
      return s;
    }
    __device__ __forceinline__ void add1(float x) { v += (double)x * (double)x; }
    __device__ __forceinline__ SumSq total() const { return SumSq{v}; }
  };
};
struct MaxAbs {
  unsigned long long v;
  static __device__ __forceinline__ MaxAbs zero() { return MaxAbs{0}; }
  static __device__ __forceinline__ MaxAbs load(const MaxAbs* p) { return MaxAbs{__ldcg(&p->v)}; }
  __device__ __forceinline__ unsigned long long bits() const { return v; }
  __device__ __forceinline__ void join(const MaxAbs& o) { v = max((unsigned)v, (unsigned)o.v); }
  __device__ __forceinline__ MaxAbs peer(int o) const { return MaxAbs{__shfl_xor_sync(0xffffffffu, (unsigned)v, o)}; }
  __device__ __forceinline__ double norm() const { return (double)__uint_as_float((unsigned)v); }

  template <int kType>
  struct Part {
    unsigned wide = 0, pairs = 0;   // bits of |x| in fp32; two 16-bit ones, compared as they are
    __device__ __forceinline__ void add(const Words<8>& r) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (kType == GRAD_F32) wide = max(wide, r.x[k] & 0x7fffffffu);
        else pairs = __vmaxu2(pairs, r.x[k] & 0x7fff7fffu);
      }
    }
    __device__ __forceinline__ void add1(float x) { wide = max(wide, __float_as_uint(x) & 0x7fffffffu); }
    __device__ __forceinline__ MaxAbs total() {
      if constexpr (kType != GRAD_F32) {
        float x[2];
        Elem<kType>::unpack(pairs, x);
        add1(x[0]);
        add1(x[1]);
      }
      return MaxAbs{wide};
    }
  };
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

// Elements [e0, e1) of a tensor by kStride threads: single ones up to the
// first 32-byte boundary, then 32 bytes at a time, two in flight per thread
// (four made blocks wait: 3.5 GB in units of 16 KB took 531 us, two 469), then
// the rest.
template <class Acc, int kType, int kStride>
__device__ __forceinline__ Acc unit_norm(const void* base, long long e0, long long e1, int tid, bool once) {
  typedef Elem<kType> E;
  typedef typename E::T T;
  constexpr int kStep = norm_step(kType);
  typename Acc::template Part<kType> a;
  const T* p = static_cast<const T*>(base) + e0;
  const int n = (int)(e1 - e0);
  const int head = min((int)((-reinterpret_cast<uintptr_t>(p) & 31) / sizeof(T)), n);
  const int nv = (n - head) / kStep;
  const Words<8>* q = reinterpret_cast<const Words<8>*>(p + head);
  int i = tid;
  for (; i + kStride < nv; i += 2 * kStride) {
    Words<8> r[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) r[k] = load_words(q + i + k * kStride, once);
#pragma unroll
    for (int k = 0; k < 2; ++k) a.add(r[k]);
  }
  if (i < nv) a.add(load_words(q + i, once));
  if (tid < head) a.add1(E::get(p, tid));
  const int t = head + nv * kStep + tid;
  if (t < n) a.add1(E::get(p, t));
  return a.total();
}

template <class Acc, int kStride>
__device__ __forceinline__ Acc unit_norm(int type, const void* base, long long e0, long long e1, int tid,
                                         bool once) {
  switch (type) {
    case GRAD_F32: return unit_norm<Acc, GRAD_F32, kStride>(base, e0, e1, tid, once);
    case GRAD_BF16: return unit_norm<Acc, GRAD_BF16, kStride>(base, e0, e1, tid, once);
    default: return unit_norm<Acc, GRAD_F16, kStride>(base, e0, e1, tid, once);
  }
}

// Eight blocks an SM: 3.5 GB of bf16 took 480 us with 30 registers a thread,
// 495 with the 38 that the compiler would take.
template <class Acc, int kCap>
__global__ void __launch_bounds__(kThreads, 8) g1_norm(const __grid_constant__ GradTable<kCap> t, int unit,
                                                       int keep_from, Acc* __restrict__ partials) {
  const int blk = blockIdx.x;
  const int i = find_tensor(t.units, blk);
  const unsigned long long meta = t.meta[i];
  const UnitRange r = unit_range(meta, blk - t.units.unit0[i], unit);
  dep_wait();
  dep_release();
  const Acc a = block_join<Acc, kThreads>(
      unit_norm<Acc, kThreads>(grad_src(meta), t.src[i], r.e0, r.e1, threadIdx.x, blk < keep_from));
  if (threadIdx.x == 0) partials[blk] = a;
}

// min(1, max_norm / (norm + 1e-6)); NaN stays NaN, no bound is 1.
__device__ __forceinline__ float clip_scale(double norm, double max_norm) {
  if (isinf(max_norm)) return 1.0f;
  const double c = max_norm / (norm + 1e-6);
  return c >= 1.0 ? 1.0f : (float)c;
}

// p's address in the shared memory of block `rank` of the cluster, and the
// cluster's barrier.
__device__ __forceinline__ uint32_t peer_shared(const void* p, int rank) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p), r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ void store_peer(uint32_t a, unsigned long long bits) {
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(a), "l"(bits) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

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

// The first cluster (of the launch that has `out`): the norm of everything and
// its clip multiplier. Other blocks: a warp per tensor. 53,000 partials take
// one block 8 us, a cluster of eight 2.
template <class Acc, int kCap>
__global__ void __cluster_dims__(kClusterBlocks, 1, 1) __launch_bounds__(kFinishThreads)
    g2_finish(const __grid_constant__ SpanTable<kCap> t, const Acc* all, long long nunits, double max_norm,
              float* __restrict__ out, const Acc* partials, float* __restrict__ per_tensor, int followed) {
  __shared__ Acc sums[kClusterBlocks];
  dep_wait();
  if (followed) dep_release();
  if (blockIdx.x >= kClusterBlocks) {
    const int i = (int)(blockIdx.x - kClusterBlocks) * (kFinishThreads / 32) + (int)(threadIdx.x >> 5);
    if (i < t.count) tensor_norm(t.unit0, i, partials, per_tensor);
    return;
  }
  if (out == nullptr) return;
  cluster_arrive();   // every block runs before another writes into the first
  constexpr int kAll = kClusterBlocks * kFinishThreads;
  Acc a = Acc::zero();
  long long i = (long long)blockIdx.x * kFinishThreads + threadIdx.x;
  for (; i + 7 * kAll < nunits; i += 8 * kAll) {
    Acc b[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) b[k] = Acc::load(all + i + k * kAll);
#pragma unroll
    for (int k = 0; k < 8; ++k) a.join(b[k]);
  }
  for (; i < nunits; i += kAll) a.join(Acc::load(all + i));
  a = block_join<Acc, kFinishThreads>(a);
  __syncwarp();
  cluster_wait();
  if (threadIdx.x == 0) store_peer(peer_shared(&sums[blockIdx.x], 0), a.bits());
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    Acc s = sums[0];
    for (int k = 1; k < kClusterBlocks; ++k) s.join(sums[k]);
    const double norm = s.norm();
    out[0] = (float)norm;
    out[1] = clip_scale(norm, max_norm);
  }
}

// ---------------------------------------------------------------------------
// Clipped copy
// ---------------------------------------------------------------------------

// dst = s * src over a unit: an fp32 product, rounded to dst's type.
template <int kSrc, int kDst, int kStride>
__device__ __forceinline__ void unit_scale(const void* src, void* dst, const UnitRange& u, float s, int tid,
                                           bool once) {
  typedef Elem<kSrc> S;
  typedef Elem<kDst> D;
  constexpr int kStep = scale_step(kSrc, kDst);
  const long long b = u.e0 + u.head, nv = (u.e1 - b) / kStep;
  const typename S::T* in = static_cast<const typename S::T*>(src) + b;
  typename D::T* out = static_cast<typename D::T*>(dst) + b;
  for (long long i = tid; i < nv; i += kStride) {
    float x[kStep];
    load_floats<kSrc, kStep>(in + i * kStep, x, once);
#pragma unroll
    for (int k = 0; k < kStep; ++k) x[k] *= s;
    store_floats<kDst, kStep>(out + i * kStep, x, once);
  }
  const long long e = b + nv * kStep + tid;
  if (e < u.e1) D::put(dst, e, S::get(src, e) * s);
#pragma unroll 4
  for (long long h = u.e0 + tid; h < b; h += kStride) D::put(dst, h, S::get(src, h) * s);
}

template <int kSrc, int kStride>
__device__ __forceinline__ void unit_scale_to(int dst_type, const void* src, void* dst, const UnitRange& u, float s,
                                              int tid, bool once) {
  switch (dst_type) {
    case GRAD_F32: unit_scale<kSrc, GRAD_F32, kStride>(src, dst, u, s, tid, once); break;
    case GRAD_BF16: unit_scale<kSrc, GRAD_BF16, kStride>(src, dst, u, s, tid, once); break;
    default: unit_scale<kSrc, GRAD_F16, kStride>(src, dst, u, s, tid, once); break;
  }
}

template <int kStride>
__device__ __forceinline__ void unit_scale(unsigned long long meta, const void* src, void* dst, const UnitRange& u,
                                           float s, int tid, bool once) {
  if (s == 1.0f && src == dst) return;   // in place and inside the bound: nothing changes
  switch (grad_src(meta)) {
    case GRAD_F32: unit_scale_to<GRAD_F32, kStride>(grad_dst(meta), src, dst, u, s, tid, once); break;
    case GRAD_BF16: unit_scale_to<GRAD_BF16, kStride>(grad_dst(meta), src, dst, u, s, tid, once); break;
    default: unit_scale_to<GRAD_F16, kStride>(grad_dst(meta), src, dst, u, s, tid, once); break;
  }
}

template <int kCap>
__global__ void __launch_bounds__(kThreads) g3_scale(const __grid_constant__ ScaleTable<kCap> t, int unit, int once,
                                                     const float* __restrict__ scale) {
  // Last unit first: what the norm's pass read last is still in L2.
  const int blk = (int)(gridDim.x - 1 - blockIdx.x);
  const int i = find_tensor(t.units, blk);
  const unsigned long long meta = t.meta[i];
  const UnitRange r = unit_range(meta, blk - t.units.unit0[i], unit);
  dep_wait();
  unit_scale<kThreads>(meta, t.src[i], t.dst[i], r, __ldcg(scale), threadIdx.x, once != 0);
}

// ---------------------------------------------------------------------------
// Small lists: norm, and clipped copy, in one kernel on one cluster
// ---------------------------------------------------------------------------

// A small list costs launches, not bytes: here one cluster does everything,
// and its barrier takes the place of the second and third launch. A warp takes
// a unit of 1024 elements and writes its partial into every block's shared
// memory; after the barrier every block adds them all, in the same order, to
// have the multiplier. A call of 25 fp32 tensors, 2^17 elements: 5.7 us against
// 8.3 (norm), 6.1 against 10.5 (clip into other tensors). Replayed from a graph
// the two or three launches are level (3.7 against 4.1 us, 6.1 against 5.8):
// they overlap. At 2^18 elements the cluster's eight SMs are too few (norm: 5.3
// us against 4.4).
constexpr int kSmallThreads = 1024;
constexpr int kSmallUnits = (int)(kGradSmallNumel >> kGradSmallUnit) + kGradCapLarge;

template <class Acc, int kCap, bool kScale>
__global__ void __cluster_dims__(kClusterBlocks, 1, 1) __launch_bounds__(kSmallThreads)
    g5_small(const __grid_constant__ ScaleTable<kCap> t, double max_norm, float* __restrict__ out,
             float* __restrict__ per_tensor) {
  __shared__ Acc partials[kSmallUnits];
  __shared__ float shared_scale;
  const int lane = threadIdx.x & 31;
  const int warp = (int)(threadIdx.x >> 5) * kClusterBlocks + (int)blockIdx.x;   // over the cluster, blocks in turn
  constexpr int kWarps = kClusterBlocks * kSmallThreads / 32;
  const int nunits = t.units.unit0[t.units.count];
  cluster_arrive();   // every block of the cluster runs before another writes into it
  dep_wait();
  bool started = false;
  for (int u = warp; u < nunits; u += kWarps) {
    const int i = find_tensor(t.units, u);
    const unsigned long long meta = t.meta[i];
    const UnitRange r = unit_range(meta, u - t.units.unit0[i], kGradSmallUnit);
    Acc a = unit_norm<Acc, 32>(grad_src(meta), t.src[i], r.e0, r.e1, lane, false);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a.join(a.peer(o));
    __syncwarp();
    if (!started) cluster_wait();
    started = true;
    if (lane < kClusterBlocks) store_peer(peer_shared(&partials[u], lane), a.bits());
  }
  __syncwarp();
  if (!started) cluster_wait();
  cluster_arrive();
  cluster_wait();
  if (kScale || blockIdx.x == 0) {
    Acc a = Acc::zero();
    for (int u = threadIdx.x; u < nunits; u += kSmallThreads) a.join(partials[u]);
    a = block_join<Acc, kSmallThreads>(a);
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
      const int i = find_tensor(t.units, u);
      const unsigned long long meta = t.meta[i];
      const UnitRange r = unit_range(meta, u - t.units.unit0[i], kGradSmallUnit);
      unit_scale<32>(meta, t.src[i], t.dst[i], r, s, lane, false);
    }
  } else if (per_tensor != nullptr) {
    for (int i = warp; i < t.units.count; i += kWarps) {
      Acc a = Acc::zero();
      for (int u = t.units.unit0[i] + lane; u < t.units.unit0[i + 1]; u += 32) a.join(partials[u]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) a.join(a.peer(o));
      if (lane == 0) per_tensor[i] = (float)a.norm();
    }
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

// A unit: 8 elements at a time, 32 bytes of each fp32 tensor.
template <int kType>
__device__ __forceinline__ void unit_adamw(float* p, const void* g, float* m, float* v, const UnitRange& u,
                                           const AdamW& f, bool once) {
  typedef Elem<kType> E;
  constexpr int kStep = kAdamStep;
  const long long b = u.e0 + u.head, nv = (u.e1 - b) / kStep;
  for (long long i = threadIdx.x; i < nv; i += kThreads) {
    const long long e = b + i * kStep;
    float gx[kStep], px[kStep], mx[kStep], vx[kStep];
    load_floats<kType, kStep>(static_cast<const typename E::T*>(g) + e, gx, once);
    load_floats<GRAD_F32, kStep>(p + e, px, once);
    load_floats<GRAD_F32, kStep>(m + e, mx, once);
    load_floats<GRAD_F32, kStep>(v + e, vx, once);
#pragma unroll
    for (int k = 0; k < kStep; ++k) f(px[k], mx[k], vx[k], gx[k]);
    store_floats<GRAD_F32, kStep>(p + e, px, once);
    store_floats<GRAD_F32, kStep>(m + e, mx, once);
    store_floats<GRAD_F32, kStep>(v + e, vx, once);
  }
  const long long e = b + nv * kStep + threadIdx.x;
  if (e < u.e1) f(p[e], m[e], v[e], E::get(g, e));
#pragma unroll 2
  for (long long h = u.e0 + threadIdx.x; h < b; h += kThreads) f(p[h], m[h], v[h], E::get(g, h));
}

template <int kCap>
__global__ void __launch_bounds__(kThreads) g4_adamw(const __grid_constant__ AdamTable<kCap> t, int unit,
                                                     const __grid_constant__ AdamArgs a) {
  const int blk = (int)(gridDim.x - 1 - blockIdx.x);   // as g3_scale: what was read last is still in L2
  const int i = find_tensor(t.units, blk);
  const unsigned long long meta = t.meta[i];
  const UnitRange r = unit_range(meta, blk - t.units.unit0[i], unit);
  AdamW f{a.decay, a.b1, a.omb1, a.b2, a.omb2, a.eps, a.step_size, a.rsqrt_bc2, 1.0f};
  dep_wait();
  if (a.grad_scale != nullptr) f.gscale = __ldcg(a.grad_scale);
  if (a.step != nullptr) {
    // 1 - beta^t = -expm1(t log beta), by every thread: t log beta is rounded
    // once and expm1f is off by an ulp, so the corrections are off by 3 and
    // 1.5 roundings, the factors made of them by 5 and 3.5. (One thread's pow
    // in fp64 held its block up: 2.09 ms for 537 M elements, 2.01 without.)
    const double t = (double)__ldcg(a.step);
    f.step_size = a.lr / -expm1f((float)(t * a.log_beta1));
    f.rsqrt_bc2 = 1.0f / sqrtf(-expm1f((float)(t * a.log_beta2)));
  }
  switch (grad_src(meta)) {
    case GRAD_F32: unit_adamw<GRAD_F32>(t.p[i], t.g[i], t.m[i], t.v[i], r, f, a.once != 0); break;
    case GRAD_BF16: unit_adamw<GRAD_BF16>(t.p[i], t.g[i], t.m[i], t.v[i], r, f, a.once != 0); break;
    default: unit_adamw<GRAD_F16>(t.p[i], t.g[i], t.m[i], t.v[i], r, f, a.once != 0); break;
  }
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------

// A launch that may be scheduled while the kernel before it drains (it waits
// for that kernel's end before its first access). The arguments are of the
// kernel's own types, so that the tables are not copied on the way.
template <class... P, class... A>
cudaError_t launch_dep(void (*kernel)(P...), unsigned grid, unsigned block, cudaStream_t st, const A&... args) {
  static_assert((std::is_same<typename std::remove_const<P>::type, A>::value && ...), "arguments of the kernel's types");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  void* ptr[] = {const_cast<void*>(static_cast<const void*>(&args))...};
  return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kernel), ptr);
}

// Index of n tensors; units(i) is the number of tensor i's units.
template <int kCap, class Units>
void fill_index(UnitIndex<kCap>& x, int n, Units units) {
  x.count = (unsigned short)n;
  x.unit0[0] = 0;
  for (int i = 0; i < n; ++i) x.unit0[i + 1] = x.unit0[i] + units(i);
  const int total = x.unit0[n];
  x.shift = 0;
  if (total == 0) return;   // nothing will look anything up
  while ((total - 1) >> x.shift >= kBuckets) ++x.shift;
  const int end = ((total - 1) >> x.shift) + 1;   // buckets in use
  int k = 0;
  for (int i = 0; i < n; ++i)
    for (; k < end && (long long)k << x.shift < x.unit0[i + 1]; ++k) x.tensor_of[k] = (unsigned short)i;
  x.tensor_of[end] = (unsigned short)(n - 1);
}

template <int kCap>
void fill(ScaleTable<kCap>& t, const GradItem* it, int n, int unit) {
  for (int i = 0; i < n; ++i) {
    t.src[i] = it[i].src;
    t.dst[i] = it[i].dst;
    t.meta[i] = grad_meta(it[i].numel, it[i].stype, it[i].dtype, it[i].scale_phase);
  }
  fill_index(t.units, n, [&](int i) { return grad_units(it[i].numel, it[i].scale_phase, unit); });
}

template <class Acc, int kCap>
cudaError_t norm_launch(const GradItem* it, int n, int unit, int keep, double* partials, cudaStream_t st, int* units) {
  GradTable<kCap> t;
  for (int i = 0; i < n; ++i) {
    t.src[i] = it[i].src;
    t.meta[i] = grad_meta(it[i].numel, it[i].stype, it[i].dtype, it[i].norm_phase);
  }
  fill_index(t.units, n, [&](int i) { return grad_units(it[i].numel, it[i].norm_phase, unit); });
  *units = t.units.unit0[n];
  if (*units == 0) return cudaSuccess;
  return launch_dep(g1_norm<Acc, kCap>, (unsigned)*units, kThreads, st, t, unit, *units - keep,
                    reinterpret_cast<Acc*>(partials));
}

template <class Acc, int kCap>
cudaError_t finish_launch(const GradItem* it, int n, int unit, const double* all, long long nunits, double max_norm,
                          float* out, const double* partials, float* per_tensor, int followed, cudaStream_t st) {
  SpanTable<kCap> t;
  t.count = n;
  t.unit0[0] = 0;
  for (int i = 0; i < n; ++i) t.unit0[i + 1] = t.unit0[i] + grad_units(it[i].numel, it[i].norm_phase, unit);
  const int per_block = kFinishThreads / 32, per_cluster = per_block * kClusterBlocks;
  const unsigned grid = (unsigned)(kClusterBlocks * (1 + (n + per_cluster - 1) / per_cluster));
  return launch_dep(g2_finish<Acc, kCap>, grid, kFinishThreads, st, t, reinterpret_cast<const Acc*>(all), nunits,
                    max_norm, out, reinterpret_cast<const Acc*>(partials), per_tensor, followed);
}

template <int kCap>
cudaError_t scale_launch(const GradItem* it, int n, int unit, int once, const float* scale, cudaStream_t st,
                         int* units) {
  ScaleTable<kCap> t;
  fill(t, it, n, unit);
  *units = t.units.unit0[n];
  if (*units == 0) return cudaSuccess;
  return launch_dep(g3_scale<kCap>, (unsigned)*units, kThreads, st, t, unit, once, scale);
}

template <class Acc, int kCap>
cudaError_t small_launch(const GradItem* it, int n, bool scale, double max_norm, float* out,
                         float* per_tensor, cudaStream_t st) {
  ScaleTable<kCap> t;
  fill(t, it, n, kGradSmallUnit);
  return launch_dep(scale ? g5_small<Acc, kCap, true> : g5_small<Acc, kCap, false>, kClusterBlocks, kSmallThreads, st, t,
                    max_norm, out, per_tensor);
}

template <int kCap>
cudaError_t adamw_launch(const AdamItem* it, int n, int unit, const AdamArgs& a, cudaStream_t st) {
  AdamTable<kCap> t;
  for (int i = 0; i < n; ++i) {
    t.p[i] = it[i].p;
    t.g[i] = it[i].g;
    t.m[i] = it[i].m;
    t.v[i] = it[i].v;
    t.meta[i] = grad_meta(it[i].numel, it[i].gtype, GRAD_F32, it[i].phase);
  }
  fill_index(t.units, n, [&](int i) { return grad_units(it[i].numel, it[i].phase, unit); });
  return launch_dep(g4_adamw<kCap>, (unsigned)t.units.unit0[n], kThreads, st, t, unit, a);
}

template <class Acc>
cudaError_t norm_for(const GradItem* it, int n, int unit, int keep, double* partials, cudaStream_t st, int* units) {
  if (n <= kGradCapSmall) return norm_launch<Acc, kGradCapSmall>(it, n, unit, keep, partials, st, units);
  if (n <= kGradCapMid) return norm_launch<Acc, kGradCapMid>(it, n, unit, keep, partials, st, units);
  if (n <= kGradCapLarge) return norm_launch<Acc, kGradCapLarge>(it, n, unit, keep, partials, st, units);
  return norm_launch<Acc, kNormCap>(it, n, unit, keep, partials, st, units);
}

template <class Acc>
cudaError_t finish_for(const GradItem* it, int n, int unit, const double* all, long long nunits, double max_norm,
                       float* out, const double* partials, float* per_tensor, int followed, cudaStream_t st) {
  if (!per_tensor) n = 0;
  const auto launch = n <= kGradCapSmall   ? finish_launch<Acc, kGradCapSmall>
                      : n <= kGradCapLarge ? finish_launch<Acc, kGradCapLarge>
                                           : finish_launch<Acc, kNormCap>;
  return launch(it, n, unit, all, nunits, max_norm, out, partials, per_tensor, followed, st);
}

template <class Acc>
cudaError_t small_for(const GradItem* it, int n, bool scale, double max_norm, float* out,
                      float* per_tensor, cudaStream_t st) {
  if (n <= kGradCapSmall) return small_launch<Acc, kGradCapSmall>(it, n, scale, max_norm, out, per_tensor, st);
  if (n <= kGradCapMid) return small_launch<Acc, kGradCapMid>(it, n, scale, max_norm, out, per_tensor, st);
  return small_launch<Acc, kGradCapLarge>(it, n, scale, max_norm, out, per_tensor, st);
}

}  // namespace

cudaError_t launch_grad_norm(const GradItem* it, int n, int unit, int keep, int kind, double* partials,
                             cudaStream_t st, int* units) {
  return kind == GRAD_NORM_INF ? norm_for<MaxAbs>(it, n, unit, keep, partials, st, units)
                               : norm_for<SumSq>(it, n, unit, keep, partials, st, units);
}

cudaError_t launch_grad_finish(const GradItem* it, int n, int unit, int kind, const double* all, long long nunits,
                               double max_norm, float* out, const double* partials, float* per_tensor,
                               bool followed, cudaStream_t st) {
  return kind == GRAD_NORM_INF
             ? finish_for<MaxAbs>(it, n, unit, all, nunits, max_norm, out, partials, per_tensor, followed, st)
             : finish_for<SumSq>(it, n, unit, all, nunits, max_norm, out, partials, per_tensor, followed, st);
}

cudaError_t launch_grad_small(const GradItem* it, int n, int kind, bool scale, double max_norm,
                              float* out, float* per_tensor, cudaStream_t st) {
  return kind == GRAD_NORM_INF ? small_for<MaxAbs>(it, n, scale, max_norm, out, per_tensor, st)
                               : small_for<SumSq>(it, n, scale, max_norm, out, per_tensor, st);
}

cudaError_t launch_grad_scale(const GradItem* it, int n, int unit, int once, const float* scale, cudaStream_t st,
                              int* units) {
  if (n <= kGradCapSmall) return scale_launch<kGradCapSmall>(it, n, unit, once, scale, st, units);
  if (n <= kGradCapMid) return scale_launch<kGradCapMid>(it, n, unit, once, scale, st, units);
  if (n <= kGradCapLarge) return scale_launch<kGradCapLarge>(it, n, unit, once, scale, st, units);
  return scale_launch<kScaleCap>(it, n, unit, once, scale, st, units);
}

cudaError_t launch_adamw(const AdamItem* it, int n, int unit, const AdamArgs& a, cudaStream_t st) {
  if (n <= kGradCapSmall) return adamw_launch<kGradCapSmall>(it, n, unit, a, st);
  if (n <= kGradCapMid) return adamw_launch<kGradCapMid>(it, n, unit, a, st);
  if (n <= kGradCapLarge) return adamw_launch<kGradCapLarge>(it, n, unit, a, st);
  return adamw_launch<kAdamCap>(it, n, unit, a, st);
}

}  // namespace muon
