// Host-side launch interfaces of the CUDA kernels (internal to the library).
#pragma once

#include <cstdint>
#include <string>
#include <cuda_runtime.h>

#include "common.cuh"

namespace muon {

// Grouped elementwise launch: one block per chunk of kElemChunk elements.
struct ElemLaunch {
  const MatPlan* plans = nullptr;     // device
  const MatBind* binds = nullptr;     // device
  const long long* prefix = nullptr;  // device, count + 1 entries
  int count = 0;
  long long block_base = 0;           // first chunk of the launch (0 for a whole set)
  long long nblocks = 0;              // chunks in the launch (prefix[count] for a whole set)
};

// partials == nullptr: one double atomic per block into sumsq; else each
// block stores its partial at partials[block] and launch_reduce_partials
// adds them per matrix in a fixed order (bitwise reproducible norms).
// grad_scale (device, or NULL = 1) multiplies every gradient as it is read.
cudaError_t launch_momentum_norm(const ElemLaunch& L, int ysel, float beta, int nesterov, double* sumsq,
                                 double* partials, DevStatus* status, int check_nonfinite, bool fp32_out,
                                 const float* grad_scale, cudaStream_t st);
cudaError_t launch_reduce_partials(const ElemLaunch& L, int m0, int m1, const double* partials, double* sumsq,
                                   cudaStream_t st);
cudaError_t launch_apply(const ElemLaunch& L, int osel, float lr, float wd, int scale_mode, float extra_scale,
                         const double* sumsq, bool fp32_in, cudaStream_t st);
// QK-Clip: rows of head h scaled by sqrt(tau / s_max[h]) when s_max[h] > tau.
cudaError_t launch_qk_clip(float* w, long long rows, long long cols, int head_rows, const float* s_max, float tau,
                           cudaStream_t st);

cudaError_t launch_scale_copy(const ElemLaunch& L, int isel, int osel, const double* sumsq, bool fp32,
                              cudaStream_t st);

// Newton-Schulz phases. PHASE_SYM is the product of two symmetric s x s
// buffers used by the Gram form of the iteration.
enum NsPhase : int { PHASE_GRAM = 0, PHASE_POLY = 1, PHASE_COMB = 2, PHASE_SYM = 3 };

// The s x s buffers of a matrix: the Gram A and polynomial B of the plan,
// and T and B1, used only by the Gram form.
enum SymBuf : int { SB_A = 0, SB_B = 1, SB_T = 2, SB_B1 = 3, SB_NONE = -1 };

struct GramBufs {
  void* t;
  void* b1;
};
// T (K-major 128- and 256-row boxes), B1 (same), then the 32 x 32 store
// boxes of T and B1.
// Gram-form maps per matrix: T K128, T K256, B1 K128, B1 K256, T store,
// B1 store, T 64 x 64 (M/N-major loads), B1 64 x 64.
constexpr int kGramMapsPerMat = 8;

// Operands and epilogue of one launch beyond the phase itself.
struct PhaseSpec {
  int poly_out = SB_B;                 // POLY: where B = aI + bA + cA^2 goes (a = 0 in the Gram form)
  int sym_l = SB_A, sym_r = SB_A;      // SYM: D = L R (both symmetric)
  int sym_out = SB_T;
  int aux1 = SB_NONE, aux2 = SB_NONE;  // SYM: out = D + e1 aux1 + e2 aux2
  float e1 = 0.0f, e2 = 0.0f;
  int comb_b = SB_B;                   // COMB: left operand (SB_B or SB_T)
};

// Tensor maps of one matrix (bf16 path). Each CUtensorMap is 128 bytes and
// must be 64-byte aligned in global memory.
struct alignas(64) TmapBlob {
  unsigned char bytes[128];
};
// Index of each map inside a matrix's block of kMapsPerMat maps.
// X-buffer maps come in triples (K-major 128-row box, K-major 256-row box,
// MN-major 64x64 box): X0 at 0, X1 at 3. A caller input buffer has its own
// triple per matrix in a separate table.
enum MapIdx : int {
  MAP_X0 = 0, MAP_X1 = 3,
  MAP_K128 = 0, MAP_K256 = 1, MAP_MN = 2,   // offsets inside a triple
  MAP_A_K128 = 6, MAP_A_K256 = 7,
  MAP_B_K128 = 8, MAP_B_K256 = 9,
  // 32 x 32 boxes with 64-byte swizzle for the epilogue's bulk stores
  MAP_X0_ST = 10, MAP_X1_ST = 11, MAP_A_ST = 12, MAP_B_ST = 13,
  // 64 x 64 boxes of A and B for M/N-major loads: the single-CTA kernel
  // writes only the upper 256-block triangle of a symmetric buffer and reads
  // the blocks below it transposed from there
  MAP_A_MN = 14, MAP_B_MN = 15,
  kMapsPerMat = 16,
  kInMapsPerMat = 3
};

// The parameter update p' = p (1 - lr wd) - lr scale O taken into the last
// combine's epilogue: O (rounded to bf16, as the separate apply pass reads
// it) is not stored; 32 x 32 blocks of p are bulk-loaded into shared memory,
// updated there and bulk-stored back through `p_maps` of the launch.
struct ApplyArgs {
  int on = 0;
  float lr = 0.0f, wd = 0.0f;
  int scale_mode = 0;
  float extra_scale = 1.0f;
};

struct NsLaunch {
  const MatPlan* plans = nullptr;     // device
  const MatBind* binds = nullptr;     // device
  const TmapBlob* maps = nullptr;     // device, kMapsPerMat per matrix (workspace)
  const TmapBlob* in_maps = nullptr;  // device, kInMapsPerMat per matrix (caller input) or NULL
  const int4* tiles = nullptr;        // device tile list of the phase
  int ntiles = 0;
  const double* sumsq = nullptr;      // device or NULL
  DevStatus* status = nullptr;        // device
  int grid = 0;                       // persistent CTAs
  unsigned long long timeout_ns = 0;
  const TmapBlob* gmaps = nullptr;   // device, kGramMapsPerMat per matrix (Gram form only)
  int tma_store = 0;                 // 1: the *_ST store maps are present, stage outputs
                                     //    in shared memory and write them with bulk stores
  const GramBufs* gbufs = nullptr;   // device, one per matrix (Gram form only)
  int max_s = 1 << 30;               // largest s = min(m, n) of the listed matrices, or an
                                     // upper bound (the polynomial's identity form needs < 2048)
  ApplyArgs apply;                   // COMB only: update p instead of storing O
  const TmapBlob* p_maps = nullptr;  // device, one fp32 32 x 32 map of p per matrix (apply only)
};

// Small-matrix path: one CTA per listed matrix runs every iteration on chip.
struct NsSmallLaunch {
  const MatPlan* plans;      // device
  const MatBind* binds;      // device
  const TmapBlob* maps;      // device, kMapsPerMat per matrix
  const TmapBlob* in_maps;   // device, kInMapsPerMat per matrix or NULL
  const int* mats;           // device list of matrix indices
  int nmats;
  const double* sumsq;       // device or NULL
  DevStatus* status;         // device
  unsigned long long timeout_ns;
  int max_l = 1 << 30;       // largest max(m, n) of the listed matrices (<= 128: compact kernel)
};

// abc: ns_steps rows of (a, b, c).
cudaError_t launch_ns_small(const NsSmallLaunch& L, int ns_steps, int src_sel, int final_sel, const float* abc,
                            cudaStream_t st);
int ns_small_smem_bytes();

cudaError_t launch_ns_phase_pair(const NsLaunch& L, int phase, int src_sel, int dst_sel, int first, float a,
                                 float b, float c, cudaStream_t st);
int ns_pair_smem_bytes();
int ns_pair_clusters_resident();

cudaError_t launch_ns_phase_bf16(const NsLaunch& L, int phase, int src_sel, int dst_sel, int first, float a,
                                 float b, float c, cudaStream_t st, const PhaseSpec& spec = PhaseSpec());

// fp32 debug Newton-Schulz: one launch per matrix and phase.
cudaError_t launch_ns_phase_fp32(const MatPlan& mp_host, int mat, int phase, const float* src, float* dst,
                                 const double* sumsq, int first, float a, float b, float c, cudaStream_t st);

int ns_bf16_smem_bytes();

// ---------------------------------------------------------------------------
// Operators on lists of gradients (grad_ops.cu)
// ---------------------------------------------------------------------------

enum GradType : int { GRAD_F32 = 0, GRAD_BF16 = 1, GRAD_F16 = 2 };   // muon_dtype
enum GradNorm : int { GRAD_NORM_L2 = 0, GRAD_NORM_INF = 1 };         // muon_norm_kind

// One tensor of a list: numel = 0 for a skipped one. The phase is the number
// of elements after which every pointer is on the boundary of the kernels'
// accesses, kNoPhase if there is none.
struct GradItem {
  const void* src;
  void* dst;          // clipped copy only
  long long numel;
  int stype, dtype;
  int norm_phase, scale_phase;   // of src alone; of src and dst
};
struct AdamItem {
  float* p;
  const void* g;
  float* m;
  float* v;
  long long numel;
  int gtype;
  int phase;
};
constexpr int kNoPhase = 31;
// Elements that a thread takes at once: 32 bytes of the wider type.
constexpr int kAdamStep = 8;
__host__ __device__ constexpr int norm_step(int src) { return src == GRAD_F32 ? 8 : 16; }
__host__ __device__ constexpr int scale_step(int src, int dst) { return src == GRAD_F32 || dst == GRAD_F32 ? 8 : 16; }
// Elements from p to a boundary of `step` elements.
inline int phase_of(const void* p, int type, int step) {
  return (int)(-(reinterpret_cast<uintptr_t>(p) >> (type == GRAD_F32 ? 2 : 1)) & (uintptr_t)(step - 1));
}
inline void set_phases(GradItem& x) {
  const int step = scale_step(x.stype, x.dtype), h = phase_of(x.src, x.stype, step);
  x.norm_phase = phase_of(x.src, x.stype, norm_step(x.stype));
  x.scale_phase = phase_of(x.dst, x.dtype, step) == h ? h : kNoPhase;
}
inline void set_phases(AdamItem& x) {
  const int h = phase_of(x.p, GRAD_F32, kAdamStep);
  x.phase = phase_of(x.m, GRAD_F32, kAdamStep) == h && phase_of(x.v, GRAD_F32, kAdamStep) == h &&
                    phase_of(x.g, x.gtype, kAdamStep) == h
                ? h
                : kNoPhase;
}

// Tables that travel as kernel arguments (at most 32,764 bytes of them). A
// launch takes the smallest table that the list fits: 31 KB of arguments cost
// the host 2.2 us more than 3 KB, 11 KB 1.1 us.
constexpr int kGradCapSmall = 64;
constexpr int kGradCapMid = 256;
constexpr int kGradCapLarge = 512;
constexpr int kNormCap = 1536;    // 20 bytes a tensor, and 0.5 KB of index
constexpr int kScaleCap = 1088;   // 28
constexpr int kAdamCap = 704;     // 44
constexpr int kGradUnits = 65536; // at most this many blocks, and one more per tensor, share a norm
// Lists up to this size take one kernel on one cluster (launch_grad_small).
constexpr long long kGradSmallNumel = 1 << 17;
constexpr int kGradSmallUnit = 10;   // log2 of the elements a warp takes there

// numel (48 bits) | source type (2) | destination type (2) | phase (5)
__host__ __device__ inline unsigned long long grad_meta(long long numel, int stype, int dtype, int phase) {
  return (unsigned long long)numel | ((unsigned long long)stype << 48) | ((unsigned long long)dtype << 50) |
         ((unsigned long long)phase << 52);
}
__host__ __device__ inline long long grad_numel(unsigned long long m) { return (long long)(m & 0xffffffffffffull); }
__host__ __device__ inline int grad_src(unsigned long long m) { return (int)(m >> 48) & 3; }
__host__ __device__ inline int grad_dst(unsigned long long m) { return (int)(m >> 50) & 3; }
__host__ __device__ inline int grad_phase(unsigned long long m) { return (int)(m >> 52) & 31; }
// Units of a tensor. They are counted from its phase (the first one takes the
// elements before it too), so that only a tensor's first and last unit have
// elements outside the wide accesses: a second pass of a block over a few
// elements costs as much time as its first.
__host__ __device__ inline int grad_units(long long numel, int phase, int log2_unit) {
  if (numel == 0) return 0;
  const long long rest = numel - (phase == kNoPhase ? 0 : phase), unit = 1ll << log2_unit;
  return rest <= unit ? 1 : (int)((rest + unit - 1) >> log2_unit);
}
struct UnitRange {
  long long e0, e1;   // elements
  int head;           // the first ones, before the boundary; all of them without a phase
};
__host__ __device__ inline UnitRange unit_range(unsigned long long meta, int k, int log2_unit) {
  const int phase = grad_phase(meta);
  const long long numel = grad_numel(meta), first = phase == kNoPhase ? 0 : phase;
  UnitRange r;
  r.e0 = k == 0 ? 0 : first + ((long long)k << log2_unit);
  r.e1 = first + ((long long)(k + 1) << log2_unit);
  if (r.e1 > numel) r.e1 = numel;
  const int n = (int)(r.e1 - r.e0);
  r.head = phase == kNoPhase ? n : k > 0 ? 0 : phase < n ? phase : n;
  return r;
}

// Where every tensor's units begin, and where to look for a unit's tensor: the
// units fall into at most kBuckets buckets of 2^shift, and tensor_of[k] holds
// the first unit of bucket k. A block then finds its tensor among those of a
// bucket instead of the whole list: mostly two or three dependent reads of its
// arguments; log2 of the tensors in a bucket at most (about 10, where a large
// table's units make the buckets so wide that one holds all the vectors).
constexpr int kBuckets = 256;
template <int kCap>
struct UnitIndex {
  int unit0[kCap + 1];
  unsigned short tensor_of[kBuckets + 1];
  unsigned short count;
  int shift;
};
template <int kCap>
struct GradTable {
  const void* src[kCap];
  unsigned long long meta[kCap];
  UnitIndex<kCap> units;
};
template <int kCap>
struct ScaleTable {
  const void* src[kCap];
  void* dst[kCap];
  unsigned long long meta[kCap];
  UnitIndex<kCap> units;
};
template <int kCap>
struct AdamTable {
  float* p[kCap];
  const void* g[kCap];
  float* m[kCap];
  float* v[kCap];
  unsigned long long meta[kCap];
  UnitIndex<kCap> units;
};
template <int kCap>
struct SpanTable {
  int unit0[kCap + 1];
  int count;
};

struct AdamArgs {
  double log_beta1, log_beta2;      // with lr, for a step number on the device
  float lr;
  float decay, eps;                 // 1 - lr wd
  float b1, omb1, b2, omb2;         // beta1, 1 - beta1, ...
  float step_size, rsqrt_bc2;       // lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t); unused with `step`
  const long long* step;            // device step number, or NULL
  const float* grad_scale;          // device multiplier of the gradients, or NULL
  int once;                         // nothing of the lists is read again soon
};

// Each launches one kernel over up to the table's capacity of tensors, in
// units of 2^unit elements; *units receives their number (0: no launch).
// Partial k of the launch is the norm of its unit k.
// The last `keep` units stay in L2 where they can, for the pass that follows.
cudaError_t launch_grad_norm(const GradItem* it, int n, int unit, int keep, int kind, double* partials,
                             cudaStream_t st, int* units);
// out (or NULL): norm and clip multiplier over all `nunits` partials at `all`.
// per_tensor (or NULL): norms of these n tensors, whose partials start at `partials`.
// followed: another kernel of the same call comes next on the stream.
cudaError_t launch_grad_finish(const GradItem* it, int n, int unit, int kind, const double* all, long long nunits,
                               double max_norm, float* out, const double* partials, float* per_tensor,
                               bool followed, cudaStream_t st);
// Both of the above, and with `scale` the clipped copy too, in one kernel:
// lists of up to kGradCapLarge tensors and kGradSmallNumel elements.
cudaError_t launch_grad_small(const GradItem* it, int n, int kind, bool scale, double max_norm, float* out,
                              float* per_tensor, cudaStream_t st);
// once: nothing of the list is read again soon.
cudaError_t launch_grad_scale(const GradItem* it, int n, int unit, int once, const float* scale, cudaStream_t st,
                              int* units);
cudaError_t launch_adamw(const AdamItem* it, int n, int unit, const AdamArgs& a, cudaStream_t st);

// Sets the calling thread's muon_last_error text.
void record_last_error(const std::string& msg);

}  // namespace muon
