// Shared pieces of the drafter-training kernels (top logits, distillation,
// linear cross entropy): argument blocks, launchers, and the access to
// vocabulary rows of any alignment.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../sv_common.hpp"

namespace sv {

typedef uint32_t vu32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr float LOG2E = 1.44269504088896340736f;

// Maximum of a set of logits and the sum of exp of their distances to it
// (base 2 of the tempered distance). Empty: (-inf, 0).
struct MaxSum {
  float m, s;
};

// exp2 by the transcendental unit (v_exp_f32: about 1 ulp, results below
// 2^-126 flushed to 0, exp2(-inf) = 0).
__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// Two sets as one; c = log2(e) / T. NaN sums stay NaN.
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float c) {
  const float m = fmaxf(a.m, b.m);
  const float ref = m == -INFINITY ? 0.0f : m;   // both empty: 0 + 0
  MaxSum r;
  r.m = m;
  r.s = a.s * fast_exp2((a.m - ref) * c) + b.s * fast_exp2((b.m - ref) * c);
  return r;
}

__device__ __forceinline__ MaxSum wave_join(MaxSum v, float c) {
#pragma unroll
  for (int off = WAVE / 2; off > 0; off >>= 1) {
    MaxSum o;
    o.m = __shfl_xor(v.m, off, WAVE);
    o.s = __shfl_xor(v.s, off, WAVE);
    v = join(v, o, c);
  }
  return v;
}

// The block's set in every thread; scratch holds NT / WAVE entries. The order
// of the joins is fixed.
template <int NT>
__device__ __forceinline__ MaxSum block_join(MaxSum v, MaxSum* scratch, float c) {
  v = wave_join(v, c);
  __syncthreads();
  if ((threadIdx.x & (WAVE - 1)) == 0) scratch[threadIdx.x / WAVE] = v;
  __syncthreads();
  MaxSum r = scratch[0];
#pragma unroll
  for (int i = 1; i < NT / WAVE; ++i) r = join(r, scratch[i], c);
  return r;
}

// A row of V logits at any element alignment, seen as `head` single elements,
// `nvec` aligned 16-byte groups of EPV elements, and a tail shorter than a group.
template <typename Elem>
struct Row {
  static constexpr int EPV = 16 / (int)sizeof(Elem);
  const Elem* p;
  int V, head, nvec;
  __device__ __forceinline__ Row(const void* base, int64_t stride, int64_t r, int V_) {
    p = (const Elem*)base + r * stride;
    V = V_;
    const int off = (int)(((16u - ((uint32_t)(uintptr_t)p & 15u)) & 15u) / sizeof(Elem));
    head = off < V ? off : V;
    nvec = (V - head) / EPV;
  }
  __device__ __forceinline__ vu32x4 vec(int j) const {
    return __builtin_nontemporal_load((const vu32x4*)(p + head) + j);
  }
  __device__ __forceinline__ int tail() const { return V - head - nvec * EPV; }
  __device__ __forceinline__ int tail0() const { return head + nvec * EPV; }
};

__device__ __forceinline__ float to_f32(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ float to_f32(const float* p) { return *p; }

// The elements of one 16-byte group.
__device__ __forceinline__ void unpack(const vu32x4& w, float (&z)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    z[2 * i] = __uint_as_float(w[i] << 16);
    z[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack(const vu32x4& w, float (&z)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) z[i] = __uint_as_float(w[i]);
}

// Rounds to nearest even once, as a cast of the float32 result would.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const f32x2 v = {lo, hi};
  const bf16x2 r = __builtin_convertvector(v, bf16x2);
  return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ vu32x4 pack(const float (&z)[8]) {
  vu32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_bf16(z[2 * i], z[2 * i + 1]);
  return w;
}
__device__ __forceinline__ vu32x4 pack(const float (&z)[4]) {
  vu32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(z[i]);
  return w;
}
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = (uint16_t)pack_bf16(v, 0.0f); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

// A thread's running set while it streams a row: the sum is kept as
// sum exp2(z c - ref), ref a whole number, so that a logit costs one fused
// multiply-add, one exp2 and one addition. The reference is next to m c when it is
// set, and set again only when a logit lies 2^30 above it (float32 holds sums of
// 2^31 such terms): a reference that followed every new maximum would be moved in
// nearly every step, since one lane of the 64 is enough. The fused product rounds z c - ref
// once. From 2^24 on (masks of -1e9 and below, temperatures next to 0) a float next to m c
// may lie more than 1 from it, from 2^32 on so far that exp2 of the difference is 0 or
// infinite: there ref is +inf as a mark and the sum is kept relative to m.
constexpr float REF_RANGE = 0x1p24f;

struct Running {
  float m = -INFINITY;        // largest logit
  float limit = -INFINITY;    // a larger one sets a new reference
  float ref = 0.0f, s = 0.0f;

  __device__ __forceinline__ MaxSum set(float c) const {
    MaxSum r{m, s};
    if (ref != INFINITY && m != -INFINITY) r.s = s * fast_exp2(__builtin_fmaf(-m, c, ref));
    return r;
  }
  // vm: larger than limit. m and s are those before it.
  __device__ __forceinline__ void raise(float vm, float c) {
    float t = set(c).s;
    t *= fast_exp2((m - vm) * c);   // m = -inf: t is 0
    if (fabsf(vm * c) < REF_RANGE) {
      ref = rintf(vm * c);
      limit = vm + 30.0f / c;
      s = t * fast_exp2(__builtin_fmaf(vm, c, -ref));
    } else {
      ref = INFINITY;
      limit = vm;
      s = t;
    }
  }
  // vm: the largest of the N logits (NaN do not count; they make the sum NaN).
  template <int N>
  __device__ __forceinline__ void add(const float (&z)[N], float vm, float c) {
    if (vm > limit) raise(vm, c);
    m = fmaxf(m, vm);
    float e[N];
    if (!__any(ref == INFINITY)) {
#pragma unroll
      for (int i = 0; i < N; ++i) e[i] = fast_exp2(__builtin_fmaf(z[i], c, -ref));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        e[i] = fast_exp2(ref == INFINITY ? (z[i] - m) * c : __builtin_fmaf(z[i], c, -ref));
    }
#pragma unroll
    for (int w = N / 2; w > 0; w >>= 1)
#pragma unroll
      for (int i = 0; i < w; ++i) e[i] += e[i + w];
    s += e[0];
  }
  template <int N>
  __device__ __forceinline__ void add(const float (&z)[N], float c) {
    add(z, largest(z), c);
  }
  template <int N>
  static __device__ __forceinline__ float largest(const float (&z)[N]) {
    float vm = z[0];
#pragma unroll
    for (int i = 1; i < N; ++i) vm = fmaxf(vm, z[i]);
    return vm;
  }
};

// ------------------------------------------------------------ held rows

// A workgroup of HOLD_THREADS keeps a whole row in registers, NV 16-byte groups a
// thread: 152 of 256 registers at NV = 38, so one workgroup fills a CU and walks
// over rows r, r + grid, ... . A group's registers take the next row's group as
// soon as the row's last pass over it is done, so that the next row arrives while
// this one is finished. NV = 20 leaves two workgroups a CU short of registers (33
// spilled), but rows that need it are slower one a CU (2000 rows of 40,000 in float32, with
// the gradient: 145 us, one a CU 160); those that 16 hold are faster there (4096 rows of 50,257
// in bfloat16: 222 us, in 20 230; 500 of 32,000 in float32: 30 and 36).
constexpr int HOLD_THREADS = 512;
constexpr int HOLD_SIZES = 4;
constexpr int HOLD_NV[HOLD_SIZES] = {10, 16, 20, 38};
// Workgroups a CU holds at once, by their registers.
constexpr int HOLD_PER_CU[HOLD_SIZES] = {2, 2, 2, 1};
constexpr int HOLD_CUS = 256;

// Index into HOLD_NV for rows of V logits of es bytes, or -1: too long.
inline int hold_size(int64_t V, int es) {
  for (int i = 0; i < HOLD_SIZES; ++i)
    if (V * es <= (int64_t)HOLD_NV[i] * HOLD_THREADS * 16) return i;
  return -1;
}

// One row of it: the groups, and in the threads below 32 the elements before the
// first and behind the last whole group (threads 0.. and 16..).
template <typename Elem, int NV>
struct Held {
  static constexpr int EPV = 16 / (int)sizeof(Elem);
  vu32x4 w[NV];
  float edge;
  // Index of the thread's i-th group, made anew: the compiler would else keep NV of
  // them across the rows.
  static __device__ __forceinline__ int index(int i) {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return i * HOLD_THREADS + t;
  }
  __device__ __forceinline__ void load_group(const Row<Elem>& row, int i) {
    const uint32_t j = (uint32_t)index(i);
    // a whole step needs no test of its lanes; a row is below 2^31 bytes
    const auto at = (const vu32x4*)((const char*)(row.p + row.head) + j * 16u);
    if ((i + 1) * HOLD_THREADS <= row.nvec) w[i] = __builtin_nontemporal_load(at);
    else w[i] = (int)j < row.nvec ? __builtin_nontemporal_load(at)
                                  : (vu32x4)(sizeof(Elem) == 2 ? 0xFF80FF80u : 0xFF800000u);   // -inf
  }
  // The group's elements, unpacked anew: the compiler would else keep those of an
  // earlier pass, twice the registers.
  __device__ __forceinline__ void get(int i, float (&z)[EPV]) {
    asm volatile("" : "+v"(w[i]));
    unpack(w[i], z);
  }
  static __device__ __forceinline__ int edge_id(const Row<Elem>& row) {
    const int t = threadIdx.x;
    if (t < row.head) return t;
    if (t >= 16 && t - 16 < row.tail()) return row.tail0() + t - 16;
    return -1;
  }
  __device__ __forceinline__ void load_edge(const Row<Elem>& row) {
    const int id = edge_id(row);
    edge = id >= 0 ? to_f32(row.p + id) : -INFINITY;
  }
  __device__ __forceinline__ void load(const Row<Elem>& row) {
    load_edge(row);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * HOLD_THREADS < row.nvec) load_group(row, i);
  }
};

// ------------------------------------------------------------ top logits

constexpr int TOP_THREADS = 256;
constexpr int TOP_STEP = TOP_THREADS * 8;   // most candidates one group a thread can add
constexpr int TOP_CAP = 12 * TOP_THREADS;    // candidates held in LDS
constexpr int TOP_MAX_K = 1024;
constexpr int TOP_THIN = 1024;              // candidates that are thinned without a cut

struct TopArgs {
  const void* logits;
  int64_t stride;
  int R, V, K;
  int parts;          // workgroups per row
  float c;            // log2(e) / T
  float temperature;
  int32_t* ids;       // [R][K]
  float* values;      // [R][K]
  float* lse;         // [R] or nullptr
  uint64_t* keys;     // [R][parts][K] when parts > 1
  MaxSum* sums;       // [R][parts] when parts > 1
};
int launch_top_logits(const TopArgs& a, int bf16, hipStream_t s);

// ------------------------------------------------------------ distillation

constexpr int DIS_MAX_K = 1024;

struct DistillArgs {
  const void* logits;
  int64_t stride;
  const int32_t* ids;        // [R][K] teacher's ids
  const float* tl;           // [R][K] teacher's logits
  const float* tlse;         // [R] or nullptr: renormalised over the kept slots
  const float* weight;       // [R] or nullptr (1): d total / d loss
  int R, V, K;
  int parts;                 // workgroups per row
  float inv_t, c;            // 1 / T, log2(e) / T
  double inv_t64;
  float* loss;               // [R] or nullptr (backward alone)
  float* stats;              // [R][2]: largest logit, log of the sum; or nullptr
  void* grad;                // [R][V] or nullptr
  int64_t grad_stride;
  MaxSum* sums;              // [R][parts] when parts > 1
  int hold;                  // index into HOLD_NV: rows are held in registers; -1: streamed
};
int launch_distill(const DistillArgs& a, int bf16, hipStream_t s);
int launch_distill_backward(const DistillArgs& a, int bf16, hipStream_t s);

// ------------------------------------------------------------ linear cross entropy

constexpr int CE_LINE = 128;       // most bytes of a row that one step of the products takes
constexpr int CE_MAX_D = 1 << 22;

struct CeTile {
  int bm, bn;
  int per_cu, per_cu_dz;   // workgroups that a CU holds at once, by LDS; of the products of dz
};
CeTile ce_tile(int64_t M, int64_t N, int planes);

// One product C[m][n] = sum_k A[m][k] B[n][k]. An operand lies
// in memory as [row][k] or, where the epilogue takes it transposed, as [k][row];
// rows of memory start on 16 bytes and can be read in whole groups of 16 bytes.
struct CeGemm {
  const void *A, *B;
  int64_t lda, ldb;          // strides of memory's rows, elements, at most CE_MAX_D
  int64_t plane_a, plane_b;  // distance of an operand's parts: three of float32, two of dz of bfloat16
  int M, N, K;               // rows of A and B, depth
  int planes;                // 1: bfloat16 operands (dz in two parts); 3: float32 in bfloat16 parts; 0: float32 as it is
  int splits;                // workgroups that share one tile's depth
  CeTile tile;
};

struct CeStatsOut {
  const int32_t* labels;
  int v0, V;                 // id of A's row 0
  MaxSum* partial;           // [tiles of A][N]
  float* zlabel;             // [N]
};
struct CeDzOut {
  const int32_t* labels;
  const float* stats;        // [N][2]
  const float* grad_loss;    // [N] or nullptr
  int v0, V;
  void* dz;                  // [parts][N][ldz] bfloat16, or [N][ldz] float; zeros behind the last token
  int64_t ldz, plane_dz;
};
struct CeAccOut {
  float* acc;                // [splits][N][ld]
  int64_t ld, split_stride;
  int add;                   // 0: the first piece of the vocabulary
};
struct CeMatOut {
  void* out;                 // [N][M], row stride ld, float32 or bfloat16
  int64_t ld;
  int bf16;
};

// Rows as the products take them: [planes][rows][ld] bfloat16, or [rows][ld] float
// (planes 0); zeros from cols to ld.
struct CePack {
  const void* src;           // [rows][cols], float32 or bfloat16
  int64_t stride;
  int bf16;
  int rows, cols;
  int planes;
  void* dst;
  int64_t ld, plane;
};

int launch_ce_pack(const CePack& p, hipStream_t s);
int launch_ce_stats(const CeGemm& g, const CeStatsOut& o, hipStream_t s);
int launch_ce_dz(const CeGemm& g, const CeDzOut& o, hipStream_t s);
int launch_ce_acc(const CeGemm& g, const CeAccOut& o, hipStream_t s);
int launch_ce_mat(const CeGemm& g, const CeMatOut& o, hipStream_t s);
int launch_ce_join(const MaxSum* partial, const float* zlabel, const int32_t* labels, int tiles,
                   int N, int V, float* loss, float* stats, hipStream_t s);
int launch_ce_sum(const float* acc, int splits, int64_t split_stride, int64_t ld, int N, int D,
                  void* out, int64_t out_stride, int bf16, hipStream_t s);

}  // namespace sv
