// Shared pieces of the drafter-training kernels (top logits, distillation,
// linear cross entropy): argument blocks, launchers, and the access to
// vocabulary rows of any alignment.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sv_common.hpp"

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

// Adds n logits to a running set: the maximum of the new ones first, so that
// the sum is rescaled at most once. NaN logits do not enter the maximum and
// make the sum NaN.
template <int N>
__device__ __forceinline__ void add_logits(MaxSum& a, const float (&z)[N], float c) {
  float vm = z[0];
#pragma unroll
  for (int i = 1; i < N; ++i) vm = fmaxf(vm, z[i]);
  if (vm > a.m) {
    a.s *= fast_exp2((a.m - vm) * c);   // a.m = -inf: a.s is 0
    a.m = vm;
  }
  const float ref = a.m == -INFINITY ? 0.0f : a.m;
#pragma unroll
  for (int i = 0; i < N; ++i) a.s += fast_exp2((z[i] - ref) * c);
}

// ------------------------------------------------------------ top logits

constexpr int TOP_THREADS = 512;
constexpr int TOP_STEP = TOP_THREADS * 8;   // most candidates one step can add
constexpr int TOP_CAP = 6144;               // candidates held in LDS
constexpr int TOP_MAX_K = 1024;

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
  float temperature, inv_t, c;
  float* loss;               // [R] or nullptr (backward alone)
  float* stats;              // [R][2]: largest logit, log of the sum; or nullptr
  void* grad;                // [R][V] or nullptr
  int64_t grad_stride;
  MaxSum* sums;              // [R][parts] when parts > 1
};
int launch_distill(const DistillArgs& a, int bf16, hipStream_t s);
int launch_distill_backward(const DistillArgs& a, int bf16, hipStream_t s);

// ------------------------------------------------------------ linear cross entropy

constexpr int CE_BK = 64;          // depth of one step of the products, in bfloat16
constexpr int CE_MAX_D = 1 << 22;

// One product C[m][n] = sum_k A[m][k] B[n][k] of bfloat16 parts. An operand lies
// in memory as [row][k] or, where the epilogue takes it transposed, as [k][row];
// rows of memory start on 16 bytes and can be read in whole groups of 8 elements.
struct CeGemm {
  const uint16_t *A, *B;
  int64_t lda, ldb;          // strides of memory's rows, elements, at most CE_MAX_D
  int64_t plane_a, plane_b;  // distance of a float32 operand's three parts
  int M, N, K;               // rows of A and B, depth
  int parts;                 // 1: bfloat16 operands; 6: products of float32's parts
  int splits;                // workgroups that share one tile's depth
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
  uint16_t* dz;              // [planes][N][ldz], zeros behind the piece's last token
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
  int vec;                   // rows of four can be stored at once
};

// Rows as the products take them: [planes][rows][ld] bfloat16, zeros from cols to ld.
struct CePack {
  const void* src;           // [rows][cols], float32 or bfloat16
  int64_t stride;
  int bf16;
  int rows, cols;
  int planes;
  uint16_t* dst;
  int64_t ld, plane;
};

// Tile shapes by the rows of B: see linear_ce.hip.
int ce_tile_m(int rows_b);
int ce_tile_n(int rows_b);
int ce_tiles_per_cu(int rows_b);   // workgroups of that shape a CU holds at once

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
