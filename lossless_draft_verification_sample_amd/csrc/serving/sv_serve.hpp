// Shared pieces of the kernels for the verification pass's rows (rotary positions,
// the 8-bit cache, attention over it, logit adjustments): argument blocks,
// launchers, access to rows of any alignment, and the cache's layout.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../sv_common.hpp"

namespace sv {

typedef uint32_t su32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t su32x4 __attribute__((ext_vector_type(4)));
typedef float sf32x2 __attribute__((ext_vector_type(2)));
typedef float sf32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 sbf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 sbf16x8 __attribute__((ext_vector_type(8)));

// The same at any alignment of their elements: the hardware loads and stores
// vectors at any address, so no row needs a head of single elements.
typedef su32x4 __attribute__((aligned(2))) su32x4_any;
typedef su32x2 __attribute__((aligned(2))) su32x2_any;

struct Strides {
  int64_t b, n, h;
};

// -------------------------------------------------------------------- the cache

constexpr int CACHE_BLOCK = 32;     // tokens of a block, which share a scale
constexpr int BRICK = 1024;         // bytes of 32 tokens by 32 dimensions
constexpr int CACHE_MAX_D = 256;
constexpr float E4M3_MAX = 448.0f;

// Byte of token s and dimension d (0..31 both) in a brick of keys or of values.
__host__ __device__ __forceinline__ int key_byte(int s, int d) {
  return 256 * (d >> 3) + 16 * (4 * (s >> 3) + (s & 3)) + 8 * ((s >> 2) & 1) + (d & 7);
}
__host__ __device__ __forceinline__ int value_byte(int s, int d) {
  return 256 * (s >> 3) + 16 * (d & 15) + 8 * (d >> 4) + (s & 7);
}

struct Cache {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  int pages, heads, per_log2, bricks, D;   // blocks of a page: 1 << per_log2
};

// Where the positions of a batch's requests lie.
struct Batch {
  const int32_t* table;
  int width;
  const int32_t* first;   // position of row 0 (NULL: 0)
  const int32_t* rows;    // NULL: N
  int B, N;
  int capacity;           // width * page size, at most 2^30
};

struct Span {
  int first, rows;
  bool bad;
};
__device__ __forceinline__ Span span_of(const Batch& a, int b) {
  Span s;
  s.first = a.first ? a.first[b] : 0;
  s.rows = a.rows ? a.rows[b] : a.N;
  s.bad = s.first < 0 || s.rows < 0 || s.rows > a.N || s.first > a.capacity - s.rows;
  return s;
}

// -------------------------------------------------------------------- elements

__device__ __forceinline__ float elem(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ float elem(const float* p) { return *p; }

// Rounds to nearest even once.
__device__ __forceinline__ uint32_t round_bf16x2(float lo, float hi) {
  const sf32x2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, sbf16x2));
}
__device__ __forceinline__ void put(uint16_t* p, float x) { *p = (uint16_t)round_bf16x2(x, 0.0f); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }

// 8 consecutive elements at any alignment.
__device__ __forceinline__ void load8(const uint16_t* p, float (&x)[8]) {
  const su32x4 w = *(const su32x4_any*)p;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const su32x4 a = *(const su32x4_any*)p, b = *(const su32x4_any*)(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = __uint_as_float(a[i]);
    x[4 + i] = __uint_as_float(b[i]);
  }
}
// bfloat16 past the caches' older contents: for results that are written in whole lines and not read again soon.
__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8]) {
  su32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = round_bf16x2(x[2 * i], x[2 * i + 1]);
  __builtin_nontemporal_store(w, (su32x4_any*)p);
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  su32x4 a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = __float_as_uint(x[i]);
    b[i] = __float_as_uint(x[4 + i]);
  }
  *(su32x4_any*)p = a;
  *(su32x4_any*)(p + 4) = b;
}

// Four e4m3 codes as float32.
__device__ __forceinline__ void codes4(uint32_t w, float* x) {
  const sf32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
  x[0] = a[0];
  x[1] = a[1];
  x[2] = b[0];
  x[3] = b[1];
}

// Bits of the bytes that are NaN codes (0x7F, 0xFF), one a byte at bit 0.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  const uint32_t x = (w & 0x7F7F7F7Fu) ^ 0x7F7F7F7Fu;       // 0 in a byte of NaN
  return (((x + 0x7F7F7F7Fu) >> 7) & 0x01010101u) ^ 0x01010101u;
}
__device__ __forceinline__ su32x4 nan_codes(su32x4 w) {
  return su32x4{nan_codes(w[0]), nan_codes(w[1]), nan_codes(w[2]), nan_codes(w[3])};
}
// The bytes of a lane's codes (8 tokens of a dimension, twice) of the first `left` tokens.
__device__ __forceinline__ su32x4 tokens_before(int left) {
  const uint32_t lo = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
  const uint32_t hi = left >= 8 ? ~0u : left <= 4 ? 0u : (1u << (8 * (left - 4))) - 1u;
  return su32x4{lo, hi, lo, hi};
}

// -------------------------------------------------------------------- launchers

struct RotateArgs {
  const void *q, *k;
  void *oq, *ok;
  Strides qs, ks, oqs, oks;
  int B, N, qh, kh, D, R;
  const double* freqs;
  float scale;
  int inter, inverse, bf16;
  const int32_t* first;
  const int32_t* rows;
};
int launch_rotate(const RotateArgs& a, hipStream_t st);

struct CacheRowsArgs {
  Cache c;
  Batch t;
  void *k, *v;        // rows: read by a write, written by a read
  Strides ks, vs;
  int blocks;         // blocks that N rows can touch
  int which;          // bit 0: keys, bit 1: values
  int bf16;
};
int launch_cache_write(const CacheRowsArgs& a, hipStream_t st);
int launch_cache_read(const CacheRowsArgs& a, hipStream_t st);

constexpr int AT_THREADS = 256, AT_WAVES = AT_THREADS / WAVE;
// How the N * group columns (row, query head) of a cache head are spread: NT tiles of
// 16 columns a wave, `across` waves of a workgroup side by side (the others share out the
// tokens), and `sets` workgroups.
struct AttendShape {
  int cols, nt, across, sets;
  int cols_set;       // columns of a set: 16 * nt * across
  int grid;           // workgroups at most
  int single;         // 1: a workgroup a unit
  int may_single, units;
  int join_cols;      // columns that a workgroup of the join takes
  int join_split;     // 1: its threads share out a column's parts
  int lds;            // bytes of LDS
};
// Workgroups of a CU, which is waves of a SIMD: by the registers of a lane (sums, a block's
// values and the next one's codes, scores and weights, the rest).
constexpr int attend_per_cu(int bricks, int nt) {
  const int need = 8 * bricks * nt + 16 * bricks + 22 * nt + 36;
  return need <= 126 ? 4 : need <= 166 ? 3 : need <= 264 ? 2 : 1;
}
// Groups of 16 dimensions that the waves of a workgroup join at a time, in 4 KB of LDS a tile each.
constexpr int attend_round(int bricks, int nt) {
  int n = 12 / nt;
  while (2 * bricks % n) --n;
  return n;
}
struct AttendArgs {
  Cache c;
  Batch t;
  const void* q;
  void* out;
  Strides qs, os;
  float* lse;
  int qh, group, window, bf16;
  uint32_t group_inv; // 2^32 / group, rounded up: a column's row is the product's upper half
  float scale2;       // scale * log2 e
  AttendShape s;
  int32_t* record;    // [B][heads][sets][2]: the first workgroup of a unit, and how many
  float* partial;     // [grid][2]: [cols_set][bricks * 32] sums, [cols_set][2] references and sums of weights
};
int launch_attend(const AttendArgs& a, hipStream_t st);

constexpr int ADJ_CHUNK = 4096, ADJ_THREADS = 256;
struct AdjustArgs {
  const void* z;
  void* out;
  Strides zs, os;
  int B, N, V, bf16;
  const int32_t *rows, *tokens, *history, *prompt, *bias_ids;
  int n_tokens, n_history, n_prompt, n_bias;
  const float *repetition, *frequency, *presence, *bias;
  const uint32_t* allowed;
  int chunks, row_groups;
};
int launch_adjust(const AdjustArgs& a, hipStream_t st);

}  // namespace sv
