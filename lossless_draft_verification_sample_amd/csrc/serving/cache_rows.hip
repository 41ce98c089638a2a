// The 8-bit cache: rows of keys and values quantised into the blocks that they fall
// into, and read back.
//
// A block (32 tokens of a head) has one scale, the smallest power of two that brings its
// largest value within e4m3's 448. A power of two makes value = scale * code exact in
// bfloat16, so that nothing is rounded when the cache is read, and costs no
// precision: e4m3 keeps its relative step down to 2^-6 of the block's largest value's
// binade either way. Since the scale depends on what the block holds alone, rows
// that it held before are decoded, and coded again at the new scale with the new ones.
//
// Bound by memory. One workgroup takes a block's keys or values: its threads read 8
// dimensions of two tokens each, the largest value goes through a block reduction, and the
// codes are put in the block's order in LDS, from where 16 bytes a thread are stored.

#include <math.h>

#include "sv_serve.hpp"

namespace sv {
namespace {

constexpr int NTH = 256;
constexpr int MAX_UNITS = CACHE_MAX_D / 32 * 64 / NTH;   // pairs of tokens by 8 dimensions, a thread

struct Where {
  int b, h, block;
  bool values;
};
// Heads are fastest: neighbouring workgroups read neighbouring parts of the same rows.
__device__ __forceinline__ Where where(const CacheRowsArgs& a) {
  const int kinds = a.which == 3 ? 2 : 1;
  uint32_t i = blockIdx.x;
  Where w;
  w.h = i % a.c.heads;
  i /= a.c.heads;
  w.values = kinds == 2 ? i % 2 : a.which == 2;
  i /= kinds;
  w.block = i % a.blocks;
  w.b = i / a.blocks;
  return w;
}

// 2^e, smallest with amax <= 448 * 2^e = 1.75 * 2^(e + 8).
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u);
  return e < -126 ? -126 : e;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// `most`: 448, or 240 at the scale 2^120, whose 256 is beyond float32.
__device__ __forceinline__ uint32_t code4(const float* x, float inv, float most) {
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = fabsf(x[i]) < INFINITY ? __builtin_amdgcn_fmed3f(x[i] * inv, -most, most) : NAN;
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  return __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
}

template <typename E>
__global__ __launch_bounds__(NTH) void write_kernel(CacheRowsArgs a) {
  __shared__ uint8_t block[CACHE_MAX_D / 32 * BRICK];
  __shared__ float top[NTH / WAVE];
  const Where w = where(a);
  const Span s = span_of(a.t, w.b);
  if (s.bad || s.rows == 0) return;
  const int end = s.first + s.rows, t0 = (s.first / CACHE_BLOCK + w.block) * CACHE_BLOCK;
  if (t0 >= end) return;
  const int blk = t0 / CACHE_BLOCK, in_page = blk & ((1 << a.c.per_log2) - 1);
  const int page = a.t.table[(int64_t)w.b * a.t.width + (blk >> a.c.per_log2)];
  if ((uint32_t)page >= (uint32_t)a.c.pages) return;
  const int64_t at = (((int64_t)page * a.c.heads + w.h) << a.c.per_log2) + in_page;
  const int bytes = a.c.bricks * BRICK, tid = threadIdx.x;
  uint8_t* mem = (w.values ? a.c.v : a.c.k) + at * bytes;
  float* scale = (w.values ? a.c.vs : a.c.ks) + at;
  const bool held = t0 < s.first;                     // rows from before
  const bool whole = !held && t0 + CACHE_BLOCK <= end;
  float old_scale = 0.0f;
  if (!whole) {
    for (int i = tid * 16; i < bytes; i += NTH * 16) *(su32x4*)(block + i) = *(const su32x4*)(mem + i);
    if (held) old_scale = *scale;
    __syncthreads();
  }
  const Strides st = w.values ? a.vs : a.ks;
  const E* rows = (const E*)(w.values ? a.v : a.k) + w.b * st.b + w.h * st.h;
  const int units = a.c.bricks * 64;
  float x[MAX_UNITS][2][8];
  float amax = 0.0f;
#pragma unroll
  for (int n = 0; n < MAX_UNITS; ++n) {
    const int u = tid + n * NTH;
    if (u >= units) break;
    // a unit: dimensions 8 d8 .. + 7 of tokens s0 and s0 + 4
    const int d8 = u % (a.c.bricks * 4), m = u / (a.c.bricks * 4);
    const int d = d8 * 8, s0 = 8 * (m >> 2) + (m & 3);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int tok = s0 + 4 * half, pos = t0 + tok;
      float(&y)[8] = x[n][half];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = 0.0f;
      if (pos >= end) continue;
      if (pos >= s.first) {
        const E* p = rows + (pos - s.first) * st.n + d;
        if (d + 8 <= a.c.D) {
          load8(p, y);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (d + e < a.c.D) y[e] = elem(p + e);
        }
      } else {
        const uint8_t* brick = block + (d / 32) * BRICK;
        uint32_t lo = 0, hi = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t c = brick[w.values ? value_byte(tok, d % 32 + e) : key_byte(tok, d % 32 + e)];
          if (e < 4) lo |= c << (8 * e);
          else hi |= c << (8 * (e - 4));
        }
        codes4(lo, y);
        codes4(hi, y + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = d + e < a.c.D ? y[e] * old_scale : 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(y[e]) < INFINITY ? fabsf(y[e]) : 0.0f);
    }
  }
#pragma unroll
  for (int off = WAVE / 2; off; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off, WAVE));
  if (tid % WAVE == 0) top[tid / WAVE] = amax;
  __syncthreads();   // also: every old code has been read
#pragma unroll
  for (int i = 0; i < NTH / WAVE; ++i) amax = fmaxf(amax, top[i]);
  const int ex = amax > 0.0f ? scale_exponent(amax) : 0;
  const float inv = pow2(-ex), most = ex == 120 ? 240.0f : E4M3_MAX;
#pragma unroll
  for (int n = 0; n < MAX_UNITS; ++n) {
    const int u = tid + n * NTH;
    if (u >= units) break;
    const int d8 = u % (a.c.bricks * 4), m = u / (a.c.bricks * 4);
    const int d = d8 * 8, s0 = 8 * (m >> 2) + (m & 3);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int tok = s0 + 4 * half;
      if (t0 + tok >= end) continue;
      uint8_t* brick = block + (d / 32) * BRICK;
      const uint32_t lo = code4(x[n][half], inv, most), hi = code4(x[n][half] + 4, inv, most);
      if (w.values) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          brick[value_byte(tok, d % 32 + e)] = (uint8_t)((e < 4 ? lo : hi) >> (8 * (e & 3)));
      } else {
        *(su32x2*)(brick + key_byte(tok, d % 32)) = su32x2{lo, hi};
      }
    }
  }
  __syncthreads();
  for (int i = tid * 16; i < bytes; i += NTH * 16) *(su32x4*)(mem + i) = *(const su32x4*)(block + i);
  if (tid == 0) *scale = pow2(ex);
}

template <typename E>
__global__ __launch_bounds__(NTH) void read_kernel(CacheRowsArgs a) {
  __shared__ uint8_t block[CACHE_MAX_D / 32 * BRICK];
  const Where w = where(a);
  Span s = span_of(a.t, w.b);
  if (s.bad) {
    s.first = 0;
    s.rows = a.t.N;
  }
  const int end = s.first + s.rows, t0 = (s.first / CACHE_BLOCK + w.block) * CACHE_BLOCK;
  if (t0 >= end) return;
  const int blk = t0 / CACHE_BLOCK, in_page = blk & ((1 << a.c.per_log2) - 1), tid = threadIdx.x;
  const int page = s.bad ? -1 : a.t.table[(int64_t)w.b * a.t.width + (blk >> a.c.per_log2)];
  const bool known = (uint32_t)page < (uint32_t)a.c.pages;
  float scale = NAN;
  if (known) {
    const int64_t at = (((int64_t)page * a.c.heads + w.h) << a.c.per_log2) + in_page;
    const int bytes = a.c.bricks * BRICK;
    const uint8_t* mem = (w.values ? a.c.v : a.c.k) + at * bytes;
    scale = (w.values ? a.c.vs : a.c.ks)[at];
    for (int i = tid * 16; i < bytes; i += NTH * 16) *(su32x4*)(block + i) = *(const su32x4*)(mem + i);
  }
  __syncthreads();
  const Strides st = w.values ? a.vs : a.ks;
  E* rows = (E*)(w.values ? a.v : a.k) + w.b * st.b + w.h * st.h;
  const int per = a.c.bricks * 4;
  for (int u = tid; u < per * CACHE_BLOCK; u += NTH) {
    const int d = u % per * 8, tok = u / per, pos = t0 + tok;
    if (pos < s.first || pos >= end || d >= a.c.D) continue;
    float y[8];
    if (known) {
      const uint8_t* brick = block + (d / 32) * BRICK;
      uint32_t lo = 0, hi = 0;
      if (w.values) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t c = brick[value_byte(tok, d % 32 + e)];
          if (e < 4) lo |= c << (8 * e);
          else hi |= c << (8 * (e - 4));
        }
      } else {
        const su32x2 c = *(const su32x2*)(brick + key_byte(tok, d % 32));
        lo = c[0];
        hi = c[1];
      }
      codes4(lo, y);
      codes4(hi, y + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= scale;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = NAN;
    }
    E* p = rows + (pos - s.first) * st.n + d;
    if (d + 8 <= a.c.D) {
      store8(p, y);
    } else {
      for (int e = 0; e < 8; ++e)
        if (d + e < a.c.D) put(p + e, y[e]);
    }
  }
}

int64_t grid_of(const CacheRowsArgs& a) {
  return (int64_t)a.t.B * a.blocks * a.c.heads * (a.which == 3 ? 2 : 1);
}

}  // namespace

int launch_cache_write(const CacheRowsArgs& a, hipStream_t st) {
  const dim3 grid((uint32_t)grid_of(a));
  if (a.bf16) write_kernel<uint16_t><<<grid, NTH, 0, st>>>(a);
  else write_kernel<float><<<grid, NTH, 0, st>>>(a);
  return hipGetLastError() != hipSuccess;
}

int launch_cache_read(const CacheRowsArgs& a, hipStream_t st) {
  const dim3 grid((uint32_t)grid_of(a));
  if (a.bf16) read_kernel<uint16_t><<<grid, NTH, 0, st>>>(a);
  else read_kernel<float><<<grid, NTH, 0, st>>>(a);
  return hipGetLastError() != hipSuccess;
}

}  // namespace sv
