// The 8-bit cache: rows of keys and values quantised into the blocks that they fall
// into, and read back.
//
// A block (32 tokens of a head) has one scale, the smallest power of two that brings its
// largest value within e4m3's 448. A power of two makes value = scale * code exact in
// bfloat16, so that nothing is rounded when the cache is read, and costs no
// precision: e4m3 keeps its relative step for values down to 2^-14 of the block's
// largest either way. Since the scale depends on what the block holds alone, rows
// that it held before are decoded, and coded again at the new scale with the new ones.
//
// Bound by memory where prompts are written, by the latency of a chain of reads (lengths, page,
// block) in a round of few rows. One workgroup takes a block's keys or values. Its threads hold the
// block's codes, 16 bytes each as they lie; the new rows come 8 dimensions a thread; the largest
// value goes through a block reduction, for which old codes need no decoding; and the new codes go
// to their places through LDS. Old codes are made again only where the scale changes, and parts of
// the block that hold no new row are then the only ones not written. Rows that are read back go past the caches'
// older contents, and so do the codes then: two prefixes of 32,768 rows of eight heads of 128 come at 5.7 TB/s (61.6 us;
// 68.2 through the caches; five pairs of prefixes in turn, whose codes no cache holds, the same). A round whose rows change every
// block's scale 12.5 us instead of 10.8. Four prompts of up to 4,096 such rows, written and read back: 40.3 us, 4.1 TB/s (44.2; with the
// rows that a write reads and the codes that it writes past them too, 42.2).

#include <math.h>

#include "sv_serve.hpp"

namespace sv {
namespace {

// A round of few rows is bound by how many waves are started, most of them for little: where the
// rows can touch at most FEW_BLOCKS blocks, a workgroup takes all of a request's, one after
// the other (most requests touch one less than the most), and has two waves up to 128 dimensions. (A
// write for 128 requests of nine rows and eight heads with a workgroup a block and four waves:
// 14.8 us, now 11.3; prompts of 4,096 rows with two waves 31.0 us instead of 29.3.)
constexpr int FEW_BLOCKS = 4;
constexpr bool wide(int bricks) { return bricks > 4; }
template <bool FEW, bool WIDE>
struct Shape {
  static constexpr int NTH = FEW && !WIDE ? 128 : 256, MAX_D = WIDE ? 256 : 128;
  static constexpr int CHUNKS = MAX_D / 32 * 64 / NTH;          // 16 bytes of codes, a thread
  static constexpr int UNITS = CACHE_BLOCK * MAX_D / 8 / NTH;   // 8 dimensions of a row, a thread
};
int blocks_of_wg(const CacheRowsArgs& a) { return a.blocks <= FEW_BLOCKS ? a.blocks : 1; }

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
  w.block = 0;
  w.b = i;
  if (a.blocks > FEW_BLOCKS) {
    w.block = i % a.blocks;
    w.b = i / a.blocks;
  }
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

// The bytes of a chunk (16 bytes of a block as they lie, chunk q * 16 + m of a brick) that hold
// tokens from `from` on and before `to`.
__device__ __forceinline__ su32x4 bytes_of(bool values, int chunk, int from, int to) {
  const int m = chunk & 15, q = chunk >> 4 & 3;
  if (values) return tokens_before(to - 8 * q) & ~tokens_before(from - 8 * q);
  const int s = 8 * (m >> 2) + (m & 3);       // and s + 4
  const uint32_t a = s >= from && s < to ? ~0u : 0u, b = s + 4 >= from && s + 4 < to ? ~0u : 0u;
  return su32x4{a, a, b, b};
}

// The bytes of a chunk whose dimensions lie within the head.
__device__ __forceinline__ su32x4 bytes_within(bool values, int chunk, int D) {
  const int d = 32 * (chunk >> 6), m = chunk & 15, q = chunk >> 4 & 3;
  if (!values) return tokens_before(D - (d + 8 * q));      // as many bytes as dimensions
  const uint32_t a = d + m < D ? ~0u : 0u, b = d + 16 + m < D ? ~0u : 0u;
  return su32x4{a, a, b, b};
}

template <typename E, bool FEW, bool WIDE>
__device__ __forceinline__ void write_block(const CacheRowsArgs& a, const Where& w, const Span& s, int t0,
                                            uint8_t (*fresh)[Shape<FEW, WIDE>::MAX_D + 8], float* top) {
  constexpr int NTH = Shape<FEW, WIDE>::NTH, MAX_CHUNKS = Shape<FEW, WIDE>::CHUNKS, MAX_UNITS = Shape<FEW, WIDE>::UNITS;
  const int end = s.first + s.rows;
  const int blk = t0 / CACHE_BLOCK, in_page = blk & ((1 << a.c.per_log2) - 1);
  const int page = a.t.table[(int64_t)w.b * a.t.width + (blk >> a.c.per_log2)];
  const int tid = threadIdx.x;
  // new rows from .. to - 1 of the block; those before `from` are kept
  const int from = s.first > t0 ? s.first - t0 : 0, to = end - t0 < CACHE_BLOCK ? end - t0 : CACHE_BLOCK;
  const Strides st = w.values ? a.vs : a.ks;
  const E* rows = (const E*)(w.values ? a.v : a.k) + w.b * st.b + w.h * st.h + (t0 - s.first) * st.n;
  const int per_row = a.c.bricks * 4, units = (to - from) * per_row, chunks = a.c.bricks * 64;
  float x[MAX_UNITS][8], amax = 0.0f;
#pragma unroll
  for (int n = 0; n < MAX_UNITS; ++n) {
    const int u = tid + n * NTH;
    if (u >= units) break;
    const int row = u / per_row, d = (u - row * per_row) * 8;
    const E* p = rows + (from + row) * st.n + d;
    if (d + 8 <= a.c.D) {
      load8(p, x[n]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[n][e] = d + e < a.c.D ? elem(p + e) : 0.0f;
    }
  }
  if ((uint32_t)page >= (uint32_t)a.c.pages) return;
  const int64_t at = (((int64_t)page * a.c.heads + w.h) << a.c.per_log2) + in_page;
  su32x4* mem = (su32x4*)((w.values ? a.c.v : a.c.k) + at * (a.c.bricks * BRICK));
  float* scale = (w.values ? a.c.vs : a.c.ks) + at;
  const bool whole = from == 0 && to == CACHE_BLOCK;
  su32x4 code[MAX_CHUNKS];
  float old_scale = 0.0f;
  if (!whole) {
#pragma unroll
    for (int n = 0; n < MAX_CHUNKS; ++n)
      if (tid + n * NTH < chunks) code[n] = mem[tid + n * NTH];
    if (a.c.D % 32) {
#pragma unroll
      for (int n = 0; n < MAX_CHUNKS; ++n) {
        const int chunk = tid + n * NTH;
        if (chunk < chunks) code[n] &= bytes_within(w.values, chunk, a.c.D) | ~bytes_of(w.values, chunk, 0, from);
      }
    }
    if (from) {
      old_scale = *scale;
      uint32_t most = 0;     // codes without their sign are in the order of their values
#pragma unroll
      for (int n = 0; n < MAX_CHUNKS; ++n) {
        if (tid + n * NTH >= chunks) break;
        su32x4 c = code[n] & bytes_of(w.values, tid + n * NTH, 0, from);
        c &= ~(nan_codes(c) * 255u) & 0x7F7F7F7Fu;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint32_t b = c[e / 4] >> (8 * (e & 3)) & 255u;
          most = b > most ? b : most;
        }
      }
      float y[4];
      codes4(most, y);
      amax = fabsf(y[0] * old_scale) < INFINITY ? fabsf(y[0] * old_scale) : 0.0f;
    }
  }
#pragma unroll
  for (int n = 0; n < MAX_UNITS; ++n) {
    if (tid + n * NTH >= units) break;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[n][e]) < INFINITY ? fabsf(x[n][e]) : 0.0f);
  }
#pragma unroll
  for (int off = WAVE / 2; off; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off, WAVE));
  if (tid % WAVE == 0) top[tid / WAVE] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NTH / WAVE; ++i) amax = fmaxf(amax, top[i]);
  const int ex = amax > 0.0f ? scale_exponent(amax) : 0;
  const float inv = pow2(-ex), most = ex == 120 ? 240.0f : E4M3_MAX, new_scale = pow2(ex);
#pragma unroll
  for (int n = 0; n < MAX_UNITS; ++n) {
    const int u = tid + n * NTH;
    if (u >= units) break;
    const int row = u / per_row, d = (u - row * per_row) * 8;
    *(su32x2*)&fresh[from + row][d] = su32x2{code4(x[n], inv, most), code4(x[n] + 4, inv, most)};
  }
  __syncthreads();
  const bool again = from && old_scale != new_scale;
#pragma unroll
  for (int n = 0; n < MAX_CHUNKS; ++n) {
    const int chunk = tid + n * NTH;
    if (chunk >= chunks) break;
    const int c = chunk >> 6, q = chunk >> 4 & 3, m = chunk & 15;
    const su32x4 now = bytes_of(w.values, chunk, from, to);
    const bool some = (now[0] | now[1] | now[2] | now[3]) != 0;
    if (!some && !again) continue;
    su32x4 out = whole ? su32x4{0, 0, 0, 0} : code[n];
    if (again) {
      const su32x4 kept = bytes_of(w.values, chunk, 0, from) & bytes_within(w.values, chunk, a.c.D);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float y[4];
        codes4(out[e], y);
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] *= old_scale;
        out[e] = (out[e] & ~kept[e]) | (code4(y, inv, most) & kept[e]);
      }
    }
    if (some) {
      su32x4 in{0, 0, 0, 0};
      if (w.values) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int tok = 8 * q + e;
          if (tok < from || tok >= to) continue;
          in[e >> 2] |= (uint32_t)fresh[tok][32 * c + m] << (8 * (e & 3));
          in[2 + (e >> 2)] |= (uint32_t)fresh[tok][32 * c + 16 + m] << (8 * (e & 3));
        }
      } else {
        const int tok = 8 * (m >> 2) + (m & 3), d = 32 * c + 8 * q;
        const su32x2 lo = *(const su32x2*)&fresh[tok][d], hi = *(const su32x2*)&fresh[tok + 4][d];
        in = su32x4{lo[0], lo[1], hi[0], hi[1]};
      }
      out = (out & ~now) | (in & now);
    }
    mem[chunk] = out;
  }
  if (tid == 0) *scale = new_scale;
}

template <typename E, bool FEW, bool WIDE>
__global__ __launch_bounds__((Shape<FEW, WIDE>::NTH)) void write_kernel(CacheRowsArgs a) {
  using S = Shape<FEW, WIDE>;
  __shared__ __attribute__((aligned(16))) uint8_t fresh[CACHE_BLOCK][S::MAX_D + 8];   // new codes, row by row
  __shared__ float top[S::NTH / WAVE];
  const Where w = where(a);
  const Span s = span_of(a.t, w.b);
  if (s.bad || s.rows == 0) return;
  for (int t0 = (s.first / CACHE_BLOCK + w.block) * CACHE_BLOCK; t0 < s.first + s.rows; t0 += CACHE_BLOCK) {
    write_block<E, FEW, WIDE>(a, w, s, t0, fresh, top);
    if (!FEW) return;
    __syncthreads();
  }
}

template <typename E, bool FEW, bool WIDE>
__device__ __forceinline__ void read_block(const CacheRowsArgs& a, const Where& w, const Span& s, int t0, uint8_t* block) {
  constexpr int NTH = Shape<FEW, WIDE>::NTH;
  const int end = s.first + s.rows;
  const int blk = t0 / CACHE_BLOCK, in_page = blk & ((1 << a.c.per_log2) - 1), tid = threadIdx.x;
  const int page = s.bad ? -1 : a.t.table[(int64_t)w.b * a.t.width + (blk >> a.c.per_log2)];
  const bool known = (uint32_t)page < (uint32_t)a.c.pages;
  float scale = NAN;
  if (known) {
    const int64_t at = (((int64_t)page * a.c.heads + w.h) << a.c.per_log2) + in_page;
    const int bytes = a.c.bricks * BRICK;
    const uint8_t* mem = (w.values ? a.c.v : a.c.k) + at * bytes;
    scale = (w.values ? a.c.vs : a.c.ks)[at];
    for (int i = tid * 16; i < bytes; i += NTH * 16) *(su32x4*)(block + i) = __builtin_nontemporal_load((const su32x4*)(mem + i));
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

template <typename E, bool FEW, bool WIDE>
__global__ __launch_bounds__((Shape<FEW, WIDE>::NTH)) void read_kernel(CacheRowsArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t block[Shape<FEW, WIDE>::MAX_D / 32 * BRICK];
  const Where w = where(a);
  Span s = span_of(a.t, w.b);
  if (s.bad) {
    s.first = 0;
    s.rows = a.t.N;
  }
  for (int t0 = (s.first / CACHE_BLOCK + w.block) * CACHE_BLOCK; t0 < s.first + s.rows; t0 += CACHE_BLOCK) {
    read_block<E, FEW, WIDE>(a, w, s, t0, block);
    if (!FEW) return;
    __syncthreads();
  }
}

int64_t grid_of(const CacheRowsArgs& a) {
  return (int64_t)a.t.B * (a.blocks / blocks_of_wg(a)) * a.c.heads * (a.which == 3 ? 2 : 1);
}

template <bool WRITE, typename E, bool FEW, bool WIDE>
int launch(const CacheRowsArgs& a, hipStream_t st) {
  const dim3 grid((uint32_t)grid_of(a)), threads(Shape<FEW, WIDE>::NTH);
  if constexpr (WRITE) write_kernel<E, FEW, WIDE><<<grid, threads, 0, st>>>(a);
  else read_kernel<E, FEW, WIDE><<<grid, threads, 0, st>>>(a);
  return hipGetLastError() != hipSuccess;
}
template <bool WRITE, typename E>
int launch(const CacheRowsArgs& a, hipStream_t st) {
  if (a.blocks <= FEW_BLOCKS)
    return wide(a.c.bricks) ? launch<WRITE, E, true, true>(a, st) : launch<WRITE, E, true, false>(a, st);
  return wide(a.c.bricks) ? launch<WRITE, E, false, true>(a, st) : launch<WRITE, E, false, false>(a, st);
}
template <bool WRITE>
int launch(const CacheRowsArgs& a, hipStream_t st) {
  return a.bf16 ? launch<WRITE, uint16_t>(a, st) : launch<WRITE, float>(a, st);
}

}  // namespace

int launch_cache_write(const CacheRowsArgs& a, hipStream_t st) { return launch<true>(a, st); }
int launch_cache_read(const CacheRowsArgs& a, hipStream_t st) { return launch<false>(a, st); }

}  // namespace sv
