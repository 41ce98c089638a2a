// Attention of a round's rows over the 8-bit cache.
//
// For each cache head the N rows of a request and the `group` query heads that share it make
// C = N * group columns. With K a block's keys (32 tokens), Q the columns' queries:
//   S = K Q            16x16x32 matrix instructions, tokens by columns
//   P = exp2(c S - r)  c = k_scale * scale * log2 e, r the column's reference
//   O += V^T P         dimensions by columns, V = v_scale * code; l += sum P
// Keys become bfloat16, which holds their codes and bfloat16 queries exactly. For bfloat16
// outputs P is taken as two bfloat16 parts, each weight to 2^-17 of itself however small it is beside the
// others, and V is code * v_scale / 2^e in bfloat16, exact for powers of two within 2^-100 .. 2^30 of 2^e;
// where a scale lies above, e is moved and O with it. For float32, P v_scale is taken as three bfloat16
// parts. (P as one float16, whose steps end at 2^-24, is faster: 225 us instead of 242 for the ragged batch
// below, 184 instead of 212 for the long requests. But where one token has nearly all the weight and the
// value 0, outputs are made of the small weights, and with the others' scores 17 below its they were off by 44%.)
// A wave takes whole blocks on its own. Every operand is in place without a shuffle: the
// cache's bricks hold keys and values in the order of the instruction's A operand, and the
// tokens of a brick of keys are ordered so that the 8 tokens whose scores a lane gets are the
// 8 tokens of the lane's part of the B operand of the second product.
//
// Bound by the cache's bytes: 64 * head_dim a block for 2 * 64 * head_dim * columns
// operations. Loads go straight to registers, 16 bytes a lane and 1 KB a wave; the next
// block's keys are asked for as soon as this block's are used up, its values likewise, so
// that about one block a wave is in flight all the time. (Four requests of 131,072 tokens, 40 columns:
// 201 to 211 us, 5.2 TB/s; 128 requests of 100 to 8,192, 36 columns: 242 to 250 us with the join, 4.5 TB/s; 8,192 each, four
// columns: 354 us with all launches, 6.1 TB/s. With three tiles of columns vector instructions take 51 to 55% of the
// cycles, most on weights and their parts, and matrix instructions 29 to 34%, hardly side by side with two waves a SIMD.)
//
// The reference r is not the running maximum but a score near it, moved only when a score
// exceeds it by 8, so that weights stay below 256; so a block costs no reduction over lanes and O is rescaled hardly ever.
// Float32 holds sums relative to any such reference as exactly as relative to the maximum.
//
// Workgroups share out the blocks of all requests evenly, whatever their lengths: with T blocks
// over all units (request, cache head, set of columns), workgroup w takes blocks
// T w / W .. T (w + 1) / W - 1. Units that several workgroups share leave their parts
// (O, r, l) in the workspace, and a second kernel joins them in the order of the workgroups. Where
// 1,120 tokens at most are in reach (page table or window) and that is faster (the rule is where the host
// makes the launch's shape), a unit is one workgroup's, without workspace or join (one token of one request over
// 1,000: 14.2 us instead of 16.8).
#pragma once

#include <math.h>

#include "sv_serve.hpp"

// What no kernel writes while it runs, read through the scalar cache.
#define SCALAR __attribute__((address_space(4)))
#define GLOBAL __attribute__((address_space(1)))

namespace sv {

constexpr float AT_SLACK = 8.0f;       // how far a score may pass the reference (base 2)
constexpr float AT_FAR = 256.0f;       // 2^AT_SLACK
// The reference of a column that has seen no token: finite, so that a masked score's weight is 0,
// and lower than any that a score of float32 products can become and stay finite.
constexpr float AT_NONE = -3.40282346638528859812e38f;
// How far above and below the sums' unit a block's scale may lie (base 2): above, the sums stay finite
// for 2^30 tokens and take the new unit otherwise; below, codes stay exact in bfloat16 and the weights
// take what is left.
constexpr int AT_ABOVE = 30, AT_BELOW = 100;
constexpr int AT_LEAST = 4;            // blocks of a workgroup at least: one a wave
// What starting and ending a unit costs, in blocks, a tile: it counts in the workgroups' shares.
// (Ragged batch of 128 requests, with weights in one float16, which makes a block shorter; three tiles: 8 in all 250 us,
// 16 231, 24 227, 40 231; one tile: 8 200, 24 203.)
constexpr int AT_START = 8;

__device__ __forceinline__ float at_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// The parts of a product's operand: x = sum of PARTS bfloat16 numbers, to 2^-9, -17, -25.
template <int PARTS>
__device__ __forceinline__ void split8(const float (&x)[8], sbf16x8 (&p)[PARTS]) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
  for (int n = 0; n < PARTS; ++n) {
    su32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = round_bf16x2(r[2 * i], r[2 * i + 1]);
      if (n + 1 < PARTS) {
        r[2 * i] -= __uint_as_float(w[i] << 16);
        r[2 * i + 1] -= __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
    p[n] = __builtin_bit_cast(sbf16x8, w);
  }
}

// 8 codes times `grow`, a power of two, as bfloat16: exact from 2^-117 to 2^118.
__device__ __forceinline__ sbf16x8 codes8(uint32_t lo, uint32_t hi, float grow = 1.0f) {
  const sbf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, grow, false);
  const sbf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, grow, true);
  const sbf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, grow, false);
  const sbf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, grow, true);
  return sbf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ sf32x4 mma(sbf16x8 a, sbf16x8 b, sf32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Blocks of a request's units, and the first one.
struct Reach {
  int first, rows, block0, blocks;
  bool bad;
};
__device__ __forceinline__ Reach reach_of(const AttendArgs& a, int b) {
  const Span s = span_of(a.t, b);
  Reach r{s.first, s.rows, 0, 0, s.bad};
  if (s.bad) {             // one block whose scores are all NaN, for all N rows
    r.first = 0;
    r.rows = a.t.N;
    r.blocks = 1;
  } else if (s.rows > 0) {
    const int low = a.window && s.first + 1 > a.window ? s.first + 1 - a.window : 0;
    r.block0 = low / CACHE_BLOCK;
    r.blocks = (s.first + s.rows + CACHE_BLOCK - 1) / CACHE_BLOCK - r.block0;
  }
  return r;
}

// The first lane's value, which the compiler then keeps in scalar registers: a quotient is made
// in vector registers, and loads from an address there do not go through the scalar cache.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32 | (uint32_t)uniform((int)v));
}
__device__ __forceinline__ float uniform(float v) { return __int_as_float(uniform(__float_as_int(v))); }
// A uniform address that stays in scalar registers, with nothing of a lane's added to it ahead of
// its loop.
template <typename P>
__device__ __forceinline__ P scalar(P p) {
  asm volatile("" : "+s"(p));
  return p;
}
__device__ __forceinline__ Reach uniform(Reach r) {
  return Reach{uniform(r.first), uniform(r.rows), uniform(r.block0), uniform(r.blocks), uniform((int)r.bad) != 0};
}

__device__ __forceinline__ int64_t wave_sum64(int64_t v) {
#pragma unroll
  for (int off = WAVE / 2; off; off >>= 1) v += __shfl_xor(v, off, WAVE);
  return v;
}

// 0 / 1 bytes as bfloat16 0.0 / 1.0.
__device__ __forceinline__ sbf16x8 ones8(uint32_t lo, uint32_t hi) {
  su32x4 w;
  w[0] = ((lo & 1u) | ((lo & 0x100u) << 8)) * 0x3F80u;
  w[1] = (((lo >> 16) & 1u) | ((lo >> 8) & 0x10000u)) * 0x3F80u;
  w[2] = ((hi & 1u) | ((hi & 0x100u) << 8)) * 0x3F80u;
  w[3] = (((hi >> 16) & 1u) | ((hi >> 8) & 0x10000u)) * 0x3F80u;
  return __builtin_bit_cast(sbf16x8, w);
}

// The row of a column, by the reciprocal of the query heads that share a cache head.
__device__ __forceinline__ int row_of(const AttendArgs& a, int col) {
  return a.group == 1 ? col : (int)__umulhi((uint32_t)col, a.group_inv);
}

// Up to 4 of 4 values, `left` of them in the row.
__device__ __forceinline__ void put4(float* p, sf32x4 x, int left) {
  if (left >= 4) {
    *(su32x4_any*)p = __builtin_bit_cast(su32x4, x);
  } else {
    for (int e = 0; e < left; ++e) p[e] = x[e];
  }
}
__device__ __forceinline__ void put4(uint16_t* p, sf32x4 x, int left) {
  const su32x2 w{round_bf16x2(x[0], x[1]), round_bf16x2(x[2], x[3])};
  if (left >= 4) {
    *(su32x2_any*)p = w;
  } else {
    for (int e = 0; e < left; ++e) p[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
  }
}

// The kernel's arguments, loaded again: what only the end of a segment needs does not take
// scalar registers from the loop.
__device__ __forceinline__ const AttendArgs& fresh_args() {
  const SCALAR AttendArgs* p = (const SCALAR AttendArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const AttendArgs*)p;
}

template <int BRICKS, int NT, bool F32>
__global__ __launch_bounds__(AT_THREADS, attend_per_cu(BRICKS, NT)) void attend_kernel(AttendArgs a) {
  constexpr int QP = F32 ? 3 : 1, WP = F32 ? 3 : 2, DT = 2 * BRICKS;   // parts of queries and of weights
  extern __shared__ char lds[];
  __shared__ float stat[AT_WAVES][NT * 16][2], total[AT_WAVES * NT * 16][2];
  const int tid = threadIdx.x, lane = tid % WAVE, wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
  const int col16 = lane & 15, quad = lane >> 4;
  const int across = a.s.across, along = uniform(AT_WAVES / across);
  const int turn = uniform(wave / across), side = wave - turn * across;
  const int U = a.c.heads * a.s.sets;

  // the blocks of all requests, and this workgroup's share of them
  auto cost = [&](const Reach& r) { return r.blocks ? (int64_t)(r.blocks + AT_START * NT) * U : 0; };
  const int64_t wg = blockIdx.x;
  int64_t T = 0, W = 1, x = 0, x1 = 0;
  int64_t before = 0;      // cost of the requests before b
  int b = 0;
  if (a.s.single) {        // a unit a workgroup
    b = uniform((int)(wg / U));
    const Reach r = uniform(reach_of(a, b));
    const int n = r.blocks + AT_START * NT;
    if (r.blocks == 0) return;
    x = (int64_t)(wg - (int64_t)b * U) * n;
    x1 = x + n;
  } else {
    for (int b = lane; b < a.t.B; b += WAVE) T += cost(reach_of(a, b));
    T = uniform(wave_sum64(T));
    W = T / AT_LEAST;
    W = W < 1 ? 1 : W > (int64_t)gridDim.x ? (int64_t)gridDim.x : W;
    if (wg >= W || T == 0) return;
    x = uniform(T * wg / W);
    x1 = uniform(T * (wg + 1) / W);
  }
  // the request of x
  for (int b0 = 0; b0 < a.t.B && !a.s.single; b0 += WAVE) {
    const int64_t mine = b0 + lane < a.t.B ? cost(reach_of(a, b0 + lane)) : 0;
    int64_t upto = mine;
#pragma unroll
    for (int off = 1; off < WAVE; off <<= 1) {
      const int64_t o = __shfl_up(upto, off, WAVE);
      if (lane >= off) upto += o;
    }
    const uint64_t past = __ballot(before + upto > x);
    if (past) {
      const int l = __builtin_ctzll(past);
      b = b0 + l;
      before += __shfl(upto - mine, l, WAVE);
      break;
    }
    before += __shfl(upto, WAVE - 1, WAVE);
  }
  b = uniform(b);
  before = uniform(before);

  // A segment: this workgroup's blocks i0 .. i1 - 1 of one unit.
  Reach r = uniform(reach_of(a, b));
  int h = 0, set = 0, i0 = 0, i1 = 0;
  int64_t unit1 = 0;       // where the unit ends
  auto next = [&]() {      // the one at x or after it; false: there is none
    for (; x < x1;) {
      while (cost(r) <= x - before) {                  // also requests without blocks
        before += cost(r);
        r = uniform(reach_of(a, ++b));
      }
      const int n = r.blocks + AT_START * NT, unit = uniform((int)((x - before) / n));
      h = uniform(unit / a.s.sets);
      set = unit - h * a.s.sets;
      unit1 = before + (int64_t)(unit + 1) * n;
      const int64_t stop = x1 < unit1 ? x1 : unit1, zero = unit1 - r.blocks;
      i0 = (int)(x > zero ? x - zero : 0);
      i1 = (int)(stop - zero);
      x = stop;
      if (i1 > i0) return true;                        // not only a unit's start
    }
    return false;
  };

  // Where block i lies: its page is asked for two blocks ahead, its scales one ahead, both
  // through the scalar cache, so that no load waits for an address.
  auto page_of = [&](int i) {
    i = i < i1 ? i : i1 - 1;
    const int64_t at = r.bad ? 0 : (int64_t)b * a.t.width + ((r.block0 + i) >> a.c.per_log2);
    return uniform(*scalar((const SCALAR int32_t*)a.t.table + at));
  };
  const float scale2 = fabsf(a.scale2);
  int page_next = 0;
  int64_t at = 0;
  float ks = 0, vs = 0, ks_next = 0, vs_next = 0;
  bool lost = false, lost_next = false;
  auto locate = [&](int i) {
    lost_next = r.bad || (uint32_t)page_next >= (uint32_t)a.c.pages;
    const int page = lost_next ? 0 : page_next, in_page = (r.block0 + i) & ((1 << a.c.per_log2) - 1);
    at = uniform((((int64_t)page * a.c.heads + h) << a.c.per_log2) + in_page);
    ks_next = uniform(*scalar((const SCALAR float*)a.c.ks + at));
    vs_next = uniform(*scalar((const SCALAR float*)a.c.vs + at));
  };
  su32x4 kraw[BRICKS], vraw[BRICKS];
  auto load = [&](const uint8_t* base, su32x4 (&raw)[BRICKS]) {
    const GLOBAL uint8_t* p = scalar((const GLOBAL uint8_t*)base + at * (BRICKS * BRICK));
#pragma unroll
    for (int c = 0; c < BRICKS; ++c) raw[c] = __builtin_nontemporal_load((const GLOBAL su32x4*)(p + (uint32_t)(lane * 16) + c * BRICK));
  };
  int i = 0;
  auto start = [&]() {     // the wave's first block of a segment
    i = i0 + turn;
    if (i < i1) {
      page_next = page_of(i);
      locate(i);
      page_next = page_of(i + along);
      load(a.c.k, kraw);
      load(a.c.v, vraw);
    }
  };

  if (!next()) return;
  start();
  for (;;) {
    // queries into LDS, in the order of the B operand: [part][tile][brick][lane] 16 bytes; the
    // loads of four go out together
    {
      const AttendArgs& z = fresh_args();
      const int items = across * NT * BRICKS * WAVE;
      for (int n0 = tid; n0 < items; n0 += 4 * AT_THREADS) {
        float y[4][8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int n = n0 + k * AT_THREADS, l = n % WAVE, c = n / WAVE % BRICKS, t = n / WAVE / BRICKS;
          const int col = set * z.s.cols_set + t * 16 + (l & 15), d = 32 * c + 8 * (l >> 4);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[k][e] = 0.0f;
          if (n < items && col < z.s.cols && d < z.c.D) {
            const int j = row_of(z, col), g = col - j * z.group;
            const int64_t from = b * z.qs.b + j * z.qs.n + (int64_t)(h * z.group + g) * z.qs.h + d;
            if (d + 8 <= z.c.D) {
              if constexpr (F32) load8((const float*)z.q + from, y[k]);
              else load8((const uint16_t*)z.q + from, y[k]);
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (d + e < z.c.D)
                  y[k][e] = F32 ? elem((const float*)z.q + from + e) : elem((const uint16_t*)z.q + from + e);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int n = n0 + k * AT_THREADS;
          if (n >= items) break;
          if (z.scale2 < 0.0f) {      // so that a score's factor is never negative
#pragma unroll
            for (int e = 0; e < 8; ++e) y[k][e] = -y[k][e];
          }
          sbf16x8 p[QP];
          split8<QP>(y[k], p);
#pragma unroll
          for (int m = 0; m < QP; ++m) ((sbf16x8*)lds)[m * items + n] = p[m];
        }
      }
    }
    __syncthreads();

    sf32x4 O[NT][DT];
    float l[NT], sub[NT];                                // sub: the column's reference
    bool settled = false;                                // every column has one
    // What the sums are relative to: 2^(eref - 127), the first block's scale, or a larger one's.
    int eref = (int)(__float_as_uint(vs_next) >> 23 & 255);
    if (F32 || lost_next || eref == 0 || eref == 255) eref = 127;
    int last[NT];                                        // the last position a column sees
    const int col0 = (set * across + side) * NT * 16;    // this wave's first column
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int k = 0; k < DT; ++k) O[t][k] = sf32x4{0, 0, 0, 0};
      l[t] = 0.0f;
      sub[t] = AT_NONE;
      last[t] = r.bad ? 0 : r.first + row_of(a, col0 + t * 16 + col16);   // bad: position 0 is NaN to all
    }
    const int end = r.first + r.rows;
    const int open0 = a.window ? end - a.window : 0;     // from here to r.first all rows see all
    const sbf16x8* qf = (const sbf16x8*)lds + side * NT * BRICKS * WAVE + lane;
    const int q_part = across * NT * BRICKS * WAVE;

    for (; i < i1; i += along) {
      // the queries are read from LDS for every block, not kept in registers that the sums need
      if constexpr (NT * BRICKS * QP > 8) asm volatile("" ::: "memory");
      const int t0 = (r.block0 + i) * CACHE_BLOCK;
      ks = ks_next * scale2;
      lost = lost_next;
      vs = lost ? 1.0f : vs_next;                        // the scale read then is another block's, or nobody's
      // some row does not see some token here, or the page is unknown
      const bool edge = t0 + CACHE_BLOCK - 1 > r.first || t0 < open0 || lost;
      const int64_t here = at;
      bool nan_values = false;
      if (edge) {
        // values of tokens that no row sees may be anything, and NaN times 0 is NaN
#pragma unroll
        for (int c = 0; c < BRICKS; ++c) {
          vraw[c] &= tokens_before(end - (t0 + 8 * quad));
          const su32x4 nan = nan_codes(vraw[c]);
          nan_values |= (nan[0] | nan[1] | nan[2] | nan[3]) != 0;
          vraw[c] &= ~(nan * 255u);
        }
        nan_values = __any(nan_values);
      }
      // the codes become numbers first, so that the next block is asked for with the whole of this
      // one's work ahead
      sbf16x8 kf[BRICKS][2], vf[BRICKS][2];
#pragma unroll
      for (int c = 0; c < BRICKS; ++c) {
        kf[c][0] = codes8(kraw[c][0], kraw[c][1]);
        kf[c][1] = codes8(kraw[c][2], kraw[c][3]);
      }
      int up = 0;
      float rho = vs;                                    // what v_scale has besides 2^up; 0, infinities, NaN
      const int ev = (int)(__float_as_uint(vs) >> 23 & 255);
      if (!F32 && vs != 0.0f && ev != 255) {
        if (ev - eref > AT_ABOVE) {
          const float f = ldexpf(1.0f, eref - ev);
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < DT; ++k) O[t][k] *= f;
          eref = ev;
        }
        up = ev - eref < -AT_BELOW ? -AT_BELOW : ev - eref;
        rho = ldexpf(vs, 127 - eref - up);
      }
      const float grow = __uint_as_float((uint32_t)(127 + up) << 23);
#pragma unroll
      for (int c = 0; c < BRICKS; ++c) {
        vf[c][0] = codes8(vraw[c][0], vraw[c][1], grow);
        vf[c][1] = codes8(vraw[c][2], vraw[c][3], grow);
      }
      if (i + along < i1) {
        locate(i + along);
        page_next = page_of(i + 2 * along);
        load(a.c.k, kraw);
        load(a.c.v, vraw);
      }

      sf32x4 S[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) S[t][0] = S[t][1] = sf32x4{0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < BRICKS; ++c) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int n = 0; n < QP; ++n) {
            const sbf16x8 q = qf[n * q_part + (t * BRICKS + c) * WAVE];
            S[t][0] = mma(kf[c][0], q, S[t][0]);
            S[t][1] = mma(kf[c][1], q, S[t][1]);
          }
        }
      }

      if (edge) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int pos = t0 + 8 * quad + e;
            float x = lost ? NAN : S[t][e >> 2][e & 3] * ks;
            if (pos > last[t] || (a.window && pos <= last[t] - a.window)) x = -INFINITY;
            S[t][e >> 2][e & 3] = x;
          }
        ks = 1.0f;
        if (nan_values) {
          // NaN values that some row sees, and maybe not all: they were taken out of the product,
          // and a product of their places with the rows' sight says whose sums are NaN
          const GLOBAL uint8_t* p = scalar((const GLOBAL uint8_t*)a.c.v + here * (BRICKS * BRICK));
#pragma unroll
          for (int c = 0; c < BRICKS; ++c) {
            const su32x4 code = *(const GLOBAL su32x4*)(p + (uint32_t)(lane * 16) + c * BRICK);
            const su32x4 nan = nan_codes(code & tokens_before(end - (t0 + 8 * quad)));
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              float one[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) one[e] = S[t][e >> 2][e & 3] != -INFINITY ? 1.0f : 0.0f;
              sbf16x8 seen[1];
              split8<1>(one, seen);
              const sf32x4 zero{0, 0, 0, 0};
              const sf32x4 n0 = mma(ones8(nan[0], nan[1]), seen[0], zero);
              const sf32x4 n1 = mma(ones8(nan[2], nan[3]), seen[0], zero);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (n0[e] > 0.0f) O[t][2 * c][e] = NAN;
                if (n1[e] > 0.0f) O[t][2 * c + 1][e] = NAN;
              }
            }
          }
        }
      }

      // Weights, and where a column has no reference yet, or a score exceeds it by more than the
      // slack, its reference first.
      float w[NT][8];
      for (bool move = !settled;;) {
        if (move) {
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const sf32x4 x = S[t][0], y = S[t][1];
            float m = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])));
            m *= ks;
            m = fmaxf(m, __shfl_xor(m, 16, WAVE));
            m = fmaxf(m, __shfl_xor(m, 32, WAVE));
            const bool none = sub[t] == AT_NONE;
            if (m > sub[t] + AT_SLACK || (none && m > -INFINITY)) {
              const float f = none ? 1.0f : at_exp2(sub[t] - m);
#pragma unroll
              for (int k = 0; k < DT; ++k) O[t][k] *= f;
              l[t] *= f;
              sub[t] = m;
            }
          }
        }
        float most = 0.0f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            w[t][e] = at_exp2(__builtin_fmaf(S[t][e >> 2][e & 3], ks, -sub[t]));
            most = fmaxf(most, w[t][e]);
          }
        if (move || !__any(most > AT_FAR)) break;
        move = true;
      }
      if (!edge) settled = true;

#pragma unroll
      for (int t = 0; t < NT; ++t)
        l[t] += ((w[t][0] + w[t][1]) + (w[t][2] + w[t][3])) + ((w[t][4] + w[t][5]) + (w[t][6] + w[t][7]));
      if (rho != 1.0f) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 8; ++e) w[t][e] *= rho;
      }
      // tile by tile, so that the parts take the weights' registers
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        sbf16x8 pf[WP];
        split8<WP>(w[t], pf);
#pragma unroll
        for (int n = 0; n < WP; ++n)
#pragma unroll
          for (int c = 0; c < BRICKS; ++c) {
            O[t][2 * c] = mma(vf[c][0], pf[n], O[t][2 * c]);
            O[t][2 * c + 1] = mma(vf[c][1], pf[n], O[t][2 * c + 1]);
          }
      }
    }

    // The next segment's first block is asked for before this one's end is dealt with.
    const bool whole = i0 == 0 && i1 == r.blocks;
    const int slot = i0 == 0, was_b = b, was_h = h, was_set = set, was_rows = r.rows;
    if (i0 == 0 && tid == 0 && !a.s.single) {
      const AttendArgs& z = fresh_args();
      const int64_t unit_id = ((int64_t)b * z.c.heads + h) * z.s.sets + set;
      z.record[2 * unit_id] = (int32_t)wg;
      z.record[2 * unit_id + 1] = (int32_t)((unit1 * W + T - 1) / T - 1 - wg) + 1;
    }
    const bool more_segments = next();
    if (more_segments) start();

    // the waves' parts joined, in the order of the waves
    const AttendArgs z = fresh_args();       // a copy: loaded once, whatever is stored
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      l[t] += __shfl_xor(l[t], 16, WAVE);
      l[t] += __shfl_xor(l[t], 32, WAVE);
      if (quad == 0) {
        // -inf: it saw nothing
        stat[wave][t * 16 + col16][0] = sub[t] == AT_NONE && l[t] == 0.0f ? -INFINITY : sub[t];
        stat[wave][t * 16 + col16][1] = l[t];
      }
    }
    __syncthreads();       // the queries are free too
    float* part = z.partial + (wg * 2 + slot) * ((int64_t)z.s.cols_set * (BRICKS * 32 + 2));
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float ms[AT_WAVES], ls[AT_WAVES], M = -INFINITY, L = 0.0f;
#pragma unroll
      for (int k = 0; k < AT_WAVES; ++k) {
        const int from = k < along ? k * across + side : wave;
        ms[k] = k < along ? stat[from][t * 16 + col16][0] : -INFINITY;
        ls[k] = stat[from][t * 16 + col16][1];
        M = M != M || ms[k] != ms[k] ? NAN : fmaxf(M, ms[k]);
      }
#pragma unroll
      for (int k = 0; k < AT_WAVES; ++k) L += ms[k] == -INFINITY ? 0.0f : at_exp2(ms[k] - M) * ls[k];
      const float mine = stat[wave][t * 16 + col16][0];
      const float f = at_exp2(mine - M) * ldexpf(1.0f, eref - 127);
#pragma unroll
      for (int k = 0; k < DT; ++k) O[t][k] = mine == -INFINITY ? sf32x4{0, 0, 0, 0} : O[t][k] * f;
      if (turn == 0 && quad == 0) {
        const int col = (side * NT + t) * 16 + col16;
        total[col][0] = 1.0f / L;
        total[col][1] = (M + __log2f(L)) * 0.69314718055994530942f;
        if (!whole) {
          float* ml = part + (int64_t)z.s.cols_set * (BRICKS * 32);
          ml[2 * col] = M;
          ml[2 * col + 1] = L;
        }
      }
    }
    sf32x4* sums = (sf32x4*)lds;                 // [wave][16 dimensions of CH][NT][lane]
    constexpr int CH = attend_round(BRICKS, NT);
#pragma unroll
    for (int d0 = 0; d0 < DT; d0 += CH) {
#pragma unroll
      for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int t = 0; t < NT; ++t) sums[((wave * CH + k) * NT + t) * WAVE + lane] = O[t][d0 + k];
      __syncthreads();
      constexpr int STEP = NT >= 3 || BRICKS >= 5 ? 1 : 2;       // items together, where registers are left
      const int items = across * CH * NT * WAVE;
      for (int n0 = tid; n0 < items; n0 += STEP * AT_THREADS) {
        sf32x4 o[STEP], other[STEP][AT_WAVES - 1];
#pragma unroll
        for (int m = 0; m < STEP; ++m) {
          const int n = n0 + m * AT_THREADS < items ? n0 + m * AT_THREADS : n0;
          o[m] = sums[n];
#pragma unroll
          for (int k = 1; k < AT_WAVES; ++k) other[m][k - 1] = sums[(k < along ? k * items : 0) + n];
        }
#pragma unroll
        for (int m = 0; m < STEP; ++m) {
          const int n = n0 + m * AT_THREADS;
          if (STEP > 1 && n >= items) break;
#pragma unroll
          for (int k = 1; k < AT_WAVES; ++k) o[m] += k < along ? other[m][k - 1] : sf32x4{0, 0, 0, 0};
          const int ln = n % WAVE, t = n / WAVE % NT, k = n / WAVE / NT % CH, sd = n / WAVE / NT / CH;
          const int d = 16 * (d0 + k) + 4 * (ln >> 4), in_set = (sd * NT + t) * 16 + (ln & 15);
          const int col = was_set * z.s.cols_set + in_set, j = row_of(z, col);
          if (!whole) {
            *(sf32x4*)(part + (int64_t)in_set * (BRICKS * 32) + d) = o[m];
          } else if (col < z.s.cols && j < was_rows) {
            const int head = was_h * z.group + col - j * z.group;
            const int64_t to = was_b * z.os.b + j * z.os.n + (int64_t)head * z.os.h + d;
            o[m] *= total[in_set][0];
            if constexpr (F32) put4((float*)z.out + to, o[m], z.c.D - d);
            else put4((uint16_t*)z.out + to, o[m], z.c.D - d);
            if (z.lse && d == 0) z.lse[((int64_t)was_b * z.t.N + j) * z.qh + head] = total[in_set][1];
          }
        }
      }
      __syncthreads();
    }
    if (!more_segments) break;
  }
}

// Launchers by type, dispatched on bricks and tiles.
int launch_attend_bf16(const AttendArgs& a, hipStream_t st);
int launch_attend_f32(const AttendArgs& a, hipStream_t st);

template <int BRICKS, bool F32>
int launch_attend_bricks(const AttendArgs& a, hipStream_t st) {
  const dim3 g(a.s.grid), n(AT_THREADS);
  switch (a.s.nt) {
    case 1: attend_kernel<BRICKS, 1, F32><<<g, n, a.s.lds, st>>>(a); break;
    case 2: attend_kernel<BRICKS, 2, F32><<<g, n, a.s.lds, st>>>(a); break;
    case 3:
      if constexpr (BRICKS <= 4) attend_kernel<BRICKS, 3, F32><<<g, n, a.s.lds, st>>>(a);
      else return 1;
      break;
    case 4:
      if constexpr (BRICKS <= 4) attend_kernel<BRICKS, 4, F32><<<g, n, a.s.lds, st>>>(a);
      else return 1;
      break;
    default: return 1;
  }
  return hipGetLastError() != hipSuccess;
}
template <bool F32>
int launch_attend_typed(const AttendArgs& a, hipStream_t st) {
  switch (a.c.bricks) {
    case 1: return launch_attend_bricks<1, F32>(a, st);
    case 2: return launch_attend_bricks<2, F32>(a, st);
    case 3: return launch_attend_bricks<3, F32>(a, st);
    case 4: return launch_attend_bricks<4, F32>(a, st);
    case 5: return launch_attend_bricks<5, F32>(a, st);
    case 6: return launch_attend_bricks<6, F32>(a, st);
    case 7: return launch_attend_bricks<7, F32>(a, st);
    case 8: return launch_attend_bricks<8, F32>(a, st);
  }
  return 1;
}

}  // namespace sv
