// Attention of a round's rows over the 8-bit cache.
//
// For each cache head the N rows of a request and the `group` query heads that share it make
// C = N * group columns. With K a block's keys (32 tokens), Q the columns' queries:
//   S = K Q            16x16x32 matrix instructions, tokens by columns
//   P = exp2(c S - r)  c = k_scale * scale * log2 e, r the column's reference
//   O += V^T (v_scale P)   dimensions by columns, l += sum P
// A wave takes whole blocks on its own. Every operand is in place without a shuffle: the
// cache's bricks hold keys and values in the order of the instruction's A operand, and the
// tokens of a brick of keys are ordered so that the 8 tokens whose scores a lane gets are the
// 8 tokens of the lane's part of the B operand of the second product.
//
// Bound by the cache's bytes: 64 * head_dim a block for 2 * 64 * head_dim * columns
// operations. Loads go straight to registers, 16 bytes a lane and 1 KB a wave; the next
// block's keys are asked for as soon as this block's are used up, its values likewise, so
// that about one block a wave is in flight all the time.
//
// The reference r is not the running maximum but a score near it, moved only when a score
// exceeds it by 2^16; so a block costs no reduction over lanes and O is rescaled hardly ever.
// Float32 holds sums relative to any such reference as exactly as relative to the maximum.
//
// Workgroups share out the blocks of all requests evenly, whatever their lengths: with T blocks
// over all units (request, cache head, set of columns), workgroup w takes blocks
// T w / W .. T (w + 1) / W - 1. Units that several workgroups share leave their parts
// (O, r, l) in the workspace, and a second kernel joins them in the order of the workgroups.
#pragma once

#include <math.h>

#include "sv_serve.hpp"

namespace sv {

constexpr float AT_SLACK = 16.0f;      // how far a score may pass the reference (base 2)
constexpr int AT_LEAST = 4;            // blocks of a workgroup at least: one a wave

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

// 8 codes as bfloat16, which holds them exactly.
__device__ __forceinline__ sbf16x8 codes8(uint32_t lo, uint32_t hi) {
  const sbf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const sbf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const sbf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const sbf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
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

__device__ __forceinline__ int64_t wave_sum64(int64_t v) {
#pragma unroll
  for (int off = WAVE / 2; off; off >>= 1) v += __shfl_xor(v, off, WAVE);
  return v;
}

// Bits of the bytes that are NaN codes (0x7F, 0xFF), one a byte at bit 0.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  const uint32_t x = (w & 0x7F7F7F7Fu) ^ 0x7F7F7F7Fu;       // 0 in a byte of NaN
  return (((x + 0x7F7F7F7Fu) >> 7) & 0x01010101u) ^ 0x01010101u;
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

constexpr int at_waves_per_simd(int bricks, int nt) {
  // registers of a lane: sums, a block's codes, scores and parts, the rest
  const int need = 8 * bricks * nt + 8 * bricks + 16 * nt + 56;
  return need <= 128 ? 4 : need <= 168 ? 3 : need <= 256 ? 2 : 1;
}

template <int BRICKS, int NT, bool F32>
__global__ __launch_bounds__(AT_THREADS, at_waves_per_simd(BRICKS, NT)) void attend_kernel(AttendArgs a) {
  constexpr int QP = F32 ? 3 : 1, PP = F32 ? 3 : 2, DT = 2 * BRICKS;
  extern __shared__ char lds[];
  __shared__ float stat[AT_WAVES][NT * 16][2];
  const int tid = threadIdx.x, lane = tid % WAVE, wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
  const int col16 = lane & 15, quad = lane >> 4;
  const int across = a.s.across, along = AT_WAVES / across;
  const int side = wave % across, turn = wave / across;
  const int U = a.c.heads * a.s.sets;

  // the blocks of all requests, and this workgroup's share of them
  int64_t T = 0;
  for (int b = lane; b < a.t.B; b += WAVE) T += (int64_t)reach_of(a, b).blocks * U;
  T = wave_sum64(T);
  int64_t W = T / AT_LEAST;
  W = W < 1 ? 1 : W > (int64_t)gridDim.x ? (int64_t)gridDim.x : W;
  const int64_t wg = blockIdx.x;
  if (wg >= W || T == 0) return;
  int64_t x = T * wg / W;
  const int64_t x1 = T * (wg + 1) / W;
  if (x >= x1) return;
  // the request of block x
  int64_t before = 0;      // blocks of the requests before b
  int b = 0;
  for (int b0 = 0; b0 < a.t.B; b0 += WAVE) {
    const int64_t mine = b0 + lane < a.t.B ? (int64_t)reach_of(a, b0 + lane).blocks * U : 0;
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
  b = __builtin_amdgcn_readfirstlane(b);

  while (x < x1) {
    // a segment: this workgroup's blocks of one unit
    Reach r = reach_of(a, b);
    while ((int64_t)r.blocks * U <= x - before) {      // also requests without blocks
      before += (int64_t)r.blocks * U;
      r = reach_of(a, ++b);
    }
    const int unit = (int)((x - before) / r.blocks);
    const int64_t unit0 = before + (int64_t)unit * r.blocks;
    const int i0 = (int)(x - unit0);
    const int i1 = (int)((x1 < unit0 + r.blocks ? x1 : unit0 + r.blocks) - unit0);
    const int h = unit / a.s.sets, set = unit % a.s.sets;
    const int col0 = (set * across + side) * NT * 16;   // this wave's first column
    const int C = a.s.cols;

    // queries into LDS, in the order of the B operand: [part][tile][brick][lane] 16 bytes
    {
      const int tiles = across * NT;
      for (int i = tid; i < tiles * BRICKS * WAVE; i += AT_THREADS) {
        const int l = i % WAVE, c = i / WAVE % BRICKS, t = i / WAVE / BRICKS;
        const int col = set * a.s.cols_set + t * 16 + (l & 15), d = 32 * c + 8 * (l >> 4);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = 0.0f;
        if (col < C && d < a.c.D) {
          const int j = col / a.group, g = col % a.group;
          const int64_t at = b * a.qs.b + j * a.qs.n + (int64_t)(h * a.group + g) * a.qs.h + d;
          if (d + 8 <= a.c.D) {
            if constexpr (F32) load8((const float*)a.q + at, y);
            else load8((const uint16_t*)a.q + at, y);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (d + e < a.c.D) y[e] = F32 ? elem((const float*)a.q + at + e) : elem((const uint16_t*)a.q + at + e);
          }
        }
        sbf16x8 p[QP];
        split8<QP>(y, p);
#pragma unroll
        for (int n = 0; n < QP; ++n) ((sbf16x8*)lds)[n * tiles * BRICKS * WAVE + i] = p[n];
      }
    }
    __syncthreads();

    sf32x4 O[NT][DT];
    float l[NT], sub[NT], thr[NT];
    int last[NT];                                        // the last position a column sees
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < DT; ++i) O[t][i] = sf32x4{0, 0, 0, 0};
      l[t] = sub[t] = 0.0f;
      thr[t] = -INFINITY;
      last[t] = r.first + (col0 + t * 16 + col16) / a.group;
    }
    const int end = r.first + r.rows;
    const int open0 = a.window ? end - a.window : 0;     // from here to r.first all rows see all
    const sbf16x8* qf = (const sbf16x8*)lds + side * NT * BRICKS * WAVE + lane;
    const int q_part = across * NT * BRICKS * WAVE;

    su32x4 kraw[BRICKS], vraw[BRICKS];
    float ks = 0, vs = 0, ks_next = 0, vs_next = 0;
    bool lost = false, lost_next = false;
    // asks for a block's keys; where it lies is kept for its values
    int64_t at_next = 0;
    auto locate = [&](int i) {
      const int blk = r.block0 + i;
      int page = r.bad ? -1 : a.t.table[(int64_t)b * a.t.width + (blk >> a.c.per_log2)];
      page = __builtin_amdgcn_readfirstlane(page);
      lost_next = (uint32_t)page >= (uint32_t)a.c.pages;
      if (lost_next) page = 0;
      at_next = (((int64_t)page * a.c.heads + h) << a.c.per_log2) + (blk & ((1 << a.c.per_log2) - 1));
      ks_next = a.c.ks[at_next];
      vs_next = lost_next ? 1.0f : a.c.vs[at_next];
    };
    auto load = [&](const uint8_t* base, su32x4 (&raw)[BRICKS]) {
      const su32x4* p = (const su32x4*)(base + at_next * (BRICKS * BRICK)) + lane;
#pragma unroll
      for (int c = 0; c < BRICKS; ++c) raw[c] = p[c * WAVE];
    };
    int i = i0 + turn;
    if (i < i1) {
      locate(i);
      load(a.c.k, kraw);
      load(a.c.v, vraw);
    }
    for (; i < i1; i += along) {
      const int t0 = (r.block0 + i) * CACHE_BLOCK;
      ks = ks_next * a.scale2;
      vs = vs_next;
      lost = lost_next;
      const bool more = i + along < i1;
      if (more) locate(i + along);

      sf32x4 S[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) S[t][0] = S[t][1] = sf32x4{0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < BRICKS; ++c) {
        const sbf16x8 k0 = codes8(kraw[c][0], kraw[c][1]), k1 = codes8(kraw[c][2], kraw[c][3]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int n = 0; n < QP; ++n) {
            const sbf16x8 q = qf[n * q_part + (t * BRICKS + c) * WAVE];
            S[t][0] = mma(k0, q, S[t][0]);
            S[t][1] = mma(k1, q, S[t][1]);
          }
        }
      }
      if (more) load(a.c.k, kraw);

      // whether some row does not see some token here, or the page is unknown
      const bool edge = t0 + CACHE_BLOCK - 1 > r.first || t0 < open0 || lost;
      float p[NT][8], most[NT];
      bool moved = false;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[t][e] = S[t][e >> 2][e & 3] * ks;
        if (edge) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int pos = t0 + 8 * quad + e;
            if (lost) p[t][e] = NAN;
            if (pos > last[t] || (a.window && pos <= last[t] - a.window)) p[t][e] = -INFINITY;
          }
        }
        most[t] = fmaxf(fmaxf(fmaxf(p[t][0], p[t][1]), fmaxf(p[t][2], p[t][3])),
                        fmaxf(fmaxf(p[t][4], p[t][5]), fmaxf(p[t][6], p[t][7])));
        moved |= most[t] > thr[t];
      }
      if (__any(moved)) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float m = most[t];
          m = fmaxf(m, __shfl_xor(m, 16, WAVE));
          m = fmaxf(m, __shfl_xor(m, 32, WAVE));
          if (m > thr[t]) {
            const float f = thr[t] == -INFINITY ? 1.0f : at_exp2(sub[t] - m);
#pragma unroll
            for (int k = 0; k < DT; ++k) O[t][k] *= f;
            l[t] *= f;
            sub[t] = m;
            thr[t] = m + AT_SLACK;
          }
        }
      }
      // values of tokens that no row sees may be anything, and NaN times 0 is NaN
      uint32_t nan0[BRICKS], nan1[BRICKS], nan2[BRICKS], nan3[BRICKS];
      bool some_nan = false;
      if (edge) {
        const int left = end - (t0 + 8 * quad);
        const uint32_t m0 = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
        const uint32_t m1 = left >= 8 ? ~0u : left <= 4 ? 0u : (1u << (8 * (left - 4))) - 1u;
#pragma unroll
        for (int c = 0; c < BRICKS; ++c) {
          vraw[c][0] &= m0;
          vraw[c][1] &= m1;
          vraw[c][2] &= m0;
          vraw[c][3] &= m1;
          nan0[c] = nan_codes(vraw[c][0]);
          nan1[c] = nan_codes(vraw[c][1]);
          nan2[c] = nan_codes(vraw[c][2]);
          nan3[c] = nan_codes(vraw[c][3]);
          some_nan |= (nan0[c] | nan1[c] | nan2[c] | nan3[c]) != 0;
          vraw[c][0] &= ~(nan0[c] * 255u);
          vraw[c][1] &= ~(nan1[c] * 255u);
          vraw[c][2] &= ~(nan2[c] * 255u);
          vraw[c][3] &= ~(nan3[c] * 255u);
        }
        some_nan = __any(some_nan);
      }
      sbf16x8 pf[NT][PP];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool seen = p[t][e] != -INFINITY;
          w[e] = at_exp2(p[t][e] - sub[t]);
          l[t] += w[e];
          w[e] = edge && !seen ? 0.0f : w[e] * vs;
          p[t][e] = seen ? 1.0f : 0.0f;
        }
        split8<PP>(w, pf[t]);
      }
#pragma unroll
      for (int c = 0; c < BRICKS; ++c) {
        const sbf16x8 v0 = codes8(vraw[c][0], vraw[c][1]), v1 = codes8(vraw[c][2], vraw[c][3]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int n = 0; n < PP; ++n) {
            O[t][2 * c] = mma(v0, pf[t][n], O[t][2 * c]);
            O[t][2 * c + 1] = mma(v1, pf[t][n], O[t][2 * c + 1]);
          }
        }
      }
      if (some_nan) {
        // how many NaN values each column sees of each dimension
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          sbf16x8 seen[1];
          split8<1>(p[t], seen);
#pragma unroll
          for (int c = 0; c < BRICKS; ++c) {
            const sf32x4 zero{0, 0, 0, 0};
            const sf32x4 n0 = mma(ones8(nan0[c], nan1[c]), seen[0], zero);
            const sf32x4 n1 = mma(ones8(nan2[c], nan3[c]), seen[0], zero);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (n0[e] > 0.0f) O[t][2 * c][e] = NAN;
              if (n1[e] > 0.0f) O[t][2 * c + 1][e] = NAN;
            }
          }
        }
      }
      if (more) load(a.c.v, vraw);
    }

    // the waves' parts joined, in the order of the waves
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      l[t] += __shfl_xor(l[t], 16, WAVE);
      l[t] += __shfl_xor(l[t], 32, WAVE);
      if (quad == 0) {
        stat[wave][t * 16 + col16][0] = thr[t] == -INFINITY && l[t] == 0.0f ? -INFINITY : sub[t];
        stat[wave][t * 16 + col16][1] = l[t];
      }
    }
    __syncthreads();       // the queries are free too
    float f[NT][AT_WAVES], M[NT], L[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      M[t] = -INFINITY;
      bool nan = false;
      for (int k = 0; k < along; ++k) {
        const float m = stat[k * across + side][t * 16 + col16][0];
        M[t] = fmaxf(M[t], m);
        nan |= m != m;
      }
      if (nan) M[t] = NAN;
      L[t] = 0.0f;
#pragma unroll
      for (int k = 0; k < AT_WAVES; ++k) {
        f[t][k] = -1.0f;
        if (k < along) {
          const float m = stat[k * across + side][t * 16 + col16][0];
          f[t][k] = m == -INFINITY ? -1.0f : at_exp2(m - M[t]);    // -1: it saw nothing
          if (m != -INFINITY) L[t] += f[t][k] * stat[k * across + side][t * 16 + col16][1];
        }
      }
    }
    const bool all = i0 == 0 && i1 == r.blocks;
    const int64_t unit_id = ((int64_t)b * a.c.heads + h) * a.s.sets + set;
    float* part = a.partial + (wg * 2 + (i0 == 0 ? 1 : 0)) * ((int64_t)a.s.cols_set * (a.c.D + 2));
    if (i0 == 0 && tid == 0) {
      const int64_t y = unit0 + r.blocks - 1;
      a.record[2 * unit_id] = (int32_t)wg;
      a.record[2 * unit_id + 1] = (int32_t)(((y + 1) * W + T - 1) / T - 1 - wg) + 1;
    }
    if (!all && turn == 0 && quad == 0) {
      float* ml = part + (int64_t)a.s.cols_set * a.c.D;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int col = (side * NT + t) * 16 + col16;
        ml[2 * col] = M[t];
        ml[2 * col + 1] = L[t];
      }
    }
    sf32x4* sums = (sf32x4*)lds;                 // [wave][tile of a dimension's 16][NT][lane]
    constexpr int CH = 2;                        // tiles of dimensions a round
#pragma unroll
    for (int d0 = 0; d0 < DT; d0 += CH) {
#pragma unroll
      for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int t = 0; t < NT; ++t) sums[((wave * CH + k) * NT + t) * WAVE + lane] = O[t][d0 + k];
      __syncthreads();
#pragma unroll
      for (int kt = 0; kt < CH * NT; ++kt) {
        if (kt % along != turn) continue;
        const int k = kt / NT, t = kt % NT;
        sf32x4 o{0, 0, 0, 0};
#pragma unroll
        for (int n = 0; n < AT_WAVES; ++n)
          if (n < along) {
            const sf32x4 y = sums[(((n * across + side) * CH + k) * NT + t) * WAVE + lane];
            if (!(f[t][n] < 0.0f)) o += y * f[t][n];
          }
        const int d = 16 * (d0 + k) + 4 * quad, in_set = (side * NT + t) * 16 + col16;
        const int col = set * a.s.cols_set + in_set;
        if (!all) {
          for (int e = 0; e < 4; ++e)
            if (d + e < a.c.D) part[(int64_t)in_set * a.c.D + d + e] = o[e];
        } else if (col < C && col / a.group < r.rows) {
          const int j = col / a.group, g = col % a.group;
          const int64_t at = b * a.os.b + j * a.os.n + (int64_t)(h * a.group + g) * a.os.h + d;
          const float inv = 1.0f / L[t];
          for (int e = 0; e < 4; ++e)
            if (d + e < a.c.D) {
              if constexpr (F32) put((float*)a.out + at + e, o[e] * inv);
              else put((uint16_t*)a.out + at + e, o[e] * inv);
            }
          if (a.lse && d0 + k == 0 && quad == 0)
            a.lse[((int64_t)b * a.t.N + j) * a.qh + h * a.group + g] =
                (M[t] + __log2f(L[t])) * 0.69314718055994530942f;
        }
      }
      __syncthreads();
    }
    x = unit0 + i1;
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
