// Rotary positions: every head's first R dimensions turned in pairs by the angle
// position * freqs[i].
//
// Bound by memory: each element is read and written once, with three float32
// operations. The angle is the only expensive part (a float64 product, its reduction to
// a quarter of a turn, a sine and a cosine), and all heads of a row share it, so a workgroup
// takes whole rows: the R/2 sines and cosines of its rows go to LDS once. float64 holds an
// angle of 2^31 positions to 2^-22; float32 would lose 2^-7 of a turn at 131,072. (1,152 rows of 40
// heads of 128 bfloat16: 7.9 us, 3.0 TB/s, one round of workgroups; 4,593 rows of 16 heads of 96 float32:
// 12.5 us, 4.5 TB/s.)

#include <math.h>

#include "sv_serve.hpp"

namespace sv {
namespace {

constexpr int NTH = 256;
constexpr int MAX_R2 = 512;        // R / 2

// Cosines and sines of this workgroup's rows, times the scale.
__device__ __forceinline__ void make_turns(const RotateArgs& a, sf32x2* turn, int64_t row0, int rows) {
  const int R2 = a.R / 2;
  for (int i = threadIdx.x; i < rows * R2; i += NTH) {
    const int64_t row = row0 + i / R2;
    const int b = (int)(row / a.N), j = (int)(row - (int64_t)b * a.N);
    const double at = (double)((int64_t)(a.first ? a.first[b] : 0) + j);
    // In quarters of a turn, less whole ones: exact up to the product's own rounding. What is left, [-1/2, 1/2], becomes
    // float32, so that a sine or cosine near 0 is as exact, relative to itself, as any other.
    const double t = at * (a.freqs[i % R2] * 0.63661977236758134308), whole = rint(t);
    float u, v;
    sincospif(0.5f * (float)(t - whole), &u, &v);
    // which quarter: whole mod 4, in float64 since whole may be beyond 32 bits
    const int quarter = (int)(whole - 4.0 * floor(0.25 * whole));
    const float s = (quarter & 1 ? v : u) * (quarter & 2 ? -1.0f : 1.0f);
    const float c = (quarter & 1 ? u : v) * (quarter == 1 || quarter == 2 ? -1.0f : 1.0f);
    turn[i] = sf32x2{c * a.scale, (a.inverse ? -s : s) * a.scale};
  }
}

__device__ __forceinline__ void turn_pair(float& x, float& y, sf32x2 cs) {
  const float u = __builtin_fmaf(x, cs[0], -(y * cs[1])), v = __builtin_fmaf(y, cs[0], x * cs[1]);
  x = u;
  y = v;
}

// Where a unit of work lies: a head of a row, and what of it.
template <typename E>
struct Item {
  const E* x;
  E* y;
  int row, unit;
  bool bad;
};
template <typename E>
__device__ __forceinline__ bool item_of(const RotateArgs& a, int64_t row0, int rows, int units, int i, Item<E>* it) {
  const int heads = a.qh + a.kh, per = heads * units, r = i / per, h = (i - r * per) / units;
  if (r >= rows) return false;
  it->row = r;
  it->unit = i - r * per - h * units;
  const int b = (int)((row0 + r) / a.N), j = (int)(row0 + r - (int64_t)b * a.N);
  const int used = a.rows ? a.rows[b] : a.N;
  it->bad = used < 0 || used > a.N;
  if (j >= used && !it->bad) return false;
  const bool isq = h < a.qh;
  const Strides xs = isq ? a.qs : a.ks, ys = isq ? a.oqs : a.oks;
  const int k = isq ? h : h - a.qh;
  it->x = (const E*)(isq ? a.q : a.k) + b * xs.b + j * xs.n + k * xs.h;
  it->y = (E*)(isq ? a.oq : a.ok) + b * ys.b + j * ys.n + k * ys.h;
  return true;
}

// 16 bytes of float32, or of bfloat16, as float32.
__device__ __forceinline__ void open16(const su32x4& w, float (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(w[i]);
}
__device__ __forceinline__ void open16(const su32x4& w, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ su32x4 close16(const float (&x)[4]) {
  return su32x4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
}
__device__ __forceinline__ su32x4 close16(const float (&x)[8]) {
  return su32x4{round_bf16x2(x[0], x[1]), round_bf16x2(x[2], x[3]), round_bf16x2(x[4], x[5]), round_bf16x2(x[6], x[7])};
}

// A unit is two times 16 bytes, of both halves or one after the other, and of the rest of a head too; where
// R/2 or the rest ends inside a unit, that one goes element by element (24,288 rows of 36 heads of 126
// bfloat16: 166 us; a pair a thread for the whole row 248; that unit's elements asked for together 182). Every thread asks for its first MINE units before the angles
// are made.
template <typename E, bool INTER>
__global__ __launch_bounds__(NTH) void rotate_vec_kernel(RotateArgs a, int per_wg, int64_t base) {
  constexpr int W = 16 / (int)sizeof(E), MINE = 2;
  __shared__ __attribute__((aligned(16))) sf32x2 turn[MAX_R2];
  const int R2 = a.R / 2, tid = threadIdx.x;
  const int64_t total = (int64_t)a.B * a.N, row0 = base + (int64_t)blockIdx.x * per_wg;
  const int rows = (int)(total - row0 < per_wg ? total - row0 : per_wg);
  const int pairs = (R2 + W - 1) / W, rest = a.D - a.R;
  const int copies = a.oq == a.q && a.ok == a.k && !a.rows ? 0 : (rest + 2 * W - 1) / (2 * W);
  const int units = pairs + copies, items = rows * (a.qh + a.kh) * units;
  for (int i0 = tid, first = 1; first || i0 - tid < items; i0 += MINE * NTH, first = 0) {
    su32x4 lo[MINE], hi[MINE];
    Item<E> it[MINE];
    bool there[MINE];
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
      there[k] = item_of(a, row0, rows, units, i0 + k * NTH, &it[k]);
      if (!there[k]) continue;
      const int u = it[k].unit, d = u < pairs ? (INTER ? 2 * u * W : u * W) : a.R + (u - pairs) * 2 * W;
      const int d1 = u < pairs && !INTER ? R2 + u * W : d + W;
      if (u < pairs ? (u + 1) * W <= R2 : d1 + W <= a.D) {
        lo[k] = *(const su32x4_any*)(it[k].x + d);
        hi[k] = *(const su32x4_any*)(it[k].x + d1);
      }
    }
    if (first) {
      make_turns(a, turn, row0, rows);
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
      if (!there[k]) continue;
      const int u = it[k].unit;
      if (u < pairs && (u + 1) * W > R2) {
        for (int i = u * W; i < R2; ++i) {
          const int p = INTER ? 2 * i : i, q = INTER ? p + 1 : R2 + i;
          float x = elem(it[k].x + p), y = elem(it[k].x + q);
          turn_pair(x, y, turn[it[k].row * R2 + i]);
          put(it[k].y + p, it[k].bad ? NAN : x);
          put(it[k].y + q, it[k].bad ? NAN : y);
        }
      } else if (u < pairs) {
        float x[W], y[W];
        open16(lo[k], x);
        open16(hi[k], y);
        const sf32x2* cs = turn + it[k].row * R2 + u * W;
        if constexpr (INTER) {
#pragma unroll
          for (int e = 0; e < W; e += 2) {
            turn_pair(x[e], x[e + 1], cs[e / 2]);
            turn_pair(y[e], y[e + 1], cs[W / 2 + e / 2]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < W; ++e) turn_pair(x[e], y[e], cs[e]);
        }
        if (it[k].bad) {
#pragma unroll
          for (int e = 0; e < W; ++e) x[e] = y[e] = NAN;
        }
        *(su32x4_any*)(it[k].y + (INTER ? 2 * u * W : u * W)) = close16(x);
        *(su32x4_any*)(it[k].y + (INTER ? 2 * u * W + W : R2 + u * W)) = close16(y);
      } else {
        const int d = a.R + (u - pairs) * 2 * W;
        if (d + 2 * W <= a.D && !it[k].bad) {
          *(su32x4_any*)(it[k].y + d) = lo[k];
          *(su32x4_any*)(it[k].y + d + W) = hi[k];
        } else {
          for (int e = d; e < d + 2 * W && e < a.D; ++e) {
            if (it[k].bad) put(it[k].y + e, NAN);
            else it[k].y[e] = it[k].x[e];
          }
        }
      }
    }
  }
}

// R/2 below a unit: a pair a thread, then the rest element by element. (8,192 rows of 40 heads of 128 bfloat16 with R = 8:
// 168 us; with R = 16 by the kernel above 32.)
template <typename E, bool INTER>
__global__ __launch_bounds__(NTH) void rotate_any_kernel(RotateArgs a, int per_wg, int64_t base) {
  __shared__ sf32x2 turn[MAX_R2];
  const int R2 = a.R / 2;
  const int64_t total = (int64_t)a.B * a.N, row0 = base + (int64_t)blockIdx.x * per_wg;
  const int rows = (int)(total - row0 < per_wg ? total - row0 : per_wg);
  make_turns(a, turn, row0, rows);
  __syncthreads();
  const int units = R2 + a.D - a.R, items = rows * (a.qh + a.kh) * units;
  for (int i = threadIdx.x; i < items; i += NTH) {
    Item<E> it;
    if (!item_of(a, row0, rows, units, i, &it)) continue;
    if (it.unit < R2) {
      const int p = INTER ? 2 * it.unit : it.unit, q = INTER ? p + 1 : R2 + p;
      float x = elem(it.x + p), y = elem(it.x + q);
      turn_pair(x, y, turn[it.row * R2 + it.unit]);
      put(it.y + p, it.bad ? NAN : x);
      put(it.y + q, it.bad ? NAN : y);
    } else {
      const int d = a.R + it.unit - R2;
      if (it.bad) put(it.y + d, NAN);
      else it.y[d] = it.x[d];
    }
  }
}

template <typename E, bool INTER>
int launch(const RotateArgs& a, hipStream_t st) {
  constexpr int W = 16 / (int)sizeof(E);
  const int R2 = a.R / 2;
  const bool vec = R2 >= W;
  // rows of a workgroup: two units a thread, the angles' room in LDS, and workgroups for the CUs
  const int64_t total = (int64_t)a.B * a.N, units = (a.qh + a.kh) * (int64_t)((a.D + 2 * W - 1) / (2 * W));
  int64_t per = 2 * NTH / units;
  if (per > total / 512) per = total / 512;
  if (R2 && per > MAX_R2 / R2) per = MAX_R2 / R2;
  if (per > 8) per = 8;
  if (per < 1) per = 1;
  // a launch has fewer than 2^32 threads, so rows without end take several
  for (int64_t base = 0; base < total; base += per << 22) {
    const int64_t left = (total - base + per - 1) / per;
    const int grid = (int)(left < 1 << 22 ? left : 1 << 22);
    if (vec) rotate_vec_kernel<E, INTER><<<grid, NTH, 0, st>>>(a, (int)per, base);
    else rotate_any_kernel<E, INTER><<<grid, NTH, 0, st>>>(a, (int)per, base);
    if (hipGetLastError() != hipSuccess) return 1;
  }
  return 0;
}

}  // namespace

int launch_rotate(const RotateArgs& a, hipStream_t st) {
  if (a.bf16) return a.inter ? launch<uint16_t, true>(a, st) : launch<uint16_t, false>(a, st);
  return a.inter ? launch<float, true>(a, st) : launch<float, false>(a, st);
}

}  // namespace sv
