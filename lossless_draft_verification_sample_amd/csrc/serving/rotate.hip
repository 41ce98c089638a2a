// Rotary positions: every head's first R dimensions turned in pairs by the angle
// position * freqs[i].
//
// Bound by memory: each element is read and written once, with three float32
// operations. The angle is the only expensive part (a float64 product, its reduction to
// one turn, a sine and a cosine), and all heads of a row share it, so a workgroup
// takes whole rows: the R/2 sines and cosines of its rows go to LDS once. float64 holds an
// angle of 2^31 positions to 2^-22; float32 would lose 2^-7 of a turn at 131,072.

#include <math.h>

#include "sv_serve.hpp"

namespace sv {
namespace {

constexpr int NTH = 256;
constexpr int MAX_R2 = 512;        // R / 2
constexpr int MAX_ROWS = 8;        // rows of a workgroup

template <typename E>
struct Side {
  const E* x;
  E* y;
  Strides xs, ys;
};

template <int W, typename E>
__device__ __forceinline__ void get(const E* p, float (&x)[W]) {
  if constexpr (W == 8) {
    load8(p, x);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) x[i] = elem(p + i);
  }
}
template <int W, typename E>
__device__ __forceinline__ void set(E* p, const float (&x)[W]) {
  if constexpr (W == 8) {
    store8(p, x);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) put(p + i, x[i]);
  }
}

// W pairs a unit; whole units of 8 elements of what is not turned.
template <typename E, bool INTER, int W>
__global__ __launch_bounds__(NTH) void rotate_kernel(RotateArgs a, int per_wg) {
  __shared__ sf32x2 turn[MAX_ROWS * 64 > MAX_R2 ? MAX_ROWS * 64 : MAX_R2];
  const int R2 = a.R / 2, tid = threadIdx.x;
  const int64_t total = (int64_t)a.B * a.N, row0 = (int64_t)blockIdx.x * per_wg;
  for (int i = tid; i < per_wg * R2; i += NTH) {
    const int64_t row = row0 + i / R2;
    if (row >= total) break;
    const int b = (int)(row / a.N), j = (int)(row % a.N);
    const double at = (double)((int64_t)(a.first ? a.first[b] : 0) + j);
    // in turns, to [-1/2, 1/2]: exact up to the product's own rounding
    const double t = at * (a.freqs[i % R2] * 0.15915494309189533577);
    const float r = (float)(t - rint(t));
    float s, c;
    sincospif(2.0f * r, &s, &c);
    turn[i] = sf32x2{c * a.scale, (a.inverse ? -s : s) * a.scale};
  }
  __syncthreads();
  const int heads = a.qh + a.kh;
  const int pairs = R2 / W, rest = a.D - a.R, units = pairs + (rest + 7) / 8;
  for (int r = 0; r < per_wg; ++r) {
    const int64_t row = row0 + r;
    if (row >= total) return;
    const int b = (int)(row / a.N), j = (int)(row % a.N);
    const int used = a.rows ? a.rows[b] : a.N;
    const bool bad = used < 0 || used > a.N;
    if (j >= used && !bad) continue;
    for (int i = tid; i < heads * units; i += NTH) {
      const int head = i / units, u = i - head * units;
      const bool isq = head < a.qh;
      const int h = isq ? head : head - a.qh;
      const Strides xs = isq ? a.qs : a.ks, ys = isq ? a.oqs : a.oks;
      const E* x = (const E*)(isq ? a.q : a.k) + b * xs.b + j * xs.n + h * xs.h;
      E* y = (E*)(isq ? a.oq : a.ok) + b * ys.b + j * ys.n + h * ys.h;
      if (u < pairs) {
        const int p = u * W;
        float lo[W], hi[W], o0[W], o1[W];
        if constexpr (INTER) {
          float both[2 * W];
          if constexpr (W == 4) {
            load8(x + 2 * p, both);
          } else {
            get<2 * W>(x + 2 * p, both);
          }
#pragma unroll
          for (int e = 0; e < W; ++e) {
            lo[e] = both[2 * e];
            hi[e] = both[2 * e + 1];
          }
        } else {
          get<W>(x + p, lo);
          get<W>(x + R2 + p, hi);
        }
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const sf32x2 cs = turn[r * R2 + p + e];
          o0[e] = bad ? NAN : __builtin_fmaf(lo[e], cs[0], -(hi[e] * cs[1]));
          o1[e] = bad ? NAN : __builtin_fmaf(hi[e], cs[0], lo[e] * cs[1]);
        }
        if constexpr (INTER) {
          float both[2 * W];
#pragma unroll
          for (int e = 0; e < W; ++e) {
            both[2 * e] = o0[e];
            both[2 * e + 1] = o1[e];
          }
          set<2 * W>(y + 2 * p, both);
        } else {
          set<W>(y + p, o0);
          set<W>(y + R2 + p, o1);
        }
      } else {
        const int d = a.R + (u - pairs) * 8;
        if (x == y && !bad) continue;
        for (int e = 0; e < 8 && d + e < a.D; ++e) {
          if (bad) put(y + d + e, NAN);
          else y[d + e] = x[d + e];
        }
      }
    }
  }
}

template <typename E, bool INTER>
int launch(const RotateArgs& a, hipStream_t st) {
  const int R2 = a.R / 2;
  int per = R2 ? MAX_R2 / R2 : MAX_ROWS;
  if (per > 4) per = 4;
  const int64_t total = (int64_t)a.B * a.N;
  const int grid = (int)((total + per - 1) / per);
  if (INTER ? R2 % 4 == 0 : R2 % 8 == 0)
    rotate_kernel<E, INTER, INTER ? 4 : 8><<<grid, NTH, 0, st>>>(a, per);
  else if (R2 % 2 == 0)
    rotate_kernel<E, INTER, 2><<<grid, NTH, 0, st>>>(a, per);
  else
    rotate_kernel<E, INTER, 1><<<grid, NTH, 0, st>>>(a, per);
  return hipGetLastError() != hipSuccess;
}

}  // namespace

int launch_rotate(const RotateArgs& a, hipStream_t st) {
  if (a.bf16) return a.inter ? launch<uint16_t, true>(a, st) : launch<uint16_t, false>(a, st);
  return a.inter ? launch<float, true>(a, st) : launch<float, false>(a, st);
}

}  // namespace sv
