// The attention kernel for bfloat16 queries, and the join of units that several workgroups
// shared.

#include "attend_kernel.hpp"

namespace sv {
namespace {

constexpr int JOIN_THREADS = 256, JOIN_PARTS = 16, JOIN_ITEMS = 6;

// Joins columns of a unit: out = sum_w 2^(r_w - M) O_w / sum_w 2^(r_w - M) l_w over its
// workgroups w. Threads first take a column each, for the weights of 16 parts at a time, then four
// dimensions of a column each. Bound by the latency of a chain of reads; units of one workgroup
// end at once.
template <bool F32>
__global__ __launch_bounds__(JOIN_THREADS) void join_kernel(AttendArgs a) {
  __shared__ float weight[JOIN_PARTS][AT_MAX_COLS], sum[AT_MAX_COLS];
  const int per = (a.s.cols_set + a.join_cols - 1) / a.join_cols, tid = threadIdx.x;
  const int unit = blockIdx.x / per;
  const int set = unit % a.s.sets, h = unit / a.s.sets % a.c.heads, b = unit / a.s.sets / a.c.heads;
  const int w0 = a.record[2 * unit], count = a.record[2 * unit + 1];   // only if it has blocks
  const Reach r = reach_of(a, b);
  if (r.blocks == 0 || count <= 1) return;
  const int c0 = blockIdx.x % per * a.join_cols;
  int cols = a.join_cols;                                 // that exist, with rows that are used
  if (cols > a.s.cols_set - c0) cols = a.s.cols_set - c0;
  const int rest = r.rows * a.group - (set * a.s.cols_set + c0);
  if (cols > rest) cols = rest;
  const int dp = a.c.bricks * 32, quads = dp / 4;
  const int64_t size = (int64_t)a.s.cols_set * (dp + 2), head = (int64_t)a.s.cols_set * dp;
  // the first workgroup's part holds the unit's start
  auto part = [&](int n) { return a.partial + ((int64_t)(w0 + n) * 2 + (n == 0 ? 1 : 0)) * size; };
  float M = -INFINITY, L = 0.0f;
  if (tid < cols) {
    bool nan = false;
#pragma unroll 4
    for (int n = 0; n < count; ++n) {
      const float m = part(n)[head + 2 * (c0 + tid)];
      M = fmaxf(M, m);
      nan |= m != m;
    }
    if (nan) M = NAN;
  }
  for (int i0 = 0; i0 < cols * quads; i0 += JOIN_ITEMS * JOIN_THREADS) {
    sf32x4 o[JOIN_ITEMS] = {};
    L = 0.0f;
    for (int n0 = 0; n0 < count; n0 += JOIN_PARTS) {
      const int some = count - n0 < JOIN_PARTS ? count - n0 : JOIN_PARTS;
      __syncthreads();
      if (tid < cols) {
#pragma unroll 4
        for (int n = 0; n < some; ++n) {
          const sf32x2 ml = *(const sf32x2*)(part(n0 + n) + head + 2 * (c0 + tid));
          const float f = ml[0] == -INFINITY ? -1.0f : at_exp2(ml[0] - M);      // -1: it saw nothing
          if (ml[0] != -INFINITY) L += f * ml[1];
          weight[n][tid] = f;
        }
        sum[tid] = L;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < JOIN_ITEMS; ++k) {
        const int i = i0 + k * JOIN_THREADS + tid;
        if (i >= cols * quads) break;
        const int c = i / quads, q = i - c * quads;
#pragma unroll 4
        for (int n = 0; n < some; ++n) {
          const float f = weight[n][c];
          const sf32x4 x = *(const sf32x4*)(part(n0 + n) + (int64_t)(c0 + c) * dp + 4 * q);
          if (!(f < 0.0f)) o[k] += x * f;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < JOIN_ITEMS; ++k) {
      const int i = i0 + k * JOIN_THREADS + tid;
      if (i >= cols * quads) break;
      const int c = i / quads, d = 4 * (i - c * quads), col = set * a.s.cols_set + c0 + c;
      const int j = row_of(a, col), g = col - j * a.group;
      const int64_t at = b * a.os.b + j * a.os.n + (int64_t)(h * a.group + g) * a.os.h + d;
      o[k] *= 1.0f / sum[c];
      if constexpr (F32) put4((float*)a.out + at, o[k], a.c.D - d);
      else put4((uint16_t*)a.out + at, o[k], a.c.D - d);
    }
  }
  if (a.lse && tid < cols) {
    const int col = set * a.s.cols_set + c0 + tid, j = row_of(a, col), g = col - j * a.group;
    a.lse[((int64_t)b * a.t.N + j) * a.qh + h * a.group + g] = (M + __log2f(L)) * 0.69314718055994530942f;
  }
}

}  // namespace

int launch_attend_bf16(const AttendArgs& a, hipStream_t st) { return launch_attend_typed<false>(a, st); }

int launch_attend(const AttendArgs& a, hipStream_t st) {
  if (a.bf16 ? launch_attend_bf16(a, st) : launch_attend_f32(a, st)) return 1;
  const int per = (a.s.cols_set + a.join_cols - 1) / a.join_cols;
  const dim3 grid((uint32_t)((int64_t)a.t.B * a.c.heads * a.s.sets * per));
  if (a.bf16) join_kernel<false><<<grid, JOIN_THREADS, 0, st>>>(a);
  else join_kernel<true><<<grid, JOIN_THREADS, 0, st>>>(a);
  return hipGetLastError() != hipSuccess;
}

}  // namespace sv
