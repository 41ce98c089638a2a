// The attention kernel for bfloat16 queries, and the join of units that several workgroups
// shared.

#include "attend_kernel.hpp"

namespace sv {
namespace {

constexpr int JOIN_WAVES = 4;

// A wave joins a column: out = sum_w 2^(r_w - M) O_w / sum_w 2^(r_w - M) l_w over the unit's
// workgroups w. Bound by the latency of reading the parts, which are few.
template <bool F32>
__global__ __launch_bounds__(JOIN_WAVES * WAVE) void join_kernel(AttendArgs a) {
  const int per = (a.s.cols_set + JOIN_WAVES - 1) / JOIN_WAVES;
  const int unit = blockIdx.x / per, lane = threadIdx.x % WAVE;
  const int in_set = blockIdx.x % per * JOIN_WAVES + threadIdx.x / WAVE;
  const int set = unit % a.s.sets, h = unit / a.s.sets % a.c.heads, b = unit / a.s.sets / a.c.heads;
  const Reach r = reach_of(a, b);
  const int col = set * a.s.cols_set + in_set, j = col / a.group, g = col % a.group;
  if (r.blocks == 0 || in_set >= a.s.cols_set || col >= a.s.cols || j >= r.rows) return;
  const int w0 = a.record[2 * unit], count = a.record[2 * unit + 1];
  if (count <= 1) return;
  const int64_t size = (int64_t)a.s.cols_set * (a.c.D + 2), head = (int64_t)a.s.cols_set * a.c.D;
  // the first workgroup's part holds the unit's start
  auto part = [&](int n) { return a.partial + ((int64_t)(w0 + n) * 2 + (n == 0 ? 1 : 0)) * size; };
  float M = -INFINITY;
  bool nan = false;
  for (int n = lane; n < count; n += WAVE) {
    const float m = part(n)[head + 2 * in_set];
    M = fmaxf(M, m);
    nan |= m != m;
  }
#pragma unroll
  for (int off = WAVE / 2; off; off >>= 1) M = fmaxf(M, __shfl_xor(M, off, WAVE));
  if (__any(nan)) M = NAN;
  float L = 0.0f, o[CACHE_MAX_D / WAVE] = {};
  for (int n = 0; n < count; ++n) {
    const float* p = part(n);
    const float m = p[head + 2 * in_set];
    if (m == -INFINITY) continue;
    const float f = at_exp2(m - M);
    L += f * p[head + 2 * in_set + 1];
#pragma unroll
    for (int k = 0; k < CACHE_MAX_D / WAVE; ++k) {
      const int d = k * WAVE + lane;
      if (d < a.c.D) o[k] += f * p[(int64_t)in_set * a.c.D + d];
    }
  }
  const int64_t at = b * a.os.b + j * a.os.n + (int64_t)(h * a.group + g) * a.os.h;
#pragma unroll
  for (int k = 0; k < CACHE_MAX_D / WAVE; ++k) {
    const int d = k * WAVE + lane;
    if (d < a.c.D) {
      if constexpr (F32) put((float*)a.out + at + d, o[k] / L);
      else put((uint16_t*)a.out + at + d, o[k] / L);
    }
  }
  if (a.lse && lane == 0)
    a.lse[((int64_t)b * a.t.N + j) * a.qh + h * a.group + g] = (M + __log2f(L)) * 0.69314718055994530942f;
}

}  // namespace

int launch_attend_bf16(const AttendArgs& a, hipStream_t st) { return launch_attend_typed<false>(a, st); }

int launch_attend(const AttendArgs& a, hipStream_t st) {
  if (a.bf16 ? launch_attend_bf16(a, st) : launch_attend_f32(a, st)) return 1;
  const int per = (a.s.cols_set + JOIN_WAVES - 1) / JOIN_WAVES;
  const dim3 grid((uint32_t)((int64_t)a.t.B * a.c.heads * a.s.sets * per));
  if (a.bf16) join_kernel<false><<<grid, JOIN_WAVES * WAVE, 0, st>>>(a);
  else join_kernel<true><<<grid, JOIN_WAVES * WAVE, 0, st>>>(a);
  return hipGetLastError() != hipSuccess;
}

}  // namespace sv
