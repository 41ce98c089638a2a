// The attention kernel for bfloat16 queries, and the join of units that several workgroups
// shared.

#include "attend_kernel.hpp"

namespace sv {
namespace {

constexpr int JOIN_THREADS = 256, JOIN_AHEAD = 8;

// Joins columns of a unit: out = sum_w 2^(r_w - M) O_w / sum_w 2^(r_w - M) l_w over its
// workgroups w. A thread takes four dimensions of a column through the parts, with the running
// maximum of r_w, so that what it reads depends on nothing but the unit's record: the parts'
// references, sums of weights and sums are asked for together, eight parts at a time (weights
// first, in LDS, then the sums: 7.2 us instead of 4.1 for one token of one request, whose
// reads are a chain). Where units have many parts, GROUPS threads share out those of an item and join
// theirs in LDS, in order (one request of 131,072 tokens, one row, 96 parts: 64 -> 53.5 us with both kernels). Units
// of one workgroup end at once.
template <bool F32, int GROUPS>
__global__ __launch_bounds__(JOIN_THREADS) void join_kernel(AttendArgs a) {
  constexpr int ITEMS = JOIN_THREADS / GROUPS;
  __shared__ float stat[GROUPS > 1 ? JOIN_THREADS : 1][2];
  __shared__ sf32x4 sums[GROUPS > 1 ? JOIN_THREADS : 1];
  const int per = (a.s.cols_set + a.s.join_cols - 1) / a.s.join_cols, tid = threadIdx.x;
  const int item = tid % ITEMS, group = GROUPS == 1 ? 0 : tid / ITEMS;
  const int unit = blockIdx.x / per, slice = blockIdx.x - unit * per;
  const int uh = unit / a.s.sets, set = unit - uh * a.s.sets, b = uh / a.c.heads, h = uh - b * a.c.heads;
  const int w0 = a.record[2 * unit], count = a.record[2 * unit + 1];   // only if it has blocks
  const Reach r = reach_of(a, b);
  if (r.blocks == 0 || count <= 1) return;
  const int c0 = slice * a.s.join_cols, dp = a.c.bricks * 32, quads = dp / 4;
  const int64_t size = (int64_t)a.s.cols_set * (dp + 2), head = (int64_t)a.s.cols_set * dp;
  // the first workgroup's part holds the unit's start: the other of its two
  const float* parts = a.partial + (int64_t)w0 * 2 * size;
  for (int i0 = 0; i0 < a.s.join_cols * quads; i0 += ITEMS) {
    const int i = i0 + item, c = c0 + i / quads, d = 4 * (i % quads), col = set * a.s.cols_set + c, j = row_of(a, col);
    const bool there = i < a.s.join_cols * quads && c < a.s.cols_set && col < a.s.cols && j < r.rows;
    if (GROUPS == 1 && !there) return;
    const int upto = GROUPS == 1 || there ? count : 0;
    float M = -INFINITY, L = 0.0f;
    sf32x4 o{0, 0, 0, 0};
    for (int n0 = group; n0 < upto; n0 += JOIN_AHEAD * GROUPS) {
      sf32x2 ml[JOIN_AHEAD];
      sf32x4 x[JOIN_AHEAD];
#pragma unroll
      for (int k = 0; k < JOIN_AHEAD; ++k) {
        ml[k] = sf32x2{-INFINITY, 0.0f};                    // it saw nothing
        if (n0 + k * GROUPS >= count) continue;
        const int n = n0 + k * GROUPS;
        const float* p = parts + (2 * n + (n == 0 ? 1 : 0)) * size;
        ml[k] = *(const sf32x2*)(p + head + 2 * c);
        x[k] = *(const sf32x4*)(p + (int64_t)c * dp + d);
      }
      float most = M;
#pragma unroll
      for (int k = 0; k < JOIN_AHEAD; ++k) most = most != most || ml[k][0] != ml[k][0] ? NAN : fmaxf(most, ml[k][0]);
      const float f = M == -INFINITY ? 0.0f : at_exp2(M - most);
      L *= f;
      o *= f;
      M = most;
#pragma unroll
      for (int k = 0; k < JOIN_AHEAD; ++k) {
        if (ml[k][0] == -INFINITY) continue;
        const float g = at_exp2(ml[k][0] - M);
        L += g * ml[k][1];
        o += x[k] * g;
      }
    }
    if constexpr (GROUPS > 1) {
      if (i0) __syncthreads();
      stat[tid][0] = M;
      stat[tid][1] = L;
      sums[tid] = o;
      __syncthreads();
      if (group || !there) continue;
      for (int k = 1; k < GROUPS; ++k) {
        const float m = stat[k * ITEMS + item][0];
        M = M != M || m != m ? NAN : fmaxf(M, m);
      }
      L = 0.0f;
      o = sf32x4{0, 0, 0, 0};
      for (int k = 0; k < GROUPS; ++k) {
        const float m = stat[k * ITEMS + item][0];
        if (m == -INFINITY) continue;
        const float g = at_exp2(m - M);
        L += g * stat[k * ITEMS + item][1];
        o += sums[k * ITEMS + item] * g;
      }
    }
    const int head_of = h * a.group + col - j * a.group;
    o *= 1.0f / L;
    const int64_t to = b * a.os.b + j * a.os.n + (int64_t)head_of * a.os.h + d;
    if constexpr (F32) put4((float*)a.out + to, o, a.c.D - d);
    else put4((uint16_t*)a.out + to, o, a.c.D - d);
    if (a.lse && d == 0)
      a.lse[((int64_t)b * a.t.N + j) * a.qh + head_of] = (M + __log2f(L)) * 0.69314718055994530942f;
  }
}

template <bool F32>
void launch_join(const AttendArgs& a, hipStream_t st) {
  const int per = (a.s.cols_set + a.s.join_cols - 1) / a.s.join_cols;
  const dim3 grid((uint32_t)((int64_t)a.t.B * a.c.heads * a.s.sets * per));
  if (a.s.join_split) join_kernel<F32, JOIN_AHEAD><<<grid, JOIN_THREADS, 0, st>>>(a);
  else join_kernel<F32, 1><<<grid, JOIN_THREADS, 0, st>>>(a);
}

}  // namespace

int launch_attend_bf16(const AttendArgs& a, hipStream_t st) { return launch_attend_typed<false>(a, st); }

int launch_attend(const AttendArgs& a, hipStream_t st) {
  if (a.bf16 ? launch_attend_bf16(a, st) : launch_attend_f32(a, st)) return 1;
  if (a.s.single) return 0;
  if (a.bf16) launch_join<false>(a, st);
  else launch_join<true>(a, st);
  return hipGetLastError() != hipSuccess;
}

}  // namespace sv
