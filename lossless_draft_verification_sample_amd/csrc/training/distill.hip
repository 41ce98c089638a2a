// Distillation of a student row z from a teacher's kept logits (t_k, id_k):
//   p_k = exp(t_k / T - L),  L = log sum_k exp(t_k / T) or the teacher's own
//   log-normaliser;  q = softmax(z / T) over the vocabulary;  P = sum_k p_k
//   loss = sum_k p_k (log p_k - log q_{id_k})
//   d loss / d z_v = (P q_v - p_v) / T,  p_v = sum of the p_k with id_k = v.
// The row's statistics are its largest logit m and logsum = log sum exp((z - m) / T),
// kept apart: their sum would lose logsum where m is large.
//
// Bound: reading the row for the loss, and reading and writing it for the
// gradient. The dense part P q_v is streamed; the K slots are written after it
// by the workgroup that owns their part of the row, so nothing is added
// atomically and repeated ids give one sum.

#include "sv_train.hpp"

namespace sv {

namespace {

constexpr int DIS_THREADS = 512;

struct DisLds {
  int32_t id[DIS_MAX_K];
  float p[DIS_MAX_K];
  double lp[DIS_MAX_K];
  float zid[DIS_MAX_K];     // student logits of the slots, read before they are overwritten
  float red[DIS_THREADS / WAVE];
  double red64[DIS_THREADS / WAVE];
  MaxSum scratch[DIS_THREADS / WAVE];
};

// A slot is filled when its id is a token and its logit is not -inf. (Not its tempered
// logit: that may pass float32's range, but its mass is made in float64.)
__device__ __forceinline__ bool filled(const DistillArgs& a, int32_t id, float t) {
  return id >= 0 && id < a.V && t != -INFINITY;
}

// A row of -inf. One of NaN, or of NaN and -inf, has the largest logit -inf too (NaN do not
// count in a maximum), but a sum of NaN.
__device__ __forceinline__ bool rules_out_all(float m, double logsum) {
  return m == -INFINITY && logsum == -INFINITY;
}

// The loss's terms p (log p - log q) are differences of logarithms that nearly agree
// for the tokens that count, and there are few of them: they are made in float64.
// log q of a kept token with logit z, of a row with these statistics.
__device__ __forceinline__ double log_q(const DistillArgs& a, float z, float m, double logsum) {
  return rules_out_all(m, logsum) ? (double)-INFINITY : ((double)z - (double)m) * a.inv_t64 - logsum;
}

// Teacher's masses of row r into LDS (an empty slot: id -1, mass 0); returns P.
// log p_k, which the loss needs besides, comes back through L.lp: the distance to the
// largest logit less the log of the sum, which would be lost in their sum where the
// logits are large (a teacher row of one far value).
__device__ float teacher(const DistillArgs& a, DisLds& L, int64_t r) {
  const int tid = threadIdx.x;
  float tm = -INFINITY;
  for (int k = tid; k < a.K; k += DIS_THREADS) {
    const int32_t id = a.ids[r * a.K + k];
    const float t = a.tl[r * a.K + k];
    const bool ok = filled(a, id, t);
    L.id[k] = ok ? id : -1;
    L.p[k] = t;
    if (ok) tm = fmaxf(tm, t);
  }
  double lse;
  if (a.tlse) {
    tm = 0.0f;
    lse = a.tlse[r];
  } else {
    tm = block_max<DIS_THREADS>(tm, L.red);
    double s = 0.0;
    for (int k = tid; k < a.K; k += DIS_THREADS)
      if (L.id[k] >= 0) s += exp(((double)L.p[k] - (double)tm) * a.inv_t64);
    s = block_sum<DIS_THREADS>(s, L.red64);
    lse = log(s);
  }
  float P = 0.0f;
  for (int k = tid; k < a.K; k += DIS_THREADS) {
    const double lp = ((double)L.p[k] - (double)tm) * a.inv_t64 - lse;
    L.lp[k] = lp;
    L.p[k] = L.id[k] >= 0 ? (float)exp(lp) : 0.0f;
    P += L.p[k];
  }
  return block_sum<DIS_THREADS>(P, L.red);
}

// loss of row r from its statistics; teacher() has run. All threads get it.
template <typename Elem>
__device__ float row_loss(const DistillArgs& a, DisLds& L, const Row<Elem>& row, float m,
                          double logsum) {
  double l = 0.0;
  for (int k = threadIdx.x; k < a.K; k += DIS_THREADS) {
    const double p = L.id[k] >= 0 ? exp(L.lp[k]) : 0.0;
    if (!(p == 0.0))   // an empty slot, or a mass that is 0: no part in the loss
      l += p * (L.lp[k] - log_q(a, to_f32(row.p + L.id[k]), m, logsum));
  }
  return (float)block_sum<DIS_THREADS>(l, L.red64);
}

// Running set of the groups [v0, v1) of the row, with its head and tail in the
// first and last part.
template <typename Elem>
__device__ MaxSum row_set(const DistillArgs& a, DisLds& L, const Row<Elem>& row, int part, int v0,
                          int v1) {
  constexpr int EPV = Row<Elem>::EPV;
  constexpr int AHEAD = 4;
  const int tid = threadIdx.x;
  Running run;
  float one[1];
  if (part == 0 && tid < row.head) {
    one[0] = to_f32(row.p + tid);
    run.add(one, a.c);
  }
  if (part == a.parts - 1 && tid < row.tail()) {
    one[0] = to_f32(row.p + row.tail0() + tid);
    run.add(one, a.c);
  }
  int j = v0 + tid;
  for (; j + (AHEAD - 1) * DIS_THREADS < v1; j += AHEAD * DIS_THREADS) {
    vu32x4 w[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) w[i] = row.vec(j + i * DIS_THREADS);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      float z[EPV];
      unpack(w[i], z);
      run.add(z, a.c);
    }
  }
  for (; j < v1; j += DIS_THREADS) {
    float z[EPV];
    unpack(row.vec(j), z);
    run.add(z, a.c);
  }
  return block_join<DIS_THREADS>(run.set(a.c), L.scratch, a.c);
}

// The dense part of a row's gradient, w / T P q_v, as scale exp2(z c - ref): ref is the
// whole number next to (m / T + logsum) log2 e, and what the rounding leaves is in the
// scale (from REF_RANGE on, see Running: relative to m).
struct Density {
  float g, scale, ref, m;
  bool none;   // nothing to learn from: no teacher mass, or a row that rules out every token
  __device__ __forceinline__ Density(const DistillArgs& a, float P, float weight, float m_, float logsum) {
    m = m_;
    g = weight * a.inv_t;
    none = P == 0.0f || rules_out_all(m, logsum);
    const float ls2 = logsum * LOG2E;
    if (fabsf(m * a.c) < REF_RANGE) {
      ref = rintf(__builtin_fmaf(m, a.c, ls2));
      scale = g * P * fast_exp2(__builtin_fmaf(-m, a.c, ref) - ls2);
    } else {
      ref = INFINITY;
      scale = g * P * fast_exp2(-ls2);
    }
  }
  template <int N>
  __device__ __forceinline__ void apply(float (&z)[N], float c) const {
    if (none) {
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = 0.0f;
    } else if (ref != INFINITY) {   // of the row: the same in every thread
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = scale * fast_exp2(__builtin_fmaf(z[i], c, -ref));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = scale * fast_exp2((z[i] - m) * c);
    }
  }
};

// Gradient of the groups [v0, v1) (and head or tail); teacher() has run.
template <typename Elem>
__device__ void row_grad(const DistillArgs& a, DisLds& L, const Row<Elem>& row, int64_t r, int part,
                         int v0, int v1, float P, float m, float logsum) {
  constexpr int EPV = Row<Elem>::EPV;
  const int tid = threadIdx.x;
  Elem* out = (Elem*)a.grad + r * a.grad_stride;
  const Density d(a, P, a.weight ? a.weight[r] : 1.0f, m, logsum);
  const int lo = part == 0 ? 0 : row.head + v0 * EPV;
  const int hi = part == a.parts - 1 ? a.V : row.head + v1 * EPV;
  // the slots' student logits, before an in-place gradient overwrites them
  for (int k = tid; k < a.K; k += DIS_THREADS) {
    const int id = L.id[k];
    if (id >= lo && id < hi) L.zid[k] = to_f32(row.p + id);
  }
  __syncthreads();
  // the output row has its own alignment; a store takes any
  const bool same = (((uintptr_t)out ^ (uintptr_t)row.p) & 15u) == 0;
  auto single = [&](int v) {
    float z[1] = {to_f32(row.p + v)};
    d.apply(z, a.c);
    put(out + v, z[0]);
  };
  if (part == 0 && tid < row.head) single(tid);
  if (part == a.parts - 1 && tid < row.tail()) single(row.tail0() + tid);
  for (int j = v0 + tid; j < v1; j += DIS_THREADS) {
    float z[EPV];
    unpack(row.vec(j), z);
    d.apply(z, a.c);
    Elem* o = out + row.head + (int64_t)j * EPV;
    const vu32x4 w = pack(z);
    if (same) __builtin_nontemporal_store(w, (vu32x4*)o);
    else __builtin_memcpy(o, &w, 16);
  }
  __syncthreads();   // orders the dense writes before the slots'
  if (d.none) return;
  for (int k = tid; k < a.K; k += DIS_THREADS) {
    const int id = L.id[k];
    if (id < lo || id >= hi) continue;
    float p = 0.0f;
    for (int j = 0; j < a.K; ++j) p += L.id[j] == id ? L.p[j] : 0.0f;
    float z[1] = {L.zid[k]};
    d.apply(z, a.c);
    put(out + id, z[0] - d.g * p);
  }
}

template <typename Elem>
__device__ __forceinline__ void part_of(const Row<Elem>& row, int parts, int part, int* v0, int* v1) {
  const int per = (row.nvec + parts - 1) / parts;
  *v0 = min(row.nvec, part * per);
  *v1 = min(row.nvec, *v0 + per);
}

__device__ __forceinline__ double log_of(const MaxSum& s) {
  return s.m == -INFINITY && s.s == 0.0f ? (double)-INFINITY : log((double)s.s);
}

// One workgroup a row: statistics, loss, gradient.
template <typename Elem>
__global__ __launch_bounds__(DIS_THREADS) void distill_row_kernel(DistillArgs a) {
  __shared__ DisLds L;
  const int64_t r = blockIdx.x;
  const Row<Elem> row(a.logits, a.stride, r, a.V);
  const MaxSum s = row_set(a, L, row, 0, 0, row.nvec);
  const double logsum = log_of(s);
  const float P = teacher(a, L, r);
  const float loss = row_loss(a, L, row, s.m, logsum);
  if (threadIdx.x == 0) {
    a.loss[r] = loss;
    if (a.stats) {
      a.stats[2 * r] = s.m;
      a.stats[2 * r + 1] = (float)logsum;
    }
  }
  if (a.grad) row_grad(a, L, row, r, 0, 0, row.nvec, P, s.m, (float)logsum);
}

// Few rows: the statistics of a part of a row ...
template <typename Elem>
__global__ __launch_bounds__(DIS_THREADS) void distill_part_kernel(DistillArgs a) {
  __shared__ DisLds L;
  const int64_t r = blockIdx.x / a.parts;
  const int part = blockIdx.x % a.parts;
  const Row<Elem> row(a.logits, a.stride, r, a.V);
  int v0, v1;
  part_of(row, a.parts, part, &v0, &v1);
  const MaxSum s = row_set(a, L, row, part, v0, v1);
  if (threadIdx.x == 0) a.sums[blockIdx.x] = s;
}

// ... the join of a row's parts and its loss ...
template <typename Elem>
__global__ __launch_bounds__(DIS_THREADS) void distill_join_kernel(DistillArgs a) {
  __shared__ DisLds L;
  const int64_t r = blockIdx.x;
  const Row<Elem> row(a.logits, a.stride, r, a.V);
  MaxSum s{-INFINITY, 0.0f};
  if ((int)threadIdx.x < a.parts) s = a.sums[r * a.parts + threadIdx.x];
  s = block_join<DIS_THREADS>(s, L.scratch, a.c);
  const double logsum = log_of(s);
  teacher(a, L, r);
  const float loss = row_loss(a, L, row, s.m, logsum);
  if (threadIdx.x == 0) {
    a.loss[r] = loss;
    a.stats[2 * r] = s.m;
    a.stats[2 * r + 1] = (float)logsum;
  }
}

// ... and the gradient of a part, from the statistics.
template <typename Elem>
__global__ __launch_bounds__(DIS_THREADS) void distill_grad_kernel(DistillArgs a) {
  __shared__ DisLds L;
  const int64_t r = blockIdx.x / a.parts;
  const int part = blockIdx.x % a.parts;
  const Row<Elem> row(a.logits, a.stride, r, a.V);
  int v0, v1;
  part_of(row, a.parts, part, &v0, &v1);
  const float P = teacher(a, L, r);
  row_grad(a, L, row, r, part, v0, v1, P, a.stats[2 * r], a.stats[2 * r + 1]);
}

struct DisHoldLds {
  int32_t id[DIS_MAX_K];
  float p[DIS_MAX_K];
  float red[HOLD_THREADS / WAVE];
  double red64[HOLD_THREADS / WAVE];
  MaxSum scratch[HOLD_THREADS / WAVE];
};

// Many rows that fit a CU's registers: each is read once, for the statistics, the
// loss and the gradient.
template <typename Elem, int SIZE>
__global__ __launch_bounds__(HOLD_THREADS, 2 * HOLD_PER_CU[SIZE]) void distill_hold_kernel(DistillArgs a) {
  constexpr int NV = HOLD_NV[SIZE];
  constexpr int EPV = Held<Elem, NV>::EPV;
  constexpr int SLOTS = DIS_MAX_K / HOLD_THREADS;
  __shared__ DisHoldLds L;
  const int tid = threadIdx.x;
  Held<Elem, NV> h;
  int32_t id[SLOTS];     // this thread's slots of the row: id (-1: empty),
  float t[SLOTS], zs[SLOTS];   // teacher's logit, student's logit
  auto slots = [&](int64_t r) {
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int k = tid + i * HOLD_THREADS;
      id[i] = k < a.K ? a.ids[r * a.K + k] : -1;
      t[i] = k < a.K ? a.tl[r * a.K + k] : 0.0f;
    }
  };
  auto gather = [&](const Row<Elem>& row) {
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      if (!filled(a, id[i], t[i])) id[i] = -1;
      zs[i] = id[i] >= 0 ? to_f32(row.p + id[i]) : 0.0f;
    }
  };
  int64_t r = blockIdx.x;
  Row<Elem> row(a.logits, a.stride, r, a.V);
  slots(r);
  h.load(row);
  gather(row);
  while (true) {
    const int64_t next = r + gridDim.x;
    const bool more = next < a.R;
    const Row<Elem> after(a.logits, a.stride, more ? next : r, a.V);
    Running run;
    {
      const float one[1] = {h.edge};
      run.add(one, a.c);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i * HOLD_THREADS < row.nvec) {
        float z[EPV];
        h.get(i, z);
        run.add(z, a.c);
      }
    }
    const MaxSum sum = block_join<HOLD_THREADS>(run.set(a.c), L.scratch, a.c);
    const float m = sum.m;
    const double logsum = log_of(sum);

    double lse;   // log p_k: as teacher()'s
    float tm = 0.0f;
    if (a.tlse) {
      lse = a.tlse[r];
    } else {
      double ts = 0.0;
      tm = -INFINITY;
#pragma unroll
      for (int i = 0; i < SLOTS; ++i)
        if (id[i] >= 0) tm = fmaxf(tm, t[i]);
      tm = block_max<HOLD_THREADS>(tm, L.red);
#pragma unroll
      for (int i = 0; i < SLOTS; ++i)
        if (id[i] >= 0) ts += exp(((double)t[i] - (double)tm) * a.inv_t64);
      lse = log(block_sum<HOLD_THREADS>(ts, L.red64));
    }
    float P = 0.0f;
    double loss = 0.0;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int k = tid + i * HOLD_THREADS;
      const double lp = ((double)t[i] - (double)tm) * a.inv_t64 - lse;
      const double p = id[i] >= 0 ? exp(lp) : 0.0;
      P += (float)p;
      if (!(p == 0.0))   // an empty slot, or a mass that is 0: no part in the loss
        loss += p * (lp - log_q(a, zs[i], m, logsum));
      if (k < a.K) {
        L.id[k] = id[i];
        L.p[k] = (float)p;
      }
    }
    loss = block_sum<HOLD_THREADS>(loss, L.red64);
    if (tid == 0) {
      a.loss[r] = (float)loss;
      a.stats[2 * r] = m;
      a.stats[2 * r + 1] = (float)logsum;
    }
    P = block_sum<HOLD_THREADS>(P, L.red);
    Elem* out = (Elem*)a.grad + r * a.grad_stride;
    const Density d(a, P, a.weight ? a.weight[r] : 1.0f, m, (float)logsum);
    // this row's slots stay in registers; the next row's are on their way
    int32_t mine[SLOTS];
    float mz[SLOTS];
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      mine[i] = id[i];
      mz[i] = zs[i];
    }
    if (more) slots(next);
    const bool same = (((uintptr_t)out ^ (uintptr_t)row.p) & 15u) == 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i * HOLD_THREADS < row.nvec) {
        const int j = h.index(i);
        float z[EPV];
        h.get(i, z);
        d.apply(z, a.c);
        if (j < row.nvec) {
          Elem* o = out + row.head + (int64_t)j * EPV;
          const vu32x4 g = pack(z);
          if (same) __builtin_nontemporal_store(g, (vu32x4*)o);
          else __builtin_memcpy(o, &g, 16);
        }
      }
      if (more && i * HOLD_THREADS < after.nvec) h.load_group(after, i);
    }
    const int edge = Held<Elem, NV>::edge_id(row);
    if (edge >= 0) {
      float z[1] = {h.edge};
      d.apply(z, a.c);
      put(out + edge, z[0]);
    }
    if (more) {
      h.load_edge(after);
      gather(after);
    }
    __syncthreads();   // orders the dense writes before the slots'
    if (!d.none) {
#pragma unroll
      for (int i = 0; i < SLOTS; ++i) {
        if (mine[i] < 0) continue;
        float p = 0.0f;
        for (int j = 0; j < a.K; ++j) p += L.id[j] == mine[i] ? L.p[j] : 0.0f;
        float z[1] = {mz[i]};
        d.apply(z, a.c);
        put(out + mine[i], z[0] - d.g * p);
      }
    }
    if (!more) break;
    r = next;
    row = after;
  }
}

template <typename Elem>
int distill(const DistillArgs& a, bool backward, hipStream_t st) {
  const dim3 block(DIS_THREADS), rows((uint32_t)a.R), all((uint32_t)a.R * (uint32_t)a.parts);
  if (!backward && a.hold >= 0) {
    const int most = HOLD_CUS * HOLD_PER_CU[a.hold];
    const dim3 grid((uint32_t)(a.R < most ? a.R : most)), held(HOLD_THREADS);
    if (a.hold == 0)
      hipLaunchKernelGGL((distill_hold_kernel<Elem, 0>), grid, held, 0, st, a);
    else if (a.hold == 1)
      hipLaunchKernelGGL((distill_hold_kernel<Elem, 1>), grid, held, 0, st, a);
    else if (a.hold == 2)
      hipLaunchKernelGGL((distill_hold_kernel<Elem, 2>), grid, held, 0, st, a);
    else
      hipLaunchKernelGGL((distill_hold_kernel<Elem, 3>), grid, held, 0, st, a);
  } else if (!backward && a.parts == 1) {
    hipLaunchKernelGGL(distill_row_kernel<Elem>, rows, block, 0, st, a);
  } else {
    if (!backward) {
      hipLaunchKernelGGL(distill_part_kernel<Elem>, all, block, 0, st, a);
      hipLaunchKernelGGL(distill_join_kernel<Elem>, rows, block, 0, st, a);
    }
    if (a.grad) hipLaunchKernelGGL(distill_grad_kernel<Elem>, all, block, 0, st, a);
  }
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace

int launch_distill(const DistillArgs& a, int bf16, hipStream_t st) {
  return bf16 ? distill<uint16_t>(a, false, st) : distill<float>(a, false, st);
}
int launch_distill_backward(const DistillArgs& a, int bf16, hipStream_t st) {
  return bf16 ? distill<uint16_t>(a, true, st) : distill<float>(a, true, st);
}

}  // namespace sv
