// The k largest logits of a vocabulary row and its log-normaliser
//   lse = log sum_v exp(z_v / T)
// in one pass over the row.
//
// A candidate is one 64-bit number: the order-preserving key of its value in
// the upper half, the complement of its id in the lower, so that keys are
// unique and the larger key is the larger logit, or the lower id among equals.
// A workgroup streams its part of a row in steps of 512 groups of 16 bytes; a
// logit above the running threshold is appended to a list in LDS. When the
// next step might not fit, the list is cut to its k largest by a radix
// selection (8 bits a level, from the top, ending as soon as a bin's border is
// the cut), and the threshold rises to the k-th value. Ids rise along the
// stream, so an equal logit that comes later never replaces a listed one and
// the threshold test is a strict comparison. The first step appends everything
// and cuts; from then on about k of every 4096 logits pass. The worst order
// (rising logits) cuts after every step: slow, but right.
//
// Bound: the read of the row. Rows are split over `parts` workgroups when there
// are few of them; the second kernel joins their lists and sums.

#include "sv_train.hpp"

namespace sv {

namespace {

struct TopLds {
  uint64_t buf[TOP_CAP];
  uint32_t hist[256];
  int added[3];         // entries appended by a step, slots in rotation
  int kept;
  int sel_bin, sel_above, sel_count;
  MaxSum scratch[TOP_THREADS / WAVE];
};

__device__ __forceinline__ uint64_t make_key(float z, int id) {
  return ((uint64_t)f32_key(z) << 32) | (uint32_t)~(uint32_t)id;
}

// Appends the lane's flagged entries: one LDS atomic a wave.
template <int N>
__device__ __forceinline__ void append(const float (&z)[N], uint32_t flags, int id0, int base,
                                       int* counter, uint64_t* buf) {
  if (!__any(flags != 0)) return;
  const int n = __popc(flags);
  const int incl = wave_scan_dpp((int32_t)n, (int32_t)0, [](int32_t x, int32_t y) { return x + y; });
  int at = 0;
  if ((threadIdx.x & (WAVE - 1)) == WAVE - 1) at = atomicAdd(counter, incl);
  at = base + lane63((int32_t)at) + incl - n;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if ((flags >> i) & 1u) buf[at++] = make_key(z[i], id0 + i);
}

// Cuts the list of n > K entries to its K largest. Returns a value no greater
// than the smallest kept one, above which later logits still count.
__device__ float cut(TopLds& L, int n, int K, bool bf16, int V) {
  constexpr int PER = TOP_CAP / TOP_THREADS;
  const int tid = threadIdx.x;
  uint64_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = tid + i * TOP_THREADS;
    key[i] = j < n ? L.buf[j] : 0ull;   // 0 is below every candidate
  }
  uint64_t mask = 0, pref = 0;
  int rem = K;
  for (int shift = 56; shift >= 0; shift -= 8) {
    // bits that what is above them decides: the low half of a bfloat16's key,
    // and the high byte of an id below 2^24
    if (bf16 && (shift == 40 || shift == 32)) continue;
    if (shift == 24 && V <= (1 << 24)) continue;
    __syncthreads();
    if (tid < 256) L.hist[tid] = 0;
    if (tid == 0) L.kept = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (key[i] && (key[i] & mask) == pref) atomicAdd(&L.hist[(uint32_t)(key[i] >> shift) & 255u], 1u);
    __syncthreads();
    if (tid < WAVE) {   // bins from the top, four a lane
      int h[4], sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += h[i] = (int)L.hist[255 - 4 * tid - i];
      const int incl =
          wave_scan_dpp((int32_t)sum, (int32_t)0, [](int32_t x, int32_t y) { return x + y; });
      int above = incl - sum;
      if (above < rem && incl >= rem) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (above < rem && above + h[i] >= rem) {
            L.sel_bin = 255 - 4 * tid - i;
            L.sel_above = above;
            L.sel_count = h[i];
          }
          above += h[i];
        }
      }
    }
    __syncthreads();
    mask |= 0xFFull << shift;
    pref |= (uint64_t)(uint32_t)L.sel_bin << shift;
    rem -= L.sel_above;
    if (L.sel_count == rem) break;
  }
  uint32_t flags = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (key[i] && (key[i] & mask) >= pref) flags |= 1u << i;
  const int cnt = __popc(flags);
  const int incl = wave_scan_dpp((int32_t)cnt, (int32_t)0, [](int32_t x, int32_t y) { return x + y; });
  int at = 0;
  if ((tid & (WAVE - 1)) == WAVE - 1) at = atomicAdd(&L.kept, incl);
  at = lane63((int32_t)at) + incl - cnt;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if ((flags >> i) & 1u) L.buf[at++] = key[i];
  __syncthreads();
  const uint32_t vk = (uint32_t)(pref >> 32);
  return vk < 0x00800000u ? -INFINITY : f32_from_key(vk);   // below: no finite value's key
}

// Writes entries 0..K-1 of the list in descending order through `out(rank, key)`;
// ranks past the list's n <= K entries get key 0.
template <typename Out>
__device__ __forceinline__ void write_sorted(TopLds& L, int n, int K, Out out) {
  for (int i = threadIdx.x; i < K; i += TOP_THREADS) {
    if (i >= n) {
      out(i, 0ull);
      continue;
    }
    const uint64_t mine = L.buf[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += L.buf[j] > mine;
    out(rank, mine);
  }
}

__device__ __forceinline__ void put_entry(const TopArgs& a, int64_t r, int rank, uint64_t key) {
  a.ids[r * a.K + rank] = key ? (int32_t)~(uint32_t)key : -1;
  a.values[r * a.K + rank] = key ? f32_from_key((uint32_t)(key >> 32)) : -INFINITY;
}

// lse of a set whose sum is in base-2 exponents of c; m / T is exact where
// T = 1, and -inf for an empty row.
__device__ __forceinline__ float row_lse(const MaxSum& s, float temperature) {
  if (s.m == -INFINITY) return s.s == 0.0f ? -INFINITY : s.s;   // empty; NaN only
  return s.m / temperature + logf(s.s);
}

template <typename Elem>
__global__ __launch_bounds__(TOP_THREADS) void top_scan_kernel(TopArgs a) {
  __shared__ TopLds L;
  constexpr int EPV = Row<Elem>::EPV;
  constexpr int AHEAD = 4;
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x / a.parts;
  const int part = blockIdx.x % a.parts;
  const Row<Elem> row(a.logits, a.stride, r, a.V);
  const int per = (row.nvec + a.parts - 1) / a.parts;
  const int v0 = min(row.nvec, part * per), v1 = min(row.nvec, v0 + per);

  if (tid < 3) L.added[tid] = 0;
  __syncthreads();
  int base = 0, slot = 0;      // entries listed, counter of this step
  float tau = -INFINITY;
  MaxSum sum{-INFINITY, 0.0f};

  auto step = [&](const float (&z)[EPV], int id0) {
    uint32_t flags = 0;
#pragma unroll
    for (int i = 0; i < EPV; ++i) flags |= (z[i] > tau ? 1u : 0u) << i;
    append(z, flags, id0, base, &L.added[slot], L.buf);
    add_logits(sum, z, a.c);
    __syncthreads();
    base += L.added[slot];
    // the counter two steps on: everyone has read it, nobody adds to it yet
    const int next = slot == 2 ? 0 : slot + 1;
    if (tid == 0) L.added[next == 2 ? 0 : next + 1] = 0;
    slot = next;
    if (base > TOP_CAP - TOP_STEP && base > a.K) {
      tau = cut(L, base, a.K, sizeof(Elem) == 2, a.V);
      base = a.K;
    }
  };
  auto singles = [&](int n, int first) {
    float z[EPV];
#pragma unroll
    for (int i = 0; i < EPV; ++i) z[i] = -INFINITY;
    if (tid < n) z[0] = to_f32(row.p + first + tid);
    step(z, first + tid);
  };

  if (part == 0 && row.head) singles(row.head, 0);
  vu32x4 cur[AHEAD], nxt[AHEAD];
  const uint32_t lowest = sizeof(Elem) == 2 ? 0xFF80FF80u : 0xFF800000u;   // -inf
  auto fetch = [&](vu32x4 (&w)[AHEAD], int b) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int j = b + i * TOP_THREADS + tid;
      w[i] = j < v1 ? row.vec(j) : (vu32x4)(lowest);
    }
  };
  fetch(cur, v0);
  for (int b = v0; b < v1; b += AHEAD * TOP_THREADS) {
    fetch(nxt, b + AHEAD * TOP_THREADS);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (b + i * TOP_THREADS < v1) {
        float z[EPV];
        unpack(cur[i], z);
        step(z, row.head + (b + i * TOP_THREADS + tid) * EPV);
      }
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) cur[i] = nxt[i];
  }
  if (part == a.parts - 1 && row.tail()) singles(row.tail(), row.tail0());

  __syncthreads();
  if (base > a.K) {
    cut(L, base, a.K, sizeof(Elem) == 2, a.V);
    base = a.K;
  }
  if (a.parts == 1) {
    write_sorted(L, base, a.K, [&](int k, uint64_t key) { put_entry(a, r, k, key); });
  } else {
    uint64_t* out = a.keys + ((int64_t)blockIdx.x) * a.K;
    for (int i = tid; i < a.K; i += TOP_THREADS) out[i] = i < base ? L.buf[i] : 0ull;
  }
  sum = block_join<TOP_THREADS>(sum, L.scratch, a.c);
  if (tid == 0) {
    if (a.parts > 1) a.sums[blockIdx.x] = sum;
    else if (a.lse) a.lse[r] = row_lse(sum, a.temperature);
  }
}

// Joins the parts of one row; parts * K <= TOP_CAP.
__global__ __launch_bounds__(TOP_THREADS) void top_join_kernel(TopArgs a, int bf16) {
  __shared__ TopLds L;
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x;
  const int n = a.parts * a.K;
  const uint64_t* in = a.keys + r * n;
  if (tid == 0) L.added[0] = 0;
  __syncthreads();
  for (int i0 = 0; i0 < n; i0 += TOP_THREADS) {
    const int i = i0 + tid;
    const uint64_t key = i < n ? in[i] : 0ull;
    if (key) L.buf[atomicAdd(&L.added[0], 1)] = key;
  }
  MaxSum sum{-INFINITY, 0.0f};
  if (tid < a.parts) sum = a.sums[r * a.parts + tid];
  sum = block_join<TOP_THREADS>(sum, L.scratch, a.c);
  int have = L.added[0];
  if (have > a.K) {
    cut(L, have, a.K, bf16 != 0, a.V);
    have = a.K;
  }
  write_sorted(L, have, a.K, [&](int k, uint64_t key) { put_entry(a, r, k, key); });
  if (tid == 0 && a.lse) a.lse[r] = row_lse(sum, a.temperature);
}

}  // namespace

int launch_top_logits(const TopArgs& a, int bf16, hipStream_t st) {
  const dim3 grid((uint32_t)a.R * (uint32_t)a.parts), block(TOP_THREADS);
  if (bf16) hipLaunchKernelGGL(top_scan_kernel<uint16_t>, grid, block, 0, st, a);
  else hipLaunchKernelGGL(top_scan_kernel<float>, grid, block, 0, st, a);
  if (a.parts > 1) hipLaunchKernelGGL(top_join_kernel, dim3(a.R), block, 0, st, a, bf16);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace sv
