// The k largest logits of a vocabulary row and its log-normaliser
//   lse = log sum_v exp(z_v / T)
// in one pass over the row.
//
// A candidate is one 64-bit number: the order-preserving key of its value in
// the upper half, the complement of its id in the lower, so that keys are
// unique and the larger key is the larger logit, or the lower id among equals.
// A workgroup streams its part of a row, four 16-byte groups a thread at a time (a
// stretch). The first six stretches (the lead) give a threshold: with one maximum a
// thread, the k-th largest of the 256 maxima is at most the k-th largest logit, and
// few logits exceed it while k is well below 256; beyond k = 64 each of a thread's four
// positions has its own. Groups of the lead whose maximum exceeds the threshold are
// noted, and in the later stretches those that hold a logit above it; the noted groups are
// read again, their logits tested and listed as candidates in LDS when 512 have come
// together, and at the end. (Listing each logit on the spot took more instructions than
// the sum, because nearly every 64 groups hold one: 190 us for 1152 rows of 151,936 in
// bfloat16.) When the list grows it is cut to its k largest, by a search of the k-th
// value that every wave makes for itself, or, from 1024 entries on, by a radix selection
// (8 bits a level, from the top, ending as soon as a bin's border is the cut), and the
// threshold rises to the k-th value. Ids rise along the stream, so an equal logit that
// comes later never replaces a listed one and the test is strict. Rising or equal logits
// only mean more cuts.
//
// Bound: the read of the row. Rows are split over `parts` workgroups when there
// are few of them; the second kernel joins their lists and sums.

#include "sv_train.hpp"

namespace sv {

namespace {

constexpr int TOP_NOTES = 1536;
constexpr int TOP_LEAD = 6;                              // stretches of the lead ...
constexpr int TOP_LEAD_K = 512;                          // ... for k up to here; else one
constexpr int TOP_FEW = 64;                              // k up to here: maxima of threads, else of groups
constexpr int TOP_AHEAD = 4;                             // groups a thread in a stretch
constexpr int TOP_STRETCH = TOP_AHEAD * TOP_THREADS;     // groups; most that one can note

static_assert(TOP_THREADS == 256, "one bin of a digit a thread");
static_assert(TOP_LEAD * TOP_STRETCH * 4 <= TOP_CAP * 8, "the lead's maxima take the list's place");
static_assert(TOP_NOTES >= TOP_STRETCH + TOP_THREADS, "a stretch's notes next to those waiting");

struct TopLds {
  uint64_t buf[TOP_CAP];
  uint32_t hist[256];
  int added[3];         // entries appended by a step, slots in rotation
  uint32_t noted[TOP_NOTES];
  int notes[3];         // groups noted by a stretch, slots in rotation
  int kept;
  int sel_bin, sel_above, sel_count;
  MaxSum scratch[TOP_THREADS / WAVE];
};

__device__ __forceinline__ uint64_t make_key(float z, int id) {
  return ((uint64_t)f32_key(z) << 32) | (uint32_t)~(uint32_t)id;
}

// Appends the lane's flagged entries: one LDS atomic a wave, all lanes taking part.
template <int N>
__device__ __forceinline__ void append(const float (&z)[N], uint32_t flags, int id0, int base,
                                       int* counter, uint64_t* buf) {
  const int n = __popc(flags);
  const int incl = wave_scan_dpp((int32_t)n, (int32_t)0, [](int32_t x, int32_t y) { return x + y; });
  int at = 0;
  if ((threadIdx.x & (WAVE - 1)) == WAVE - 1) at = atomicAdd(counter, incl);
  at = base + lane63((int32_t)at) + incl - n;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if ((flags >> i) & 1u) buf[at++] = make_key(z[i], id0 + i);
}

// The value of a key that was found bit by bit from the top. The search leaves the low half
// of a bfloat16's key 0, but negative values have ones there: without them the value would
// lie just below its own logits, and later ones equal to it would be listed again (1,152 rows
// of 151,936 whose first half is -1e9, 64 kept: 1,575 us instead of 270).
__device__ __forceinline__ float found_value(uint32_t key, bool bf16) {
  if (key < 0x00800000u) return -INFINITY;   // no finite value's key
  return f32_from_key(bf16 && key < 0x80000000u ? key | 0xFFFFu : key);
}

// A value below v with none of the row's between (-inf below -inf); below the
// zeros, which are equal, it is the negated least normal number.
__device__ __forceinline__ float below(float v) {
  const uint32_t k = f32_key(v);
  if (v == 0.0f) return -0x1p-126f;
  return k <= 0x00800000u ? -INFINITY : f32_from_key(k - 1);
}

// The largest key, or one that few more reach, that at least K of the wave's 64 N
// keys reach; bit by bit from the top.
template <int N>
__device__ __forceinline__ uint32_t reached(const uint32_t (&v)[N], int K, bool bf16) {
  uint32_t key = 0;
  for (uint32_t bit = 1u << 31; bit >= (bf16 ? 1u << 16 : 1u); bit >>= 1) {
    const uint32_t trial = key | bit;
    int n = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) n += __popcll(__ballot(v[j] >= trial));
    if (n >= K) {
      key = trial;
      if (n <= K + K / 8) break;
    }
  }
  return key;
}

// A value that at least K of the N maxima (keys) exceed and few more; -inf where fewer
// are finite. Every wave finds it for itself.
template <int N>
__device__ __forceinline__ float threshold(const uint32_t* maxima, int K, bool bf16) {
  uint32_t v[N / WAVE];
#pragma unroll
  for (int j = 0; j < N / WAVE; ++j) v[j] = maxima[j * WAVE + (threadIdx.x & (WAVE - 1))];
  const uint32_t key = reached(v, K, bf16);
  return key < 0x00800000u ? -INFINITY : below(found_value(key, bf16));
}

// Cuts the list of n > K entries to its K largest. Returns a value no greater
// than the smallest kept one, above which later logits still count.
__attribute__((noinline)) __device__ float cut(TopLds& L, int n, int K, bool bf16, int V) {
  constexpr int PER = TOP_CAP / TOP_THREADS;
  const int tid = threadIdx.x;
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
#pragma unroll 2
    for (int j = tid; j < n; j += TOP_THREADS) {
      const uint64_t key = L.buf[j];
      if ((key & mask) == pref) atomicAdd(&L.hist[(uint32_t)(key >> shift) & 255u], 1u);
    }
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
  uint64_t key[PER];
  uint32_t flags = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = tid + i * TOP_THREADS;
    key[i] = j < n ? L.buf[j] : 0ull;
    if (j < n && (key[i] & mask) >= pref) flags |= 1u << i;
  }
  __syncthreads();   // the list is rewritten in place
  const int cnt = __popc(flags);
  const int incl = wave_scan_dpp((int32_t)cnt, (int32_t)0, [](int32_t x, int32_t y) { return x + y; });
  int at = 0;
  if ((tid & (WAVE - 1)) == WAVE - 1) at = atomicAdd(&L.kept, incl);
  at = lane63((int32_t)at) + incl - cnt;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if ((flags >> i) & 1u) L.buf[at++] = key[i];
  __syncthreads();
  return found_value((uint32_t)(pref >> 32), bf16);
}

// Thins the list of K < n <= TOP_THIN entries to those at or above a value that at
// least K reach: the K largest and what comes close. Without a barrier a level, unlike
// cut: every wave searches the value for itself. Returns the new length; *tau: a value
// above which later logits still count.
__device__ __forceinline__ int thin(TopLds& L, int n, int K, bool bf16, float* tau) {
  constexpr int PER = TOP_THIN / WAVE, MINE = TOP_THIN / TOP_THREADS;
  const int tid = threadIdx.x, lane = tid & (WAVE - 1);
  uint32_t v[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i)
    v[i] = i * WAVE + lane < n ? (uint32_t)(L.buf[i * WAVE + lane] >> 32) : 0u;   // 0: below every value
  uint64_t mine[MINE];
#pragma unroll
  for (int i = 0; i < MINE; ++i) mine[i] = i * TOP_THREADS + tid < n ? L.buf[i * TOP_THREADS + tid] : 0ull;
  const uint32_t key = reached(v, K, bf16);
  if (tid == 0) L.kept = 0;
  __syncthreads();   // the list is rewritten in place
#pragma unroll
  for (int i = 0; i < MINE; ++i)
    if (mine[i] && (uint32_t)(mine[i] >> 32) >= key) L.buf[atomicAdd(&L.kept, 1)] = mine[i];
  __syncthreads();
  *tau = found_value(key, bf16);
  return L.kept;
}

// Passes the list's K largest in descending order to `out(rank, key)`, key 0 for ranks
// past its n entries: up to 256 by counting the larger ones (the keys are unique),
// more by a bitonic sort. Ends without a barrier.
template <typename Out>
__device__ __forceinline__ void write_sorted(TopLds& L, int n, int K, Out out) {
  const int tid = threadIdx.x;
  if (n <= TOP_THREADS) {
    const uint64_t mine = tid < n ? L.buf[tid] : 0ull;
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) rank += L.buf[j] > mine;
    if (tid < n && rank < K) out(rank, mine);
    for (int i = n + tid; i < K; i += TOP_THREADS) out(i, 0ull);
    return;
  }
  int P = 2 * TOP_THREADS;
  while (P < n) P *= 2;
  for (int i = n + tid; i < P; i += TOP_THREADS) L.buf[i] = 0ull;
  __syncthreads();
  for (int size = 2; size <= P; size *= 2) {
    for (int step = size / 2; step > 0; step /= 2) {
      for (int i = tid; i < P / 2; i += TOP_THREADS) {
        const int lo = 2 * i - (i & (step - 1)), hi = lo + step;
        const uint64_t x = L.buf[lo], y = L.buf[hi];
        if ((x < y) == ((lo & size) == 0)) {
          L.buf[lo] = y;
          L.buf[hi] = x;
        }
      }
      __syncthreads();
    }
  }
  for (int i = tid; i < K; i += TOP_THREADS) out(i, i < P ? L.buf[i] : 0ull);
}

// The list's length once it is short enough to be sorted, K at least where it had K.
__device__ __forceinline__ int shorten(TopLds& L, int n, int K, bool bf16, int V) {
  float tau;
  if (n > K && n > TOP_THREADS && n <= TOP_THIN) n = thin(L, n, K, bf16, &tau);
  if (n > K && n > TOP_THREADS) {   // more than fit, or many equal values
    cut(L, n, K, bf16, V);
    n = K;
  }
  return n;
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
__global__ __launch_bounds__(TOP_THREADS, 5) void top_scan_kernel(TopArgs a) {
  __shared__ TopLds L;
  constexpr int EPV = Row<Elem>::EPV;
  constexpr bool BF16 = sizeof(Elem) == 2;
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x / a.parts;
  const int part = blockIdx.x % a.parts;
  const Row<Elem> row(a.logits, a.stride, r, a.V);
  const int per = (row.nvec + a.parts - 1) / a.parts;
  const int v0 = min(row.nvec, part * per), v1 = min(row.nvec, v0 + per);

  if (tid < 3) L.added[tid] = L.notes[tid] = 0;
  __syncthreads();
  int listed = 0, noted = 0;
  int slot = 0, note_slot = 0;   // counters of this step and this stretch
  float tau = -INFINITY;
  Running run;

  // Adds up what the workgroup counted in counters[slot], in every thread, and gets
  // the next counter ready: the one two turns on, which everyone has read and
  // nobody adds to yet.
  auto close = [&](int* counters, int& at) {
    __syncthreads();
    const int n = counters[at];
    const int after = at == 2 ? 0 : at + 1;
    if (tid == 0) counters[after == 2 ? 0 : after + 1] = 0;
    at = after;
    return n;
  };
  auto offer = [&](const float (&z)[EPV], int id0) {
    if (__any(Running::largest(z) > tau)) {
      uint32_t flags = 0;
#pragma unroll
      for (int i = 0; i < EPV; ++i) flags |= (z[i] > tau ? 1u : 0u) << i;
      append(z, flags, id0, listed, &L.added[slot], L.buf);
    }
    listed += close(L.added, slot);
  };
  // The elements before the first whole group and behind the last (one a thread).
  auto singles = [&](int n, int id0) {
    float z[EPV];
#pragma unroll
    for (int i = 1; i < EPV; ++i) z[i] = -INFINITY;
    z[0] = tid < n ? to_f32(row.p + id0 + tid) : -INFINITY;
    run.add(z, z[0], a.c);
    offer(z, id0 + tid);
  };

  const uint32_t lowest = BF16 ? 0xFF80FF80u : 0xFF800000u;   // -inf
  vu32x4 cur[TOP_AHEAD], nxt[TOP_AHEAD];
  auto fetch = [&](int b) {
#pragma unroll
    for (int i = 0; i < TOP_AHEAD; ++i) {
      const int j = b + i * TOP_THREADS + tid;
      nxt[i] = j < v1 ? row.vec(j) : (vu32x4)(lowest);
    }
  };
  // The lead: only the sum, the groups' maxima (kept in the list's place) and, per
  // thread and position in a stretch, the maximum over the lead's stretches.
  uint32_t* maxima = (uint32_t*)L.buf;
  const int lead = v0 + (a.K <= TOP_LEAD_K ? TOP_LEAD : 1) * TOP_STRETCH;
  float best[TOP_AHEAD];
#pragma unroll
  for (int i = 0; i < TOP_AHEAD; ++i) best[i] = -INFINITY;
  fetch(v0);
  int b = v0;
  for (int at = tid; b < v1 && b < lead; b += TOP_STRETCH, at += TOP_STRETCH) {
#pragma unroll
    for (int i = 0; i < TOP_AHEAD; ++i) cur[i] = nxt[i];
    fetch(b + TOP_STRETCH);
#pragma unroll
    for (int i = 0; i < TOP_AHEAD; ++i) {
      float z[EPV];
      unpack(cur[i], z);
      const float vm = Running::largest(z);
      maxima[at + i * TOP_THREADS] = f32_key(vm);
      best[i] = fmaxf(best[i], vm);
      run.add(z, vm, a.c);
    }
  }
  if (v0 < v1) {
    const bool few = a.K <= TOP_FEW;
    if (few) {
      L.noted[tid] = f32_key(Running::largest(best));
    } else {
#pragma unroll
      for (int i = 0; i < TOP_AHEAD; ++i) L.noted[i * TOP_THREADS + tid] = f32_key(best[i]);
    }
    __syncthreads();
    tau = few ? threshold<TOP_THREADS>(L.noted, a.K, BF16) : threshold<TOP_STRETCH>(L.noted, a.K, BF16);
    __syncthreads();
    const uint32_t key = f32_key(tau);
    for (int at = tid, j = v0 + tid; j - tid < b; j += TOP_THREADS, at += TOP_THREADS)
      if (maxima[at] > key) {   // this thread's own
        const int n = atomicAdd(&L.notes[note_slot], 1);
        if (n < TOP_NOTES) L.noted[n] = (uint32_t)j;
      }
    noted = close(L.notes, note_slot);
    if (noted > TOP_NOTES) {   // many equal logits: the lead once more, a stretch at a time
      noted = 0;
      b = v0;
      fetch(v0);
    }
  }
  const int summed = min(lead, v1);
  if (part == 0 && row.head) singles(row.head, 0);
  while (true) {
    if (noted > TOP_NOTES - TOP_STRETCH || (b >= v1 && noted > 0)) {
      // the noted groups, one a thread at a time
      auto load = [&](int n, int* at) {
        *at = n < noted ? (int)L.noted[n] : -1;
        return *at >= 0 ? row.vec(*at) : (vu32x4)(lowest);
      };
      // Notes come in no order, so that after a cut among them a logit equal to the
      // k-th may still have a lower id: until all are listed, equal ones pass.
      const float strict = tau;
      float higher = -INFINITY;
      int at, at2;
      vu32x4 w = load(tid, &at);
      for (int k = 0; k < noted; k += TOP_THREADS) {
        const vu32x4 w2 = load(k + TOP_THREADS + tid, &at2);
        if (listed > TOP_CAP - TOP_STEP) {   // more than K: room for all of it
          higher = fmaxf(higher, cut(L, listed, a.K, BF16, a.V));
          listed = a.K;
          tau = fmaxf(strict, below(higher));
        }
        float z[EPV];
        unpack(w, z);
        offer(z, row.head + at * EPV);
        w = w2;
        at = at2;
      }
      noted = 0;
      tau = fmaxf(strict, higher);
      // a higher threshold for what follows, or room for the row's last elements
      if (listed > a.K && (b < v1 ? listed > 2 * a.K : listed > TOP_CAP - EPV)) {
        float t;
        if (listed <= TOP_THIN) {
          listed = thin(L, listed, a.K, BF16, &t);
        } else {
          t = cut(L, listed, a.K, BF16, a.V);
          listed = a.K;
        }
        tau = fmaxf(tau, t);
      }
    }
    if (b >= v1) break;
#pragma unroll
    for (int i = 0; i < TOP_AHEAD; ++i) cur[i] = nxt[i];
    fetch(b + TOP_STRETCH);
    const bool again = b < summed;
#pragma unroll
    for (int i = 0; i < TOP_AHEAD; ++i) {
      float z[EPV];
      unpack(cur[i], z);
      const float vm = Running::largest(z);
      if (vm > tau)
        L.noted[noted + atomicAdd(&L.notes[note_slot], 1)] = (uint32_t)(b + i * TOP_THREADS + tid);
      if (!again) run.add(z, vm, a.c);
    }
    noted += close(L.notes, note_slot);
    b += TOP_STRETCH;
  }
  if (part == a.parts - 1 && row.tail()) singles(row.tail(), row.tail0());

  listed = shorten(L, listed, a.K, BF16, a.V);
  if (a.parts == 1) {
    write_sorted(L, listed, a.K, [&](int k, uint64_t key) { put_entry(a, r, k, key); });
  } else {
    uint64_t* out = a.keys + ((int64_t)blockIdx.x) * a.K;
    write_sorted(L, listed, a.K, [&](int k, uint64_t key) { out[k] = key; });
  }
  const MaxSum sum = block_join<TOP_THREADS>(run.set(a.c), L.scratch, a.c);
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
#pragma unroll 4
  for (int i = tid; i < n; i += TOP_THREADS) {
    const uint64_t key = in[i];
    if (key) L.buf[atomicAdd(&L.added[0], 1)] = key;
  }
  MaxSum sum{-INFINITY, 0.0f};
  if (tid < a.parts) sum = a.sums[r * a.parts + tid];
  sum = block_join<TOP_THREADS>(sum, L.scratch, a.c);
  const int have = shorten(L, L.added[0], a.K, bf16 != 0, a.V);
  write_sorted(L, have, a.K, [&](int k, uint64_t key) { put_entry(a, r, k, key); });
  if (tid == 0 && a.lse) a.lse[r] = row_lse(sum, a.temperature);
}

template <typename Elem>
int top_logits(const TopArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(top_scan_kernel<Elem>, dim3((uint32_t)a.R * (uint32_t)a.parts), dim3(TOP_THREADS), 0, st, a);
  if (a.parts > 1)
    hipLaunchKernelGGL(top_join_kernel, dim3(a.R), dim3(TOP_THREADS), 0, st, a, (int)(sizeof(Elem) == 2));
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace

int launch_top_logits(const TopArgs& a, int bf16, hipStream_t st) {
  return bf16 ? top_logits<uint16_t>(a, st) : top_logits<float>(a, st);
}

}  // namespace sv
