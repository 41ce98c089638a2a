// Logit adjustments: penalties of tokens that occurred, biases, and a grammar's mask.
//
// Bound by memory: a row is read and written once, with a bit a token of the mask. What
// touches a token at all is sparse (the tokens before the row, the biases), so a
// workgroup takes 4,096 tokens of the vocabulary for several rows of a request, counts the
// occurrences of those tokens in LDS, indexed by the token itself (no limit on the lists'
// lengths, no hash), and keeps a bit for each token that anything falls on. Rows then pass other
// tokens through, and a lane takes its touched tokens one by one: their arithmetic, a division
// among it, for all 8 tokens of every group with a touched one made 262 us of 1,152 rows of 151,936
// with 2,000 tokens before them (now 186, 3.9 TB/s; with a mask alone 149). The proposals before a row are counted one by one as the
// workgroup goes from row to row; a row is asked for while the one before is worked on.

#include <math.h>

#include "sv_serve.hpp"

namespace sv {
namespace {

constexpr int GROUPS = ADJ_CHUNK / 8;

// For each token of the chunk how often it occurred, whether the prompt has it, and 1 + the index
// of its last bias. SMALL: in 16 bits each, for lists of fewer than 2^15 tokens and 2^16 biases, so
// that seven workgroups fit a CU instead of four (1,152 rows of 151,936: 220 -> 186 us).
template <bool SMALL>
struct State {
  static constexpr int WORDS = SMALL ? ADJ_CHUNK / 2 : ADJ_CHUNK;
  static constexpr uint32_t PROMPT = SMALL ? 0x8000u : 0x80000000u;   // top bit of a count
  uint32_t count[WORDS], biased[WORDS];
  static __device__ __forceinline__ int word(uint32_t at) { return SMALL ? at / 2 : at; }
  static __device__ __forceinline__ int shift(uint32_t at) { return SMALL ? 16 * (at & 1) : 0; }
  __device__ __forceinline__ void clear(int tid) {
    for (int i = tid * 4; i < WORDS; i += ADJ_THREADS * 4)
      *(su32x4*)(count + i) = *(su32x4*)(biased + i) = su32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void occurs(uint32_t at) { atomicAdd(&count[word(at)], 1u << shift(at)); }
  __device__ __forceinline__ void in_prompt(uint32_t at) { atomicOr(&count[word(at)], PROMPT << shift(at)); }
  __device__ __forceinline__ void bias(uint32_t at, uint32_t which) {
    if constexpr (SMALL) {
      uint32_t* w = &biased[word(at)];
      for (uint32_t old = *w;;) {
        if ((old >> shift(at) & 0xFFFFu) >= which) break;
        const uint32_t was = atomicCAS(w, old, (old & ~(0xFFFFu << shift(at))) | which << shift(at));
        if (was == old) break;
        old = was;
      }
    } else {
      atomicMax(&biased[at], which);
    }
  }
  static __device__ __forceinline__ uint32_t half(uint32_t v, uint32_t at) {
    return SMALL ? v >> shift(at) & 0xFFFFu : v;
  }
  __device__ __forceinline__ uint32_t counted(uint32_t at) const { return half(count[word(at)], at); }
  __device__ __forceinline__ uint32_t last_bias(uint32_t at) const { return half(biased[word(at)], at); }
};

__device__ __forceinline__ void raw8(const uint16_t* p, uint16_t (&w)[8]) {
  const su32x4 v = *(const su32x4_any*)p;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[2 * i] = (uint16_t)v[i];
    w[2 * i + 1] = (uint16_t)(v[i] >> 16);
  }
}
__device__ __forceinline__ void raw8(const float* p, float (&w)[8]) { load8(p, w); }
__device__ __forceinline__ void raw_store8(uint16_t* p, const uint16_t (&w)[8]) {
  su32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (uint32_t)w[2 * i] | (uint32_t)w[2 * i + 1] << 16;
  *(su32x4_any*)p = v;
}
__device__ __forceinline__ void raw_store8(float* p, const float (&w)[8]) { store8(p, w); }
__device__ __forceinline__ uint16_t lowest(uint16_t) { return 0xFF80u; }
__device__ __forceinline__ float lowest(float) { return -INFINITY; }

constexpr int MINE = GROUPS / ADJ_THREADS;   // groups of a thread
constexpr int AHEAD = 4;                     // loads of four ids of a list that a thread keeps
constexpr int ADJ_BIASES = 1024;             // of a request, in LDS; more are read from memory

// Ids n0 + 4 (thread + 256 k) .. + 3 of a list, -1 behind its end.
template <int LOADS>
__device__ __forceinline__ void load_ids(su32x4 (&v)[LOADS], const int32_t* ids, int n, int n0) {
#pragma unroll
  for (int k = 0; k < LOADS; ++k) {
    const int i = n0 + 4 * ((int)threadIdx.x + k * ADJ_THREADS);
    v[k] = su32x4{~0u, ~0u, ~0u, ~0u};
    if (i + 4 <= n) {
      v[k] = *(const su32x4_any*)(ids + i);
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (i + e < n) v[k][e] = (uint32_t)ids[i + e];
    }
  }
}

// What a thread has of a row: its groups' logits and bits.
template <typename E>
struct Held {
  E x[MINE][8];
  uint32_t mask[MINE];
};

template <typename E, bool SMALL>
__global__ __launch_bounds__(ADJ_THREADS) void adjust_kernel(AdjustArgs a) {
  __shared__ __attribute__((aligned(16))) State<SMALL> state;
  constexpr uint32_t PROMPT = State<SMALL>::PROMPT;
  __shared__ float biases[ADJ_BIASES];
  __shared__ uint32_t touched[ADJ_CHUNK / 32];   // a bit a token
  const int tid = threadIdx.x;
  uint32_t w = blockIdx.x;
  const int chunk = w % a.chunks;
  w /= a.chunks;
  const int part = w % a.row_groups, b = w / a.row_groups;
  const int v0 = chunk * ADJ_CHUNK, nv = a.V - v0 < ADJ_CHUNK ? a.V - v0 : ADJ_CHUNK;
  const int per = (a.N + a.row_groups - 1) / a.row_groups, j0 = part * per;
  int j1 = j0 + per < a.N ? j0 + per : a.N;
  const int used = a.rows ? a.rows[b] : a.N;
  const bool bad = used < 0 || used > a.N;
  if (!bad && j1 > used) j1 = used;
  if (j0 >= j1) return;
  const E* z = (const E*)a.z + b * a.zs.b + v0;
  E* out = (E*)a.out + b * a.os.b + v0;
  if (bad) {
    for (int j = j0; j < j1; ++j)
      for (int i = tid; i < nv; i += ADJ_THREADS) put(out + j * a.os.n + i, NAN);
    return;
  }
  const int64_t words = (a.V + 31) / 32;
  auto bits_of = [&](int j, int k) -> uint32_t {
    const int g = tid + k * ADJ_THREADS;
    if (!a.allowed || g * 8 >= nv) return 0xFFu;
    return ((const uint8_t*)(a.allowed + ((int64_t)b * a.N + j) * words) + v0 / 8)[g];
  };
  // What the whole workgroup waits for first goes out together: the rows' bits, and the lists'
  // first 4,096 ids, four a load.
  const bool counts = a.repetition || a.frequency || a.presence;
  const int32_t* history = a.history + (int64_t)b * a.n_history;
  const int32_t* prompt = a.prompt + (int64_t)b * a.n_prompt;
  const int32_t* tokens = a.tokens + (int64_t)b * a.n_tokens;
  const int32_t* bias_ids = a.bias_ids + (int64_t)b * a.n_bias;
  const float* bias = a.bias + (int64_t)b * a.n_bias;
  const int n_history = counts ? a.n_history : 0, n_prompt = counts ? a.n_prompt : 0;
  const int n_tokens = counts && a.tokens ? j1 - 1 : 0;      // the proposals before the last row
  Held<E> row, next;
  uint32_t later[MINE];                                      // bits of the row after the next
#pragma unroll
  for (int k = 0; k < MINE; ++k) {
    row.mask[k] = bits_of(j0, k);
    next.mask[k] = j0 + 1 < j1 ? bits_of(j0 + 1, k) : 0;
  }
  su32x4 h[AHEAD], p[AHEAD], m[1];
  load_ids(h, history, n_history, 0);
  load_ids(p, prompt, n_prompt, 0);
  load_ids(m, bias_ids, a.n_bias, 0);
  const float theta = a.repetition ? a.repetition[b] : 1.0f;
  const float often = a.frequency ? a.frequency[b] : 0.0f, once = a.presence ? a.presence[b] : 0.0f;
  const bool in_place = a.z == a.out;
  int left[MINE];                              // tokens from a group's first to the chunk's end
  uint32_t note[MINE];                         // which of a group's tokens anything falls on
#pragma unroll
  for (int k = 0; k < MINE; ++k) {
    left[k] = nv - 8 * (tid + k * ADJ_THREADS);
    note[k] = 0;
  }
  // groups that become -inf are not read, and in place groups that stay are not touched
  auto fetch = [&](int j, Held<E>& to) {
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
      if (left[k] <= 0 || to.mask[k] == 0 || (in_place && !note[k] && to.mask[k] == 0xFFu)) continue;
      const E* q = z + j * a.zs.n + 8 * (tid + k * ADJ_THREADS);
      if (left[k] >= 8) {
        raw8(q, to.x[k]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) to.x[k][e] = e < left[k] ? q[e] : lowest(E());
      }
    }
  };
  if (!in_place) fetch(j0, row);

  if (counts || a.n_bias) {
    for (int i = tid; i < ADJ_CHUNK / 32; i += ADJ_THREADS) touched[i] = 0;
    state.clear(tid);
    for (int i = tid; i < a.n_bias && i < ADJ_BIASES; i += ADJ_THREADS) biases[i] = bias[i];
    __syncthreads();
    // f(place in the chunk, index) for the ids of a list that lie in the chunk
    auto each = [&](auto& v, const int32_t* ids, int n, auto&& f) {
      constexpr int LOADS = sizeof(v) / sizeof(v[0]);
      auto one = [&](int id, int i) {
        const uint32_t at = (uint32_t)id - (uint32_t)v0;
        if (id >= 0 && at < (uint32_t)nv && i < n) {
          f(at, i);
          atomicOr(&touched[at / 32], 1u << (at % 32));
        }
      };
      for (int n0 = 0; n0 < n; n0 += LOADS * ADJ_THREADS * 4) {
        if (n0) load_ids(v, ids, n, n0);
#pragma unroll
        for (int k = 0; k < LOADS; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) one((int)v[k][e], n0 + 4 * (tid + k * ADJ_THREADS) + e);
      }
    };
    each(h, history, n_history, [&](uint32_t at, int) { state.occurs(at); });
    each(p, prompt, n_prompt, [&](uint32_t at, int) { state.in_prompt(at); });
    each(m, bias_ids, a.n_bias, [&](uint32_t at, int i) { state.bias(at, (uint32_t)i + 1u); });
    // proposals of later rows are noted already, so that nothing is passed over
    for (int i = tid; i < n_tokens; i += ADJ_THREADS) {
      const int id = tokens[i];
      const uint32_t at = (uint32_t)id - (uint32_t)v0;
      if (id >= 0 && at < (uint32_t)nv) {
        if (i < j0) state.occurs(at);
        atomicOr(&touched[at / 32], 1u << (at % 32));
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < MINE; ++k) note[k] = ((const uint8_t*)touched)[tid + k * ADJ_THREADS];
  }
  if (in_place) fetch(j0, row);
  for (int j = j0; j < j1; ++j) {
    if (j + 1 < j1) fetch(j + 1, next);
#pragma unroll
    for (int k = 0; k < MINE; ++k) later[k] = j + 2 < j1 ? bits_of(j + 2, k) : 0;
    if (j > j0 && j - 1 < n_tokens) {
      const int id = tokens[j - 1];
      const uint32_t at = (uint32_t)id - (uint32_t)v0;
      if (id >= 0 && at < (uint32_t)nv) {
        __syncthreads();
        if (tid == 0) state.occurs(at);
        __syncthreads();
      }
    }
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
      const int g = tid + k * ADJ_THREADS;
      const uint32_t mask = row.mask[k];
      if (left[k] <= 0 || (in_place && !note[k] && mask == 0xFFu)) continue;
      E(&x)[8] = row.x[k];
      // one token of each lane at a time: few lanes have one, and those have few
      for (uint32_t bits = note[k] & mask; bits; bits &= bits - 1) {
        const int e = __builtin_ctz(bits);
        const uint32_t c = state.counted(g * 8 + e), last = state.last_bias(g * 8 + e);
        E v = x[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) v = e == i ? x[i] : v;
        float y = elem(&v);
        if (c) y = y > 0.0f ? y / theta : y * theta;
        if (c & ~PROMPT) y = y - (often * (float)(c & ~PROMPT) + once);
        if (last) y = y + (last <= ADJ_BIASES ? biases[last - 1] : bias[last - 1]);
        if (c | last) put(&v, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = e == i ? v : x[i];
      }
      if (mask != 0xFFu) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!(mask >> e & 1)) x[e] = lowest(E());
      }
      E* o = out + j * a.os.n + 8 * g;
      if (left[k] >= 8) {
        raw_store8(o, x);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < left[k]) o[e] = x[e];
      }
    }
    row = next;
#pragma unroll
    for (int k = 0; k < MINE; ++k) next.mask[k] = later[k];
  }
}

}  // namespace

int launch_adjust(const AdjustArgs& a, hipStream_t st) {
  const dim3 grid((uint32_t)((int64_t)a.chunks * a.row_groups * a.B));
  const bool small = (int64_t)a.n_history + a.n_tokens < 1 << 15 && a.n_bias < 1 << 16;
  if (a.bf16) {
    if (small) adjust_kernel<uint16_t, true><<<grid, ADJ_THREADS, 0, st>>>(a);
    else adjust_kernel<uint16_t, false><<<grid, ADJ_THREADS, 0, st>>>(a);
  } else {
    if (small) adjust_kernel<float, true><<<grid, ADJ_THREADS, 0, st>>>(a);
    else adjust_kernel<float, false><<<grid, ADJ_THREADS, 0, st>>>(a);
  }
  return hipGetLastError() != hipSuccess;
}

}  // namespace sv
