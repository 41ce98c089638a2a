// Logit adjustments: penalties of tokens that occurred, biases, and a grammar's mask.
//
// Bound by memory: a row is read and written once, with a bit a token of the mask. What
// touches a token at all is sparse (the tokens before the row, the biases), so a
// workgroup takes 4,096 tokens of the vocabulary for several rows of a request, counts the
// occurrences of those tokens in LDS, indexed by the token itself (no limit on the lists'
// lengths, no hash), and keeps a bit for each token that anything falls on. Rows then pass other
// tokens through, and a lane takes its touched tokens one by one: their arithmetic, a division
// among it, for all 8 tokens of every group with a touched one made 262 us of 1,152 rows of 151,936
// with 2,000 tokens before them instead of 220 then. The proposals before a row are counted one by one as the
// workgroup goes from row to row; a row is asked for while the one before is worked on. (Those rows now:
// 154 us, 4.7 TB/s; with a mask alone 127, 5.7 TB/s, which is more than a plain copy has.)

#include <math.h>

#include "sv_serve.hpp"

namespace sv {
namespace {

constexpr int GROUPS = ADJ_CHUNK / 8;

// For each token of the chunk how often it occurred, whether the prompt has it, and 1 + the index
// of its last bias. SMALL: in 16 bits each, for lists of fewer than 2^15 tokens and 2^16 biases, so
// that eight workgroups fit a CU instead of four (1,152 rows of 151,936: 220 -> 186 us then).
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

__device__ __forceinline__ uint32_t bits(uint16_t x) { return x; }
__device__ __forceinline__ uint32_t bits(float x) { return __float_as_uint(x); }
__device__ __forceinline__ void from_bits(uint16_t* p, uint32_t x) { *p = (uint16_t)x; }
__device__ __forceinline__ void from_bits(float* p, uint32_t x) { *p = __uint_as_float(x); }

// 8 logits as they lie, two or one to a register, so that rows which pass through cost no instructions
// (as 8 values each, 179 us instead of 157). bfloat16 rows are read once and not read again here, 1 KB a wave
// at once, so both ways go past the caches' older contents (186 -> 179 us, passed through 149 -> 138); float32 rows
// are two times 16 bytes a lane with others' between, which caches put together (322 us past them, 299 through).
template <typename E>
struct Eight {
  static constexpr int LOADS = (int)sizeof(E) / 2;
  static constexpr uint32_t LOWEST = sizeof(E) == 2 ? 0xFF80FF80u : 0xFF800000u;
  su32x4 w[LOADS];
  __device__ __forceinline__ void load(const E* p) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) w[i] = LOADS == 1 ? __builtin_nontemporal_load((const su32x4_any*)p) : ((const su32x4_any*)p)[i];
  }
  __device__ __forceinline__ void store(E* p) const {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      if constexpr (LOADS == 1) __builtin_nontemporal_store(w[i], (su32x4_any*)p);
      else ((su32x4_any*)p)[i] = w[i];
    }
  }
  // the first `left` of them
  __device__ __forceinline__ void load(const E* p, int left) {
    constexpr int PER = 4 / (int)sizeof(E);
#pragma unroll
    for (int i = 0; i < 4 * LOADS; ++i) {
      uint32_t x = 0;
#pragma unroll
      for (int e = 0; e < PER; ++e)
        if (i * PER + e < left) x |= bits(p[i * PER + e]) << (16 * e);
      w[i / 4][i % 4] = x;
    }
  }
  __device__ __forceinline__ void store(E* p, int left) const {
    constexpr int PER = 4 / (int)sizeof(E);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) from_bits(p + e, w[e / PER / 4][e / PER % 4] >> (16 * (e % PER)));
  }
  __device__ __forceinline__ uint32_t word(int i) const {
    const uint32_t a = i & 1 ? w[0][1] : w[0][0], b = i & 1 ? w[0][3] : w[0][2], lo = i & 2 ? b : a;
    if constexpr (LOADS == 1) return lo;
    const uint32_t c = i & 1 ? w[LOADS - 1][1] : w[LOADS - 1][0], d = i & 1 ? w[LOADS - 1][3] : w[LOADS - 1][2];
    return i & 4 ? (i & 2 ? d : c) : lo;
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (sizeof(E) == 4) return __uint_as_float(word(e));
    const uint32_t x = word(e >> 1);
    return __uint_as_float(e & 1 ? x & 0xFFFF0000u : x << 16);
  }
  __device__ __forceinline__ void set(int e, float y) {
    uint32_t x = __float_as_uint(y);
    int at = e;
    if constexpr (sizeof(E) == 2) {
      at = e >> 1;
      const uint32_t was = word(at), half = round_bf16x2(y, 0.0f);
      x = e & 1 ? (was & 0xFFFFu) | half << 16 : (was & 0xFFFF0000u) | half;
    }
#pragma unroll
    for (int i = 0; i < 4 * LOADS; ++i) w[i / 4][i % 4] = at == i ? x : w[i / 4][i % 4];
  }
  // -inf where a bit is clear
  __device__ __forceinline__ void keep(uint32_t mask) {
#pragma unroll
    for (int i = 0; i < 4 * LOADS; ++i) {
      uint32_t m = 0;
      if constexpr (sizeof(E) == 2) m = (mask >> (2 * i) & 1 ? 0xFFFFu : 0u) | (mask >> (2 * i) & 2 ? 0xFFFF0000u : 0u);
      else m = mask >> i & 1 ? ~0u : 0u;
      w[i / 4][i % 4] = (w[i / 4][i % 4] & m) | (LOWEST & ~m);
    }
  }
};

constexpr int MINE = GROUPS / ADJ_THREADS;   // groups of a thread
// Loads of four ids of a list that a thread keeps (4: 20 registers more and a wave less, 157 us instead of 154).
constexpr int AHEAD = 2;
constexpr int ADJ_BIASES = 768;              // of a request, in LDS; more are read from memory

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
  Eight<E> x[MINE];
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
  // first 2,048 ids, four a load.
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
      if (left[k] >= 8) to.x[k].load(q);
      else to.x[k].load(q, left[k]);
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
      Eight<E>& x = row.x[k];
      // one token of each lane at a time: few lanes have one, and those have few
      for (uint32_t bits = note[k] & mask; bits; bits &= bits - 1) {
        const int e = __builtin_ctz(bits);
        const uint32_t c = state.counted(g * 8 + e), last = state.last_bias(g * 8 + e);
        float y = x.get(e);
        if (c) y = y > 0.0f ? y / theta : y * theta;
        if (c & ~PROMPT) y = y - (often * (float)(c & ~PROMPT) + once);
        if (last) y = y + (last <= ADJ_BIASES ? biases[last - 1] : bias[last - 1]);
        if (c | last) x.set(e, y);
      }
      if (mask != 0xFFu) x.keep(mask);
      E* o = out + j * a.os.n + 8 * g;
      if (left[k] >= 8) x.store(o);
      else x.store(o, left[k]);
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
