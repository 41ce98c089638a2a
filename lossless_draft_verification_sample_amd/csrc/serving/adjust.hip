// Logit adjustments: penalties of tokens that occurred, biases, and a grammar's mask.
//
// Bound by memory: a row is read and written once, with a bit a token of the mask. What
// touches a token at all is sparse (the tokens before the row, the biases), so a
// workgroup takes 4,096 tokens of the vocabulary for several rows of a request, counts the
// occurrences of those tokens in LDS, indexed by the token itself (no limit on the lists'
// lengths, no hash), and notes which groups of 8 tokens anything falls into. Rows then pass
// groups without a note through untouched. The proposals before a row are counted one by one
// as the workgroup goes from row to row.

#include <math.h>

#include "sv_serve.hpp"

namespace sv {
namespace {

constexpr int GROUPS = ADJ_CHUNK / 8;
constexpr uint32_t PROMPT = 0x80000000u;   // top bit of a count: the prompt has the token

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

template <typename E>
__global__ __launch_bounds__(ADJ_THREADS) void adjust_kernel(AdjustArgs a) {
  __shared__ uint32_t count[ADJ_CHUNK];
  __shared__ uint32_t biased[ADJ_CHUNK];   // 1 + index of the token's last bias
  __shared__ uint8_t noted[GROUPS];
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
  const float theta = a.repetition ? a.repetition[b] : 1.0f;
  const float often = a.frequency ? a.frequency[b] : 0.0f, once = a.presence ? a.presence[b] : 0.0f;
  const bool counts = a.repetition || a.frequency || a.presence;
  const bool state = counts || a.n_bias;
  for (int g = tid; g < GROUPS; g += ADJ_THREADS) noted[g] = 0;
  if (state) {
    for (int i = tid; i < ADJ_CHUNK; i += ADJ_THREADS) count[i] = biased[i] = 0;
    __syncthreads();
    auto each = [&](const int32_t* ids, int n, auto&& f) {
      for (int i = tid; i < n; i += ADJ_THREADS) {
        const uint32_t at = (uint32_t)ids[i] - (uint32_t)v0;
        if (ids[i] >= 0 && at < (uint32_t)nv) {
          f(at, i);
          noted[at / 8] = 1;
        }
      }
    };
    if (counts) {
      each(a.history + (int64_t)b * a.n_history, a.n_history, [&](uint32_t at, int) { atomicAdd(&count[at], 1u); });
      each(a.prompt + (int64_t)b * a.n_prompt, a.n_prompt, [&](uint32_t at, int) { atomicOr(&count[at], PROMPT); });
      if (a.tokens)
        each(a.tokens + (int64_t)b * a.n_tokens, j0, [&](uint32_t at, int) { atomicAdd(&count[at], 1u); });
    }
    each(a.bias_ids + (int64_t)b * a.n_bias, a.n_bias,
         [&](uint32_t at, int i) { atomicMax(&biased[at], (uint32_t)i + 1u); });
  }
  __syncthreads();
  const bool in_place = a.z == a.out;
  const int64_t words = (a.V + 31) / 32;
  for (int j = j0; j < j1; ++j) {
    if (counts && a.tokens && j > j0) {
      const int id = a.tokens[(int64_t)b * a.n_tokens + j - 1];
      const uint32_t at = (uint32_t)id - (uint32_t)v0;
      if (id >= 0 && at < (uint32_t)nv) {
        __syncthreads();
        if (tid == 0) {
          count[at] += 1;
          noted[at / 8] = 1;
        }
        __syncthreads();
      }
    }
    const uint8_t* bits = a.allowed ? (const uint8_t*)(a.allowed + ((int64_t)b * a.N + j) * words) + v0 / 8 : nullptr;
    const E* zr = z + j * a.zs.n;
    E* o = out + j * a.os.n;
    for (int g = tid; g * 8 < nv; g += ADJ_THREADS) {
      const int n = nv - g * 8 < 8 ? nv - g * 8 : 8;
      const uint32_t mask = bits ? bits[g] : 0xFFu;
      const bool note = noted[g];
      if (in_place && !note && mask == 0xFFu) continue;
      E x[8];
      if (n == 8) {
        raw8(zr + g * 8, x);
      } else {
        for (int e = 0; e < 8; ++e) x[e] = e < n ? zr[g * 8 + e] : lowest(E());
      }
      if (note) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t c = count[g * 8 + e], k = biased[g * 8 + e];
          if (c | k) {
            float y = elem(&x[e]);
            const float n_times = (float)(c & ~PROMPT);
            if (c) y = y > 0.0f ? y / theta : y * theta;
            if (c & ~PROMPT) y = y - (often * n_times + once);
            if (k) y = y + a.bias[(int64_t)b * a.n_bias + k - 1];
            put(&x[e], y);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (!(mask >> e & 1)) x[e] = lowest(E());
      if (n == 8) {
        raw_store8(o + g * 8, x);
      } else {
        for (int e = 0; e < n; ++e) o[g * 8 + e] = x[e];
      }
    }
  }
}

}  // namespace

int launch_adjust(const AdjustArgs& a, hipStream_t st) {
  const dim3 grid((uint32_t)((int64_t)a.chunks * a.row_groups * a.B));
  if (a.bf16) adjust_kernel<uint16_t><<<grid, ADJ_THREADS, 0, st>>>(a);
  else adjust_kernel<float><<<grid, ADJ_THREADS, 0, st>>>(a);
  return hipGetLastError() != hipSuccess;
}

}  // namespace sv
