// Softmax cross entropy of a linear head without its logits. Every product is
// C[m][n] = sum_k A[m][k] B[n][k] with both operands contiguous along k, made by
// one tiled kernel whose epilogues differ:
//   stats  A = W (tokens), B = h (states): a tile's logits become each state's
//          maximum and sum of exp over the tile's tokens; a second kernel joins
//          the tiles of a state;
//   dz     the same product again: dz = g (exp(z - m - logsum) - [v = y]),
//          rounded to bfloat16, as [state][token] and as [token][state];
//   acc    A = W^T of a piece of the vocabulary, B = dz: adds to dh in float32;
//   mat    A = h^T, B = dz^T: rows of dW, complete after one product.
// The operands of the last two are transposed into the workspace first, so one
// access pattern serves all four.
//
// float32 operands are split into three bfloat16 parts x = x1 + x2 + x3 (each the
// rounding of what the parts before leave: 24 bits in all), and a product sums
// the six part products down to 2^-24 of the largest, small ones first. Six
// bfloat16 products take 6/2500 of a second per PFLOP against 1/157 for the
// float32 matrix instructions.

#include "sv_train.hpp"

namespace sv {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

typedef __attribute__((address_space(3))) void lds_void;

// s_waitcnt operand: no vector memory operation outstanding, other counters free
// (vmcnt in bits 3:0 and 15:14, expcnt in 6:4, lgkmcnt in 11:8).
constexpr int WAIT_VM0 = 0x0F70;
// Last word of a raw buffer resource: 32-bit data, no swizzle.
constexpr int RSRC_WORD3 = 0x00027000;

// Part products of float32 operands, in the order in which they are summed.
__device__ __forceinline__ void part_pair(int i, int* pa, int* pb) {
  // (3,1) (1,3) (2,2) (2,1) (1,2) (1,1)
  *pa = (0x001102 >> (4 * i)) & 15;
  *pb = (0x010120 >> (4 * i)) & 15;
}

template <int BM, int BN, int WM, int WN>
struct Tile {
  static constexpr int WAVES_M = WM, WAVES_N = WN, THREADS = WM * WN * WAVE;
  static constexpr int TM = BM / WM, TN = BN / WN;   // a wave's tile
  static constexpr int MI = TM / 16, NI = TN / 16;
  static constexpr int LA = BM * 8 / THREADS, LB = BN * 8 / THREADS;   // 16-byte loads a thread
  static constexpr int STAGE = (BM + BN) * CE_BK;    // bfloat16 elements
  static_assert(LA * THREADS == BM * 8 && LB * THREADS == BN * 8, "whole rounds of loads");
};

// Tile indices of a workgroup: consecutive workgroups go to different XCDs (8),
// so each XCD takes a run of consecutive tiles, ordered in groups of 8 rows of
// tiles that share their operands' rows in its L2.
__device__ __forceinline__ void tile_of(int id, int tiles_m, int tiles_n, int* tm, int* tn) {
  const int total = tiles_m * tiles_n;
  constexpr int XCDS = 8;
  const int q = total / XCDS, rem = total % XCDS;
  const int x = id % XCDS, y = id / XCDS;
  id = x * q + (x < rem ? x : rem) + y;
  constexpr int GROUP = 8;
  const int per = GROUP * tiles_n;
  const int g = id / per;
  const int rows = min(GROUP, tiles_m - g * GROUP);
  const int in = id - g * per;
  *tm = g * GROUP + in % rows;
  *tn = in / rows;
}

template <int BM, int BN, int WM, int WN, typename Epi>
__global__ __launch_bounds__(WM* WN* WAVE, WM* WN == 8 ? 2 : 1) void ce_gemm_kernel(
    CeGemm g, int tiles_m, int tiles_n, typename Epi::Args ea) {
#if defined(__HIP_DEVICE_COMPILE__)   // buffer resources exist on the device side only
  using T = Tile<BM, BN, WM, WN>;
  __shared__ __align__(16) uint16_t lds[2 * T::STAGE];
  const int tid = threadIdx.x, lane = tid & (WAVE - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
  const int wm = wave / WN, wn = wave % WN;
  int tm, tn;
  tile_of(blockIdx.x, tiles_m, tiles_n, &tm, &tn);
  const int m0 = tm * BM, n0 = tn * BN;
  // rows past the end repeat the last one; a tile may lie behind it altogether
  const int mb = min(m0, g.M - 1), nb = min(n0, g.N - 1);

  // This thread's loads: row of the tile, and the 16-byte slot it fills. Slot s
  // of row r holds group s ^ (r & 7), which spreads a fragment's rows over banks.
  uint32_t offa[T::LA], offb[T::LB];
#pragma unroll
  for (int i = 0; i < T::LA; ++i) {
    const int c = i * T::THREADS + tid, row = c >> 3, grp = (c & 7) ^ (row & 7);
    offa[i] = (uint32_t)(min(row, g.M - 1 - mb) * g.lda + grp * 8) * 2u;
  }
#pragma unroll
  for (int i = 0; i < T::LB; ++i) {
    const int c = i * T::THREADS + tid, row = c >> 3, grp = (c & 7) ^ (row & 7);
    offb[i] = (uint32_t)(min(row, g.N - 1 - nb) * g.ldb + grp * 8) * 2u;
  }
  const uint16_t* rowa = g.A + (int64_t)mb * g.lda;
  const uint16_t* rowb = g.B + (int64_t)nb * g.ldb;

  // steps of this split
  const int steps_k = g.K / CE_BK;
  const int total = steps_k * g.parts;
  const int per = (total + g.splits - 1) / g.splits;
  const int first = min(total, (int)blockIdx.y * per), last = min(total, first + per);

  // Loads go straight into LDS: per lane a 32-bit offset from the tile's first
  // row, per step a scalar one. next_*: what is to be loaded next.
  int next_pair = first / steps_k, next_k = (first - next_pair * steps_k) * CE_BK;
  auto issue = [&](int stage) {
    int pa = 0, pb = 0;
    if (g.parts > 1) part_pair(next_pair, &pa, &pb);
    const auto ra = __builtin_amdgcn_make_buffer_rsrc((void*)(rowa + pa * g.plane_a), 0, -1, RSRC_WORD3);
    const auto rb = __builtin_amdgcn_make_buffer_rsrc((void*)(rowb + pb * g.plane_b), 0, -1, RSRC_WORD3);
    uint16_t* la = lds + stage * T::STAGE + wave * WAVE * 8;
    uint16_t* lb = la + BM * CE_BK;
#pragma unroll
    for (int i = 0; i < T::LA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(la + i * T::THREADS * 8), 16, (int)offa[i],
                                               next_k * 2, 0, 0);
#pragma unroll
    for (int i = 0; i < T::LB; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(lb + i * T::THREADS * 8), 16, (int)offb[i],
                                               next_k * 2, 0, 0);
    next_k += CE_BK;
    if (next_k == g.K) {
      next_k = 0;
      ++next_pair;
    }
  };

  f32x4 acc[T::MI][T::NI];
#pragma unroll
  for (int i = 0; i < T::MI; ++i)
#pragma unroll
    for (int j = 0; j < T::NI; ++j) acc[i][j] = (f32x4)(0.0f);

  const int fr = lane & 15, fk = lane >> 4;
  const int grp0 = (fk ^ (fr & 7)) * 8, grp1 = ((4 + fk) ^ (fr & 7)) * 8;
  auto step = [&](int s, int stage) {
    // this stage has arrived for every wave, and every wave is done with the other
    __builtin_amdgcn_s_waitcnt(WAIT_VM0);
    __syncthreads();
    if (s + 1 < last) issue(stage ^ 1);
    const uint16_t* la = lds + stage * T::STAGE + (wm * T::TM + fr) * CE_BK;
    const uint16_t* lb = lds + stage * T::STAGE + BM * CE_BK + (wn * T::TN + fr) * CE_BK;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const int grp = kk ? grp1 : grp0;
      bf16x8 fa[T::MI], fb[T::NI];
#pragma unroll
      for (int j = 0; j < T::NI; ++j) fb[j] = *(const bf16x8*)(lb + j * 16 * CE_BK + grp);
#pragma unroll
      for (int i = 0; i < T::MI; ++i) fa[i] = *(const bf16x8*)(la + i * 16 * CE_BK + grp);
#pragma unroll
      for (int i = 0; i < T::MI; ++i)
#pragma unroll
        for (int j = 0; j < T::NI; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
    }
    // Order of issue: all of B's fragments and two of A's, then each row of
    // matrix instructions with the fragment read that the row after the next needs.
    constexpr int MFMA = 0x008, DS_READ = 0x100;
    if constexpr (T::MI > 2) {
      __builtin_amdgcn_sched_group_barrier(DS_READ, T::NI + 2, 0);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
        for (int i = 0; i < T::MI - 2; ++i) {
          __builtin_amdgcn_sched_group_barrier(MFMA, T::NI, 0);
          __builtin_amdgcn_sched_group_barrier(DS_READ, 1, 0);
        }
        if (kk == 0) {
          __builtin_amdgcn_sched_group_barrier(MFMA, T::NI, 0);
          __builtin_amdgcn_sched_group_barrier(DS_READ, T::NI, 0);
          __builtin_amdgcn_sched_group_barrier(MFMA, T::NI, 0);
          __builtin_amdgcn_sched_group_barrier(DS_READ, 2, 0);
        } else {
          __builtin_amdgcn_sched_group_barrier(MFMA, 2 * T::NI, 0);
        }
      }
    }
  };
  if (first < last) issue(0);
  int s = first;
  for (; s + 1 < last; s += 2) {
    step(s, 0);
    step(s + 1, 1);
  }
  if (s < last) step(s, 0);
  __syncthreads();
  Epi::template run<T>(ea, g, acc, m0 + wm * T::TM, n0 + wn * T::TN, tm, wm, wn, lane, (char*)lds);
#endif
}

// Element i of acc[mi][ni] of lane l is C[m][n] with
//   m = m_wave + 16 mi + 4 (l / 16) + i,  n = n_wave + 16 ni + l % 16.

struct EpiStats {
  typedef CeStatsOut Args;
  template <typename T, typename Acc>
  static __device__ __forceinline__ void run(const Args& o, const CeGemm& g, Acc& acc, int mw, int nw,
                                             int tm, int wm, int wn, int lane, char* lds) {
    const int fr = lane & 15, fk = lane >> 4;
    MaxSum* red = (MaxSum*)lds;   // [waves along m][columns of the tile]
    constexpr int cols = T::TN * T::WAVES_N;
#pragma unroll
    for (int j = 0; j < T::NI; ++j) {
      const int n = nw + 16 * j + fr;
      const int lab = n < g.N ? o.labels[n] - o.v0 : -1;
      MaxSum s{-INFINITY, 0.0f};
#pragma unroll
      for (int i = 0; i < T::MI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int m = mw + 16 * i + 4 * fk + e;
          if (m >= g.M) acc[i][j][e] = -INFINITY;
          s.m = fmaxf(s.m, acc[i][j][e]);
          if (m == lab && m < g.M && n < g.N) o.zlabel[n] = acc[i][j][e];
        }
      const float ref = s.m == -INFINITY ? 0.0f : s.m;
#pragma unroll
      for (int i = 0; i < T::MI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s.s += fast_exp2((acc[i][j][e] - ref) * LOG2E);
#pragma unroll
      for (int off = 16; off < WAVE; off <<= 1) {
        MaxSum t;
        t.m = __shfl_xor(s.m, off, WAVE);
        t.s = __shfl_xor(s.s, off, WAVE);
        s = join(s, t, LOG2E);
      }
      if (fk == 0) red[wm * cols + wn * T::TN + 16 * j + fr] = s;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < cols; c += T::THREADS) {
      MaxSum s = red[c];
#pragma unroll
      for (int w = 1; w < T::WAVES_M; ++w) s = join(s, red[w * cols + c], LOG2E);
      const int n = nw - wn * T::TN + c;
      if (n < g.N) o.partial[(int64_t)tm * g.N + n] = s;
    }
  }
};

__device__ __forceinline__ void split3(float x, uint16_t (&p)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    uint32_t b = pack_bf16(x, 0.0f) & 0xFFFFu;
    // finite values next to the largest would round to infinity: cut them
    if ((b & 0x7FFFu) == 0x7F80u && fabsf(x) < INFINITY) b = __float_as_uint(x) >> 16;
    p[i] = (uint16_t)b;
    // nothing is left of an infinity
    x = (b & 0x7FFFu) == 0x7F80u ? 0.0f : x - bf16_to_f32(b);
  }
}

struct EpiDz {
  typedef CeDzOut Args;
  template <typename T, typename Acc>
  static __device__ __forceinline__ void run(const Args& o, const CeGemm& g, Acc& acc, int mw, int nw,
                                             int, int, int, int lane, char*) {
    const int fr = lane & 15, fk = lane >> 4;
#pragma unroll
    for (int j = 0; j < T::NI; ++j) {
      const int n = nw + 16 * j + fr;
      if (n >= o.n_pad) continue;
      int lab = -1;
      float m = 0.0f, ls2 = 0.0f, gl = 0.0f;
      if (n < g.N) {
        const int l = o.labels[n];
        if (l >= 0 && l < o.V) {
          lab = l - o.v0;
          m = o.stats[2 * (int64_t)n];
          ls2 = o.stats[2 * (int64_t)n + 1] * LOG2E;
          gl = o.grad_loss ? o.grad_loss[n] : 1.0f;
        }
      }
#pragma unroll
      for (int i = 0; i < T::MI; ++i) {
        const int r = mw + 16 * i + 4 * fk;
        float d[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float q = fast_exp2((acc[i][j][e] - m) * LOG2E - ls2);
          if (r + e == lab) q -= 1.0f;
          // a row left out, and what lies behind the last state or token, is 0
          d[e] = gl == 0.0f || r + e >= g.M ? 0.0f : gl * q;
        }
        for (int p = 0; p < o.planes; ++p) {
          uint16_t h[4];
          if (o.planes == 1) {
            const uint32_t lo = pack_bf16(d[0], d[1]), hi = pack_bf16(d[2], d[3]);
            h[0] = (uint16_t)lo;
            h[1] = (uint16_t)(lo >> 16);
            h[2] = (uint16_t)hi;
            h[3] = (uint16_t)(hi >> 16);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint16_t t[3];
              split3(d[e], t);
              h[e] = p == 0 ? t[0] : p == 1 ? t[1] : t[2];
            }
          }
          if (o.dz && n < g.N && r < o.ldz) {   // ldz is a multiple of 4
            uint2 w;
            w.x = (uint32_t)h[0] | ((uint32_t)h[1] << 16);
            w.y = (uint32_t)h[2] | ((uint32_t)h[3] << 16);
            *(uint2*)(o.dz + p * o.plane_dz + (int64_t)n * o.ldz + r) = w;
          }
          if (o.dzt) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (r + e < g.M) o.dzt[p * o.plane_dzt + (int64_t)(r + e) * o.ldt + n] = h[e];
          }
        }
      }
    }
  }
};

struct EpiAcc {
  typedef CeAccOut Args;
  template <typename T, typename Acc>
  static __device__ __forceinline__ void run(const Args& o, const CeGemm& g, Acc& acc, int mw, int nw,
                                             int, int, int, int lane, char*) {
    const int fr = lane & 15, fk = lane >> 4;
    float* base = o.acc + (int64_t)blockIdx.y * o.split_stride;
#pragma unroll
    for (int j = 0; j < T::NI; ++j) {
      const int n = nw + 16 * j + fr;
      if (n >= g.N) continue;
#pragma unroll
      for (int i = 0; i < T::MI; ++i) {
        const int r = mw + 16 * i + 4 * fk;
        if (r >= o.ld) continue;   // ld is M rounded up to 4
        f32x4* p = (f32x4*)(base + (int64_t)n * o.ld + r);
        f32x4 v = acc[i][j];
        if (o.add) v += *p;
        *p = v;
      }
    }
  }
};

struct EpiMat {
  typedef CeMatOut Args;
  template <typename T, typename Acc>
  static __device__ __forceinline__ void run(const Args& o, const CeGemm& g, Acc& acc, int mw, int nw,
                                             int, int, int, int lane, char*) {
    const int fr = lane & 15, fk = lane >> 4;
#pragma unroll
    for (int j = 0; j < T::NI; ++j) {
      const int n = nw + 16 * j + fr;
      if (n >= g.N) continue;
#pragma unroll
      for (int i = 0; i < T::MI; ++i) {
        const int r = mw + 16 * i + 4 * fk;
        const f32x4 v = acc[i][j];
        if (o.bf16) {
          uint16_t* p = (uint16_t*)o.out + (int64_t)n * o.ld + r;
          if (o.vec && r + 3 < g.M) {
            *(uint2*)p = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (r + e < g.M) put(p + e, v[e]);
          }
        } else {
          float* p = (float*)o.out + (int64_t)n * o.ld + r;
          if (o.vec && r + 3 < g.M) {
            *(f32x4*)p = v;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (r + e < g.M) p[e] = v[e];
          }
        }
      }
    }
  }
};

// ---------------------------------------------------------------- packing

__device__ __forceinline__ void load_parts(const CePack& p, int64_t r, int c, uint16_t (&h)[3]) {
  if (p.bf16) h[0] = ((const uint16_t*)p.src)[r * p.stride + c];
  else split3(((const float*)p.src)[r * p.stride + c], h);
}

__global__ __launch_bounds__(256) void ce_pack_kernel(CePack p) {
  const int64_t r = blockIdx.y + (int64_t)blockIdx.z * 65535;
  if (r >= p.rows) return;
  for (int64_t c = blockIdx.x * 256 + threadIdx.x; c < p.ld; c += (int64_t)gridDim.x * 256) {
    uint16_t h[3] = {0, 0, 0};
    if (c < p.cols) load_parts(p, r, (int)c, h);
    for (int k = 0; k < p.planes; ++k) p.dst[k * p.plane + r * p.ld + c] = h[k];
  }
}

// 64 x 64 tiles through LDS.
__global__ __launch_bounds__(256) void ce_transpose_kernel(CePack p, int tiles_c) {
  __shared__ uint16_t t[64][66];
  const int64_t r0 = (int64_t)(blockIdx.x / tiles_c) * 64;
  const int c0 = (int)(blockIdx.x % tiles_c) * 64;
  const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
  for (int k = 0; k < p.planes; ++k) {
    for (int i = y; i < 64; i += 4) {
      uint16_t h[3] = {0, 0, 0};
      if (r0 + i < p.rows && c0 + x < p.cols) load_parts(p, r0 + i, c0 + x, h);
      t[i][x] = h[k];
    }
    __syncthreads();
    for (int i = y; i < 64; i += 4)
      if (c0 + i < p.cols && r0 + x < p.ld) p.dst[k * p.plane + (int64_t)(c0 + i) * p.ld + r0 + x] = t[x][i];
    __syncthreads();
  }
}

// ---------------------------------------------------------------- joins

// 32 states a workgroup; 8 threads a state take every eighth tile.
__global__ __launch_bounds__(256) void ce_join_kernel(const MaxSum* partial, const float* zlabel,
                                                      const int32_t* labels, int tiles, int N, int V,
                                                      float* loss, float* stats) {
  __shared__ MaxSum red[8][32];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int64_t n = (int64_t)blockIdx.x * 32 + x;
  MaxSum s{-INFINITY, 0.0f};
  if (n < N)
    for (int t = y; t < tiles; t += 8) s = join(s, partial[(int64_t)t * N + n], LOG2E);
  red[y][x] = s;
  __syncthreads();
  if (y || n >= N) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) s = join(s, red[i][x], LOG2E);
  const float logsum = logf(s.s);
  stats[2 * n] = s.m;
  stats[2 * n + 1] = logsum;
  const int32_t l = labels[n];
  loss[n] = l >= 0 && l < V ? logsum - (zlabel[n] - s.m) : 0.0f;
}

__global__ __launch_bounds__(256) void ce_sum_kernel(const float* acc, int splits, int64_t split_stride,
                                                     int64_t ld, int D, void* out, int64_t out_stride,
                                                     int bf16) {
  const int64_t n = blockIdx.x;
  for (int d = threadIdx.x; d < D; d += 256) {
    float v = acc[n * ld + d];
    for (int s = 1; s < splits; ++s) v += acc[s * split_stride + n * ld + d];
    if (bf16) put((uint16_t*)out + n * out_stride + d, v);
    else ((float*)out)[n * out_stride + d] = v;
  }
}

// cover: rows of B's side that the tiles have to reach (its padding, if any).
template <typename Epi>
int gemm(const CeGemm& g, const typename Epi::Args& ea, int cover, hipStream_t st) {
  const int bm = ce_tile_m(g.N), bn = ce_tile_n(g.N);
  const int tiles_m = (g.M + bm - 1) / bm;
  const int tiles_n = (cover + bn - 1) / bn;
  const dim3 grid((uint32_t)tiles_m * (uint32_t)tiles_n, (uint32_t)g.splits);
#define CE_LAUNCH(BM, BN, WM, WN) \
  hipLaunchKernelGGL((ce_gemm_kernel<BM, BN, WM, WN, Epi>), grid, dim3(WM * WN * WAVE), 0, st, g, tiles_m, tiles_n, ea)
  if (bn == 32) CE_LAUNCH(256, 32, 4, 1);
  else if (bn == 128) CE_LAUNCH(128, 128, 2, 2);
  else CE_LAUNCH(256, 256, 2, 4);
#undef CE_LAUNCH
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace

int ce_tile_m(int rows_b) { return rows_b <= 32 || rows_b > 128 ? 256 : 128; }
int ce_tile_n(int rows_b) { return rows_b <= 32 ? 32 : rows_b <= 128 ? 128 : 256; }

int launch_ce_stats(const CeGemm& g, const CeStatsOut& o, hipStream_t st) { return gemm<EpiStats>(g, o, g.N, st); }
int launch_ce_dz(const CeGemm& g, const CeDzOut& o, hipStream_t st) { return gemm<EpiDz>(g, o, o.dzt ? o.n_pad : g.N, st); }
int launch_ce_acc(const CeGemm& g, const CeAccOut& o, hipStream_t st) { return gemm<EpiAcc>(g, o, g.N, st); }
int launch_ce_mat(const CeGemm& g, const CeMatOut& o, hipStream_t st) { return gemm<EpiMat>(g, o, g.N, st); }

int launch_ce_pack(const CePack& p, bool transposed, hipStream_t st) {
  if (transposed) {
    const int tiles_c = (p.cols + 63) / 64;
    const int64_t tiles_r = (p.ld + 63) / 64;
    hipLaunchKernelGGL(ce_transpose_kernel, dim3((uint32_t)(tiles_r * tiles_c)), dim3(256), 0, st, p, tiles_c);
  } else {
    const int64_t bx = (p.ld + 255) / 256;
    const dim3 grid((uint32_t)(bx < 64 ? bx : 64), (uint32_t)(p.rows < 65535 ? p.rows : 65535),
                    (uint32_t)((p.rows + 65534) / 65535));
    hipLaunchKernelGGL(ce_pack_kernel, grid, dim3(256), 0, st, p);
  }
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_ce_join(const MaxSum* partial, const float* zlabel, const int32_t* labels, int tiles,
                   int N, int V, float* loss, float* stats, hipStream_t st) {
  hipLaunchKernelGGL(ce_join_kernel, dim3((uint32_t)((N + 31) / 32)), dim3(256), 0, st, partial, zlabel,
                     labels, tiles, N, V, loss, stats);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_ce_sum(const float* acc, int splits, int64_t split_stride, int64_t ld, int N, int D,
                  void* out, int64_t out_stride, int bf16, hipStream_t st) {
  hipLaunchKernelGGL(ce_sum_kernel, dim3((uint32_t)N), dim3(256), 0, st, acc, splits, split_stride, ld, D,
                     out, out_stride, bf16);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace sv
