// Softmax cross entropy of a linear head without its logits. Every product is
// C[m][n] = sum_k A[m][k] B[n][k], made by one tiled kernel whose epilogues differ:
//   stats  A = W (tokens), B = h (states): a tile's logits become each state's
//          maximum and sum of exp over the tile's tokens; a second kernel joins
//          the tiles of a state;
//   dz     the same product again: dz = g (exp(z - m - logsum) - [v = y]),
//          as [state][token] of a piece of the vocabulary;
//   acc    A = W^T of the piece, B = dz: adds to dh in float32;
//   mat    A = h^T, B = dz^T: rows of dW, complete after one product.
// The last two read their transposed operands from W, h and dz as they lie in
// memory; the transposition happens in the read from LDS.
//
// dz of bfloat16 matrices is float32 taken as two bfloat16 parts, dz = d1 + d2, which hold it
// to 2^-16: the gradients' own rounding is the only one to bfloat16 that they show. In one
// part, half the work, their error against 64 bits is 2.4e-3 instead of the 1.66e-3 of
// that rounding (4,096 states of 4,096 over 151,936 tokens). A step of the product takes both
// parts of a stretch of depth, so that the matrix instructions of two products share the
// fragments of W or h.
//
// float32 operands, by the number of states (CE_F32_STATES):
//   few   as they are, with the float32 matrix instructions: what bounds these calls is
//         the read of W, 4 bytes an element;
//   many  split into three bfloat16 parts x = x1 + x2 + x3 (each the rounding of what
//         the parts before leave: 24 bits in all); a product sums the six part products
//         down to 2^-24 of the largest. Six bfloat16 products take 6/2500 of a second
//         per PFLOP against 1/157 for the float32 instructions, but the parts have to be
//         written first, 6 bytes an element.

#include "sv_train.hpp"

namespace sv {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int vs32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// s_waitcnt operand: no vector memory operation outstanding, other counters free
// (vmcnt in bits 3:0 and 15:14, expcnt in 6:4, lgkmcnt in 11:8).
constexpr int WAIT_VM0 = 0x0F70;
// Last word of a raw buffer resource: 32-bit data, no swizzle.
constexpr int RSRC_WORD3 = 0x00027000;
// Range of the buffer resources, and the offset of a load that shall read zeros.
// A tile's own offsets stay below it: 255 rows of at most 2^22 bfloat16, or 127 of
// as many float elements.
constexpr uint32_t BEYOND = 0x80000000u;

template <int BM, int BN, int WM, int WN>
struct Tile {
  static constexpr int WAVES_M = WM, WAVES_N = WN, THREADS = WM * WN * WAVE;
  static constexpr int TM = BM / WM, TN = BN / WN;   // a wave's tile
  static constexpr int MI = TM / 16, NI = TN / 16;
};

// Sixteen bytes of depth of one row.
template <typename E>
struct Frag {
  typedef bf16x8 type;
};
template <>
struct Frag<float> {
  typedef f32x4 type;
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

// Thread of the workgroup, made anew from the lane counter: kept in a register
// across the products it would cost them one.
__device__ __forceinline__ int thread_again(int wave) {
  return wave * WAVE + (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
}

// One 16-byte group a lane from base + byte_off into LDS at `lds`, lanes in order;
// an offset from BEYOND on reads as zeros. Asynchronous: it counts as a vector
// memory operation, and the caller waits for it (WAIT_VM0).
// In assembly because the compiler, which cannot tell the two halves of LDS apart,
// else waits for it before the next transposing read (dW 632 instead of 450 us a
// piece of 16,384 tokens at 4,096 states of 4,096, with dz in one part). It has no result register. m0 is
// no register the compiler allocates (it warns that it cannot keep a value there), but
// it does place writes of m0 of its own, and the clobber tells it where they end.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy_to_lds(uint64_t base, uint32_t byte_off, uint32_t lds) {
  const vs32x4 rsrc = {(int)(uint32_t)base, (int)(uint32_t)(base >> 32), (int)BEYOND, RSRC_WORD3};
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(lds), "v"(byte_off), "s"(rsrc) : "memory", "m0");
}
#pragma clang diagnostic pop

// One operand of a tile, of bfloat16 (uint16_t) or float elements: how ROWS rows by one
// step of depth (LINE bytes of a row) get from memory into LDS, and its fragments
// from there: per lane 16 bytes of depth of one row.
//   plain       memory [row][k]: LDS row of 8 (LINE 128) or 4 (64) groups of 16 bytes;
//               slot s of row r holds group s ^ spread(r), so that a fragment's 16
//               rows spread over the banks.
//   transposed  memory [k][row]: LDS as in memory. bfloat16: a fragment is made by the
//               transposing LDS read, which gives lane i of 16 the i-th of 16 columns of
//               4 consecutive k; blocks of 16 columns (32 bytes) are permuted by
//               block ^ f(k), f from bits 0, 1 and 3 of k: the 16 k that one read
//               touches are then spread over the banks. float: four reads of one element
//               each; blocks of 16 columns (64 bytes) are permuted by bits 2 and 3 of k.
// Groups behind the depth, or (transposed) behind the last row, are loaded from
// beyond the buffer resource's range, which reads as zero.
template <typename E, bool TRANS, int ROWS, int LINE, int FRAGS, int THREADS>
struct Side {
  static constexpr int LOADS = ROWS * LINE / 16 / THREADS;      // 16-byte loads a thread
  static_assert(LOADS * THREADS * 16 == ROWS * LINE, "whole rounds of loads");
  static constexpr int ES = sizeof(E);
  static constexpr int EPG = 16 / ES;                           // elements of a group
  static constexpr int DEPTH = LINE / ES;                       // elements of a step
  static constexpr int PARTS = LINE / 64;                       // fragments of a row's step
  static constexpr int GROUPS = TRANS ? ROWS / EPG : LINE / 16; // of a line of LDS
  static constexpr int BLOCK = 16 / EPG;                        // groups of 16 columns
  static constexpr int READS = !TRANS ? 1 : ES == 2 ? 2 : 4;    // LDS reads a fragment
  typedef typename Frag<E>::type F;
  uint32_t off[LOADS];              // of this thread's loads from the tile's first row, bytes
  uint32_t at[TRANS ? FRAGS : PARTS];   // in LDS, bytes. transposed: per fragment; plain: per part of the depth

  static __device__ __forceinline__ int line(int i, int tid) { return (i * THREADS + tid) / GROUPS; }
  static __device__ __forceinline__ int twist(int k) {
    return (ES == 2 ? (k & 3) | ((k >> 3) & 1) << 2 : (k >> 2) & 3) & (GROUPS / BLOCK - 1);
  }
  static __device__ __forceinline__ int spread(int row) { return LINE == 128 ? row & 7 : (row >> 1) & 3; }
  static __device__ __forceinline__ int group(int i, int tid) {
    const int slot = (i * THREADS + tid) % GROUPS, l = line(i, tid);
    if (!TRANS) return slot ^ spread(l);
    return (slot / BLOCK ^ twist(l)) * BLOCK + slot % BLOCK;
  }

  // base: first row of the tile; rows, ld: of the operand; wave_row: first row of
  // this wave's fragments in the tile.
  __device__ __forceinline__ void init(int base, int rows, int64_t ld, int wave_row, int lane) {
    const int fr = lane & 15, fk = lane >> 4;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int l = line(i, threadIdx.x), gr = group(i, threadIdx.x);
      if (TRANS) off[i] = base + gr * EPG < rows ? (uint32_t)(l * ld + gr * EPG) * ES : BEYOND;
      else off[i] = (uint32_t)(min(l, rows - 1 - base) * ld + gr * EPG) * ES;   // rows past the end repeat
    }
    if (TRANS) {
      const int k = ES == 2 ? fk * 8 + (fr >> 2) : fk * 4;
      const int f = twist(k), in = ES == 2 ? (fr & 3) * 4 : fr;
#pragma unroll
      for (int i = 0; i < FRAGS; ++i)
        at[i] = (uint32_t)(k * ROWS + ((wave_row / 16 + i) ^ f) * 16 + in) * ES;
    } else {
#pragma unroll
      for (int kk = 0; kk < PARTS; ++kk)
        at[kk] = (uint32_t)((wave_row + fr) * LINE + ((kk * 4 + fk) ^ spread(fr)) * 16);
    }
  }
  // Loads the tile's depth k.. of the operand that begins at p (the tile's first
  // row, k = 0); depth: where the operand ends.
  __device__ __forceinline__ void load(const E* p, int64_t ld, int k, int depth, uint32_t lds, int wave) {
    const uint64_t base = (uint64_t)(uintptr_t)(p + (TRANS ? (int64_t)k * ld : (int64_t)k));
    if (k + DEPTH <= depth) {
#pragma unroll
      for (int i = 0; i < LOADS; ++i) copy_to_lds(base, off[i], lds + i * THREADS * 16);
    } else {   // the operand's last, shorter step
      const int tid = thread_again(wave);
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const bool in = k + (TRANS ? line(i, tid) : group(i, tid) * EPG) < depth;
        copy_to_lds(base, in ? off[i] : BEYOND, lds + i * THREADS * 16);
      }
    }
  }
  __device__ __forceinline__ F frag(const char* lds, int i, int kk) const {
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (!TRANS) {
      return *(const F*)(lds + at[kk] + i * 16 * LINE);
    } else if constexpr (ES == 2) {
      const char* p = lds + at[i] + kk * 32 * ROWS * ES;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * ROWS * ES));
      return __builtin_bit_cast(F, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const char* p = lds + at[i] + kk * 16 * ROWS * ES;
      F v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = *(const float*)(p + e * ROWS * ES);
      return v;
    }
#else
    return F{};
#endif
  }
};

// C += A B over the 16 bytes of depth of a fragment pair: 32 of bfloat16, or 16 of
// float32, whose four instructions take element e of every lane: the same k in A and B.
__device__ __forceinline__ f32x4 multiply(const bf16x8& a, const bf16x8& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 multiply(const f32x4& a, const f32x4& b, f32x4 c) {
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
  return c;
}

// LINE: bytes of a row that one step takes. Where B is dz in two parts, a step takes both.
template <typename E, int BM, int BN, int WM, int WN, int LINE, typename Epi>
__global__ __launch_bounds__(WM* WN* WAVE, WM* WN == 8 ? 2 : 1) void ce_gemm_kernel(
    CeGemm g, int tiles_m, int tiles_n, typename Epi::Args ea) {
  using T = Tile<BM, BN, WM, WN>;
  constexpr int PB = Epi::OF_DZ && sizeof(E) == 2 ? 2 : 1;   // parts of B
  constexpr int PLANE_A = BM * LINE, PLANE_B = BN * LINE, STAGE = PLANE_A + PB * PLANE_B;
  constexpr int KK = LINE / 64;                              // fragments of a row's step
  __shared__ __align__(16) char lds[2 * STAGE];
  const int tid = threadIdx.x, lane = tid & (WAVE - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
  const int wm = wave / WN, wn = wave % WN;
  int tm, tn;
  tile_of(blockIdx.x, tiles_m, tiles_n, &tm, &tn);
  const int m0 = tm * BM, n0 = tn * BN;

  Side<E, Epi::TRANS_A, BM, LINE, T::MI, T::THREADS> sa;
  Side<E, Epi::TRANS_B, BN, LINE, T::NI, T::THREADS> sb;
  sa.init(m0, g.M, g.lda, wm * T::TM, lane);
  sb.init(n0, g.N, g.ldb, wn * T::TN, lane);
  const E* pa = (const E*)g.A + (Epi::TRANS_A ? (int64_t)m0 : m0 * g.lda);
  const E* pb = (const E*)g.B + (Epi::TRANS_B ? (int64_t)n0 : n0 * g.ldb);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(lds_void*)lds);

  // steps of this split; next_k: what is to be loaded next
  constexpr int DEPTH = decltype(sa)::DEPTH;
  const int total = (g.K + DEPTH - 1) / DEPTH;
  const int per = (total + g.splits - 1) / g.splits;
  const int first = min(total, (int)blockIdx.y * per), last = min(total, first + per);
  int next_k = first * DEPTH;
  auto issue = [&](int stage) {
    const uint32_t la = lds0 + stage * STAGE + wave * WAVE * 16;
    sa.load(pa, g.lda, next_k, g.K, la, wave);
#pragma unroll
    for (int q = 0; q < PB; ++q)
      sb.load(pb + q * g.plane_b, g.ldb, next_k, g.K, la + PLANE_A + q * PLANE_B, wave);
    next_k += DEPTH;
  };

  f32x4 acc[T::MI][T::NI];
#pragma unroll
  for (int i = 0; i < T::MI; ++i)
#pragma unroll
    for (int j = 0; j < T::NI; ++j) acc[i][j] = (f32x4)(0.0f);

  auto step = [&](int s, int stage) {
    // this stage has arrived for every wave, and every wave is done with the other
    __builtin_amdgcn_s_waitcnt(WAIT_VM0);
    __syncthreads();
    if (s + 1 < last) issue(stage ^ 1);
    const char* la = lds + stage * STAGE;
    const char* lb = la + PLANE_A;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      typename Frag<E>::type fa[T::MI], fb[PB][T::NI];
#pragma unroll
      for (int q = 0; q < PB; ++q)
#pragma unroll
        for (int j = 0; j < T::NI; ++j) fb[q][j] = sb.frag(lb + q * PLANE_B, j, kk);
#pragma unroll
      for (int i = 0; i < T::MI; ++i) fa[i] = sa.frag(la, i, kk);
#pragma unroll
      for (int i = 0; i < T::MI; ++i)
#pragma unroll
        for (int q = 0; q < PB; ++q)
#pragma unroll
          for (int j = 0; j < T::NI; ++j) acc[i][j] = multiply(fa[i], fb[q][j], acc[i][j]);
    }
    // Order of issue: all of B's fragments and two of A's, then each row of
    // matrix instructions with the fragment reads that the row after the next needs.
    constexpr int MFMA = 0x008, DS_READ = 0x100, ROW = T::NI * PB;
    constexpr int RA = decltype(sa)::READS, RB = decltype(sb)::READS * PB;
    if constexpr (T::MI > 2 && sizeof(E) == 2) {
      __builtin_amdgcn_sched_group_barrier(DS_READ, RB * T::NI + 2 * RA, 0);
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
#pragma unroll
        for (int i = 0; i < T::MI - 2; ++i) {
          __builtin_amdgcn_sched_group_barrier(MFMA, ROW, 0);
          __builtin_amdgcn_sched_group_barrier(DS_READ, RA, 0);
        }
        if (kk + 1 < KK) {
          __builtin_amdgcn_sched_group_barrier(MFMA, ROW, 0);
          __builtin_amdgcn_sched_group_barrier(DS_READ, RB * T::NI, 0);
          __builtin_amdgcn_sched_group_barrier(MFMA, ROW, 0);
          __builtin_amdgcn_sched_group_barrier(DS_READ, 2 * RA, 0);
        } else {
          __builtin_amdgcn_sched_group_barrier(MFMA, 2 * ROW, 0);
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
  Epi::template run<T>(ea, g, acc, m0 + wm * T::TM, n0 + wn * T::TN, tm, wm, wn, lane, lds);
}

// float32 operands in three bfloat16 parts: a step takes 32 of depth of all six, so that
// 96 matrix instructions share 24 fragments (one pair of parts at a time, over the whole
// depth, they share 12 each, and LDS bounds it). Parts are numbered from the largest; the
// order within a step is by B's part, so that the first products need few fragments.
// A step of 512 states of 1,024 over 32,000 tokens takes 773 us, one pair at a time 882.
// The lower tile is for dh and dW of up to 128 columns (3,000 states of 64, 32,000 tokens:
// 1,150 us, in the higher one 1,911).
template <int BM, int BN, int WM, int WN, typename Epi>
__global__ __launch_bounds__(WM* WN* WAVE, 2) void ce_split_kernel(CeGemm g, int tiles_m, int tiles_n,
                                                                   typename Epi::Args ea) {
  constexpr int LINE = 64;
  using T = Tile<BM, BN, WM, WN>;
  constexpr int PLANE_A = BM * LINE, PLANE_B = BN * LINE, STAGE = 3 * (PLANE_A + PLANE_B);
  __shared__ __align__(16) char lds[2 * STAGE];
  const int lane = threadIdx.x & (WAVE - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;
  int tm, tn;
  tile_of(blockIdx.x, tiles_m, tiles_n, &tm, &tn);
  const int m0 = tm * BM, n0 = tn * BN;

  Side<uint16_t, Epi::TRANS_A, BM, LINE, T::MI, T::THREADS> sa;
  Side<uint16_t, Epi::TRANS_B, BN, LINE, T::NI, T::THREADS> sb;
  sa.init(m0, g.M, g.lda, wm * T::TM, lane);
  sb.init(n0, g.N, g.ldb, wn * T::TN, lane);
  const uint16_t* pa = (const uint16_t*)g.A + (Epi::TRANS_A ? (int64_t)m0 : m0 * g.lda);
  const uint16_t* pb = (const uint16_t*)g.B + (Epi::TRANS_B ? (int64_t)n0 : n0 * g.ldb);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(lds_void*)lds);

  constexpr int DEPTH = decltype(sa)::DEPTH;
  const int total = (g.K + DEPTH - 1) / DEPTH;
  const int per = (total + g.splits - 1) / g.splits;
  const int first = min(total, (int)blockIdx.y * per), last = min(total, first + per);
  int next_k = first * DEPTH;
  auto issue = [&](int stage) {
    const uint32_t la = lds0 + stage * STAGE + wave * WAVE * 16;
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      sa.load(pa + p * g.plane_a, g.lda, next_k, g.K, la + p * PLANE_A, wave);
      sb.load(pb + p * g.plane_b, g.ldb, next_k, g.K, la + 3 * PLANE_A + p * PLANE_B, wave);
    }
    next_k += DEPTH;
  };

  f32x4 acc[T::MI][T::NI];
#pragma unroll
  for (int i = 0; i < T::MI; ++i)
#pragma unroll
    for (int j = 0; j < T::NI; ++j) acc[i][j] = (f32x4)(0.0f);

  auto step = [&](int s, int stage) {
    // this stage has arrived for every wave, and every wave is done with the other
    __builtin_amdgcn_s_waitcnt(WAIT_VM0);
    __syncthreads();
    if (s + 1 < last) issue(stage ^ 1);
    const char* la = lds + stage * STAGE;
    const char* lb = la + 3 * PLANE_A;
    bf16x8 fb[3][T::NI];
#pragma unroll
    for (int i = 0; i < T::MI; ++i) {
      bf16x8 fa[3];
#pragma unroll
      for (int p = 0; p < 3; ++p) fa[p] = sa.frag(la + p * PLANE_A, i, 0);
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        if (i == 0) {
#pragma unroll
          for (int j = 0; j < T::NI; ++j) fb[q][j] = sb.frag(lb + q * PLANE_B, j, 0);
        }
#pragma unroll
        for (int p = 2 - q; p >= 0; --p)
#pragma unroll
          for (int j = 0; j < T::NI; ++j) acc[i][j] = multiply(fa[p], fb[q][j], acc[i][j]);
      }
    }
    // Order of issue: what the first products need, then each group of matrix
    // instructions with the reads that the group after the next needs.
    constexpr int MFMA = 0x008, DS_READ = 0x100, N = T::NI;
    constexpr int RA = decltype(sa)::READS * 3, RB = decltype(sb)::READS * N;
    __builtin_amdgcn_sched_group_barrier(DS_READ, RA + 2 * RB, 0);
    __builtin_amdgcn_sched_group_barrier(MFMA, 3 * N, 0);
    __builtin_amdgcn_sched_group_barrier(DS_READ, RB, 0);
    __builtin_amdgcn_sched_group_barrier(MFMA, 2 * N, 0);
#pragma unroll
    for (int i = 1; i < T::MI; ++i) {
      __builtin_amdgcn_sched_group_barrier(DS_READ, RA, 0);
      __builtin_amdgcn_sched_group_barrier(MFMA, 6 * N, 0);
    }
    __builtin_amdgcn_sched_group_barrier(MFMA, N, 0);
  };
  if (first < last) issue(0);
  int s = first;
  for (; s + 1 < last; s += 2) {
    step(s, 0);
    step(s + 1, 1);
  }
  if (s < last) step(s, 0);
  __syncthreads();
  Epi::template run<T>(ea, g, acc, m0 + wm * T::TM, n0 + wn * T::TN, tm, wm, wn, lane, lds);
}

// Element i of acc[mi][ni] of lane l is C[m][n] with
//   m = m_wave + 16 mi + 4 (l / 16) + i,  n = n_wave + 16 ni + l % 16.

struct EpiStats {
  typedef CeStatsOut Args;
  static constexpr bool TRANS_A = false, TRANS_B = false, OF_DZ = false;
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

// PARTS: bfloat16 parts that dz is written in (each the rounding of what the parts before
// leave), or 0: float32.
template <int PARTS>
struct EpiDz {
  typedef CeDzOut Args;
  static constexpr bool TRANS_A = false, TRANS_B = false, OF_DZ = false;
  template <typename T, typename Acc>
  static __device__ __forceinline__ void run(const Args& o, const CeGemm& g, Acc& acc, int mw, int nw,
                                             int, int, int, int lane, char*) {
    const int fr = lane & 15, fk = lane >> 4;
#pragma unroll
    for (int j = 0; j < T::NI; ++j) {
      const int n = nw + 16 * j + fr;
      int lab = n < g.N ? o.labels[n] : -1;
      float m = 0.0f, ls2 = 0.0f, gl = 0.0f;
      if (lab >= 0 && lab < o.V) {
        lab -= o.v0;
        m = o.stats[2 * (int64_t)n];
        ls2 = o.stats[2 * (int64_t)n + 1] * LOG2E;
        gl = o.grad_loss ? o.grad_loss[n] : 1.0f;
      }
      uint16_t* row = (uint16_t*)o.dz + (int64_t)n * o.ldz;
#pragma unroll
      for (int i = 0; i < T::MI; ++i) {
        const int r = mw + 16 * i + 4 * fk;
        float d[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float q = fast_exp2((acc[i][j][e] - m) * LOG2E - ls2);
          if (r + e == lab) q -= 1.0f;
          // a state left out, and what lies behind the last token, is 0
          d[e] = gl == 0.0f || r + e >= g.M ? 0.0f : gl * q;
        }
        if (PARTS == 0 && n < g.N && r < o.ldz)
          *(f32x4*)((float*)o.dz + (int64_t)n * o.ldz + r) = (f32x4){d[0], d[1], d[2], d[3]};
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
          const uint2 w = make_uint2(pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3]));
          if (n < g.N && r < o.ldz) *(uint2*)(row + p * o.plane_dz + r) = w;   // ldz is a multiple of 4
          if (p + 1 < PARTS) {   // what the next part has to hold
            d[0] -= __uint_as_float(w.x << 16);
            d[1] -= __uint_as_float(w.x & 0xFFFF0000u);
            d[2] -= __uint_as_float(w.y << 16);
            d[3] -= __uint_as_float(w.y & 0xFFFF0000u);
          }
        }
      }
    }
  }
};

struct EpiAcc {
  typedef CeAccOut Args;
  static constexpr bool TRANS_A = true, TRANS_B = false, OF_DZ = true;
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
  static constexpr bool TRANS_A = true, TRANS_B = true, OF_DZ = true;
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
        // four columns at once, whatever their alignment
        if (o.bf16) {
          uint16_t* p = (uint16_t*)o.out + (int64_t)n * o.ld + r;
          if (r + 3 < g.M) {
            const uint2 w = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
            __builtin_memcpy(p, &w, 8);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (r + e < g.M) put(p + e, v[e]);
          }
        } else {
          float* p = (float*)o.out + (int64_t)n * o.ld + r;
          if (r + 3 < g.M) {
            __builtin_memcpy(p, &v, 16);
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

// Four columns a thread, read at once whatever their alignment.
__global__ __launch_bounds__(256) void ce_pack_kernel(CePack p) {
  const int64_t quads = p.ld / 4, all = quads * p.rows;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / quads;
    const int c = (int)(i - r * quads) * 4;
    uint16_t h[3][4] = {};
    if (p.bf16) {
      const uint16_t* src = (const uint16_t*)p.src + r * p.stride + c;
      if (c + 3 < p.cols) {
        __builtin_memcpy(h[0], src, 8);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < p.cols) h[0][e] = src[e];
      }
    } else {
      const float* src = (const float*)p.src + r * p.stride + c;
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (c + 3 < p.cols) {
        __builtin_memcpy(v, src, 16);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < p.cols) v[e] = src[e];
      }
      if (p.planes == 0) {   // as they are
        *(f32x4*)((float*)p.dst + r * p.ld + c) = (f32x4){v[0], v[1], v[2], v[3]};
        continue;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint16_t t[3];
        split3(v[e], t);
        h[0][e] = t[0];
        h[1][e] = t[1];
        h[2][e] = t[2];
      }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (k < p.planes) {
        const uint2 w = make_uint2(h[k][0] | ((uint32_t)h[k][1] << 16), h[k][2] | ((uint32_t)h[k][3] << 16));
        *(uint2*)((uint16_t*)p.dst + k * p.plane + r * p.ld + c) = w;
      }
  }
}

// ---------------------------------------------------------------- joins

// A workgroup joins X states; 256 / X threads a state take every so many-th tile.
template <int X>
__global__ __launch_bounds__(256) void ce_join_kernel(const MaxSum* partial, const float* zlabel,
                                                      const int32_t* labels, int tiles, int N, int V,
                                                      float* loss, float* stats) {
  constexpr int Y = 256 / X;
  __shared__ MaxSum red[Y][X];
  const int x = threadIdx.x % X, y = threadIdx.x / X;
  const int64_t n = (int64_t)blockIdx.x * X + x;
  MaxSum s{-INFINITY, 0.0f};
  if (n < N) {
    int t = y;
    for (; t + 3 * Y < tiles; t += 4 * Y) {
      MaxSum p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = partial[(int64_t)(t + i * Y) * N + n];
      s = join(s, join(join(p[0], p[1], LOG2E), join(p[2], p[3], LOG2E), LOG2E), LOG2E);
    }
    for (; t < tiles; t += Y) s = join(s, partial[(int64_t)t * N + n], LOG2E);
  }
#pragma unroll
  for (int half = Y / 2; half > 0; half >>= 1) {
    red[y][x] = s;
    __syncthreads();
    if (y < half) s = join(s, red[y + half][x], LOG2E);
    __syncthreads();
  }
  if (y || n >= N) return;
  const float logsum = logf(s.s);
  stats[2 * n] = s.m;
  stats[2 * n + 1] = logsum;
  const int32_t l = labels[n];
  loss[n] = l >= 0 && l < V ? logsum - (zlabel[n] - s.m) : 0.0f;
}

// Sums the splits of dh in order, four columns a thread.
__global__ __launch_bounds__(256) void ce_sum_kernel(const float* acc, int splits, int64_t split_stride,
                                                     int64_t ld, int64_t quads, int N, int D, void* out,
                                                     int64_t out_stride, int bf16) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t n = i / quads;
  if (n >= N) return;
  const int d = (int)(i - n * quads) * 4;
  const f32x4* p = (const f32x4*)(acc + n * ld + d);
  const int64_t step = split_stride / 4;
  f32x4 v = *p;
#pragma unroll 8
  for (int s = 1; s < splits; ++s) v += p[s * step];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (d + e < D) {
      if (bf16) put((uint16_t*)out + n * out_stride + d + e, v[e]);
      else ((float*)out)[n * out_stride + d + e] = v[e];
    }
}

template <typename Epi, typename EpiSplit, typename EpiF32>
int gemm(const CeGemm& g, const typename Epi::Args& ea, hipStream_t st) {
  const CeTile t = g.tile;
  const int tiles_m = (g.M + t.bm - 1) / t.bm;
  const int tiles_n = (g.N + t.bn - 1) / t.bn;
  const dim3 grid((uint32_t)tiles_m * (uint32_t)tiles_n, (uint32_t)g.splits);
  // both parts of dz at a depth of 64 do not fit LDS twice in the largest tile
  constexpr int WIDE = Epi::OF_DZ ? CE_LINE / 2 : CE_LINE;
#define CE_LAUNCH(E, BM, BN, WM, WN, LINE, EPI) \
  hipLaunchKernelGGL((ce_gemm_kernel<E, BM, BN, WM, WN, LINE, EPI>), grid, dim3(WM * WN * WAVE), 0, st, g, tiles_m, tiles_n, ea)
  if (g.planes == 3) {
    if (t.bm == 64)
      hipLaunchKernelGGL((ce_split_kernel<64, 128, 2, 2, EpiSplit>), grid, dim3(256), 0, st, g, tiles_m, tiles_n, ea);
    else
      hipLaunchKernelGGL((ce_split_kernel<256, 128, 4, 2, EpiSplit>), grid, dim3(512), 0, st, g, tiles_m, tiles_n, ea);
  } else if (g.planes == 0) {
    if (t.bn == 32) CE_LAUNCH(float, 64, 32, 4, 1, CE_LINE, EpiF32);
    else CE_LAUNCH(float, 128, 64, 2, 2, CE_LINE, EpiF32);
  } else if (t.bn == 32) {
    CE_LAUNCH(uint16_t, 64, 32, 4, 1, CE_LINE, Epi);
  } else if (t.bn == 64) {
    CE_LAUNCH(uint16_t, 128, 64, 2, 2, CE_LINE, Epi);
  } else {
    CE_LAUNCH(uint16_t, 256, 256, 2, 4, WIDE, Epi);
  }
#undef CE_LAUNCH
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace

// Tiles of bfloat16 and of float32 as it is, by the rows of B (states, or tokens for dW). Few rows leave the read of A as
// the bound, and many small workgroups in flight keep it busy: logits of 151,936
// tokens of 1,024 at 17 rows take 52 us in 64 x 32, 55 in 128 x 32, 59 in 256 x 32; at
// 64 rows 69 us in 128 x 64, 78 in 128 x 128; at 128 rows of 2,048 187 us in 128 x 64, 193 in
// 128 x 128, 204 in 256 x 128. From there on products bound it, and the largest tile
// reads LDS least: 1,300 TFLOP/s in 256 x 256, 930 in 256 x 128, 910 to 1,010 in 128 x 128.
// dh and dW of less than 128 columns (the rows of A) take the smaller tile too.
CeTile ce_tile(int64_t M, int64_t N, int planes) {
  if (planes == 3) return M <= 128 ? CeTile{64, 128, 2, 2} : CeTile{256, 128, 1, 1};
  const bool parts = planes == 1;   // dz in two
  if (N <= 32) return CeTile{64, 32, 6, parts ? 5 : 6};
  if (N <= 128 || M <= 128 || planes == 0) return CeTile{128, 64, 3, parts ? 2 : 3};
  return CeTile{256, 256, 1, 1};
}

int launch_ce_stats(const CeGemm& g, const CeStatsOut& o, hipStream_t st) {
  return gemm<EpiStats, EpiStats, EpiStats>(g, o, st);
}
int launch_ce_dz(const CeGemm& g, const CeDzOut& o, hipStream_t st) {
  return gemm<EpiDz<2>, EpiDz<3>, EpiDz<0>>(g, o, st);
}
int launch_ce_acc(const CeGemm& g, const CeAccOut& o, hipStream_t st) { return gemm<EpiAcc, EpiAcc, EpiAcc>(g, o, st); }
int launch_ce_mat(const CeGemm& g, const CeMatOut& o, hipStream_t st) { return gemm<EpiMat, EpiMat, EpiMat>(g, o, st); }

int launch_ce_pack(const CePack& p, hipStream_t st) {
  const int64_t blocks = (p.ld / 4 * p.rows + 255) / 256;
  const dim3 grid((uint32_t)(blocks < 16384 ? blocks : 16384));
  hipLaunchKernelGGL(ce_pack_kernel, grid, dim3(256), 0, st, p);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_ce_join(const MaxSum* partial, const float* zlabel, const int32_t* labels, int tiles,
                   int N, int V, float* loss, float* stats, hipStream_t st) {
  // few states: a workgroup each, or the tiles are read one after the other
  if (N <= 2048)
    hipLaunchKernelGGL(ce_join_kernel<1>, dim3((uint32_t)N), dim3(256), 0, st, partial, zlabel, labels, tiles,
                       N, V, loss, stats);
  else
    hipLaunchKernelGGL(ce_join_kernel<16>, dim3((uint32_t)((N + 15) / 16)), dim3(256), 0, st, partial, zlabel,
                       labels, tiles, N, V, loss, stats);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_ce_sum(const float* acc, int splits, int64_t split_stride, int64_t ld, int N, int D,
                  void* out, int64_t out_stride, int bf16, hipStream_t st) {
  const int64_t quads = ld / 4;   // ld is D rounded up to 4
  hipLaunchKernelGGL(ce_sum_kernel, dim3((uint32_t)((quads * N + 255) / 256)), dim3(256), 0, st, acc, splits,
                     split_stride, ld, quads, N, D, out, out_stride, bf16);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace sv
