// Host side of the drafter-training calls of include/spec_verify.h: argument
// checks before anything touches the device, how the work is cut into parts,
// workspace carving and the launches on the caller's stream.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../../include/spec_verify.h"
#include "sv_train.hpp"

static_assert(SV_MAX_TOP == sv::TOP_MAX_K && SV_MAX_TOP == sv::DIS_MAX_K, "kept logits per row");
static_assert(sv::TOP_CAP - sv::TOP_STEP >= sv::TOP_MAX_K, "a cut list leaves room for a group a thread");

namespace {

constexpr size_t WS_ALIGN = 256;

size_t align_up(size_t x) { return (x + WS_ALIGN - 1) / WS_ALIGN * WS_ALIGN; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

bool known(sv_dtype t) { return t == SV_F32 || t == SV_BF16; }
size_t size_of(sv_dtype t) { return t == SV_BF16 ? 2 : 4; }
bool aligned(const void* p, size_t to) { return (uintptr_t)p % to == 0; }
bool workspace_ok(const void* p, size_t have, size_t need) {
  return need == 0 || (p && aligned(p, WS_ALIGN) && have >= need);
}
bool temperature_ok(float t) { return t > 0.0f && isnormal(t); }   // 1 / t is finite too

// log2(e) / T, the factor of the kernels' exponents. One float, so that an exponent is one
// fused product: off by 2^-25 of a logit's distance to the row's largest, which for the
// tokens that count is within the rounding of the exponent itself.
float exponent_factor(float temperature) { return (float)(M_LOG2E / temperature); }

// Threads of a launch, 512 a workgroup, are counted in 32 bits.
constexpr int64_t MAX_WORKGROUPS = 1 << 23;
constexpr int64_t MAX_VOCAB_ROWS = 1 << 22;

// Carves a workspace front to back.
struct Carver {
  size_t off = 0;
  size_t take(size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes);
    return at;
  }
};

// ---------------------------------------------------------------- vocabulary rows

// Workgroups per row when there are few rows: as many as give about `total` in all,
// each with `least` bytes or more, if that takes more off a row's time than the kernel
// that joins them costs: `gain` bytes of one workgroup's streaming.
int64_t row_parts(int64_t R, int64_t bytes, int64_t total, int64_t least, int64_t gain, int64_t most) {
  int64_t p = total / R;
  if (p > bytes / least) p = bytes / least;
  if (p > most) p = most;
  return p > 1 && bytes - bytes / p >= gain ? p : 1;
}

// Top logits: a workgroup alone takes 8 bytes a nanosecond and 5 us besides, the join
// 5 to 12 us, more with more kept. 9 rows of 151,936 in bfloat16, 32 kept: 16 parts 16.6
// us, 8 parts 17.8, 4 parts 19.4; 100 rows, 64 kept: one part 44, four 26, eight 28; 400 rows:
// one 52, two 45, three 44, four 49. 331 rows of 50,257 in float32, 200 kept: one 48, two and
// three 46, four 55. 9 rows of 32,000, 32 kept: one 12.9, two 13.5, four 12.9.
struct TopLayout {
  int parts;
  size_t keys, sums, total;
};
bool top_layout(int32_t R, int32_t V, int32_t K, sv_dtype dtype, TopLayout* L) {
  if (R < 1 || R > MAX_VOCAB_ROWS || V < 1 || K < 1 || K > SV_MAX_TOP || K > V || !known(dtype)) return false;
  const int64_t most = sv::TOP_CAP / K < 64 ? sv::TOP_CAP / K : 64;   // what the join holds
  const int64_t parts = L->parts =
      (int)row_parts(R, (int64_t)V * size_of(dtype), 5 * sv::HOLD_CUS, 16000, 66000, most);
  Carver c;
  L->keys = c.take(parts > 1 ? (size_t)R * parts * K * sizeof(uint64_t) : 0);
  L->sums = c.take(parts > 1 ? (size_t)R * parts * sizeof(sv::MaxSum) : 0);
  L->total = c.off;
  return true;
}

// Distillation: a workgroup alone takes 23 bytes a nanosecond, the join 4.5 us. The loss
// of 32 rows of 151,936 in bfloat16 in 8 parts: 10.8 us, in one 17.0; of 128 in 4: 15.1,
// in one 20.2; of 400 in 2: 34, in one 27.
int distill_parts(int32_t R, int32_t V, sv_dtype dtype) {
  return (int)row_parts(R, (int64_t)V * size_of(dtype), 2 * sv::HOLD_CUS, 38000, 120000, 64);
}

// With the gradient, rows are held in registers (HOLD_NV's index) where they fit; -1:
// streamed. Not short ones, for which the walk over rows costs more than a second read
// of what the caches hold (4096 rows of 8,000 in bfloat16: held 105 us, streamed 74; of
// 32,000: 157 and 163; of 151,936: 574 and 708). Nor fewer than 96 long ones, which several
// workgroups share (32 rows of 151,936: held 31 us, in 8 parts 24; 128: 34 and 38).
int distill_hold(int32_t R, int32_t V, sv_dtype dtype) {
  const int64_t bytes = (int64_t)V * size_of(dtype);
  if (bytes < 40000 || (R < 96 && bytes > 200000)) return -1;
  return sv::hold_size(V, (int)size_of(dtype));
}

int distill_args(const void* logits, int64_t logits_stride, sv_dtype dtype, int32_t R, int32_t V,
                 const int32_t* ids, const float* tl, const float* tlse, int32_t K,
                 float temperature, void* grad, int64_t grad_stride, sv::DistillArgs* a) {
  if (!logits || !ids || !tl) return SV_EINVAL;
  if (!known(dtype)) return SV_EDTYPE;
  if (R < 1 || V < 1 || K < 1 || K > SV_MAX_TOP || !temperature_ok(temperature)) return SV_EINVAL;
  if (logits_stride < V || (grad && grad_stride < V)) return SV_EINVAL;
  if (!aligned(logits, size_of(dtype)) || !aligned(grad, size_of(dtype))) return SV_EINVAL;
  if (grad == logits && grad_stride != logits_stride) return SV_EINVAL;
  if (R > MAX_VOCAB_ROWS) return SV_ESIZE;
  a->logits = logits;
  a->stride = logits_stride;
  a->ids = ids;
  a->tl = tl;
  a->tlse = tlse;
  a->R = R;
  a->V = V;
  a->K = K;
  a->parts = distill_parts(R, V, dtype);
  a->hold = grad ? distill_hold(R, V, dtype) : -1;   // the loss alone streams faster
  a->inv_t = 1.0f / temperature;
  a->inv_t64 = 1.0 / temperature;
  a->c = exponent_factor(temperature);
  a->grad = grad;
  a->grad_stride = grad_stride;
  return SV_OK;
}

// ---------------------------------------------------------------- linear cross entropy

constexpr int64_t CE_MAX_ROWS = 1 << 22;
// Bytes of a piece's operands in the workspace. A piece is a whole number of
// rounds of tiles over the CUs (piece_rows); as many rounds as stay within
// CE_PIECE_BYTES, half of what the last-level cache holds, and at least one unless
// that takes more than CE_PIECE_MOST. dz of bfloat16 takes twice that, a part each: pieces
// of half the length make more sums of dh (8,192 states of 1,024 over 32,000 tokens 4,512 us a
// step instead of 3,386, 2,742 of 384 over 151,936 3,517 instead of 2,945).
constexpr int64_t CE_PIECE_BYTES = 128ll << 20, CE_PIECE_MOST = 1024ll << 20;
constexpr int64_t CE_PIECE_STEP = 256;    // a multiple of every tile height
constexpr int64_t CE_CUS = 256;

// Up to here states of float32 take the float32 matrix instructions (linear_ce.hip).
constexpr int64_t CE_F32_STATES = 384;

// Up to here states dW is bound by its writes, which many small tiles serve better (a step of
// 151,936 tokens of 1,408 at 128 states 756 us, with dW in 256 x 256 774; at 200 881 and 827).
constexpr int64_t CE_SHORT_DEPTH = 128;

// float32 in three parts of bfloat16: planes 3; as it is: planes 0; bfloat16: 1.
struct CeShape {
  int64_t N, D, V, kp;   // kp: row length of packed operands, whole steps of depth
  int planes;
  bool f32() const { return planes == 0; }
  int es() const { return f32() ? 4 : 2; }                   // bytes of an element of an operand
  int64_t row_bytes(int64_t n) const { return n * (planes == 3 ? 6 : es()); }
  int64_t dz_bytes(int64_t n) const { return n * (planes == 3 ? 6 : 4); }   // bfloat16: two parts
  int64_t depth() const { return sv::CE_LINE / es(); }
  int64_t per16() const { return 16 / es(); }
};
bool ce_shape(int32_t N, int32_t D, int32_t V, sv_dtype dtype, CeShape* s) {
  if (N < 1 || D < 1 || V < 1 || !known(dtype)) return false;
  if (N > CE_MAX_ROWS || D > sv::CE_MAX_D || V >= INT32_MAX - 1024) return false;
  *s = CeShape{N, D, V, 0, dtype == SV_BF16 ? 1 : N <= CE_F32_STATES ? 0 : 3};
  s->kp = round_up(D, s->depth());
  // workgroups of the products over the vocabulary and of dh, and of its sums
  const sv::CeTile t = sv::ce_tile(V, N, s->planes), h = sv::ce_tile(D, N, s->planes);
  return ceil_div(V, t.bm) * ceil_div(N, t.bn) < MAX_WORKGROUPS &&
         ceil_div(D, h.bm) * ceil_div(N, h.bn) < MAX_WORKGROUPS && ceil_div(D, 4) * N / 256 < MAX_WORKGROUPS;
}

// Tokens of a piece whose operands take `bytes` a token. Rounds do not exceed the CUs: with
// three columns of tiles, 85 rows of them make one (86 would take a second one for two
// tiles: 622 states of 2,048 over 151,936 tokens 2,734 us a step instead of 2,483).
int64_t piece_rows(const CeShape& s, int64_t bytes) {
  const sv::CeTile t = sv::ce_tile(s.V, s.N, s.planes);
  int64_t round = CE_CUS * t.per_cu / ceil_div(s.N, t.bn) * t.bm / CE_PIECE_STEP * CE_PIECE_STEP;
  if (round < CE_PIECE_STEP) round = CE_PIECE_STEP;
  int64_t rows = CE_PIECE_BYTES / bytes / round * round;
  if (rows < round) rows = round;
  const int64_t most = CE_PIECE_MOST / bytes / CE_PIECE_STEP * CE_PIECE_STEP;
  if (rows > most) rows = most;
  if (rows < 4 * CE_PIECE_STEP) rows = 4 * CE_PIECE_STEP;
  if (rows > sv::CE_MAX_D) rows = sv::CE_MAX_D;   // dz's row length
  const int64_t all = round_up(s.V, CE_PIECE_STEP);
  return rows < all ? rows : all;
}

// Tokens packed at a time. Heads whose width is whole groups of 16 bytes are read in place, but
// for odd strides, and do not get room for a long piece that only those would use: one
// state of 4,096 over 128,256 tokens had a workspace of 768 MB, its logits take 0.5. Odd strides
// pay for it in launches that do not fill the CUs: 17 states of 4,096 over 151,936 tokens, rows
// 4,099 apart, 880 us instead of 836, 200 states 1,410 instead of 970, a step of 64 of float32
// over 32,000 1,882 instead of 1,087. Other widths are packed by every call, which has the whole
// piece.
int64_t packed_rows(const CeShape& s, int64_t piece) {
  if (s.planes == 3 || s.D % s.per16()) return piece;
  int64_t rows = CE_PIECE_BYTES / s.row_bytes(s.kp) / CE_PIECE_STEP * CE_PIECE_STEP;
  if (rows < 4 * CE_PIECE_STEP) rows = 4 * CE_PIECE_STEP;
  return rows < piece ? rows : piece;
}

struct CeForward {
  int64_t piece;               // tokens a piece where the weight is packed
  size_t partial, zlabel, hidden, weight, total;
};
CeForward ce_forward(const CeShape& s) {
  CeForward f;
  Carver c;
  f.piece = packed_rows(s, piece_rows(s, s.row_bytes(s.kp)));
  f.partial = c.take((size_t)(ceil_div(s.V, sv::ce_tile(s.V, s.N, s.planes).bm) * s.N) * sizeof(sv::MaxSum));
  f.zlabel = c.take((size_t)s.N * sizeof(float));
  f.hidden = c.take((size_t)(s.N * s.row_bytes(s.kp)));
  f.weight = c.take((size_t)(f.piece * s.row_bytes(s.kp)));
  f.total = c.off;
  return f;
}

// dh has few tiles and a long depth, a piece of the vocabulary: workgroups that share a
// tile's depth. The fewest microseconds of a piece: rounds of workgroups over the CUs, and
// the sums that every split reads and writes. As many splits as give each CU its fill
// take a round too many instead: 622 states of 2,048 over 151,936 tokens 2,934 us a step
// instead of 2,499, 2,742 of 384 3,231 instead of 2,832.
int dh_splits(const CeShape& s, int64_t piece, int64_t ld) {
  const sv::CeTile t = sv::ce_tile(s.D, s.N, s.planes);
  const int64_t tiles = ceil_div(s.D, t.bm) * ceil_div(s.N, t.bn), places = CE_CUS * t.per_cu_dz;
  const int64_t steps = piece / s.depth() * (s.planes == 3 || t.bm == 256 ? 2 : 1);
  const double rate = s.planes == 1 ? 1200e6 : s.planes == 3 ? 180e6 : 120e6;   // flop a us
  const double tile_us = 2.0 * t.bm * t.bn * piece * (s.planes == 1 ? 2 : 1) / (rate / places);
  const double sum_us = 2.0 * s.N * ld * 4 / 5e6;   // at 5 TB/s
  int64_t most = steps / 4, fit = CE_PIECE_BYTES / (s.N * ld * 4);
  if (most > fit) most = fit;
  int64_t best = 1;
  double least = INFINITY;
  auto offer = [&](int64_t n) {
    n = n > most ? most : n;
    n = n < 1 ? 1 : n;
    const double us = (double)ceil_div(tiles * n, places) / n * tile_us + n * sum_us;
    if (us < least) {
      least = us;
      best = n;
    }
  };
  // the most splits of so many rounds, and where the sums weigh as much as the product
  const int64_t rounds = ceil_div(tiles, places);
  for (int64_t r = rounds; r < rounds + 8; ++r) offer(r * places / tiles);
  offer((int64_t)sqrt(tile_us / sum_us));
  return (int)best;
}

struct CeBackward {
  int64_t piece, packed, acc_ld;   // tokens a piece, and a piece that is packed
  int splits;
  size_t hidden, weight, dz, acc, total;
};
CeBackward ce_backward(const CeShape& s, bool want_h) {
  CeBackward b;
  Carver c;
  b.piece = piece_rows(s, s.row_bytes(s.N > s.kp ? s.N : s.kp));
  b.packed = packed_rows(s, b.piece);
  b.acc_ld = round_up(s.D, 4);
  b.splits = dh_splits(s, b.piece, b.acc_ld);
  b.hidden = c.take((size_t)(s.N * s.row_bytes(s.kp)));
  b.weight = c.take((size_t)(b.packed * s.row_bytes(s.kp)));
  b.dz = c.take((size_t)s.dz_bytes(s.N * b.piece));
  b.acc = c.take(want_h ? (size_t)(b.splits * s.N * b.acc_ld) * 4 : 0);
  b.total = c.off;
  return b;
}

// A matrix as the products take it: rows on 16 bytes, read in whole groups of 16 bytes.
// Used as it is where it has that form, else packed.
struct Operand {
  const void* p;
  int64_t ld, plane;
  int64_t cols;
};
bool ce_direct(const void* p, int64_t stride, const CeShape& s) {
  return s.planes != 3 && s.D % s.per16() == 0 && aligned(p, 16) && stride % s.per16() == 0 &&
         stride <= sv::CE_MAX_D;
}
int ce_operand(const void* src, int64_t stride, int64_t row0, int64_t rows, const CeShape& s,
               void* room, hipStream_t st, Operand* out) {
  const char* at = (const char*)src + row0 * stride * (s.planes == 1 ? 2 : 4);
  if (ce_direct(src, stride, s)) {
    *out = Operand{at, stride, 0, s.D};
    return 0;
  }
  const sv::CePack p{at, stride, s.planes == 1, (int)rows, (int)s.D, s.planes, room, s.kp, rows * s.kp};
  *out = Operand{room, s.kp, p.plane, s.kp};
  return sv::launch_ce_pack(p, st);
}
sv::CeGemm ce_gemm(const Operand& a, int64_t M, const Operand& b, int64_t N, int64_t K, const CeShape& s) {
  return sv::CeGemm{a.p, b.p, a.ld, b.ld, a.plane, b.plane, (int)M, (int)N, (int)K, s.planes, 1,
                    sv::ce_tile(M, N, s.planes)};
}
// Depth of the logits' product: what both operands have in whole groups.
int64_t ce_depth(const Operand& a, const Operand& b) { return a.cols < b.cols ? a.cols : b.cols; }

int ce_check(const void* hidden, int64_t hidden_stride, const void* weight, int64_t weight_stride,
             sv_dtype dtype, const int32_t* labels, int32_t N, int32_t D, int32_t V, CeShape* s) {
  if (!hidden || !weight || !labels) return SV_EINVAL;
  if (!known(dtype)) return SV_EDTYPE;
  if (N < 1 || D < 1 || V < 1 || hidden_stride < D || weight_stride < D) return SV_EINVAL;
  if (!aligned(hidden, size_of(dtype)) || !aligned(weight, size_of(dtype))) return SV_EINVAL;
  return ce_shape(N, D, V, dtype, s) ? SV_OK : SV_ESIZE;
}

}  // namespace

extern "C" {

size_t spec_verify_top_logits_workspace_bytes(int32_t R, int32_t V, int32_t K, sv_dtype dtype) {
  TopLayout L;
  return top_layout(R, V, K, dtype, &L) ? L.total : 0;
}

int spec_verify_top_logits(const void* logits, int64_t logits_stride, sv_dtype dtype, int32_t R,
                           int32_t V, int32_t K, float temperature, int32_t* out_ids,
                           float* out_values, float* out_lse, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (!logits || !out_ids || !out_values) return SV_EINVAL;
  if (!known(dtype)) return SV_EDTYPE;
  if (!temperature_ok(temperature) || logits_stride < V || !aligned(logits, size_of(dtype)))
    return SV_EINVAL;
  TopLayout L;
  if (!top_layout(R, V, K, dtype, &L)) return R > MAX_VOCAB_ROWS && V >= 1 ? SV_ESIZE : SV_EINVAL;
  if (!workspace_ok(workspace, workspace_bytes, L.total)) return SV_EWORKSPACE;
  sv::TopArgs a{};
  a.logits = logits;
  a.stride = logits_stride;
  a.R = R;
  a.V = V;
  a.K = K;
  a.parts = L.parts;
  a.c = exponent_factor(temperature);
  a.temperature = temperature;
  a.ids = out_ids;
  a.values = out_values;
  a.lse = out_lse;
  a.keys = (uint64_t*)((char*)workspace + L.keys);
  a.sums = (sv::MaxSum*)((char*)workspace + L.sums);
  return sv::launch_top_logits(a, dtype == SV_BF16, (hipStream_t)stream) ? SV_EHIP : SV_OK;
}

size_t spec_verify_distill_workspace_bytes(int32_t R, int32_t V, sv_dtype dtype) {
  if (R < 1 || R > MAX_VOCAB_ROWS || V < 1 || !known(dtype)) return 0;
  const int parts = distill_parts(R, V, dtype);
  return parts > 1 ? align_up((size_t)R * parts * sizeof(sv::MaxSum)) : 0;
}

int spec_verify_distill(const void* logits, int64_t logits_stride, sv_dtype dtype, int32_t R,
                        int32_t V, const int32_t* teacher_ids, const float* teacher_logits,
                        const float* teacher_lse, int32_t K, float temperature,
                        const float* row_weight, float* out_loss, float* out_stats, void* out_grad,
                        int64_t grad_stride, void* workspace, size_t workspace_bytes, void* stream) {
  sv::DistillArgs a{};
  if (!out_loss || !out_stats) return SV_EINVAL;
  const int rc = distill_args(logits, logits_stride, dtype, R, V, teacher_ids, teacher_logits,
                              teacher_lse, K, temperature, out_grad, grad_stride, &a);
  if (rc != SV_OK) return rc;
  if (!workspace_ok(workspace, workspace_bytes, spec_verify_distill_workspace_bytes(R, V, dtype)))
    return SV_EWORKSPACE;
  a.weight = row_weight;
  a.loss = out_loss;
  a.stats = out_stats;
  a.sums = (sv::MaxSum*)workspace;
  return sv::launch_distill(a, dtype == SV_BF16, (hipStream_t)stream) ? SV_EHIP : SV_OK;
}

int spec_verify_distill_backward(const void* logits, int64_t logits_stride, sv_dtype dtype,
                                 int32_t R, int32_t V, const int32_t* teacher_ids,
                                 const float* teacher_logits, const float* teacher_lse, int32_t K,
                                 float temperature, const float* stats, const float* grad_loss,
                                 void* out_grad, int64_t grad_stride, void* stream) {
  sv::DistillArgs a{};
  if (!stats || !out_grad) return SV_EINVAL;
  const int rc = distill_args(logits, logits_stride, dtype, R, V, teacher_ids, teacher_logits,
                              teacher_lse, K, temperature, out_grad, grad_stride, &a);
  if (rc != SV_OK) return rc;
  a.weight = grad_loss;
  a.stats = const_cast<float*>(stats);   // only read
  return sv::launch_distill_backward(a, dtype == SV_BF16, (hipStream_t)stream) ? SV_EHIP : SV_OK;
}

size_t spec_verify_linear_ce_workspace_bytes(int32_t N, int32_t D, int32_t V, sv_dtype dtype) {
  CeShape s;
  return ce_shape(N, D, V, dtype, &s) ? ce_forward(s).total : 0;
}

int spec_verify_linear_ce(const void* hidden, int64_t hidden_stride, const void* weight,
                          int64_t weight_stride, sv_dtype dtype, const int32_t* labels, int32_t N,
                          int32_t D, int32_t V, float* out_loss, float* out_stats, void* workspace,
                          size_t workspace_bytes, void* stream) {
  CeShape s;
  if (!out_loss || !out_stats) return SV_EINVAL;
  const int rc = ce_check(hidden, hidden_stride, weight, weight_stride, dtype, labels, N, D, V, &s);
  if (rc != SV_OK) return rc;
  const CeForward f = ce_forward(s);
  if (!workspace_ok(workspace, workspace_bytes, f.total)) return SV_EWORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  char* ws = (char*)workspace;
  sv::MaxSum* partial = (sv::MaxSum*)(ws + f.partial);
  float* zlabel = (float*)(ws + f.zlabel);
  Operand h, w;
  if (ce_operand(hidden, hidden_stride, 0, N, s, ws + f.hidden, st, &h)) return SV_EHIP;
  const sv::CeTile tile = sv::ce_tile(V, N, s.planes);   // of every piece: partial has a row a tile
  const int64_t piece = ce_direct(weight, weight_stride, s) ? V : f.piece;
  for (int64_t v0 = 0; v0 < V; v0 += piece) {
    const int64_t rows = V - v0 < piece ? V - v0 : piece;
    if (ce_operand(weight, weight_stride, v0, rows, s, ws + f.weight, st, &w)) return SV_EHIP;
    const sv::CeStatsOut o{labels, (int)v0, V, partial + v0 / tile.bm * N, zlabel};
    sv::CeGemm g = ce_gemm(w, rows, h, N, ce_depth(w, h), s);
    g.tile = tile;
    if (sv::launch_ce_stats(g, o, st)) return SV_EHIP;
  }
  return sv::launch_ce_join(partial, zlabel, labels, (int)ceil_div(V, tile.bm), N, V, out_loss, out_stats, st)
             ? SV_EHIP : SV_OK;
}

size_t spec_verify_linear_ce_backward_workspace_bytes(int32_t N, int32_t D, int32_t V,
                                                      sv_dtype dtype, int want_grad_hidden,
                                                      int want_grad_weight) {
  CeShape s;
  if (!want_grad_hidden && !want_grad_weight) return 0;
  return ce_shape(N, D, V, dtype, &s) ? ce_backward(s, want_grad_hidden).total : 0;
}

int spec_verify_linear_ce_backward(const void* hidden, int64_t hidden_stride, const void* weight,
                                   int64_t weight_stride, sv_dtype dtype, const int32_t* labels,
                                   const float* stats, const float* grad_loss, int32_t N, int32_t D,
                                   int32_t V, void* out_grad_hidden, int64_t grad_hidden_stride,
                                   void* out_grad_weight, int64_t grad_weight_stride,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  CeShape s;
  if (!stats || (!out_grad_hidden && !out_grad_weight)) return SV_EINVAL;
  const int rc = ce_check(hidden, hidden_stride, weight, weight_stride, dtype, labels, N, D, V, &s);
  if (rc != SV_OK) return rc;
  if ((out_grad_hidden && (grad_hidden_stride < D || !aligned(out_grad_hidden, size_of(dtype)))) ||
      (out_grad_weight && (grad_weight_stride < D || !aligned(out_grad_weight, size_of(dtype)))))
    return SV_EINVAL;
  const CeBackward b = ce_backward(s, out_grad_hidden);
  if (!workspace_ok(workspace, workspace_bytes, b.total)) return SV_EWORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  char* ws = (char*)workspace;
  const int bf16 = dtype == SV_BF16;
  const size_t es = size_of(dtype);
  void* dz = ws + b.dz;
  float* acc = (float*)(ws + b.acc);
  Operand h, w;
  if (ce_operand(hidden, hidden_stride, 0, N, s, ws + b.hidden, st, &h)) return SV_EHIP;
  const int64_t piece = ce_direct(weight, weight_stride, s) ? b.piece : b.packed;
  for (int64_t v0 = 0; v0 < V; v0 += piece) {
    const int64_t rows = V - v0 < piece ? V - v0 : piece;
    const int64_t ldz = round_up(rows, s.depth());
    if (ce_operand(weight, weight_stride, v0, rows, s, ws + b.weight, st, &w)) return SV_EHIP;
    const sv::CeDzOut o{labels, stats, grad_loss, (int)v0, V, dz, ldz, N * ldz};
    if (sv::launch_ce_dz(ce_gemm(w, rows, h, N, ce_depth(w, h), s), o, st)) return SV_EHIP;
    const Operand z{dz, ldz, N * ldz, ldz};
    if (out_grad_hidden) {
      sv::CeGemm g = ce_gemm(w, D, z, N, rows, s);
      g.splits = b.splits;
      const sv::CeAccOut ao{acc, b.acc_ld, N * b.acc_ld, v0 > 0};
      if (sv::launch_ce_acc(g, ao, st)) return SV_EHIP;
    }
    if (out_grad_weight) {
      sv::CeGemm g = ce_gemm(h, D, z, rows, N, s);
      if (N <= CE_SHORT_DEPTH && s.planes == 1) g.tile = sv::ce_tile(D, 128, s.planes);
      const sv::CeMatOut mo{(char*)out_grad_weight + v0 * grad_weight_stride * es, grad_weight_stride, bf16};
      if (sv::launch_ce_mat(g, mo, st)) return SV_EHIP;
    }
  }
  if (out_grad_hidden &&
      sv::launch_ce_sum(acc, b.splits, N * b.acc_ld, b.acc_ld, N, D, out_grad_hidden,
                        grad_hidden_stride, bf16, st))
    return SV_EHIP;
  return SV_OK;
}

}  // extern "C"
