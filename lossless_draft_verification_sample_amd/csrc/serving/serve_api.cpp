// Host side of the calls for the verification pass's rows (include/spec_verify.h):
// argument checks before anything touches the device, how work is cut into
// workgroups, workspace carving and the launches on the caller's stream.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../../include/spec_verify.h"
#include "sv_serve.hpp"

namespace {

constexpr size_t WS_ALIGN = 256;
// Threads of a launch, 256 a workgroup, are counted in 32 bits.
constexpr int64_t MAX_WORKGROUPS = 1 << 23;
constexpr int64_t MAX_TOKENS = 1 << 30;
constexpr int MAX_PAGE = 65536;
constexpr int MAX_GROUP = 4096;    // query heads that share a cache head
constexpr int CUS = 256;
constexpr int SINGLE_TOKENS = 1120;   // in reach: a workgroup may take all blocks of a unit

size_t align_up(size_t x) { return (x + WS_ALIGN - 1) / WS_ALIGN * WS_ALIGN; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool known(sv_dtype t) { return t == SV_F32 || t == SV_BF16; }
size_t size_of(sv_dtype t) { return t == SV_BF16 ? 2 : 4; }
bool aligned(const void* p, size_t to) { return (uintptr_t)p % to == 0; }

// Inputs: strides of dimensions of one entry do not matter, others are not negative.
bool readable(sv_strides s, int64_t B, int64_t N, int64_t H) {
  return (B <= 1 || s.request >= 0) && (N <= 1 || s.row >= 0) && (H <= 1 || s.head >= 0);
}
// Outputs: no two rows or heads overlap, with the dimensions in any order.
bool writable(sv_strides s, int64_t B, int64_t N, int64_t H, int64_t width) {
  int64_t step[3] = {s.request, s.row, s.head}, size[3] = {B, N, H};
  for (int i = 0; i < 3; ++i)
    if (size[i] <= 1) step[i] = INT64_MAX;      // never stepped over
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j)
      if (step[j] > step[j + 1]) {
        const int64_t a = step[j], b = size[j];
        step[j] = step[j + 1];
        size[j] = size[j + 1];
        step[j + 1] = a;
        size[j + 1] = b;
      }
  int64_t extent = width;                       // elements from the first to the last, and one
  for (int i = 0; i < 3; ++i) {
    if (size[i] <= 1) continue;
    if (step[i] < extent || step[i] > INT64_MAX / 4 / size[i]) return false;
    extent += step[i] * (size[i] - 1);
  }
  return true;
}
sv::Strides strides_of(sv_strides s) { return sv::Strides{s.request, s.row, s.head}; }
bool same(sv_strides a, sv_strides b, int64_t B, int64_t N, int64_t H) {
  return (B <= 1 || a.request == b.request) && (N <= 1 || a.row == b.row) && (H <= 1 || a.head == b.head);
}
// In place only at the same strides.
bool place_ok(const void* in, sv_strides is, const void* out, sv_strides os, int64_t B, int64_t N, int64_t H) {
  return in != out || same(is, os, B, N, H);
}

// ---------------------------------------------------------------- the cache

bool cache_shape(int64_t pages, int64_t heads, int64_t page, int64_t D) {
  return pages >= 1 && heads >= 1 && D >= 1 && D <= sv::CACHE_MAX_D && page >= sv::CACHE_BLOCK && page <= MAX_PAGE &&
         (page & (page - 1)) == 0;
}
int log2_of(int x) { return 31 - __builtin_clz((unsigned)x); }

int cache_of(const sv_cache* c, bool k, bool v, sv::Cache* out) {
  if (!c || (k && (!c->k || !c->k_scale)) || (v && (!c->v || !c->v_scale))) return SV_EINVAL;
  if (!cache_shape(c->pages, c->heads, c->page_size, c->head_dim)) return SV_EINVAL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)) return SV_EINVAL;
  *out = sv::Cache{(uint8_t*)c->k, (uint8_t*)c->v, c->k_scale, c->v_scale, c->pages, c->heads,
                   log2_of(c->page_size / sv::CACHE_BLOCK), (int)ceil_div(c->head_dim, 32), c->head_dim};
  return SV_OK;
}

int batch_of(const int32_t* table, int32_t width, const int32_t* first, const int32_t* rows, int32_t B, int32_t N,
             int32_t page, sv::Batch* out) {
  if (!table || width < 1 || B < 1 || N < 1) return SV_EINVAL;
  if (!aligned(table, 4) || !aligned(first, 4) || !aligned(rows, 4)) return SV_EINVAL;
  if ((int64_t)width * page > MAX_TOKENS || N > MAX_TOKENS) return SV_ESIZE;
  *out = sv::Batch{table, width, first, rows, B, N, width * page};
  return SV_OK;
}

int cache_rows(const sv_cache* cache, const int32_t* table, int32_t width, const int32_t* first,
               const int32_t* rows, const void* k, sv_strides ks, const void* v, sv_strides vs, sv_dtype dtype,
               int32_t B, int32_t N, bool write, sv::CacheRowsArgs* a) {
  if (write ? !k || !v : !k && !v) return SV_EINVAL;
  if (!known(dtype)) return SV_EDTYPE;
  int rc = cache_of(cache, k, v, &a->c);
  if (rc == SV_OK) rc = batch_of(table, width, first, rows, B, N, cache->page_size, &a->t);
  if (rc != SV_OK) return rc;
  const int64_t H = a->c.heads, D = a->c.D;
  for (int i = 0; i < 2; ++i) {
    const void* p = i ? v : k;
    const sv_strides s = i ? vs : ks;
    if (!p) continue;
    if (!aligned(p, size_of(dtype))) return SV_EINVAL;
    if (write ? !readable(s, B, N, H) : !writable(s, B, N, H, D)) return SV_EINVAL;
  }
  a->k = (void*)k;
  a->v = (void*)v;
  a->ks = strides_of(ks);
  a->vs = strides_of(vs);
  a->which = (k ? 1 : 0) | (v ? 2 : 0);
  a->bf16 = dtype == SV_BF16;
  // rows that start at a block's last token touch one block more
  a->blocks = (int)ceil_div((int64_t)N + sv::CACHE_BLOCK - 1, sv::CACHE_BLOCK);    // N <= 2^30
  if ((double)B * a->blocks * H * 2 >= MAX_WORKGROUPS) return SV_ESIZE;
  return SV_OK;
}

// ---------------------------------------------------------------- attention

// Whether units over a short reach are shared out as longer ones are. A unit's own workgroup has no join, but each of
// its four waves walks `across` fourths of the blocks; shared workgroups take four. A block costs 0.1 us times `block`
// (measured: 1.0 for one tile of 128 dimensions in bfloat16, 1.8 for three; float32 1.3 and 2.8), the join and its launch
// 10 us and 0.16 more a unit. Times in us, own workgroup / shared out, at 1,000 tokens but where it says so:
//   8 units of one tile 14.2 / 16.8, of three 23.9 / 19.0 (500 tokens 17.2 / 20.3), 64 of three 24.2 / 26.0, 256 24.9 / 41.5
//   heads of 256, 8 units of one tile 19.2 / 16.6
//   64 rows, four waves side by side: 3 units of three tiles 71.1 / 34.1 (500 tokens 47.9 / 38.9, 250 35.8 / 39.8),
//   24 units 76.5 / 39.4, 64 of two tiles 69.8 / 55.1 (500 tokens 46.9 / 49.4), 256 of them 74.4 / 78.7
//   float32: 8 units of one tile 16.1 / 16.8, of three 34.9 / 24.1, 64 of three 35.2 / 34.2; 8 of four 48.2 / 26.8
bool sharing_pays(int64_t tokens, int64_t units, int64_t across, int64_t nt, int64_t bricks, sv_dtype dtype) {
  const double saved = across * (ceil_div(tokens, sv::CACHE_BLOCK) / 4.0 - 1.0);
  const double block = 5.0 + (double)(bricks * nt * (dtype == SV_BF16 ? 1 : 2));
  return saved * block > 100.0 + 1.6 * units;
}

// Tiles of 16 columns: as few sets as the LDS that holds their queries allows (60 KB, so that
// two workgroups fit a CU with room to spare), then as few waves side by side as the
// registers allow, so that the others share out the tokens.
bool attend_shape(int64_t B, int64_t N, int64_t qh, int64_t heads, int64_t D, int64_t tokens, sv_dtype dtype,
                  sv::AttendShape* s) {
  if (B < 1 || N < 1 || N > SV_MAX_ROWS || qh < 1 || heads < 1 || qh % heads || D < 1 || D > sv::CACHE_MAX_D ||
      qh / heads > MAX_GROUP || tokens < 1 || tokens > MAX_TOKENS || !known(dtype) || (double)B * N * qh >= 2147483648.0)
    return false;
  const int64_t bricks = ceil_div(D, 32), parts = dtype == SV_BF16 ? 1 : 3;
  const int64_t cols = N * (qh / heads), tiles = ceil_div(cols, 16);
  const int64_t most = 60 / (bricks * parts), nt_most = bricks <= 4 ? 4 : 2;
  for (int64_t sets = 1;; ++sets) {
    const int64_t t = ceil_div(tiles, sets);
    for (int64_t across = 1; across <= 4; across *= 2) {
      const int64_t nt = ceil_div(t, across);
      if (nt > nt_most || nt * across > most) continue;
      const int64_t units = B * heads * sets;
      const int64_t cols_set = 16 * nt * across;
      // a workgroup takes four blocks at least
      const double blocks = (double)units * (ceil_div(tokens, sv::CACHE_BLOCK) + 1);
      const int64_t full = CUS * sv::attend_per_cu((int)bricks, (int)nt);
      const int64_t grid = ceil(blocks / 4) < full ? (int64_t)ceil(blocks / 4) : full;
      // Columns of a workgroup of the join: three items a thread, one where the units are few, and an
      // eighth where they have so many parts that reading them is a long chain (one request of 131,072
      // tokens, 64 parts, nine rows: 69 -> 63 us; of 4,000 tokens, 31 parts: 23 -> 20; four requests, 16 parts:
      // 184 -> 187; 16 requests, 4 parts: 33 -> 51).
      const bool split = grid >= 24 * units;
      int64_t join = cols_set;
      while (join > 1 && join * bricks * 8 > ((double)units * ceil_div(cols_set, join) >= 4 * CUS ? 768 : split ? 32 : 256))
        join = (join + 1) / 2;
      if ((double)units * ceil_div(cols_set, join) >= MAX_WORKGROUPS) return false;
      s->join_cols = (int)join;
      s->join_split = split;
      s->cols = (int)cols;
      s->nt = (int)nt;
      s->across = (int)across;
      s->sets = (int)sets;
      s->cols_set = (int)cols_set;
      const int64_t q = nt * across * bricks * parts * 1024, sums = 4096 * nt * sv::attend_round((int)bricks, (int)nt);
      s->lds = (int)(q > sums ? q : sums);
      s->units = (int)units;
      s->may_single = tokens <= SINGLE_TOKENS;
      s->single = s->may_single && !sharing_pays(tokens, units, across, nt, bricks, dtype);
      s->grid = (int)(s->single ? units : grid);
      return true;
    }
  }
}
struct AttendSpace {
  size_t record, partial, total;
};
AttendSpace attend_space(const sv::AttendShape& s, int64_t B, int64_t heads, int64_t D) {
  AttendSpace w;
  w.record = w.partial = w.total = 0;
  if (s.single) return w;
  w.partial = align_up((size_t)(B * heads * s.sets) * 2 * sizeof(int32_t));
  w.total = w.partial + align_up((size_t)s.grid * 2 * s.cols_set * (ceil_div(D, 32) * 32 + 2) * sizeof(float));
  return w;
}

}  // namespace

extern "C" {

int spec_verify_rotate(const void* q, sv_strides q_strides, const void* k, sv_strides k_strides,
                       sv_dtype dtype, int32_t B, int32_t N, int32_t q_heads, int32_t k_heads,
                       int32_t head_dim, int32_t rotary_dim, int interleaved, int inverse,
                       const double* freqs, float scale, const int32_t* kv_len,
                       const int32_t* rows, void* out_q, sv_strides out_q_strides, void* out_k,
                       sv_strides out_k_strides, void* stream) {
  if (!q || !out_q || (k_heads > 0 && (!k || !out_k)) || (rotary_dim > 0 && !freqs)) return SV_EINVAL;
  if (!known(dtype)) return SV_EDTYPE;
  if (B < 1 || N < 1 || q_heads < 1 || k_heads < 0 || head_dim < 1 || head_dim > 1024 || rotary_dim < 0 ||
      rotary_dim % 2 || rotary_dim > head_dim || !isfinite(scale))
    return SV_EINVAL;
  if ((int64_t)q_heads + k_heads > 1 << 15 || (double)B * N >= 2147483648.0) return SV_ESIZE;
  const size_t es = size_of(dtype);
  if (!aligned(q, es) || !aligned(out_q, es) || !aligned(freqs, 8) || !aligned(kv_len, 4) || !aligned(rows, 4) ||
      !readable(q_strides, B, N, q_heads) || !writable(out_q_strides, B, N, q_heads, head_dim) ||
      !place_ok(q, q_strides, out_q, out_q_strides, B, N, q_heads))
    return SV_EINVAL;
  if (k_heads > 0 &&
      (!aligned(k, es) || !aligned(out_k, es) || !readable(k_strides, B, N, k_heads) ||
       !writable(out_k_strides, B, N, k_heads, head_dim) || !place_ok(k, k_strides, out_k, out_k_strides, B, N, k_heads)))
    return SV_EINVAL;
  const sv::RotateArgs a{q, k, out_q, out_k, strides_of(q_strides), strides_of(k_strides), strides_of(out_q_strides),
                         strides_of(out_k_strides), B, N, q_heads, k_heads, head_dim, rotary_dim, freqs, scale,
                         interleaved != 0, inverse != 0, dtype == SV_BF16, kv_len, rows};
  return sv::launch_rotate(a, (hipStream_t)stream) ? SV_EHIP : SV_OK;
}

size_t spec_verify_cache_bytes(int32_t pages, int32_t heads, int32_t page_size, int32_t head_dim) {
  if (!cache_shape(pages, heads, page_size, head_dim)) return 0;
  const double all = (double)pages * heads * page_size * ceil_div(head_dim, 32) * 32;
  if (all >= 9e18) return 0;
  return (size_t)pages * heads * page_size * ceil_div(head_dim, 32) * 32;
}

int spec_verify_cache_write(const sv_cache* cache, const int32_t* page_table, int32_t table_width,
                            const int32_t* kv_len, const int32_t* rows, const void* k,
                            sv_strides k_strides, const void* v, sv_strides v_strides,
                            sv_dtype dtype, int32_t B, int32_t N, void* stream) {
  sv::CacheRowsArgs a;
  if (!kv_len) return SV_EINVAL;
  const int rc = cache_rows(cache, page_table, table_width, kv_len, rows, k, k_strides, v, v_strides, dtype, B, N,
                            true, &a);
  if (rc != SV_OK) return rc;
  return sv::launch_cache_write(a, (hipStream_t)stream) ? SV_EHIP : SV_OK;
}

int spec_verify_cache_read(const sv_cache* cache, const int32_t* page_table, int32_t table_width,
                           const int32_t* first, const int32_t* rows, void* out_k,
                           sv_strides k_strides, void* out_v, sv_strides v_strides, sv_dtype dtype,
                           int32_t B, int32_t N, void* stream) {
  sv::CacheRowsArgs a;
  const int rc = cache_rows(cache, page_table, table_width, first, rows, out_k, k_strides, out_v, v_strides, dtype, B,
                            N, false, &a);
  if (rc != SV_OK) return rc;
  return sv::launch_cache_read(a, (hipStream_t)stream) ? SV_EHIP : SV_OK;
}

size_t spec_verify_attention_workspace_bytes(int32_t B, int32_t N, int32_t q_heads, int32_t heads,
                                             int32_t head_dim, int64_t tokens, sv_dtype dtype) {
  sv::AttendShape s;
  if (!attend_shape(B, N, q_heads, heads, head_dim, tokens, dtype, &s)) return 0;
  return attend_space(s, B, heads, head_dim).total;
}

int spec_verify_attention(const void* q, sv_strides q_strides, sv_dtype dtype, int32_t B, int32_t N,
                          int32_t q_heads, const sv_cache* cache, const int32_t* page_table,
                          int32_t table_width, const int32_t* kv_len, const int32_t* rows,
                          float scale, int32_t window, void* out, sv_strides out_strides,
                          float* out_lse, void* workspace, size_t workspace_bytes, void* stream) {
  sv::AttendArgs a;
  if (!q || !out || !kv_len) return SV_EINVAL;
  if (!known(dtype)) return SV_EDTYPE;
  int rc = cache_of(cache, true, true, &a.c);
  if (rc == SV_OK) rc = batch_of(page_table, table_width, kv_len, rows, B, N, cache->page_size, &a.t);
  if (rc != SV_OK) return rc;
  if (N > SV_MAX_ROWS || q_heads < 1 || q_heads % a.c.heads || window < 0 || !isfinite(scale)) return SV_EINVAL;
  const size_t es = size_of(dtype);
  if (!aligned(q, es) || !aligned(out, es) || !aligned(out_lse, 4) || !readable(q_strides, B, N, q_heads) ||
      !writable(out_strides, B, N, q_heads, a.c.D) || q == out)
    return SV_EINVAL;
  const int64_t reach = (int64_t)window + N + sv::CACHE_BLOCK - 1;     // with the first block's rest
  const int64_t tokens = window && reach < a.t.capacity ? reach : a.t.capacity;
  if (!attend_shape(B, N, q_heads, a.c.heads, a.c.D, tokens, dtype, &a.s)) return SV_ESIZE;
  AttendSpace w = attend_space(a.s, B, a.c.heads, a.c.D);
  const bool room = workspace && aligned(workspace, WS_ALIGN) && workspace_bytes >= w.total;
  if (a.s.may_single && !a.s.single && !room) {     // without room to share it out
    a.s.single = 1;
    a.s.grid = a.s.units;
    w = attend_space(a.s, B, a.c.heads, a.c.D);
  }
  if (w.total && !room) return SV_EWORKSPACE;
  a.q = q;
  a.out = out;
  a.qs = strides_of(q_strides);
  a.os = strides_of(out_strides);
  a.lse = out_lse;
  a.qh = q_heads;
  a.group = q_heads / a.c.heads;
  // exact for columns below 2^32 / group: there are 64 * group of them and a set's filling
  a.group_inv = (uint32_t)((0x100000000ull + a.group - 1) / a.group);
  a.window = window;
  a.bf16 = dtype == SV_BF16;
  a.scale2 = (float)((double)scale * M_LOG2E);
  a.record = (int32_t*)((char*)workspace + w.record);
  a.partial = (float*)((char*)workspace + w.partial);
  return sv::launch_attend(a, (hipStream_t)stream) ? SV_EHIP : SV_OK;
}

int spec_verify_adjust_logits(const void* logits, sv_strides strides, sv_dtype dtype, int32_t B,
                              int32_t N, int32_t V, const int32_t* rows, const int32_t* tokens,
                              int32_t n_tokens, const int32_t* history, int32_t n_history,
                              const int32_t* prompt, int32_t n_prompt, const float* repetition,
                              const float* frequency, const float* presence,
                              const int32_t* bias_ids, const float* bias, int32_t n_bias,
                              const uint32_t* allowed, void* out, sv_strides out_strides,
                              void* stream) {
  if (!logits || !out) return SV_EINVAL;
  if (!known(dtype)) return SV_EDTYPE;
  if (B < 1 || N < 1 || V < 1 || n_tokens < 0 || n_history < 0 || n_prompt < 0 || n_bias < 0) return SV_EINVAL;
  if ((n_tokens > 0) != (tokens != nullptr) || (n_history > 0) != (history != nullptr) ||
      (n_prompt > 0) != (prompt != nullptr) || (n_bias > 0) != (bias_ids != nullptr) ||
      (n_bias > 0) != (bias != nullptr) || (tokens && n_tokens < N - 1))
    return SV_EINVAL;
  const size_t es = size_of(dtype);
  const void* words[] = {rows, tokens, history, prompt, repetition, frequency, presence, bias_ids, bias, allowed};
  for (const void* p : words)
    if (!aligned(p, 4)) return SV_EINVAL;
  strides.head = out_strides.head = 0;
  if (!aligned(logits, es) || !aligned(out, es) || !readable(strides, B, N, 1) || !writable(out_strides, B, N, 1, V) ||
      !place_ok(logits, strides, out, out_strides, B, N, 1))
    return SV_EINVAL;
  if (V >= INT32_MAX - 65536 || n_history >= 1 << 24 || n_prompt >= 1 << 24 || n_bias >= 1 << 24) return SV_ESIZE;
  const int64_t chunks = ceil_div(V, sv::ADJ_CHUNK);
  if ((double)chunks * B * N >= MAX_WORKGROUPS) return SV_ESIZE;
  // rows of a request in one workgroup, which counts the lists once, unless that leaves CUs idle
  int64_t groups = ceil_div(8 * CUS, chunks * B);
  if (groups > N) groups = N;
  const sv::AdjustArgs a{logits, out, strides_of(strides), strides_of(out_strides), B, N, V, dtype == SV_BF16,
                         rows, tokens, history, prompt, bias_ids, n_tokens, n_history, n_prompt, n_bias,
                         repetition, frequency, presence, bias, allowed, (int)chunks, (int)groups};
  return sv::launch_adjust(a, (hipStream_t)stream) ? SV_EHIP : SV_OK;
}

}  // extern "C"
