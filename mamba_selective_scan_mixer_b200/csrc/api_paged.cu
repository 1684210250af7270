// C ABI of the paged key-value cache: argument checks, workspace layout and the
// launch sequences.  See include/jamba.h for the contract of each call.
#include <climits>
#include <string>

#include "api.hpp"
#include "gemm_tc.cuh"
#include "pages.cuh"

using namespace jb;

namespace {

constexpr int DECODE_MAX_REP = 16;    // query heads per KV head of the one-token kernel
constexpr int MAX_SLOTS = 1 << 20;
constexpr int EXTEND_MAX_REP = 128;   // ... of the ragged kernel: one token's heads fill its rows of a tile

jamba_status geom(const jamba_pages_config* c, PageGeom* g) {
  if (!c) return fail(JAMBA_ERR_INVALID_ARG, "pages: null config");
  if (c->dtype != JAMBA_BF16) return fail(JAMBA_ERR_UNSUPPORTED, "pages: bf16 only");
  if (c->head_dim != PG_D) return fail(JAMBA_ERR_UNSUPPORTED, "pages: head_dim must be 128");
  if (c->num_pages <= 0 || c->n_kv_heads <= 0 || c->max_seqs <= 0 || c->max_pages <= 0)
    return fail(JAMBA_ERR_INVALID_ARG, "pages: sizes must be positive");
  if (c->ld_table < c->max_pages) return fail(JAMBA_ERR_INVALID_ARG, "pages: ld_table below max_pages");
  int shift = 0;
  while ((1 << shift) < c->page_size && shift < 9) ++shift;
  if (shift < 4 || shift > 8 || (1 << shift) != c->page_size)
    return fail(JAMBA_ERR_UNSUPPORTED, "pages: page_size must be 16, 32, 64, 128 or 256");
  if (((long long)c->max_pages << shift) > INT_MAX / 2)
    return fail(JAMBA_ERR_UNSUPPORTED, "pages: max_pages * page_size above 2^30 tokens");
  if (c->n_kv_heads > 1024) return fail(JAMBA_ERR_UNSUPPORTED, "pages: at most 1024 KV heads");
  if (((long long)c->num_pages * c->n_kv_heads << shift) > INT_MAX)
    return fail(JAMBA_ERR_UNSUPPORTED, "pages: more than 2^31 - 1 rows in a plane");
  if (c->max_seqs > MAX_SLOTS) return fail(JAMBA_ERR_UNSUPPORTED, "pages: at most 2^20 slots");
  *g = {c->num_pages, c->n_kv_heads, shift, c->planes, c->max_seqs, c->max_pages, c->ld_table};
  return JAMBA_OK;
}

// the last check before a launch: kernels report into the device's status word
jamba_status ready() {
  return device_error_word() ? JAMBA_OK : fail(JAMBA_ERR_CUDA, "could not allocate the device status word");
}

jamba_status check_int(const void* p, const char* name) {
  if (!p) return fail(JAMBA_ERR_INVALID_ARG, std::string(name) + " is null");
  if (reinterpret_cast<uintptr_t>(p) & 3u) return fail(JAMBA_ERR_INVALID_ARG, std::string(name) + " is misaligned");
  return JAMBA_OK;
}

// what fork, grow and compact check alike
jamba_status check_upkeep(const PageGeom& g, const void* refs, const void* table, const void* lengths, const void* ws,
                          size_t ws_bytes, const char* who) {
  JB_TRY(check_ptr(refs, "refs"));
  JB_TRY(check_int(table, "table"));
  JB_TRY(check_int(lengths, "lengths"));
  JB_TRY(check_ptr(ws, "workspace"));
  if (ws_bytes < pages_workspace_bytes(g)) return fail(JAMBA_ERR_WORKSPACE, std::string(who) + ": workspace too small");
  return JAMBA_OK;
}

jamba_status check_planes(const jamba_pages_config* c) {
  if (c->planes <= 0 || c->planes > 65535) return fail(JAMBA_ERR_INVALID_ARG, "pages: planes must be 1 .. 65535");
  return JAMBA_OK;
}

jamba_status check_heads(const PageGeom& g, int n_heads, int tokens, int max_rep) {
  if (n_heads <= 0 || n_heads % g.G)
    return fail(JAMBA_ERR_INVALID_ARG, "paged attention: n_kv_heads must divide n_heads");
  if (n_heads / g.G > max_rep)
    return fail(JAMBA_ERR_UNSUPPORTED,
                "paged attention: at most " + std::to_string(max_rep) + " query heads per KV head");
  if ((long long)tokens * n_heads > INT_MAX)
    return fail(JAMBA_ERR_UNSUPPORTED, "paged attention: tokens * heads above 2^31 - 1");
  return JAMBA_OK;
}

// whether one of `tokens` rows of `row` bytes at a, ld_a bytes apart, shares a byte with one of those at b (slices of
// one buffer may lie between one another)
bool rows_overlap(const void* a, long long ld_a, const void* b, long long ld_b, long long row, long long tokens) {
  const long long d = (long long)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a)), n = tokens - 1;
  if (tokens <= 0 || d >= n * ld_a + row || -d >= n * ld_b + row) return false;
  // row j of b against the rows of a that begin before and after it; with one stride, row 0 of b against those of a
  // on either side of it, were a to go on without end: any pair (i, j) with that difference i - j will do
  const bool same = ld_a == ld_b;
  for (long long j = 0; j <= (same ? 0 : n); ++j) {
    const long long at = d + j * ld_b;
    const long long i = at >= 0 ? at / ld_a : -((-at + ld_a - 1) / ld_a);
    for (int k = 0; k < 2; ++k) {
      const long long gap = at - (i + k) * ld_a;
      if ((same ? i + k >= -n : i + k >= 0) && i + k <= n && gap < row && -gap < row) return true;
    }
  }
  return false;
}

jamba_status check_attn_args(int n_heads, int tokens, const void* q, int ld_q, const void* k_pages,
                             const void* v_pages, const void* table, const void* lengths, const void* o, int ld_o,
                             const void* lse, const void* ws) {
  JB_TRY(check_ptr(q, "q"));
  JB_TRY(check_ptr(k_pages, "k_pages"));
  JB_TRY(check_ptr(v_pages, "v_pages"));
  JB_TRY(check_ptr(o, "o"));
  JB_TRY(check_ptr(ws, "workspace"));
  JB_TRY(check_int(table, "table"));
  JB_TRY(check_int(lengths, "lengths"));
  if (lse) JB_TRY(check_int(lse, "lse"));
  const long long row = (long long)n_heads * PG_D;
  if (ld_q < row || ld_o < row || ld_q % 8 || ld_o % 8)
    return fail(JAMBA_ERR_INVALID_ARG, "paged attention: token strides must be multiples of 8 and hold all heads");
  if (q == o || rows_overlap(q, 2ll * ld_q, o, 2ll * ld_o, 2 * row, tokens))
    return fail(JAMBA_ERR_INVALID_ARG, "paged attention: o may not overlap q");
  return JAMBA_OK;
}

struct PagedLayerWs {
  void *qkv, *attn, *o; float* opart;
  int o_splits;
  size_t total;
};
PagedLayerWs carve_layer(const jamba_attn_config& c, const PageGeom& g, int tokens, bool ragged, void* ws) {
  PagedLayerWs a;
  const int W = (c.n_heads + 2 * c.n_kv_heads) * c.head_dim, HD = c.n_heads * c.head_dim;
  a.o_splits = ragged ? 1 : choose_splits(c.d_model, tokens, HD, 64, 8);
  Carver cv(ws);
  a.qkv = cv.take((size_t)tokens * W * 2);
  a.o = cv.take((size_t)tokens * HD * 2);
  a.attn = cv.take(ragged ? paged_extend_workspace_bytes() : paged_decode_workspace_bytes(g, c.n_heads));
  a.opart = ragged ? nullptr : cv.take<float>((size_t)a.o_splits * tokens * c.d_model * 4);
  a.total = cv.off;
  return a;
}

jamba_status layer_geom(const jamba_attn_config* cfg, const jamba_pages_config* pages, int tokens, int max_rep,
                        PageGeom* g) {
  JB_TRY(check_attn_cfg(cfg));
  JB_TRY(geom(pages, g));
  if (pages->n_kv_heads != cfg->n_kv_heads)
    return fail(JAMBA_ERR_INVALID_ARG, "paged attention layer: the pages hold another number of KV heads");
  return check_heads(*g, cfg->n_heads, tokens, max_rep);
}

jamba_status check_layer_args(const jamba_attn_weights* w, const void* x, const void* residual, const void* out,
                              const void* k_pages, const void* v_pages, const void* table, const void* lengths,
                              const void* ws) {
  if (!w) return fail(JAMBA_ERR_INVALID_ARG, "paged attention layer: null weights");
  JB_TRY(check_ptr(w->w_qkv, "w_qkv"));
  JB_TRY(check_ptr(w->w_o, "w_o"));
  JB_TRY(check_ptr(x, "x"));
  JB_TRY(check_ptr(out, "out"));
  JB_TRY(check_ptr(residual, "residual", false));
  JB_TRY(check_ptr(k_pages, "k_pages"));
  JB_TRY(check_ptr(v_pages, "v_pages"));
  JB_TRY(check_ptr(ws, "workspace"));
  JB_TRY(check_int(table, "table"));
  JB_TRY(check_int(lengths, "lengths"));
  if (x == out) return fail(JAMBA_ERR_INVALID_ARG, "paged attention layer: out may not alias x");
  return JAMBA_OK;
}

}  // namespace

extern "C" {

jamba_status jamba_pages_workspace_size(const jamba_pages_config* cfg, size_t* bytes) {
  PageGeom g;
  JB_TRY(geom(cfg, &g));
  if (!bytes) return fail(JAMBA_ERR_INVALID_ARG, "pages workspace: bytes is null");
  *bytes = pages_workspace_bytes(g);
  return JAMBA_OK;
}

jamba_status jamba_pages_fork(const jamba_pages_config* cfg, const int32_t* parent, int32_t* refs, int32_t* table,
                              int32_t* lengths, void* ws, size_t ws_bytes, jamba_stream_t stream) {
  JB_RANGE("jamba_pages_fork");
  PageGeom g;
  JB_TRY(geom(cfg, &g));
  JB_TRY(check_int(parent, "parent"));
  JB_TRY(check_upkeep(g, refs, table, lengths, ws, ws_bytes, "pages fork"));
  JB_TRY(ready());
  return pages_fork(g, parent, refs, table, lengths, ws, cs(stream));
}

jamba_status jamba_pages_grow(const jamba_pages_config* cfg, const int32_t* add, void* data, int32_t* refs,
                              int32_t* table, int32_t* lengths, int32_t* granted, void* ws, size_t ws_bytes,
                              jamba_stream_t stream) {
  JB_RANGE("jamba_pages_grow");
  PageGeom g;
  JB_TRY(geom(cfg, &g));
  JB_TRY(check_planes(cfg));
  JB_TRY(check_int(add, "add"));
  JB_TRY(check_int(granted, "granted"));
  JB_TRY(check_ptr(data, "data"));
  JB_TRY(check_upkeep(g, refs, table, lengths, ws, ws_bytes, "pages grow"));
  JB_TRY(ready());
  return pages_grow(g, add, data, refs, table, lengths, granted, ws, cs(stream));
}

jamba_status jamba_pages_active(int max_seqs, const int32_t* active, const int32_t* lengths, int32_t* out,
                                jamba_stream_t stream) {
  JB_RANGE("jamba_pages_active");
  if (max_seqs <= 0 || max_seqs > MAX_SLOTS)
    return fail(JAMBA_ERR_INVALID_ARG, "pages active: max_seqs must be 1 .. 2^20");
  JB_TRY(check_int(active, "active"));
  JB_TRY(check_int(lengths, "lengths"));
  JB_TRY(check_int(out, "out"));
  return pages_active(max_seqs, active, lengths, out, cs(stream));
}

jamba_status jamba_pages_compact(const jamba_pages_config* cfg, void* data, int32_t* refs, int32_t* table,
                                 const int32_t* lengths, int32_t* remap, void* ws, size_t ws_bytes,
                                 jamba_stream_t stream) {
  JB_RANGE("jamba_pages_compact");
  PageGeom g;
  JB_TRY(geom(cfg, &g));
  JB_TRY(check_planes(cfg));
  JB_TRY(check_int(remap, "remap"));
  JB_TRY(check_ptr(data, "data"));
  JB_TRY(check_upkeep(g, refs, table, lengths, ws, ws_bytes, "pages compact"));
  JB_TRY(ready());
  return pages_compact(g, data, refs, table, lengths, remap, ws, cs(stream));
}

jamba_status jamba_paged_append(const jamba_pages_config* cfg, const void* k, const void* v, int ld_kv, int tokens,
                                const int32_t* q_start, void* k_pages, void* v_pages, const int32_t* table,
                                const int32_t* lengths, jamba_stream_t stream) {
  JB_RANGE("jamba_paged_append");
  PageGeom g;
  JB_TRY(geom(cfg, &g));
  if (tokens < 0 || (!q_start && tokens != g.S))
    return fail(JAMBA_ERR_INVALID_ARG, "paged append: tokens must be max_seqs without q_start, and not negative");
  if (q_start) JB_TRY(check_int(q_start, "q_start"));
  JB_TRY(check_ptr(k, "k"));
  JB_TRY(check_ptr(v, "v"));
  JB_TRY(check_ptr(k_pages, "k_pages"));
  JB_TRY(check_ptr(v_pages, "v_pages"));
  JB_TRY(check_int(table, "table"));
  JB_TRY(check_int(lengths, "lengths"));
  if (ld_kv < g.G * PG_D || ld_kv % 8)
    return fail(JAMBA_ERR_INVALID_ARG, "paged append: ld_kv must be a multiple of 8 and hold all heads");
  if (tokens == 0) return JAMBA_OK;
  JB_TRY(ready());
  return paged_append(g, k, v, ld_kv, tokens, q_start, k_pages, v_pages, table, lengths, cs(stream));
}

jamba_status jamba_paged_decode_workspace_size(const jamba_pages_config* cfg, int n_heads, size_t* bytes) {
  PageGeom g;
  JB_TRY(geom(cfg, &g));
  JB_TRY(check_heads(g, n_heads, g.S, DECODE_MAX_REP));
  if (!bytes) return fail(JAMBA_ERR_INVALID_ARG, "paged decode workspace: bytes is null");
  *bytes = paged_decode_workspace_bytes(g, n_heads);
  return JAMBA_OK;
}

jamba_status jamba_paged_extend_workspace_size(const jamba_pages_config* cfg, int n_heads, int tokens, size_t* bytes) {
  PageGeom g;
  JB_TRY(geom(cfg, &g));
  if (tokens < 0) return fail(JAMBA_ERR_INVALID_ARG, "paged extend workspace: negative tokens");
  JB_TRY(check_heads(g, n_heads, tokens, EXTEND_MAX_REP));
  if (!bytes) return fail(JAMBA_ERR_INVALID_ARG, "paged extend workspace: bytes is null");
  *bytes = paged_extend_workspace_bytes();
  return JAMBA_OK;
}

jamba_status jamba_paged_decode(const jamba_pages_config* cfg, int n_heads, const void* q, int ld_q,
                                const void* k_pages, const void* v_pages, const int32_t* table,
                                const int32_t* lengths, void* o, int ld_o, float* lse, void* ws, size_t ws_bytes,
                                jamba_stream_t stream) {
  JB_RANGE("jamba_paged_decode");
  PageGeom g;
  JB_TRY(geom(cfg, &g));
  JB_TRY(check_heads(g, n_heads, g.S, DECODE_MAX_REP));
  JB_TRY(check_attn_args(n_heads, g.S, q, ld_q, k_pages, v_pages, table, lengths, o, ld_o, lse, ws));
  if (ws_bytes < paged_decode_workspace_bytes(g, n_heads))
    return fail(JAMBA_ERR_WORKSPACE, "paged decode: workspace too small");
  JB_TRY(ready());
  return paged_decode(g, n_heads, q, ld_q, k_pages, v_pages, table, lengths, o, ld_o, lse, ws, cs(stream));
}

jamba_status jamba_paged_extend(const jamba_pages_config* cfg, int n_heads, const void* q, int ld_q, int tokens,
                                const int32_t* q_start, const void* k_pages, const void* v_pages,
                                const int32_t* table, const int32_t* lengths, void* o, int ld_o, float* lse,
                                void* ws, size_t ws_bytes, jamba_stream_t stream) {
  JB_RANGE("jamba_paged_extend");
  PageGeom g;
  JB_TRY(geom(cfg, &g));
  if (tokens < 0) return fail(JAMBA_ERR_INVALID_ARG, "paged extend: negative tokens");
  JB_TRY(check_heads(g, n_heads, tokens, EXTEND_MAX_REP));
  JB_TRY(check_int(q_start, "q_start"));
  JB_TRY(check_attn_args(n_heads, tokens, q, ld_q, k_pages, v_pages, table, lengths, o, ld_o, lse, ws));
  if (ws_bytes < paged_extend_workspace_bytes())
    return fail(JAMBA_ERR_WORKSPACE, "paged extend: workspace too small");
  if (tokens == 0) return JAMBA_OK;
  JB_TRY(ready());
  return paged_extend(g, n_heads, q, ld_q, tokens, q_start, k_pages, v_pages, table, lengths, o, ld_o, lse, false, ws,
                      cs(stream));
}

jamba_status jamba_attn_paged_prefill_workspace_size(const jamba_attn_config* cfg, const jamba_pages_config* pages,
                                                     int tokens, size_t* bytes) {
  PageGeom g;
  JB_TRY(layer_geom(cfg, pages, tokens, EXTEND_MAX_REP, &g));
  if (!bytes || tokens <= 0) return fail(JAMBA_ERR_INVALID_ARG, "paged attention workspace: bad argument");
  *bytes = carve_layer(*cfg, g, tokens, true, nullptr).total;
  return JAMBA_OK;
}

jamba_status jamba_attn_paged_prefill(const jamba_attn_config* cfg, const jamba_attn_weights* w,
                                      const jamba_pages_config* pages, const void* x, const void* residual, void* out,
                                      int tokens, const int32_t* q_start, void* k_pages, void* v_pages,
                                      const int32_t* table, const int32_t* lengths, void* ws, size_t ws_bytes,
                                      jamba_stream_t stream) {
  JB_RANGE("jamba_attn_paged_prefill");
  PageGeom g;
  JB_TRY(layer_geom(cfg, pages, tokens, EXTEND_MAX_REP, &g));
  if (tokens <= 0) return fail(JAMBA_ERR_INVALID_ARG, "paged attention prefill: tokens must be positive");
  JB_TRY(check_int(q_start, "q_start"));
  JB_TRY(check_layer_args(w, x, residual, out, k_pages, v_pages, table, lengths, ws));
  const jamba_attn_config& c = *cfg;
  PagedLayerWs a = carve_layer(c, g, tokens, true, ws);
  if (ws_bytes < a.total) return fail(JAMBA_ERR_WORKSPACE, "paged attention prefill: workspace too small");
  JB_TRY(ready());
  cudaStream_t s = cs(stream);
  const int dm = c.d_model, HD = c.n_heads * PG_D, KD = c.n_kv_heads * PG_D, W = HD + 2 * KD;
  bf16* qkv = reinterpret_cast<bf16*>(a.qkv);
  JB_TRY(gemm_bf16(gdesc(x, dm, w->w_qkv, dm, tokens, W, dm, EPI_BF16, qkv, W), s));
  JB_TRY(paged_append(g, qkv + HD, qkv + HD + KD, W, tokens, q_start, k_pages, v_pages, table, lengths, s));
  JB_TRY(paged_extend(g, c.n_heads, qkv, W, tokens, q_start, k_pages, v_pages, table, lengths, a.o, HD, nullptr, true,
                      a.attn, s));
  GemmDesc go = gdesc(a.o, HD, w->w_o, HD, tokens, dm, HD, EPI_BF16, out, dm);
  go.residual = residual;
  go.ldr = dm;
  JB_TRY(gemm_bf16(go, s));
  return JAMBA_OK;
}

jamba_status jamba_attn_paged_step_workspace_size(const jamba_attn_config* cfg, const jamba_pages_config* pages,
                                                  size_t* bytes) {
  PageGeom g;
  JB_TRY(layer_geom(cfg, pages, pages ? pages->max_seqs : 1, DECODE_MAX_REP, &g));
  if (!bytes) return fail(JAMBA_ERR_INVALID_ARG, "paged attention workspace: bytes is null");
  *bytes = carve_layer(*cfg, g, g.S, false, nullptr).total;
  return JAMBA_OK;
}

jamba_status jamba_attn_paged_step(const jamba_attn_config* cfg, const jamba_attn_weights* w,
                                   const jamba_pages_config* pages, const void* x, const void* residual, void* out,
                                   void* k_pages, void* v_pages, const int32_t* table, const int32_t* lengths,
                                   void* ws, size_t ws_bytes, jamba_stream_t stream) {
  JB_RANGE("jamba_attn_paged_step");
  PageGeom g;
  JB_TRY(layer_geom(cfg, pages, pages ? pages->max_seqs : 1, DECODE_MAX_REP, &g));
  JB_TRY(check_layer_args(w, x, residual, out, k_pages, v_pages, table, lengths, ws));
  const jamba_attn_config& c = *cfg;
  const int B = g.S;
  PagedLayerWs a = carve_layer(c, g, B, false, ws);
  if (ws_bytes < a.total) return fail(JAMBA_ERR_WORKSPACE, "paged attention step: workspace too small");
  JB_TRY(ready());
  cudaStream_t s = cs(stream);
  const int dm = c.d_model, HD = c.n_heads * PG_D, KD = c.n_kv_heads * PG_D, W = HD + 2 * KD;
  bf16* qkv = reinterpret_cast<bf16*>(a.qkv);
  // weights stream through the tensor cores as the 128-row side; the token batch is the N side
  GemmDesc g1 = gdesc(w->w_qkv, dm, x, dm, W, B, dm, EPI_BF16, qkv, W);
  g1.transpose_out = 1;
  g1.bn = 64;
  JB_TRY(gemm_bf16(g1, s));
  JB_TRY(paged_append(g, qkv + HD, qkv + HD + KD, W, B, nullptr, k_pages, v_pages, table, lengths, s));
  JB_TRY(paged_decode(g, c.n_heads, qkv, W, k_pages, v_pages, table, lengths, a.o, HD, nullptr, a.attn, s));
  GemmDesc g2 = gdesc(w->w_o, HD, a.o, HD, dm, B, HD, EPI_F32, a.opart, dm);
  g2.transpose_out = 1;
  g2.bn = 64;
  g2.splits = a.o_splits;
  g2.split_stride = (long long)B * dm;
  JB_TRY(gemm_bf16(g2, s));
  JB_TRY(splitk_reduce(a.opart, a.o_splits, (long long)B * dm, (long long)B * dm, residual, out, JAMBA_BF16, s));
  return JAMBA_OK;
}

}  // extern "C"
