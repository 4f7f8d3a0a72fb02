// capi.cu -- the extern "C" entry points of libspecverify: host-side argument
// checks (nothing is launched when they fail), workspace layout, dispatch.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "common.cuh"
#include "internal.h"
#include "spec_cache.h"

using namespace specv;

namespace {

thread_local char g_cuda_error[256] = "no error";

int cuda_fail(cudaError_t e)
{
    std::snprintf(g_cuda_error, sizeof g_cuda_error, "%s: %s", cudaGetErrorName(e),
                  cudaGetErrorString(e));
    return SPEC_ERR_CUDA;
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

size_t elt_bytes(int dtype) { return dtype == SPEC_BF16 ? 2 : 4; }

struct WsLayout {
    int32_t *tok, *flag;
    uint32_t *ticket;
    void *info, *part, *cand;
};

// tok [R_cap] | flag [R_cap] | ticket [B] | info [R_cap * 64 B] |
// part [R_cap * nchunk * 32 B] | cand (sampler only); 256-byte aligned
size_t ws_bytes(int32_t R_cap, int32_t B, int32_t V, int elt, bool sampling)
{
    const size_t R = static_cast<size_t>(R_cap);
    const size_t rc = R * static_cast<size_t>(chunks_per_row(V, elt));
    size_t n = 2 * align256(R * 4) + align256(static_cast<size_t>(B) * 4) + align256(R * 64) +
               align256(rc * 32);
    if (sampling) n += align256(rc * kWsCandCap * 8);
    return n;
}

WsLayout ws_layout(void *ws, int32_t R_cap, int32_t B, int32_t V, int elt, bool sampling)
{
    uint8_t *p = static_cast<uint8_t *>(ws);
    const size_t R = static_cast<size_t>(R_cap);
    const size_t rc = R * static_cast<size_t>(chunks_per_row(V, elt));
    WsLayout l = {};
    l.tok = reinterpret_cast<int32_t *>(p);
    p += align256(R * 4);
    l.flag = reinterpret_cast<int32_t *>(p);
    p += align256(R * 4);
    l.ticket = reinterpret_cast<uint32_t *>(p);
    p += align256(static_cast<size_t>(B) * 4);
    l.info = p;
    p += align256(R * 64);
    l.part = p;
    p += align256(rc * 32);
    if (sampling) l.cand = p;
    return l;
}

// checks shared by the three verify entry points
int check_batch(const spec_batch *b, const spec_outputs *o)
{
    if (!b || !o) return SPEC_ERR_INVALID_ARG;
    if (!b->logits || !b->cu_rows || !b->draft_ids) return SPEC_ERR_INVALID_ARG;
    if (!o->accepted_len || !o->out_tokens || !o->next_token) return SPEC_ERR_INVALID_ARG;
    if (b->dtype != SPEC_F32 && b->dtype != SPEC_BF16) return SPEC_ERR_UNSUPPORTED;
    if (b->V < 1 || b->ld < b->V || b->B < 1 || b->R_cap < 1) return SPEC_ERR_INVALID_ARG;
    if (b->k_max < 0) return SPEC_ERR_INVALID_ARG;
    if (b->k_max > 31) return SPEC_ERR_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(b->logits) % elt_bytes(b->dtype)) return SPEC_ERR_INVALID_ARG;
    if (static_cast<size_t>(b->V) * elt_bytes(b->dtype) > max_row_bytes()) return SPEC_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(b->R_cap) * b->ld > (int64_t(1) << 40)) return SPEC_ERR_UNSUPPORTED;
    // one CTA per (row, chunk): the grid stays below 2^31
    if (static_cast<int64_t>(b->R_cap) * chunks_per_row(b->V, static_cast<int>(elt_bytes(b->dtype))) >
        INT32_MAX)
        return SPEC_ERR_UNSUPPORTED;
    if ((o->acc == nullptr) != (o->ver == nullptr)) return SPEC_ERR_INVALID_ARG;
    return SPEC_OK;
}

VerifyParams base_params(const spec_batch *b, const spec_outputs *o, void *ws, bool sampling)
{
    VerifyParams p;
    std::memset(&p, 0, sizeof p);
    p.logits = b->logits;
    p.ld = b->ld;
    p.V = b->V;
    p.B = b->B;
    p.k_max = b->k_max;
    p.R_cap = b->R_cap;
    p.cu_rows = b->cu_rows;
    p.draft_ids = b->draft_ids;
    p.accepted_len = o->accepted_len;
    p.out_tokens = o->out_tokens;
    p.next_token = o->next_token;
    p.row_max = o->row_max;
    p.row_lse = o->row_lse;
    p.row_argmax = o->row_argmax;
    p.row_token = o->row_token;
    p.status = o->status;
    p.acc = o->acc;
    p.ver = o->ver;
    p.hist = o->hist;
    const int elt = static_cast<int>(elt_bytes(b->dtype));
    const WsLayout l = ws_layout(ws, b->R_cap, b->B, b->V, elt, sampling);
    p.ws_tok = l.tok;
    p.ws_flag = l.flag;
    p.ws_ticket = l.ticket;
    p.ws_info = l.info;
    p.ws_part = l.part;
    p.ws_cand = l.cand;
    p.nchunk = chunks_per_row(b->V, elt);
    p.n_rows = b->R_cap;
    return p;
}

int run_verify(int mode, const spec_batch *b, VerifyParams &p, cudaStream_t s)
{
    const cudaError_t e = launch_verify(mode, b->dtype, p, s);
    return e == cudaSuccess ? SPEC_OK : cuda_fail(e);
}

// Built-in scratch of spec_verify_greedy_noalloc: a device array of the
// library (zero at load).
static __device__ __align__(256) uint8_t g_noalloc_scratch[SPEC_NOALLOC_SCRATCH_BYTES];

// Device address of the scratch array in the current context (the host-side
// name of the array is not a device address; only this lookup gives one).
// Looked up on every call, never cached: after a device reset, or under a
// context other than the device's primary one, the module is loaded again
// and the array can move.
int noalloc_scratch(void **ptr)
{
    void *p = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&p, g_noalloc_scratch);
    if (e != cudaSuccess) return cuda_fail(e);
    *ptr = p;
    return SPEC_OK;
}

// ---- the 4-bit paged cache ----

// slots are 32-bit; kv heads and requests are the y and z of the grids
constexpr int32_t kMostSlots = 1 << 30, kMostHeads = 65535, kMostRequests = 65535;

// whether device arrays of 32-bit values lie on their words (null: absent)
template <typename... T> bool on_words(const T *...p)
{
    return ((reinterpret_cast<uintptr_t>(p) % 4 == 0) && ...);
}

int check_cache(const spec_cache *c, CacheView &v)
{
    if (!c || !c->pages || !c->page_table) return SPEC_ERR_INVALID_ARG;
    if (c->n_pages < 1 || c->n_pages > INT32_MAX || c->H < 1 || c->B < 1 || c->max_pages < 1)
        return SPEC_ERR_INVALID_ARG;
    if (c->page_tokens < SPEC_CACHE_BLOCK_TOKENS || c->page_tokens % SPEC_CACHE_BLOCK_TOKENS)
        return SPEC_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(c->pages) % 16 || !on_words(c->k_scale, c->v_scale, c->page_table))
        return SPEC_ERR_INVALID_ARG;
    if (c->D != 64 && c->D != 128 && c->D != 256) return SPEC_ERR_UNSUPPORTED;
    if (c->page_tokens > 65536 || c->H > kMostHeads || c->B > kMostRequests) return SPEC_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(c->max_pages) * c->page_tokens > kMostSlots) return SPEC_ERR_UNSUPPORTED;
    v.pages = static_cast<uint8_t *>(c->pages);
    v.n_pages = c->n_pages;
    v.page_tokens = c->page_tokens;
    v.H = c->H;
    v.D = c->D;
    v.k_scale = c->k_scale;
    v.v_scale = c->v_scale;
    v.B = c->B;
    v.max_pages = c->max_pages;
    v.page_table = c->page_table;
    return SPEC_OK;
}

// whether every (row, head) of a tensor starts on a 16-byte boundary
bool rows_aligned(const void *p, int64_t row, int64_t head, size_t elt)
{
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (row * static_cast<int64_t>(elt)) % 16 == 0 &&
           (head * static_cast<int64_t>(elt)) % 16 == 0;
}

int run_cache_rows(const spec_cache *cache, const spec_cache_rows *r, bool append, spec_stream stream)
{
    CacheView c;
    const int rc = check_cache(cache, c);
    if (rc != SPEC_OK) return rc;
    if (!r || !r->k || !r->v || !r->cu_rows || !r->start) return SPEC_ERR_INVALID_ARG;
    if (r->dtype != SPEC_F32 && r->dtype != SPEC_BF16) return SPEC_ERR_UNSUPPORTED;
    if (r->R_cap < 1 || r->max_rows < 1) return SPEC_ERR_INVALID_ARG;
    if (r->max_rows > (1 << 30)) return SPEC_ERR_UNSUPPORTED;
    const size_t elt = elt_bytes(r->dtype);
    if (reinterpret_cast<uintptr_t>(r->k) % elt || reinterpret_cast<uintptr_t>(r->v) % elt ||
        !on_words(r->cu_rows, r->start, r->score, r->slot_pos, r->pos0, r->status))
        return SPEC_ERR_INVALID_ARG;
    CacheRows p;
    p.k = r->k;
    p.v = r->v;
    p.k_row = r->k_row;
    p.k_head = r->k_head;
    p.v_row = r->v_row;
    p.v_head = r->v_head;
    p.R_cap = r->R_cap;
    p.max_rows = r->max_rows;
    p.cu_rows = r->cu_rows;
    p.start = r->start;
    p.score = append ? r->score : nullptr;
    p.slot_pos = append ? r->slot_pos : nullptr;
    p.pos0 = r->pos0;
    p.status = r->status;
    p.k_aligned = rows_aligned(r->k, r->k_row, r->k_head, elt);
    p.v_aligned = rows_aligned(r->v, r->v_row, r->v_head, elt);
    const cudaError_t e = launch_cache_rows(c, p, r->dtype, append, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPEC_OK : cuda_fail(e);
}

int check_attention(const spec_cache *cache, const spec_attention *a, CacheView &c, AttnParams &p)
{
    const int rc = check_cache(cache, c);
    if (rc != SPEC_OK) return rc;
    if (!a || !a->q || !a->cu_rows || !a->len) return SPEC_ERR_INVALID_ARG;
    if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_ERR_UNSUPPORTED;
    if (a->Hq < 1 || a->Hq % c.H || a->R_cap < 1 || a->k_max < 0 || a->window < 0 || a->prefix < 0)
        return SPEC_ERR_INVALID_ARG;
    if (a->k_max > 31 || a->Hq > kMostHeads) return SPEC_ERR_UNSUPPORTED;
    if (!(a->scale - a->scale == 0.f) || !(a->cap >= 0.f) || !(a->cap - a->cap == 0.f))
        return SPEC_ERR_INVALID_ARG;
    const int64_t room = static_cast<int64_t>(c.max_pages) * c.page_tokens;
    if (a->max_len < 0 || a->max_len > room) return SPEC_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(a->q) % elt_bytes(a->dtype) ||
        !on_words(a->cu_rows, a->len, a->slopes, a->slot_pos, a->status))
        return SPEC_ERR_INVALID_ARG;
    // the work's units and their multiples stay far below 2^63
    const double units = static_cast<double>(c.B) * a->Hq * (a->k_max + 1) * (room / 128 + 16);
    if (units > 1e15) return SPEC_ERR_UNSUPPORTED;
    std::memset(&p, 0, sizeof p);
    p.q = a->q;
    p.q_row = a->q_row;
    p.q_head = a->q_head;
    p.Hq = a->Hq;
    p.R_cap = a->R_cap;
    p.k_max = a->k_max;
    p.cu_rows = a->cu_rows;
    p.len = a->len;
    p.max_len = a->max_len ? a->max_len : static_cast<int32_t>(room);
    p.scale = a->scale;
    p.scale_log2 = static_cast<float>(std::fabs(static_cast<double>(a->scale)) * 1.4426950408889634);
    p.cap = a->cap;
    p.slopes = a->slopes;
    p.window = a->window;
    // no slot lies beyond room: a prefix of any size stays clear of 2^31 in the kernels' sums
    p.prefix = static_cast<int32_t>(a->prefix < room ? a->prefix : room);
    p.slot_pos = a->slot_pos;
    p.status = a->status;
    p.q_aligned = rows_aligned(a->q, a->q_row, a->q_head, elt_bytes(a->dtype));
    return SPEC_OK;
}

}  // namespace

extern "C" {

size_t spec_workspace_bytes(int32_t R_cap, int32_t B, int32_t V, int32_t dtype, int32_t sampling)
{
    if (R_cap < 1 || B < 1 || V < 1 || (dtype != SPEC_F32 && dtype != SPEC_BF16)) return 0;
    if (static_cast<size_t>(V) * elt_bytes(dtype) > max_row_bytes()) return 0;
    return ws_bytes(R_cap, B, V, static_cast<int>(elt_bytes(dtype)), sampling != 0);
}

size_t spec_draft_workspace_bytes(int32_t B, int32_t k, int32_t V, int32_t dtype)
{
    if (B < 1 || k < 1 || V < 1 || (dtype != SPEC_F32 && dtype != SPEC_BF16)) return 0;
    if (static_cast<size_t>(V) * elt_bytes(dtype) > max_row_bytes()) return 0;
    const int64_t Q = static_cast<int64_t>(B) * k;
    if (Q > INT32_MAX) return 0;
    return ws_bytes(static_cast<int32_t>(Q), 1, V, static_cast<int>(elt_bytes(dtype)), false);
}

int spec_verify_greedy(const spec_batch *batch, const spec_outputs *out, void *workspace,
                       size_t workspace_bytes, spec_stream stream)
{
    int rc = check_batch(batch, out);
    if (rc != SPEC_OK) return rc;
    if (!workspace || workspace_bytes < ws_bytes(batch->R_cap, batch->B, batch->V,
                                                     static_cast<int>(elt_bytes(batch->dtype)), false))
        return SPEC_ERR_WORKSPACE;
    VerifyParams p = base_params(batch, out, workspace, false);
    return run_verify(MODE_GREEDY, batch, p, reinterpret_cast<cudaStream_t>(stream));
}

int spec_verify_greedy_noalloc(const spec_batch *batch, const spec_outputs *out, spec_stream stream)
{
    int rc = check_batch(batch, out);
    if (rc != SPEC_OK) return rc;
    const int elt = static_cast<int>(elt_bytes(batch->dtype));
    if (ws_bytes(batch->R_cap, batch->B, batch->V, elt, false) > SPEC_NOALLOC_SCRATCH_BYTES)
        return SPEC_ERR_WORKSPACE;
    void *ws = nullptr;
    rc = noalloc_scratch(&ws);
    if (rc != SPEC_OK) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // the per-request and per-row tickets must start at zero (they are
    // adjacent in the layout); the rest is written before it is read
    const WsLayout l = ws_layout(ws, batch->R_cap, batch->B, batch->V, elt, false);
    const size_t tick = align256(static_cast<size_t>(batch->B) * 4) +
                        align256(static_cast<size_t>(batch->R_cap) * 4);
    cudaError_t e = cudaMemsetAsync(l.ticket, 0, tick, s);
    if (e != cudaSuccess) return cuda_fail(e);
    VerifyParams p = base_params(batch, out, ws, false);
    return run_verify(MODE_GREEDY, batch, p, s);
}

int spec_verify_relaxed_topk(const spec_batch *batch, const int32_t *relaxed_k,
                             const spec_outputs *out, void *workspace, size_t workspace_bytes,
                             spec_stream stream)
{
    int rc = check_batch(batch, out);
    if (rc != SPEC_OK) return rc;
    if (!relaxed_k) return SPEC_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < ws_bytes(batch->R_cap, batch->B, batch->V,
                                                     static_cast<int>(elt_bytes(batch->dtype)), false))
        return SPEC_ERR_WORKSPACE;
    VerifyParams p = base_params(batch, out, workspace, false);
    p.relaxed_k = relaxed_k;
    return run_verify(MODE_RELAXED, batch, p, reinterpret_cast<cudaStream_t>(stream));
}

int spec_verify_greedy_active(const spec_batch *batch, const int32_t *vocab_ids,
                              const spec_outputs *out, void *workspace, size_t workspace_bytes,
                              spec_stream stream)
{
    int rc = check_batch(batch, out);
    if (rc != SPEC_OK) return rc;
    if (!vocab_ids) return SPEC_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < ws_bytes(batch->R_cap, batch->B, batch->V,
                                                     static_cast<int>(elt_bytes(batch->dtype)), false))
        return SPEC_ERR_WORKSPACE;
    VerifyParams p = base_params(batch, out, workspace, false);
    p.vocab_ids = vocab_ids;
    return run_verify(MODE_GREEDY, batch, p, reinterpret_cast<cudaStream_t>(stream));
}

int spec_verify_greedy_margin(const spec_batch *batch, const spec_margin *margin,
                              const spec_outputs *out, void *workspace, size_t workspace_bytes,
                              spec_stream stream)
{
    int rc = check_batch(batch, out);
    if (rc != SPEC_OK) return rc;
    if (!margin || !margin->margin || margin->n_protected < 0 ||
        (margin->n_protected > 0 && !margin->protected_ids))
        return SPEC_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < ws_bytes(batch->R_cap, batch->B, batch->V,
                                                     static_cast<int>(elt_bytes(batch->dtype)), false))
        return SPEC_ERR_WORKSPACE;
    VerifyParams p = base_params(batch, out, workspace, false);
    p.margin = margin->margin;
    p.generated = margin->generated;
    p.protected_ids = margin->protected_ids;
    p.n_protected = margin->n_protected;
    p.from_position = margin->from_position;
    p.after_tokens = margin->after_tokens;
    return run_verify(MODE_GREEDY, batch, p, reinterpret_cast<cudaStream_t>(stream));
}

int spec_verify_sample(const spec_batch *batch, const spec_sampling *params,
                       const spec_outputs *out, void *workspace, size_t workspace_bytes,
                       spec_stream stream)
{
    int rc = check_batch(batch, out);
    if (rc != SPEC_OK) return rc;
    if (!params || !params->temperature || !params->top_k || !params->top_p || !params->min_p ||
        !params->seed)
        return SPEC_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < ws_bytes(batch->R_cap, batch->B, batch->V,
                                                     static_cast<int>(elt_bytes(batch->dtype)), true))
        return SPEC_ERR_WORKSPACE;
    VerifyParams p = base_params(batch, out, workspace, true);
    p.temperature = params->temperature;
    p.top_k = params->top_k;
    p.top_p = params->top_p;
    p.min_p = params->min_p;
    p.seed = params->seed;
    p.request_id = params->request_id;
    p.step = params->step;
    return run_verify(MODE_SAMPLE, batch, p, reinterpret_cast<cudaStream_t>(stream));
}

int spec_draft_confidence(const spec_draft *d, const spec_allocation *o, void *workspace,
                          size_t workspace_bytes, spec_stream stream)
{
    if (!d || !o || !d->draft_logits) return SPEC_ERR_INVALID_ARG;
    if (!o->conf || !o->draft_token || !o->k_alloc || !o->cu_rows || !o->row_owner ||
        !o->row_pos || !o->total_rows)
        return SPEC_ERR_INVALID_ARG;
    if (d->dtype != SPEC_F32 && d->dtype != SPEC_BF16) return SPEC_ERR_UNSUPPORTED;
    if (d->V < 1 || d->ld < d->V || d->B < 1 || d->k < 1) return SPEC_ERR_INVALID_ARG;
    if (d->k > 31) return SPEC_ERR_UNSUPPORTED;
    if (!(d->threshold == d->threshold)) return SPEC_ERR_INVALID_ARG;
    if (d->max_rows < 0) return SPEC_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(d->draft_logits) % elt_bytes(d->dtype)) return SPEC_ERR_INVALID_ARG;
    if (static_cast<size_t>(d->V) * elt_bytes(d->dtype) > max_row_bytes()) return SPEC_ERR_UNSUPPORTED;
    const int64_t Q = static_cast<int64_t>(d->B) * d->k;
    if (Q * 8 + (static_cast<int64_t>(d->B) * 4 + 1) * 4 > 200 * 1024) return SPEC_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(Q) * d->ld > (int64_t(1) << 40)) return SPEC_ERR_UNSUPPORTED;
    if (Q * chunks_per_row(d->V, static_cast<int>(elt_bytes(d->dtype))) > INT32_MAX)
        return SPEC_ERR_UNSUPPORTED;

    const int elt = static_cast<int>(elt_bytes(d->dtype));
    if (!workspace || workspace_bytes < ws_bytes(static_cast<int32_t>(Q), 1, d->V, elt, false))
        return SPEC_ERR_WORKSPACE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    VerifyParams p;
    std::memset(&p, 0, sizeof p);
    const WsLayout l = ws_layout(workspace, static_cast<int32_t>(Q), 1, d->V, elt, false);
    p.ws_tok = l.tok;
    p.ws_flag = l.flag;
    p.ws_ticket = l.ticket;
    p.ws_info = l.info;
    p.ws_part = l.part;
    p.nchunk = chunks_per_row(d->V, elt);
    p.logits = d->draft_logits;
    p.ld = d->ld;
    p.V = d->V;
    p.B = d->B;
    p.k_max = d->k;
    p.R_cap = static_cast<int32_t>(Q);
    p.n_rows = static_cast<int32_t>(Q);
    p.selected = d->selected;
    p.conf = o->conf;
    p.draft_token = o->draft_token;
    p.status = o->status;
    cudaError_t e = launch_verify(MODE_CONF, d->dtype, p, s);
    if (e != cudaSuccess) return cuda_fail(e);

    AllocParams a;
    a.conf = o->conf;
    a.draft_token = o->draft_token;
    a.B = d->B;
    a.k = d->k;
    a.threshold = d->threshold;
    a.max_rows = d->max_rows;
    a.k_alloc = o->k_alloc;
    a.cu_rows = o->cu_rows;
    a.row_owner = o->row_owner;
    a.row_pos = o->row_pos;
    a.packed_draft = o->packed_draft;
    a.total_rows = o->total_rows;
    a.status = o->status;
    e = launch_alloc(a, s);
    return e == cudaSuccess ? SPEC_OK : cuda_fail(e);
}

int spec_prefix_stats(const int32_t *accepted_len, const int32_t *cu_rows, int32_t B,
                      int32_t k_max, int64_t *acc, int64_t *ver, int64_t *hist, uint32_t *status,
                      spec_stream stream)
{
    if (!accepted_len || !cu_rows || !acc || !ver) return SPEC_ERR_INVALID_ARG;
    if (B < 1 || k_max < 0) return SPEC_ERR_INVALID_ARG;
    if (k_max > 31) return SPEC_ERR_UNSUPPORTED;
    const cudaError_t e = launch_prefix_stats(accepted_len, cu_rows, B, k_max, acc, ver, hist,
                                              status, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPEC_OK : cuda_fail(e);
}

int spec_restore_rows(const void *compact, int64_t compact_ld, int32_t R_cap,
                      const int32_t *cu_rows, int32_t B, int32_t k_max, int64_t row_bytes,
                      void *out, int64_t out_ld, uint32_t *status, spec_stream stream)
{
    if (!compact || !cu_rows || !out) return SPEC_ERR_INVALID_ARG;
    if (B < 1 || R_cap < 1 || k_max < 0 || row_bytes < 1 || compact_ld < row_bytes ||
        out_ld < row_bytes)
        return SPEC_ERR_INVALID_ARG;
    if (k_max > 31 || row_bytes > (static_cast<int64_t>(1) << 30)) return SPEC_ERR_UNSUPPORTED;
    if (row_bytes % 16 || compact_ld % 16 || out_ld % 16 ||
        reinterpret_cast<uintptr_t>(compact) % 16 || reinterpret_cast<uintptr_t>(out) % 16)
        return SPEC_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(B) * (k_max + 1) > INT32_MAX) return SPEC_ERR_UNSUPPORTED;
    const cudaError_t e = launch_restore_rows(compact, compact_ld, R_cap, cu_rows, B, k_max,
                                              row_bytes, out, out_ld, status,
                                              reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPEC_OK : cuda_fail(e);
}

int spec_cache_append(const spec_cache *cache, const spec_cache_rows *rows, spec_stream stream)
{
    return run_cache_rows(cache, rows, true, stream);
}

int spec_cache_read(const spec_cache *cache, const spec_cache_rows *rows, spec_stream stream)
{
    return run_cache_rows(cache, rows, false, stream);
}

size_t spec_cache_workspace_bytes(int32_t B, int32_t k_max, int32_t Hq, int32_t H, int32_t D,
                                  int32_t max_len)
{
    if (B < 1 || k_max < 0 || k_max > 31 || H < 1 || Hq < H || Hq % H || max_len < 1) return 0;
    if (D != 64 && D != 128 && D != 256) return 0;
    if (B > kMostRequests || Hq > kMostHeads || max_len > kMostSlots) return 0;      // (no call accepts them)
    return cache_attend_workspace(B, k_max, Hq, H, D, max_len);
}

int spec_cache_attend(const spec_cache *cache, const spec_attention *attn, void *out, float *lse,
                      void *workspace, size_t workspace_bytes, spec_stream stream)
{
    CacheView c;
    AttnParams p;
    const int rc = check_attention(cache, attn, c, p);
    if (rc != SPEC_OK) return rc;
    if (!out) return SPEC_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(out) % elt_bytes(attn->dtype) || !on_words(lse)) return SPEC_ERR_INVALID_ARG;
    // (the parts of split tasks are read 16 bytes at a time)
    if (reinterpret_cast<uintptr_t>(workspace) % 16) return SPEC_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < spec_cache_workspace_bytes(c.B, p.k_max, p.Hq, c.H, c.D, p.max_len))
        return SPEC_ERR_WORKSPACE;
    p.out = out;
    p.lse = lse;
    p.ws = workspace;
    const cudaError_t e = launch_cache_attend(c, p, attn->dtype, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPEC_OK : cuda_fail(e);
}

int spec_cache_weights(const spec_cache *cache, const spec_attention *attn, const float *lse,
                       float *score, spec_stream stream)
{
    CacheView c;
    AttnParams p;
    const int rc = check_attention(cache, attn, c, p);
    if (rc != SPEC_OK) return rc;
    if (!lse || !score || !on_words(lse, score)) return SPEC_ERR_INVALID_ARG;
    p.lse = const_cast<float *>(lse);
    p.score = score;
    const cudaError_t e = launch_cache_weights(c, p, attn->dtype, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPEC_OK : cuda_fail(e);
}

int spec_cache_evict(const spec_cache *cache, const spec_eviction *ev, spec_stream stream)
{
    CacheView c;
    const int rc = check_cache(cache, c);
    if (rc != SPEC_OK) return rc;
    if (!ev || !ev->score || !ev->len || !ev->dst_table || !ev->kept || !ev->new_len)
        return SPEC_ERR_INVALID_ARG;
    if (!on_words(ev->score, ev->slot_pos, ev->len, ev->dst_table, ev->kept, ev->new_len, ev->status))
        return SPEC_ERR_INVALID_ARG;
    if (ev->budget < 1 || ev->recent < 0 || ev->recent > ev->budget || ev->dst_pages < 1)
        return SPEC_ERR_INVALID_ARG;
    const int64_t room = static_cast<int64_t>(c.max_pages) * c.page_tokens;
    const int64_t most = ev->budget < room ? ev->budget : room;
    if (static_cast<int64_t>(ev->dst_pages) * c.page_tokens < most) return SPEC_ERR_INVALID_ARG;
    EvictParams p;
    p.score = ev->score;
    p.slot_pos = ev->slot_pos;
    p.len = ev->len;
    p.budget = ev->budget;
    p.recent = ev->recent;
    p.dst_table = ev->dst_table;
    p.dst_pages = ev->dst_pages;
    p.kept = ev->kept;
    p.new_len = ev->new_len;
    p.status = ev->status;
    const cudaError_t e = launch_cache_evict(c, p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPEC_OK : cuda_fail(e);
}

const char *spec_result_string(int code)
{
    switch (code) {
    case SPEC_OK: return "SPEC_OK";
    case SPEC_ERR_INVALID_ARG: return "SPEC_ERR_INVALID_ARG";
    case SPEC_ERR_UNSUPPORTED: return "SPEC_ERR_UNSUPPORTED";
    case SPEC_ERR_CUDA: return "SPEC_ERR_CUDA";
    case SPEC_ERR_WORKSPACE: return "SPEC_ERR_WORKSPACE";
    default: return "unknown spec_result";
    }
}

const char *spec_last_cuda_error(void) { return g_cuda_error; }

int spec_abi_version(void) { return SPEC_ABI_VERSION; }

}  // extern "C"
