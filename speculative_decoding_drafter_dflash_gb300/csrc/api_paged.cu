// C ABI entry points of the paged 4-bit KV cache and of the token log probabilities: host-side
// validation, workspace carving and launches.
#include <math.h>

#include "df_internal.cuh"

namespace df {

namespace {

#define REQ(cond, code, ...)                         \
    do {                                             \
        if (!(cond)) return fail(code, __VA_ARGS__); \
    } while (0)

int check_ptr(const void *p, unsigned align, const char *name) {
    REQ(p != nullptr, DF_EINVAL, "%s is NULL", name);
    REQ((reinterpret_cast<uintptr_t>(p) & (align - 1)) == 0, DF_EINVAL, "%s is not %u-byte aligned",
        name, align);
    return DF_OK;
}

bool power_of_two(float f) {
    int e;
    return f > 0.f && f <= 3.4028234e38f && frexpf(f, &e) == 0.5f;
}

// shape: the sizes alone (workspace queries).
int check_paged(const df_paged_kv *c, bool shape_only) {
    REQ(c, DF_EINVAL, "cache is NULL");
    REQ(c->head_dim == 64 || c->head_dim == 128 || c->head_dim == 256, DF_ESHAPE,
        "head_dim=%d must be 64, 128 or 256", c->head_dim);
    REQ(c->page_size >= 16 && c->page_size <= 256 && (c->page_size & (c->page_size - 1)) == 0,
        DF_ESHAPE, "page_size=%d must be 16, 32, 64, 128 or 256", c->page_size);
    REQ(c->n_kv_heads > 0 && c->n_kv_heads <= 4096, DF_ESHAPE, "n_kv_heads=%d", c->n_kv_heads);
    REQ(c->batch > 0 && c->batch <= kPagedMaxBatch, DF_ESHAPE, "batch=%d must be in [1, %d]", c->batch,
        kPagedMaxBatch);
    REQ(c->n_pages > 0, DF_ESHAPE, "n_pages=%d", c->n_pages);
    REQ(c->max_pages > 0 && (long long)c->max_pages * c->page_size <= (1LL << 30), DF_ESHAPE,
        "max_pages=%d (at most 2^30 rows a sequence)", c->max_pages);
    REQ(power_of_two(c->k_scale) && power_of_two(c->v_scale), DF_EINVAL,
        "k_scale=%g, v_scale=%g must be powers of two", (double)c->k_scale, (double)c->v_scale);
    if (shape_only) return DF_OK;
    DF_TRY(check_ptr(c->k_codes, 16, "k_codes"));
    DF_TRY(check_ptr(c->v_codes, 16, "v_codes"));
    DF_TRY(check_ptr(c->k_scales, 16, "k_scales"));
    DF_TRY(check_ptr(c->v_scales, 16, "v_scales"));
    DF_TRY(check_ptr(c->page_table, 4, "page_table"));
    return check_ptr(c->seq_len, 4, "seq_len");
}

int check_attention_paged(const df_paged_kv *c, int blk, int nq, bool shape_only) {
    DF_TRY(check_paged(c, shape_only));
    REQ(blk > 0, DF_ESHAPE, "blk=%d", blk);
    REQ(nq > 0 && nq % c->n_kv_heads == 0, DF_ESHAPE, "nq=%d must be a positive multiple of n_kv_heads=%d",
        nq, c->n_kv_heads);
    // places of work (32 keys of one KV head and 8 query rows, and 24 more of each such task) and row
    // indices stay in 32 bits
    const long long rows = (long long)blk * (nq / c->n_kv_heads);
    REQ(rows <= (1LL << 24), DF_ESHAPE, "blk x query heads per KV head = %lld", rows);
    const double units = ((double)c->max_pages * c->page_size / 32 + 25) * c->batch * c->n_kv_heads *
                         ((double)rows / 8 + 1);
    REQ(units < 1073741824.0, DF_ESHAPE, "%.3g pieces of 32 keys and 8 query rows (at most 2^30)", units);
    return DF_OK;
}

int check_logprobs(int R, int V, int top_k) {
    REQ(R > 0 && R <= (1 << 24), DF_ESHAPE, "R=%d", R);
    REQ(V > 0 && V <= (1 << 30), DF_ESHAPE, "V=%d", V);
    REQ(top_k >= 0 && top_k <= kLogprobsMaxTop && top_k <= V, DF_ESHAPE,
        "top_k=%d must be in [0, %d] and at most V", top_k, kLogprobsMaxTop);
    return DF_OK;
}

int check_ws(void *ws, size_t ws_bytes, size_t need) {
    REQ(ws != nullptr, DF_EWORKSPACE, "workspace is NULL (need %zu bytes)", need);
    REQ((reinterpret_cast<uintptr_t>(ws) & 255u) == 0, DF_EWORKSPACE, "workspace is not 256-byte aligned");
    REQ(ws_bytes >= need, DF_EWORKSPACE, "workspace of %zu bytes is smaller than %zu", ws_bytes, need);
    return DF_OK;
}

// Counters, then partial results.
size_t attention_carve(const df_paged_kv &c, int blk, int nq, AttnPagedArgs *a, void *ws) {
    Carve cv{static_cast<char *>(ws), 0, ~size_t(0), true};
    int *counters = cv.take<int>(kOpsCounters);
    float *part = cv.take<float>(attn_paged_part_floats(c, blk, nq));
    if (a) {
        a->counters = counters;
        a->part = part;
    }
    return cv.off;
}

size_t logprobs_carve(int R, int V, LogprobsArgs *a, void *ws) {
    Carve cv{static_cast<char *>(ws), 0, ~size_t(0), true};
    int *counters = cv.take<int>(kOpsCounters);
    char *part = cv.take<char>(logprobs_part_bytes(R, V));
    if (a) {
        a->counters = counters;
        a->part = part;
    }
    return cv.off;
}

}  // namespace

}  // namespace df

using namespace df;

extern "C" {

int df_kv_append_paged(const df_paged_kv *cache, const float *q, int ldq, int n_q_heads,
                       const float *k, int ldk, const float *v, int ldv, const float *q_norm,
                       const float *k_norm, float eps, const df_rope *rope, const int32_t *n_new,
                       int n_max, float *q_out, int32_t *d_status, df_stream_t stream) {
    clear_error();
    DF_TRY(check_paged(cache, false));
    const int d = cache->head_dim;
    REQ(n_max > 0 && (long long)n_max * cache->batch <= (1LL << 28), DF_ESHAPE, "n_max=%d", n_max);
    REQ(n_q_heads >= 0 && n_q_heads <= 65536, DF_ESHAPE, "n_q_heads=%d", n_q_heads);
    REQ((q != nullptr) == (n_q_heads > 0) && (q != nullptr) == (q_out != nullptr), DF_EINVAL,
        "q, n_q_heads and q_out go together");
    if (q) {
        DF_TRY(check_ptr(q, 16, "q"));
        DF_TRY(check_ptr(q_out, 16, "q_out"));
        REQ(ldq % 4 == 0 && ldq >= n_q_heads * d, DF_ESHAPE, "ldq=%d (a multiple of 4, >= %d)", ldq,
            n_q_heads * d);
    }
    DF_TRY(check_ptr(k, 16, "k"));
    DF_TRY(check_ptr(v, 16, "v"));
    const long long row = (long long)cache->n_kv_heads * d;
    REQ(ldk % 4 == 0 && ldk >= row, DF_ESHAPE, "ldk=%d (a multiple of 4, >= %lld)", ldk, row);
    REQ(ldv % 4 == 0 && ldv >= row, DF_ESHAPE, "ldv=%d (a multiple of 4, >= %lld)", ldv, row);
    if (q_norm) DF_TRY(check_ptr(q_norm, 4, "q_norm"));
    if (k_norm) DF_TRY(check_ptr(k_norm, 4, "k_norm"));
    REQ(eps >= 0.f && eps <= 3.4028234e38f, DF_EINVAL, "eps=%g", (double)eps);
    KvAppendArgs a;
    a.rope = df_rope{};
    if (rope) {
        REQ(rope->rotary_dim > 0 && rope->rotary_dim % 16 == 0 && rope->rotary_dim <= d, DF_ESHAPE,
            "rotary_dim=%d must be a multiple of 16 in [16, head_dim]", rope->rotary_dim);
        REQ(rope->n_axes >= 1 && rope->n_axes <= kPagedMaxAxes, DF_ESHAPE, "n_axes=%d must be in [1, %d]",
            rope->n_axes, kPagedMaxAxes);
        DF_TRY(check_ptr(rope->inv_freq, 8, "inv_freq"));
        if (rope->positions) DF_TRY(check_ptr(rope->positions, 4, "positions"));
        a.rope = *rope;
    }
    a.c = *cache;
    a.q = q;
    a.k = k;
    a.v = v;
    a.ldq = ldq;
    a.ldk = ldk;
    a.ldv = ldv;
    a.nq = n_q_heads;
    a.q_norm = q_norm;
    a.k_norm = k_norm;
    a.eps = eps;
    a.n_new = n_new;
    a.n_max = n_max;
    a.q_out = q_out;
    a.status = d_status;
    return launch_kv_append_paged(a, (cudaStream_t)stream);
}

int df_kv_gather_paged(const df_paged_kv *cache, const int32_t *start, const int32_t *n, int n_max,
                       float *k_out, float *v_out, int32_t *d_status, df_stream_t stream) {
    clear_error();
    DF_TRY(check_paged(cache, false));
    REQ(n_max > 0 && n_max <= (1 << 30), DF_ESHAPE, "n_max=%d", n_max);
    DF_TRY(check_ptr(k_out, 16, "k_out"));
    DF_TRY(check_ptr(v_out, 16, "v_out"));
    return launch_kv_gather_paged(*cache, start, n, n_max, k_out, v_out, d_status, (cudaStream_t)stream);
}

int kv_advance(int32_t *seq_len, const int32_t *n, int B, int cap, int32_t *d_status,
               df_stream_t stream) {
    clear_error();
    REQ(B > 0, DF_ESHAPE, "B=%d", B);
    REQ(cap > 0, DF_ESHAPE, "cap=%d", cap);
    REQ(seq_len && n, DF_EINVAL, "seq_len / n is NULL");
    return launch_seq_advance(seq_len, n, B, 0, cap, d_status, (cudaStream_t)stream);
}

size_t df_attention_paged_workspace_bytes(const df_paged_kv *cache, int blk, int nq) {
    if (check_attention_paged(cache, blk, nq, true) != DF_OK) return 0;
    return attention_carve(*cache, blk, nq, nullptr, nullptr);
}

int df_attention_paged(const df_paged_kv *cache, const float *q, const int32_t *n_new, int blk,
                       int nq, int causal, float *out, void *ws, size_t ws_bytes,
                       int32_t *d_status, df_stream_t stream) {
    clear_error();
    DF_TRY(check_attention_paged(cache, blk, nq, false));
    DF_TRY(check_ptr(q, 16, "q"));
    DF_TRY(check_ptr(out, 16, "out"));
    REQ(causal == 0 || causal == 1, DF_EINVAL, "causal=%d", causal);
    REQ(!causal || n_new, DF_EINVAL, "causal=1 needs n_new (which rows are the new ones)");
    DF_TRY(check_ws(ws, ws_bytes, attention_carve(*cache, blk, nq, nullptr, nullptr)));
    AttnPagedArgs a;
    attention_carve(*cache, blk, nq, &a, ws);
    a.c = *cache;
    a.q = q;
    a.n_new = n_new;
    a.blk = blk;
    a.nq = nq;
    a.causal = causal;
    a.out = out;
    a.status = d_status;
    return launch_attn_paged(a, (cudaStream_t)stream);
}

size_t df_token_logprobs_workspace_bytes(int R, int V, int top_k) {
    if (check_logprobs(R, V, top_k) != DF_OK) return 0;
    return logprobs_carve(R, V, nullptr, nullptr);
}

int df_token_logprobs(const void *logits, int logits_bf16, int R, int V, long long ld,
                      float temperature, const int32_t *tokens, float *logprob, float *entropy,
                      int top_k, int32_t *top_ids, float *top_logprobs, void *ws, size_t ws_bytes,
                      int32_t *d_status, df_stream_t stream) {
    clear_error();
    DF_TRY(check_logprobs(R, V, top_k));
    REQ(logits_bf16 == 0 || logits_bf16 == 1, DF_EINVAL, "logits_bf16=%d", logits_bf16);
    REQ(ld >= V, DF_ESHAPE, "ld=%lld < V=%d", ld, V);
    REQ(temperature > 1e-30f && temperature <= 1e30f, DF_EINVAL,
        "temperature=%g (temperature 0 is the argmax)", (double)temperature);
    DF_TRY(check_ptr(logits, logits_bf16 ? 2 : 4, "logits"));
    DF_TRY(check_ptr(tokens, 4, "tokens"));
    DF_TRY(check_ptr(logprob, 4, "logprob"));
    if (top_k > 0) {
        DF_TRY(check_ptr(top_ids, 4, "top_ids"));
        DF_TRY(check_ptr(top_logprobs, 4, "top_logprobs"));
    }
    DF_TRY(check_ws(ws, ws_bytes, logprobs_carve(R, V, nullptr, nullptr)));
    LogprobsArgs a;
    logprobs_carve(R, V, &a, ws);
    a.logits = logits;
    a.bf16 = logits_bf16;
    a.R = R;
    a.V = V;
    a.ld = ld;
    a.T = temperature;
    a.tokens = tokens;
    a.logprob = logprob;
    a.entropy = entropy;
    a.top_k = top_k;
    a.top_ids = top_ids;
    a.top_lp = top_logprobs;
    a.status = d_status;
    return launch_token_logprobs(a, (cudaStream_t)stream);
}

}  // extern "C"
