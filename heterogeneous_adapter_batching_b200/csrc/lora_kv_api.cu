// C-ABI entry points of the KV-cache and attention calls: argument checks, then
// one launcher each.  See include/lora.h for the contract of every function.
#include <cmath>

#include "lora_internal.cuh"
#include "lora_kv.cuh"

using namespace lora;

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int elem_size(int dtype) { return dtype == LORA_FP32 ? 4 : 2; }

// Row tensor checks; without tokens or heads any tensor is fine, also one that is missing or has no address.
bool rows_ok(const lora_rows_t *r, int T, int heads, int dtype) {
    if (T == 0 || heads == 0) return true;
    if (!r || !r->data || !aligned16(r->data) || r->token_stride < 0 || r->head_stride < 0) return false;
    const int64_t e = 16 / elem_size(dtype);
    return r->token_stride % e == 0 && r->head_stride % e == 0;
}

// Output rows: also apart from one another.
bool out_ok(const lora_rows_t *r, int T, int heads, int dim, int dtype) {
    return rows_ok(r, T, heads, dtype) && (T == 0 || heads == 0 || ((T < 2 || r->token_stride >= dim) && (heads < 2 || r->head_stride >= dim)));
}

// n int32 of an array; none where there is no array.
struct Span {
    const int32_t *p;
    long long n;
};
bool overlap(const Span &a, const Span &b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && x < y + 4 * (uintptr_t)b.n && y < x + 4 * (uintptr_t)a.n;
}

// Strides that a TMA descriptor takes: positive where they count, below 2^40 bytes (of 16-bit elements).
bool strides_ok(const lora_rows_t *r, int T, int heads) {
    if (T < 1) return true;
    return (T == 1 || (r->token_stride > 0 && r->token_stride < (1LL << 39))) &&
           (heads == 1 || (r->head_stride > 0 && r->head_stride < (1LL << 39)));
}

Rows rows(const lora_rows_t *r) { return r ? Rows{r->data, r->token_stride, r->head_stride} : Rows{nullptr, 0, 0}; }

int check_cache(const lora_kv_cache_t *c) {
    if (!c || !c->pages || !aligned16(c->pages) || c->page_bytes % 16 || c->num_pages < 1) return LORA_ERR_INVALID_ARG;
    const size_t need = lora_kv_block_bytes(c->kv_heads, c->head_dim, c->block_tokens);
    if (need == 0 || c->page_bytes < need) return LORA_ERR_INVALID_ARG;
    if ((long long)c->num_pages * c->block_tokens > INT32_MAX) return LORA_ERR_TOO_LARGE;
    return LORA_OK;
}

KvCache cache(const lora_kv_cache_t *c) {
    return KvCache{static_cast<unsigned char *>(c->pages), (long long)c->page_bytes, c->num_pages, c->kv_heads,
                   c->block_tokens, c->block_tokens / LORA_KV_GRANULE};
}

bool half_type(int t) { return t == LORA_BF16 || t == LORA_FP16; }

bool rope_ok(int src, int dst, int T, int dim, const int32_t *positions, const float *freq, int rot) {
    return half_type(dst) && (src == dst || src == LORA_FP32) && T >= 0 && dim >= 16 && dim <= 256 && dim % 16 == 0 &&
           rot >= 0 && rot <= dim && rot % 16 == 0 && (rot == 0 || freq) && (T == 0 || positions);
}

int layout(const LayoutArgs &a, lora_stream_t stream) {
    reset_launch_count();
    if (!a.past || !a.fresh_len || !a.table || !a.cu || !a.kv_len || (a.T > 0 && (!a.positions || !a.slots)) || a.R < 1 ||
        a.T < 0 || a.max_blocks < 1 || a.num_free < 0)
        return LORA_ERR_INVALID_ARG;
    if (a.block < 1 || a.block > 1024 || a.block % LORA_KV_GRANULE) return LORA_ERR_INVALID_ARG;
    if (a.R > LORA_KV_MAX_REQUESTS || ((long long)a.max_blocks + 1) * a.block > INT32_MAX) return LORA_ERR_TOO_LARGE;
    // Every CTA reads the inputs for itself while others write: a kv_len that is past_len would be read half updated.
    const Span in[] = {{a.past, a.R}, {a.fresh_len, a.R}, {a.req_ids, a.R}, {a.free_pages, a.num_free}, {a.free_head, 1}, {a.held, a.R}};
    const Span out[] = {{a.table, (long long)a.R * a.max_blocks}, {a.cu, a.R + 1}, {a.kv_len, a.R}, {a.positions, a.T},
                        {a.slots, a.T}, {a.ids, a.T}, {a.head_out, 1}, {a.held_out, a.R}};
    for (const Span &o : out) {
        for (const Span &i : in)
            if (overlap(o, i)) return LORA_ERR_INVALID_ARG;
        for (const Span &i : out)
            if (&i != &o && overlap(o, i)) return LORA_ERR_INVALID_ARG;
    }
    return launch_kv_layout(a, reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

size_t lora_kv_block_bytes(int kv_heads, int head_dim, int block_tokens) {
    if (kv_heads < 1 || kv_heads > 256 || (head_dim != 64 && head_dim != 128) || block_tokens < 1 || block_tokens > 1024 ||
        block_tokens % LORA_KV_GRANULE)
        return 0;
    return (size_t)kv_heads * (block_tokens / LORA_KV_GRANULE) * kv_granule_bytes(head_dim);
}

int lora_kv_layout(const int32_t *past_len, const int32_t *new_len, const int32_t *req_ids, int R, int T,
                   int block_tokens, int32_t *block_table, int max_blocks, const int32_t *free_pages, int num_free,
                   const int32_t *free_head, int32_t *cu_new, int32_t *kv_len, int32_t *positions, int32_t *slots,
                   int32_t *ids, int32_t *free_head_out, int32_t *err_dev, lora_stream_t stream) {
    return layout(LayoutArgs{past_len, new_len, req_ids, R, T, block_tokens, block_table, max_blocks, free_pages, num_free,
                             free_head, cu_new, kv_len, positions, slots, ids, free_head_out, err_dev, nullptr, nullptr},
                  stream);
}

int lora_kv_layout_held(const int32_t *past_len, const int32_t *new_len, const int32_t *req_ids, int R, int T,
                        int block_tokens, int32_t *block_table, int max_blocks, const int32_t *free_pages, int num_free,
                        const int32_t *free_head, int32_t *cu_new, int32_t *kv_len, int32_t *positions, int32_t *slots,
                        int32_t *ids, int32_t *free_head_out, const int32_t *held, int32_t *held_out, int32_t *err_dev,
                        lora_stream_t stream) {
    if (!held || !held_out) {
        reset_launch_count();
        return LORA_ERR_INVALID_ARG;
    }
    return layout(LayoutArgs{past_len, new_len, req_ids, R, T, block_tokens, block_table, max_blocks, free_pages, num_free,
                             free_head, cu_new, kv_len, positions, slots, ids, free_head_out, err_dev, held, held_out},
                  stream);
}

int lora_rope(const lora_rows_t *q, int q_heads, const lora_rows_t *k, int k_heads, int src_dtype, int T, int head_dim,
              const int32_t *positions, const float *inv_freq, int rot_dim, int interleaved, double mscale,
              const lora_rows_t *q_out, const lora_rows_t *k_out, int dst_dtype, lora_stream_t stream) {
    reset_launch_count();
    if (!rope_ok(src_dtype, dst_dtype, T, head_dim, positions, inv_freq, rot_dim) || q_heads < 0 || k_heads < 0 ||
        q_heads > 4096 || k_heads > 4096)
        return LORA_ERR_INVALID_ARG;
    if (!rows_ok(q, T, q_heads, src_dtype) || !rows_ok(k, T, k_heads, src_dtype) || !out_ok(q_out, T, q_heads, head_dim, dst_dtype) ||
        !out_ok(k_out, T, k_heads, head_dim, dst_dtype))
        return LORA_ERR_INVALID_ARG;
    if (T == 0 || q_heads + k_heads == 0) return LORA_OK;
    RopeArgs a{};
    a.q = rows(q); a.k = rows(k); a.qo = rows(q_out); a.ko = rows(k_out);
    a.hq = q_heads; a.hk = k_heads; a.has_ko = true;
    a.T = T; a.dim = head_dim; a.rot = rot_dim; a.interleaved = interleaved; a.mscale = mscale;
    a.positions = positions; a.freq = inv_freq;
    return launch_rope(a, src_dtype, dst_dtype, reinterpret_cast<cudaStream_t>(stream));
}

int lora_kv_append(const lora_rows_t *q, int q_heads, const lora_rows_t *k, const lora_rows_t *v, int src_dtype, int T,
                   const int32_t *positions, const float *inv_freq, int rot_dim, int interleaved, double mscale,
                   const int32_t *slots, const lora_kv_cache_t *kv, const lora_rows_t *q_out,
                   const lora_rows_t *k_out, const lora_rows_t *v_out, int dst_dtype, int32_t *err_dev,
                   lora_stream_t stream) {
    reset_launch_count();
    if (int rc = check_cache(kv)) return rc;
    const int h = kv->kv_heads;
    if (!rope_ok(src_dtype, dst_dtype, T, kv->head_dim, positions, inv_freq, rot_dim) || q_heads < 0 || q_heads > 4096 ||
        (T > 0 && !slots))
        return LORA_ERR_INVALID_ARG;
    if (!rows_ok(q, T, q_heads, src_dtype) || !rows_ok(k, T, h, src_dtype) || !rows_ok(v, T, h, src_dtype) ||
        !out_ok(q_out, T, q_heads, kv->head_dim, dst_dtype) || !out_ok(k_out, T, k_out ? h : 0, kv->head_dim, dst_dtype) ||
        !out_ok(v_out, T, v_out ? h : 0, kv->head_dim, dst_dtype))
        return LORA_ERR_INVALID_ARG;
    if (T == 0) return LORA_OK;
    RopeArgs a{};
    a.q = rows(q); a.k = rows(k); a.v = rows(v);
    a.qo = rows(q_out); a.ko = rows(k_out); a.vo = rows(v_out);
    a.hq = q_heads; a.hk = h; a.hv = h;
    a.has_ko = k_out != nullptr; a.has_vo = v_out != nullptr;
    a.T = T; a.dim = kv->head_dim; a.rot = rot_dim; a.interleaved = interleaved; a.mscale = mscale;
    a.positions = positions; a.freq = inv_freq; a.slots = slots; a.c = cache(kv); a.err = err_dev;
    return launch_rope(a, src_dtype, dst_dtype, reinterpret_cast<cudaStream_t>(stream));
}

int lora_kv_gather(const lora_kv_cache_t *kv, const int32_t *slots, int T, const lora_rows_t *k_out,
                   const lora_rows_t *v_out, int dst_dtype, int32_t *err_dev, lora_stream_t stream) {
    reset_launch_count();
    if (int rc = check_cache(kv)) return rc;
    if (dst_dtype < LORA_BF16 || dst_dtype > LORA_FP32 || T < 0 || (T > 0 && !slots)) return LORA_ERR_INVALID_ARG;
    if (!out_ok(k_out, T, k_out ? kv->kv_heads : 0, kv->head_dim, dst_dtype) ||
        !out_ok(v_out, T, v_out ? kv->kv_heads : 0, kv->head_dim, dst_dtype))
        return LORA_ERR_INVALID_ARG;
    if (T == 0 || (!k_out && !v_out)) return LORA_OK;
    const GatherKvArgs a{cache(kv), kv->head_dim, T, slots, rows(k_out), rows(v_out), k_out != nullptr, v_out != nullptr,
                         err_dev};
    return launch_kv_gather(a, dst_dtype, reinterpret_cast<cudaStream_t>(stream));
}

static bool group_ok(int q_heads, int kv_heads) {
    return q_heads >= 1 && kv_heads >= 1 && kv_heads <= 256 && q_heads % kv_heads == 0 && q_heads / kv_heads <= LORA_KV_MAX_GROUP;
}

size_t lora_kv_attend_workspace_size(int q_heads, int kv_heads, int head_dim, int max_q_len) {
    if (!group_ok(q_heads, kv_heads) || (head_dim != 64 && head_dim != 128) || max_q_len < 1) return 0;
    return attend_workspace(q_heads, kv_heads, head_dim, max_q_len);
}

int lora_kv_attend(const lora_rows_t *q, int T, int q_heads, int dtype, const lora_kv_cache_t *kv,
                   const int32_t *block_table, int max_blocks, const int32_t *cu_q, const int32_t *kv_len, int R,
                   int max_q_len, float scale, const lora_rows_t *out, float *lse, void *ws, size_t ws_bytes,
                   int32_t *err_dev, lora_stream_t stream) {
    reset_launch_count();
    if (int rc = check_cache(kv)) return rc;
    if (!half_type(dtype) || T < 0 || R < 1 || max_q_len < 1 || max_blocks < 1 || !group_ok(q_heads, kv->kv_heads) ||
        !block_table || !cu_q || !kv_len || !std::isfinite(scale))
        return LORA_ERR_INVALID_ARG;
    if (R > LORA_KV_MAX_REQUESTS || ((long long)max_blocks + 1) * kv->block_tokens > INT32_MAX) return LORA_ERR_TOO_LARGE;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) ||
        ws_bytes < attend_workspace(q_heads, kv->kv_heads, kv->head_dim, max_q_len))
        return LORA_ERR_WORKSPACE;
    if (T == 0) return LORA_OK;
    if ((long long)T * (q_heads / kv->kv_heads) > INT32_MAX) return LORA_ERR_TOO_LARGE;
    if (!rows_ok(q, T, q_heads, dtype) || !out_ok(out, T, q_heads, kv->head_dim, dtype)) return LORA_ERR_INVALID_ARG;
    const int group = q_heads / kv->kv_heads;
    const AttendArgs a{rows(q), rows(out), T, q_heads, kv->head_dim, dtype, cache(kv), block_table, max_blocks, cu_q,
                       kv_len, R, max_q_len, scale, lse, ws, err_dev, group, 65536u / (uint32_t)group + 1};
    return launch_kv_attend(a, reinterpret_cast<cudaStream_t>(stream));
}

static int prompt(const lora_rows_t *q, const lora_rows_t *k, const lora_rows_t *v, int Tq, int Tk, int q_heads, int kv_heads,
                  int head_dim, int dtype, const int32_t *cu_q, const int32_t *cu_k, const int32_t *kv_len, int R, float scale,
                  const lora_rows_t *out, float *lse, int32_t *err_dev, lora_stream_t stream) {
    reset_launch_count();
    if (!half_type(dtype) || Tq < 0 || Tk < 0 || R < 1 || !group_ok(q_heads, kv_heads) ||
        (head_dim != 64 && head_dim != 128) || !cu_q || !cu_k || !(scale >= 0.f && scale < INFINITY))
        return LORA_ERR_INVALID_ARG;
    if (R > LORA_KV_MAX_REQUESTS || (long long)Tq * (q_heads / kv_heads) > INT32_MAX) return LORA_ERR_TOO_LARGE;
    if (Tq == 0) return LORA_OK;
    if (!rows_ok(q, Tq, q_heads, dtype) || !out_ok(out, Tq, q_heads, head_dim, dtype) || !rows_ok(k, Tk, kv_heads, dtype) ||
        !rows_ok(v, Tk, kv_heads, dtype))
        return LORA_ERR_INVALID_ARG;
    if (!strides_ok(q, Tq, q_heads) || !strides_ok(k, Tk, kv_heads) || !strides_ok(v, Tk, kv_heads)) return LORA_ERR_INVALID_ARG;
    const PromptArgs a{rows(q), rows(k), rows(v), rows(out), Tq, Tk, q_heads, kv_heads, head_dim, dtype,
                       cu_q, cu_k, R, scale, lse, err_dev, kv_len};
    return launch_prompt(a, reinterpret_cast<cudaStream_t>(stream));
}

int lora_prompt_attend(const lora_rows_t *q, const lora_rows_t *k, const lora_rows_t *v, int Tq, int Tk, int q_heads,
                       int kv_heads, int head_dim, int dtype, const int32_t *cu_q, const int32_t *cu_k, int R,
                       float scale, const lora_rows_t *out, float *lse, int32_t *err_dev, lora_stream_t stream) {
    return prompt(q, k, v, Tq, Tk, q_heads, kv_heads, head_dim, dtype, cu_q, cu_k, nullptr, R, scale, out, lse, err_dev, stream);
}

int lora_prompt_attend_whole(const lora_rows_t *q, const lora_rows_t *k, const lora_rows_t *v, int T, int q_heads,
                             int kv_heads, int head_dim, int dtype, const int32_t *cu, const int32_t *kv_len, int R,
                             float scale, const lora_rows_t *out, float *lse, int32_t *err_dev, lora_stream_t stream) {
    if (!kv_len) {
        reset_launch_count();
        return LORA_ERR_INVALID_ARG;
    }
    return prompt(q, k, v, T, T, q_heads, kv_heads, head_dim, dtype, cu, cu, kv_len, R, scale, out, lse, err_dev, stream);
}

}  // extern "C"
