// C ABI of the calls around the attention (ac_layer_*, ac_rope_table,
// ac_qk_norm_rope, ac_cache_*): argument checks, then one or two launches of
// the kernels in ac_rope.cu and ac_cache_attn.cu.
#include <algorithm>
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdlib.h>
#include <string.h>

#include "adacluster.h"
#include "ac_layer.cuh"

using namespace ac;

struct ac_layer {
    ac_layer_config cfg;
    RopeArgs rope;     // without table and positions
    FreqArgs freq;
    int device, num_sms, elt;
    int *d_status;
    void *encode_fn;
};

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// A view's data and strides (see ac_tensor).  `out`: rows must not overlap.
bool view_ok(const ac_tensor &t, long long batch, long long n, int heads, int d, int elt, bool out) {
    if (!t.data || !aligned16(t.data)) return false;
    long long size[3] = {batch, n, heads}, stride[3] = {t.batch_stride, t.token_stride, t.head_stride};
    int m = 0;
    for (int i = 0; i < 3; i++) {
        if (size[i] <= 1) continue;
        // 2^40 elements reach past any device; token and head strides are 32-bit in
        // the kernels (64-bit products cost the gradients' kernel 7%)
        if (stride[i] < 0 || stride[i] > (i == 0 ? 1LL << 40 : 0x7fffffffLL) || (stride[i] * elt) % 16) return false;
        size[m] = size[i];
        stride[m++] = stride[i];
    }
    if (!out) return true;
    for (int i = 1; i < m; i++)
        for (int j = i; j > 0 && stride[j] < stride[j - 1]; j--) {
            std::swap(stride[j], stride[j - 1]);
            std::swap(size[j], size[j - 1]);
        }
    long long span = d;
    for (int i = 0; i < m; i++) {
        if (stride[i] < span) return false;
        span += stride[i] * (size[i] - 1);
    }
    return true;
}

// First and last byte of a view.
void span_of(const ac_tensor &t, long long batch, long long n, int heads, int d, int elt, uintptr_t &a, uintptr_t &b) {
    long long last = d;
    if (batch > 1) last += (batch - 1) * t.batch_stride;
    if (n > 1) last += (n - 1) * t.token_stride;
    if (heads > 1) last += (heads - 1) * t.head_stride;
    a = (uintptr_t)t.data;
    b = a + (uintptr_t)last * elt;
}

// An output may be its input (the same view) or lie apart from it.
bool alias_ok(const ac_tensor &x, const ac_tensor &y, long long batch, long long n, int heads, int d, int elt) {
    if (x.data == y.data && (batch <= 1 || x.batch_stride == y.batch_stride) &&
        (n <= 1 || x.token_stride == y.token_stride) && (heads <= 1 || x.head_stride == y.head_stride))
        return true;
    uintptr_t xa, xb, ya, yb;
    span_of(x, batch, n, heads, d, elt, xa, xb);
    span_of(y, batch, n, heads, d, elt, ya, yb);
    return xb <= ya || yb <= xa;
}

View view_of(const ac_tensor &t) { return View{t.data, t.batch_stride, (int)t.token_stride, (int)t.head_stride}; }

// The device check shared by every call that launches.
ac_status enter(const ac_layer *l) {
    (void)cudaGetLastError();  // a pending error of earlier work would be read back as this call's
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return AC_ERR_CUDA;
    return dev == l->device ? AC_OK : AC_ERR_INVALID_ARG;
}
ac_status leave() { return cudaGetLastError() == cudaSuccess ? AC_OK : AC_ERR_CUDA; }

// Rotation arguments of one call.
ac_status rope_of(const ac_layer *l, const float *table, const int32_t *pos, int64_t pos_batch, int batch, RopeArgs &r) {
    r = l->rope;
    if (!r.axes) return AC_OK;
    if (!table || !aligned16(table)) return AC_ERR_INVALID_ARG;
    if (pos && batch > 1 && (pos_batch < 0 || pos_batch > (int64_t(1) << 40))) return AC_ERR_INVALID_ARG;
    r.table = (const float2 *)table;
    r.pos = pos;
    r.pos_batch = pos && batch > 1 ? pos_batch : 0;
    return AC_OK;
}

long long table_pairs(const RopeArgs &r) {
    return r.axes ? r.off[r.axes - 1] + (long long)r.max[r.axes - 1] * r.np[r.axes - 1] : 0;
}

}  // namespace

extern "C" {

ac_status ac_layer_create(const ac_layer_config *cfg, ac_layer **out) {
    if (!out) return AC_ERR_INVALID_ARG;
    *out = nullptr;
    if (!cfg) return AC_ERR_INVALID_ARG;
    const ac_layer_config &g = *cfg;
    if (g.heads < 1 || g.kv_heads < 1 || g.heads % g.kv_heads) return AC_ERR_INVALID_ARG;
    if (g.heads > 4096) return AC_ERR_UNSUPPORTED;
    if (g.d != 64 && g.d != 128) return AC_ERR_UNSUPPORTED;
    if (g.dtype != AC_F32 && g.dtype != AC_BF16) return AC_ERR_INVALID_ARG;
    if (g.w_dtype != AC_F32 && g.w_dtype != AC_BF16) return AC_ERR_INVALID_ARG;
    if (g.norm != AC_NORM_NONE && g.norm != AC_NORM_RMS && g.norm != AC_NORM_LAYER) return AC_ERR_INVALID_ARG;
    if (!(g.eps >= 0.0) || !isfinite(g.eps)) return AC_ERR_INVALID_ARG;
    if (g.rope_axes < 0 || g.rope_axes > 3) return AC_ERR_INVALID_ARG;
    if (g.page_size < 0 || g.causal_block < 0 || g.window < 0) return AC_ERR_INVALID_ARG;
    if (!(g.scale >= 0.0) || !isfinite(g.scale)) return AC_ERR_INVALID_ARG;
    if (g.page_size && (g.page_size < 16 || g.page_size > 1024 || (g.page_size & (g.page_size - 1))))
        return AC_ERR_UNSUPPORTED;
    RopeArgs r;
    FreqArgs f;
    memset(&r, 0, sizeof(r));
    memset(&f, 0, sizeof(f));
    r.axes = g.rope_axes;
    if (r.axes) {
        if (g.rope_layout != AC_ROPE_INTERLEAVED && g.rope_layout != AC_ROPE_HALF) return AC_ERR_INVALID_ARG;
        if (!(g.rope_theta > 0.0) || !isfinite(g.rope_theta)) return AC_ERR_INVALID_ARG;
        const int sc = g.rope_scaling;
        if (sc != AC_ROPE_PLAIN && sc != AC_ROPE_LINEAR && sc != AC_ROPE_NTK && sc != AC_ROPE_YARN)
            return AC_ERR_INVALID_ARG;
        if (sc != AC_ROPE_PLAIN && (!(g.rope_factor >= 1.0) || !isfinite(g.rope_factor))) return AC_ERR_INVALID_ARG;
        if (sc == AC_ROPE_YARN && (g.rope_orig < 1 || !(g.rope_beta_slow >= 0.0) ||
                                   !(g.rope_beta_fast > g.rope_beta_slow) || !isfinite(g.rope_beta_fast)))
            return AC_ERR_INVALID_ARG;
        f.mag = sc == AC_ROPE_YARN ? 0.1 * log(g.rope_factor) + 1.0 : 1.0;
        r.half = g.rope_layout == AC_ROPE_HALF;
        long long off = 0, cells = 1;
        for (int a = 0; a < r.axes; a++) {
            const int D = g.rope_dims[a];
            if (D < 2 || D > g.d || (D & 1) || g.rope_max[a] < 1 || (sc == AC_ROPE_NTK && D == 2))
                return AC_ERR_INVALID_ARG;
            r.first[a] = r.pairs;
            r.np[a] = D / 2;
            r.max[a] = g.rope_max[a];
            r.off[a] = (uint32_t)off;
            off += (long long)r.max[a] * r.np[a];
            cells = std::min(cells * r.max[a], 0x7fffffffLL);
            r.pairs += D / 2;
            if (off > (1LL << 31)) return AC_ERR_UNSUPPORTED;  // a table of 16 GiB
            if (2 * r.pairs > g.d) return AC_ERR_INVALID_ARG;
            const double theta = sc == AC_ROPE_NTK ? g.rope_theta * pow(g.rope_factor, D / (D - 2.0)) : g.rope_theta;
            for (int j = 0; j < D / 2; j++) {
                double w = pow(theta, -2.0 * j / D);
                if (sc == AC_ROPE_LINEAR) w /= g.rope_factor;
                if (sc == AC_ROPE_YARN) {
                    const double turns = g.rope_orig * w / 6.283185307179586476925;
                    const double keep = std::min(
                        1.0, std::max(0.0, (turns - g.rope_beta_slow) / (g.rope_beta_fast - g.rope_beta_slow)));
                    w = w * keep + w / g.rope_factor * (1.0 - keep);
                }
                f.f[r.first[a] + j] = w;
            }
        }
        for (int a = r.axes; a < 3; a++) {
            r.first[a] = r.pairs;
            r.max[a] = 1;
        }
        r.cells = (int)cells;
        r.by1 = FastDiv(r.max[1]);
        r.by2 = FastDiv(r.max[2]);
        if (r.half && r.pairs % 8) return AC_ERR_UNSUPPORTED;
    }
    ac_layer *l = (ac_layer *)calloc(1, sizeof(ac_layer));
    if (!l) return AC_ERR_INVALID_ARG;
    l->cfg = g;
    l->rope = r;
    l->freq = f;
    l->elt = g.dtype == AC_BF16 ? 2 : 4;
    (void)cudaGetLastError();
    if (cudaGetDevice(&l->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&l->num_sms, cudaDevAttrMultiProcessorCount, l->device) != cudaSuccess ||
        cudaMalloc(&l->d_status, 8 * sizeof(int)) != cudaSuccess) {
        free(l);
        return AC_ERR_CUDA;
    }
    cudaDriverEntryPointQueryResult qr;
    // a call on a stream that does not wait for the default one must find zeros too
    if (cudaMemset(l->d_status, 0, 8 * sizeof(int)) != cudaSuccess || cudaStreamSynchronize(0) != cudaSuccess ||
        cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &l->encode_fn, cudaEnableDefault, &qr) != cudaSuccess ||
        qr != cudaDriverEntryPointSuccess || !l->encode_fn ||
        rope_setup(g.dtype, g.d, r.half, g.norm) || (g.page_size && g.dtype == AC_BF16 && cache_attn_setup(g.d))) {
        ac_layer_destroy(l);
        return AC_ERR_CUDA;
    }
    *out = l;
    return AC_OK;
}

void ac_layer_destroy(ac_layer *l) {
    if (!l) return;
    if (l->d_status) cudaFree(l->d_status);
    free(l);
}

ac_status ac_layer_workspace_size(const ac_layer *l, size_t *bytes) {
    if (!l || !bytes) return AC_ERR_INVALID_ARG;
    const size_t back = (size_t)back_ctas(l->num_sms) * 2 * l->cfg.d * sizeof(float);
    const size_t attn = l->cfg.page_size && l->cfg.dtype == AC_BF16 ? cache_attn_ws(l->num_sms, l->cfg.d) : 0;
    *bytes = (std::max(back, attn) + 255) & ~(size_t)255;
    return AC_OK;
}

ac_status ac_layer_get_status(ac_layer *l, void *stream) {
    if (!l) return AC_ERR_INVALID_ARG;
    const ac_status e = enter(l);
    if (e != AC_OK) return e;
    cudaStream_t st = (cudaStream_t)stream;
    int code = 0;
    if (cudaMemcpyAsync(&code, l->d_status, sizeof(int), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaMemsetAsync(l->d_status, 0, sizeof(int), st) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess)
        return AC_ERR_CUDA;
    return (ac_status)code;
}

ac_status ac_rope_table_size(const ac_layer *l, size_t *bytes) {
    if (!l || !bytes) return AC_ERR_INVALID_ARG;
    if (!l->rope.axes) return AC_ERR_UNSUPPORTED;
    *bytes = (size_t)table_pairs(l->rope) * sizeof(float2);
    return AC_OK;
}

ac_status ac_rope_table(ac_layer *l, float *table, void *stream) {
    if (!l || !table || !aligned16(table)) return AC_ERR_INVALID_ARG;
    if (!l->rope.axes) return AC_ERR_UNSUPPORTED;
    const ac_status e = enter(l);
    if (e != AC_OK) return e;
    k_rope_table(l->rope, l->freq, (float2 *)table, (cudaStream_t)stream);
    return leave();
}

ac_status ac_qk_norm_rope(ac_layer *l, int batch, int n, const float *table, const int32_t *pos,
                          int64_t pos_batch_stride, const ac_tensor *q, const void *w_q, const void *b_q,
                          const ac_tensor *q_out, const ac_tensor *k, const void *w_k, const void *b_k,
                          const ac_tensor *k_out, void *stream) {
    if (!l || batch < 0 || n < 0 || !q != !q_out || !k != !k_out) return AC_ERR_INVALID_ARG;
    if ((long long)batch * n > 0x3fffffffLL) return AC_ERR_UNSUPPORTED;
    RowArgs a;
    memset(&a, 0, sizeof(a));
    const ac_status re = rope_of(l, table, pos, pos_batch_stride, batch, a.rope);
    if (re != AC_OK) return re;
    const ac_tensor *in[2] = {q, k}, *out[2] = {q_out, k_out};
    const void *w[2] = {w_q, w_k}, *b[2] = {b_q, b_k};
    const int heads[2] = {l->cfg.heads, l->cfg.kv_heads}, d = l->cfg.d;
    for (int i = 0; i < 2; i++) {
        if (!in[i]) continue;
        if (batch && n &&
            (!view_ok(*in[i], batch, n, heads[i], d, l->elt, false) ||
             !view_ok(*out[i], batch, n, heads[i], d, l->elt, true) ||
             !alias_ok(*in[i], *out[i], batch, n, heads[i], d, l->elt)))
            return AC_ERR_INVALID_ARG;
        a.t[a.nt++] = RowTensor{view_of(*in[i]), view_of(*out[i]), w[i], b[i], heads[i], 0, 0};
    }
    const ac_status e = enter(l);
    if (e != AC_OK || !batch || !n || !a.nt) return e;
    a.batch = batch;
    a.n = n;
    a.by_n = FastDiv(n);
    a.norm = l->cfg.norm;
    a.w_f32 = l->cfg.w_dtype == AC_F32;
    a.eps = (float)l->cfg.eps;
    a.status = l->d_status;
    if (k_norm_rope(a, l->cfg.dtype, d, l->num_sms, (cudaStream_t)stream)) return AC_ERR_UNSUPPORTED;
    return leave();
}

ac_status ac_qk_norm_rope_backward(ac_layer *l, int batch, int n, const float *table, const int32_t *pos,
                                   int64_t pos_batch_stride, const ac_tensor *gq, const ac_tensor *q,
                                   const void *w_q, const ac_tensor *dq, void *dw_q, void *db_q, const ac_tensor *gk,
                                   const ac_tensor *k, const void *w_k, const ac_tensor *dk, void *dw_k, void *db_k,
                                   void *ws, size_t ws_bytes, void *stream) {
    if (!l || batch < 0 || n < 0 || !gq != !dq || !gk != !dk) return AC_ERR_INVALID_ARG;
    if ((long long)batch * n > 0x3fffffffLL) return AC_ERR_UNSUPPORTED;
    BackArgs a;
    memset(&a, 0, sizeof(a));
    const ac_status re = rope_of(l, table, pos, pos_batch_stride, batch, a.rope);
    if (re != AC_OK) return re;
    const bool norm = l->cfg.norm != AC_NORM_NONE;
    const ac_tensor *g[2] = {gq, gk}, *x[2] = {q, k}, *dx[2] = {dq, dk};
    const void *w[2] = {w_q, w_k};
    void *dw[2] = {dw_q, dw_k}, *db[2] = {db_q, db_k};
    const int heads[2] = {l->cfg.heads, l->cfg.kv_heads}, d = l->cfg.d;
    bool sums = false;
    for (int i = 0; i < 2; i++) {
        if (!g[i]) {
            if (dw[i] || db[i]) return AC_ERR_INVALID_ARG;
            continue;
        }
        if ((norm && !x[i]) || (!norm && (dw[i] || db[i]))) return AC_ERR_INVALID_ARG;
        if (batch && n) {
            if (!view_ok(*g[i], batch, n, heads[i], d, l->elt, false) ||
                !view_ok(*dx[i], batch, n, heads[i], d, l->elt, true) ||
                !alias_ok(*g[i], *dx[i], batch, n, heads[i], d, l->elt))
                return AC_ERR_INVALID_ARG;
            if (norm && (!view_ok(*x[i], batch, n, heads[i], d, l->elt, false) ||
                         !alias_ok(*x[i], *dx[i], batch, n, heads[i], d, l->elt)))
                return AC_ERR_INVALID_ARG;
        }
        sums = sums || dw[i] || db[i];
        a.t[i] = BackTensor{view_of(*g[i]), norm ? view_of(*x[i]) : View{nullptr, 0, 0, 0}, view_of(*dx[i]),
                            w[i], dw[i], db[i], heads[i]};
    }
    if (sums) {
        size_t need = 0;
        ac_layer_workspace_size(l, &need);
        if (!ws || !aligned16(ws) || ws_bytes < need) return AC_ERR_WORKSPACE;
    }
    const ac_status e = enter(l);
    if (e != AC_OK || (!gq && !gk)) return e;
    cudaStream_t st = (cudaStream_t)stream;
    if (!batch || !n) {
        const size_t wb = (size_t)d * (l->cfg.w_dtype == AC_F32 ? 4 : 2);
        for (int i = 0; i < 2; i++)
            if ((dw[i] && cudaMemsetAsync(dw[i], 0, wb, st) != cudaSuccess) ||
                (db[i] && cudaMemsetAsync(db[i], 0, wb, st) != cudaSuccess))
                return AC_ERR_CUDA;
        return AC_OK;
    }
    a.batch = batch;
    a.n = n;
    a.by_n = FastDiv(n);
    a.norm = l->cfg.norm;
    a.w_f32 = l->cfg.w_dtype == AC_F32;
    a.eps = (float)l->cfg.eps;
    a.part = sums ? (float *)ws : nullptr;
    a.status = l->d_status;
    if (k_norm_rope_back(a, l->cfg.dtype, d, l->num_sms, st)) return AC_ERR_UNSUPPORTED;
    return leave();
}

// The cache arguments that ac_cache_append and ac_cache_attn share.
static ac_status cache_ok(const ac_layer *l, int seqs, int tokens, const int32_t *q_start, const int32_t *kv_len,
                          const int32_t *block_table, int max_pages, int num_pages, const void *k_pages,
                          const void *v_pages) {
    if (!l || seqs < 0 || tokens < 0 || max_pages < 0 || num_pages < 0) return AC_ERR_INVALID_ARG;
    if (!l->cfg.page_size) return AC_ERR_UNSUPPORTED;
    if (seqs && (!q_start || !kv_len || (max_pages && !block_table))) return AC_ERR_INVALID_ARG;
    if (num_pages && (!k_pages || !v_pages || !aligned16(k_pages) || !aligned16(v_pages))) return AC_ERR_INVALID_ARG;
    if (tokens > 0x3fffffff || seqs > 0xffffff) return AC_ERR_UNSUPPORTED;
    // rows of a pool are addressed with 32-bit coordinates
    if ((long long)num_pages * l->cfg.kv_heads * l->cfg.page_size > 0x7fffffffLL) return AC_ERR_UNSUPPORTED;
    return AC_OK;
}

static int log2i(int v) {
    int r = 0;
    while ((1 << r) < v) r++;
    return r;
}

ac_status ac_cache_append(ac_layer *l, int seqs, int tokens, const int32_t *q_start, const int32_t *kv_len,
                          const int32_t *block_table, int max_pages, int num_pages, const float *table,
                          const int32_t *pos, const ac_tensor *k, const void *w_k, const void *b_k, const ac_tensor *v,
                          void *k_pages, void *v_pages, const ac_tensor *q, const void *w_q, const void *b_q,
                          const ac_tensor *q_out, void *stream) {
    const ac_status ce = cache_ok(l, seqs, tokens, q_start, kv_len, block_table, max_pages, num_pages, k_pages, v_pages);
    if (ce != AC_OK) return ce;
    if (!k || !v || !q != !q_out) return AC_ERR_INVALID_ARG;
    RowArgs a;
    memset(&a, 0, sizeof(a));
    const ac_status re = rope_of(l, table, pos, 0, 1, a.rope);
    if (re != AC_OK) return re;
    a.rope.line = a.rope.axes == 1;
    const int d = l->cfg.d, hk = l->cfg.kv_heads, hq = l->cfg.heads;
    if (tokens) {
        if (!view_ok(*k, 1, tokens, hk, d, l->elt, false) || !view_ok(*v, 1, tokens, hk, d, l->elt, false))
            return AC_ERR_INVALID_ARG;
        if (q && (!view_ok(*q, 1, tokens, hq, d, l->elt, false) || !view_ok(*q_out, 1, tokens, hq, d, l->elt, true) ||
                  !alias_ok(*q, *q_out, 1, tokens, hq, d, l->elt)))
            return AC_ERR_INVALID_ARG;
    }
    const ac_status e = enter(l);
    if (e != AC_OK || !seqs || !tokens) return e;
    const View kv{nullptr, 0, 0, l->cfg.page_size * d};
    View kp = kv, vp = kv;
    kp.p = k_pages;
    vp.p = v_pages;
    if (q) a.t[a.nt++] = RowTensor{view_of(*q), view_of(*q_out), w_q, b_q, hq, 0, 0};
    a.t[a.nt++] = RowTensor{view_of(*k), kp, w_k, b_k, hk, 0, 1};
    a.t[a.nt++] = RowTensor{view_of(*v), vp, nullptr, nullptr, hk, 1, 1};
    a.batch = 1;
    a.n = tokens;
    a.by_n = FastDiv(tokens);
    a.norm = l->cfg.norm;
    a.w_f32 = l->cfg.w_dtype == AC_F32;
    a.eps = (float)l->cfg.eps;
    a.status = l->d_status;
    a.page = PageArgs{q_start, kv_len, block_table, seqs, max_pages, num_pages, log2i(l->cfg.page_size), hk};
    if (k_norm_rope(a, l->cfg.dtype, d, l->num_sms, (cudaStream_t)stream)) return AC_ERR_UNSUPPORTED;
    return leave();
}

ac_status ac_cache_attn(ac_layer *l, int seqs, int tokens, int max_q, int max_kv, const int32_t *q_start,
                        const int32_t *kv_len, const int32_t *block_table, int max_pages, int num_pages,
                        const ac_tensor *q, const void *k_pages, const void *v_pages, const ac_tensor *out, float *lse,
                        void *ws, size_t ws_bytes, void *stream) {
    const ac_status ce = cache_ok(l, seqs, tokens, q_start, kv_len, block_table, max_pages, num_pages, k_pages, v_pages);
    if (ce != AC_OK) return ce;
    if (l->cfg.dtype != AC_BF16) return AC_ERR_UNSUPPORTED;
    if (!q || !out || max_q < 0 || max_kv < 0) return AC_ERR_INVALID_ARG;
    const int d = l->cfg.d, hq = l->cfg.heads;
    if (tokens && (!view_ok(*q, 1, tokens, hq, d, l->elt, false) || !view_ok(*out, 1, tokens, hq, d, l->elt, true) ||
                   !alias_ok(*q, *out, 1, tokens, hq, d, l->elt)))
        return AC_ERR_INVALID_ARG;
    // query tiles are tensor-map boxes of whole groups
    if (hq / l->cfg.kv_heads > 128 || (tokens > 1 && !q->token_stride) || (hq > 1 && !q->head_stride))
        return AC_ERR_UNSUPPORTED;
    size_t need = 0;
    ac_layer_workspace_size(l, &need);
    if (!ws || !aligned16(ws) || ws_bytes < need) return AC_ERR_WORKSPACE;
    const ac_status e = enter(l);
    if (e != AC_OK || !seqs || !tokens || !max_q) return e;
    CacheAttnArgs a;
    memset(&a, 0, sizeof(a));
    a.seqs = seqs;
    a.tokens = tokens;
    a.max_q = std::min(max_q, tokens);
    // no page can hold a key beyond these; the end of a chunk or tile of keys that
    // begins below MAX_KEYS is a 32-bit number too
    constexpr int MAX_KEYS = 0x7fff0000;
    a.max_kv = num_pages ? (int)std::min<long long>(std::min(max_kv, MAX_KEYS), (long long)max_pages * l->cfg.page_size) : 0;
    a.heads = hq;
    a.kv_heads = l->cfg.kv_heads;
    a.group = hq / l->cfg.kv_heads;
    a.D = d;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.page_log2 = log2i(l->cfg.page_size);
    a.causal_block = l->cfg.causal_block;
    a.window = l->cfg.window;
    a.scale_log2 = (float)((l->cfg.scale > 0.0 ? l->cfg.scale : 1.0 / sqrt((double)d)) * 1.4426950408889634);
    a.q_start = q_start;
    a.kv_len = kv_len;
    a.block_table = block_table;
    a.q = view_of(*q);
    a.out = view_of(*out);
    a.kp = k_pages;
    a.vp = v_pages;
    a.lse = lse;
    a.status = l->d_status;
    a.counters = l->d_status + 2;
    a.ws = ws;
    if (k_cache_attn(a, l->num_sms, l->encode_fn, (cudaStream_t)stream)) return AC_ERR_UNSUPPORTED;
    return leave();
}

}  // extern "C"
