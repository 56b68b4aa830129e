// Attention of the newest tokens of ragged sequences over a paged cache of keys
// and values, bf16.
//
// out_i = sum_j w_ij v_j / sum_j w_ij, w_ij = 2^(c q_i.k_j - m_i), c = scale
// log2(e), in one pass over the keys with the running maximum m_i and sum.
// One warp per (token, head): a lane holds D / 32 elements of q and of the sum.
#include "ac_layer.cuh"

namespace ac {
namespace {

template <int D> __global__ void __launch_bounds__(128) cache_attn_kernel(const __grid_constant__ CacheAttnArgs a) {
    constexpr int E = D / 32;
    const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (w >= (long long)a.tokens * a.heads) return;
    const int row = (int)(w / a.heads), h = (int)(w - (long long)row * a.heads);
    int lo = 0, hi = a.seqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.q_start + mid) <= row) lo = mid; else hi = mid;
    }
    const int s0 = __ldg(a.q_start + lo), s1 = __ldg(a.q_start + lo + 1);
    if (row < s0 || row >= s1) return;
    int len = __ldg(a.kv_len + lo);
    const int p = len - (s1 - s0) + (row - s0);
    const long long cap = min((long long)a.max_kv, (long long)a.max_pages << a.page_log2);
    if (row - s0 >= a.max_q || len < 0 || len > cap) {
        set_status(a.status, ST_INVALID);
        if (row - s0 >= a.max_q) return;
        len = len < 0 ? 0 : (int)cap;
    }
    int end = len, begin = 0;
    if (a.causal_block) {
        const long long e = p < 0 ? 0 : ((long long)p / a.causal_block + 1) * a.causal_block;
        end = (int)min((long long)len, e);
    }
    if (a.window) begin = (int)max(0LL, (long long)p - a.window + 1);
    const __nv_bfloat16 *q = (const __nv_bfloat16 *)a.q.p + row * a.q.sn + h * a.q.sh;
    __nv_bfloat16 *o = (__nv_bfloat16 *)a.out.p + row * a.out.sn + h * a.out.sh;
    float qv[E], acc[E];
#pragma unroll
    for (int i = 0; i < E; i++) {
        qv[i] = __bfloat162float(q[lane * E + i]) * a.scale_log2;
        acc[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    const int kvh = h / a.group;
    for (int j = begin; j < end; j++) {
        int page = __ldg(a.block_table + (long long)lo * a.max_pages + (j >> a.page_log2));
        if (page < 0 || page >= a.num_pages) {
            set_status(a.status, ST_INVALID);
            page = page < 0 ? 0 : a.num_pages - 1;
        }
        const long long r = ((((long long)page * a.kv_heads + kvh) << a.page_log2) + (j & ((1 << a.page_log2) - 1))) * D;
        const __nv_bfloat16 *k = (const __nv_bfloat16 *)a.kp + r, *v = (const __nv_bfloat16 *)a.vp + r;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < E; i++) s += qv[i] * __bfloat162float(k[lane * E + i]);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        const float mn = fmaxf(m, s);
        const float f = mn == -INFINITY ? 1.f : exp2f(m - mn), w2 = mn == -INFINITY ? 0.f : exp2f(s - mn);
        m = mn;
        l = l * f + w2;
#pragma unroll
        for (int i = 0; i < E; i++) acc[i] = acc[i] * f + w2 * __bfloat162float(v[lane * E + i]);
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
    for (int i = 0; i < E; i++) o[lane * E + i] = __float2bfloat16(acc[i] * inv);
    if (a.lse && lane == 0) a.lse[w] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace

size_t cache_attn_ws(int, int) { return 0; }

int k_cache_attn(const CacheAttnArgs &a, int, void *, cudaStream_t st) {
    const long long grid = ((long long)a.tokens * a.heads + 3) / 4;
    if (grid > 0x7fffffffLL) return -1;
    if (a.D == 64)
        cache_attn_kernel<64><<<(unsigned)grid, 128, 0, st>>>(a);
    else
        cache_attn_kernel<128><<<(unsigned)grid, 128, 0, st>>>(a);
    note_launch();
    return 0;
}

}  // namespace ac
