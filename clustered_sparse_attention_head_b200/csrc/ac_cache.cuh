// What the two kernels of the cache attention share (ac_cache_attn.cu: tiles of
// 128 rows on tcgen05; ac_cache_decode.cu: up to 16 rows).
#pragma once
#include "ac_layer.cuh"

namespace ac {

// Cluster size with which the kernel for few rows takes this call, 0: it does not.
int decode_cluster(const CacheAttnArgs &a, int num_sms);
int k_cache_decode(const CacheAttnArgs &a, int cluster, cudaStream_t st);
int cache_decode_setup(int D);

namespace {

// Keys [lo, hi) that a token at position p sees of a sequence of `len` keys.
__device__ __forceinline__ void key_range(const CacheAttnArgs &a, int p, int len, int &lo, int &hi) {
    hi = len;
    lo = 0;
    if (a.causal_block) {
        const long long e = p < 0 ? 0 : ((long long)(p / a.causal_block) + 1) * a.causal_block;
        hi = (int)min((long long)len, e);
    }
    if (a.window) lo = (int)max(0LL, (long long)p - a.window + 1);
}

// Sequence s: its rows (cut to the tensor and to max_q), the position of its
// first new token and its keys.
__device__ __forceinline__ void sequence(const CacheAttnArgs &a, int s, int &row0, int &nq, int &p0, int &len, bool report) {
    const int s0 = __ldg(a.q_start + s), s1 = __ldg(a.q_start + s + 1);
    len = __ldg(a.kv_len + s);
    p0 = len - (s1 - s0);
    row0 = max(0, s0);
    nq = max(0, min(s1, a.tokens) - row0);
    p0 += row0 - s0;
    bool bad = s0 < 0 || s1 > a.tokens || s1 < s0;
    if (nq > a.max_q) {
        nq = a.max_q;
        bad = true;
    }
    if (len < 0 || len > a.max_kv) {
        len = len < 0 ? 0 : a.max_kv;
        bad = true;
    }
    if (bad && report) set_status(a.status, ST_INVALID);
}

// 2^(a - b), 0 for a = -inf also when b is
__device__ __forceinline__ float weight(float a, float b) { return a == -INFINITY ? 0.f : ex2_approx(a - b); }

}  // namespace
}  // namespace ac
