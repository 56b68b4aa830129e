// Internal interface of the calls around the attention (ac_layer_*): argument
// blocks of the kernels in ac_rope.cu and ac_cache_attn.cu.
#pragma once
#include "ac_kernels.cuh"

namespace ac {

// [batch, token, head, d] view: data and strides in elements (token and head
// strides below 2^31).
struct View {
    const void *p;
    long long sb;
    int sn, sh;
};

// n / d for 0 <= n < 2^31 by a multiplication: with l = ceil(log2 d) and m =
// floor(2^32 (2^l - d) / d) + 1, n / d = (mulhi(n, m) + n) >> l (Granlund and
// Montgomery, "Division by Invariant Integers using Multiplication", 1994).
struct FastDiv {
    uint32_t d, m, l;
    FastDiv() = default;
    explicit FastDiv(uint32_t d_) : d(d_), l(0) {
        while ((1ull << l) < d) l++;
        m = (uint32_t)((((1ull << l) - d) << 32) / d + 1);
    }
    __device__ __forceinline__ int div(int n) const { return (int)((__umulhi((uint32_t)n, m) + (uint32_t)n) >> l); }
};

// Pair ranges and table offsets of the rotation's axes.
struct RopeArgs {
    int axes;             // 0 = no rotation
    int pairs;            // R / 2
    int half;             // layout
    int first[3], np[3];  // first pair and number of pairs of each axis
    int max[3];           // positions of each axis
    uint32_t off[3];      // first (cos, sin) of each axis in the table
    int cells;            // product of max, at most 2^31 - 1: tokens of the implicit grid
    int line;             // 1: the implicit tokens are a stream of one axis, recorded at or beyond cells
    FastDiv by1, by2;     // by max[1] and max[2]
    const float2 *table;
    const int32_t *pos;   // NULL: row-major coordinates of the token's index
    long long pos_batch;  // elements between the samples' position blocks
};

enum { NORM_NONE = 0, NORM_RMS = 1, NORM_LAYER = 2 };

// One tensor of the norm and rotation: x [token, head] rows to y.
struct RowTensor {
    View x, y;
    const void *w, *b;  // [d] in the weights' type, or NULL
    int heads;
    int copy;           // 1: rows are copied (values on the way into the cache)
    int paged;          // 1: y is a cache pool
};

// Where the new tokens of a paged cache go.
struct PageArgs {
    const int32_t *q_start, *kv_len, *block_table;
    int seqs, max_pages, num_pages, page_log2, kv_heads;
};

struct RowArgs {
    RowTensor t[3];
    int nt;
    int batch, n;      // tokens = batch * n rows of heads
    FastDiv by_n;
    int norm, w_f32;
    float eps;
    RopeArgs rope;
    PageArgs page;     // seqs = 0: dense
    int *status;
};

struct BackTensor {
    View g, x, dx;
    const void *w;
    void *dw, *db;
    int heads;
};
struct BackArgs {
    BackTensor t[2];
    int batch, n;
    FastDiv by_n;
    int norm, w_f32;
    float eps;
    RopeArgs rope;
    int ctas[2];       // CTAs of each tensor
    int run;           // heads per item
    FastDiv by_runs[2];  // by the items of a tile, per tensor
    float *part;       // [ctas, 2, d] partial sums of dw and db
    int *status;
};

// Freq of every pair (double) and the factor on cosine and sine.
struct FreqArgs {
    double f[64];
    double mag;
};

// A kernel that reads what the one before it on the stream wrote, launched while
// that one still runs: it begins with after_previous(), which waits for it.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
void launch_after(void (*fn)(P...), unsigned grid, unsigned block, cudaStream_t st, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.stream = st;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    // an error stays pending for the caller's check
    if (cudaLaunchKernelEx(&cfg, fn, P(args)...) == cudaSuccess) note_launch();
}

// ---- ac_rope.cu
void k_rope_table(const RopeArgs &r, const FreqArgs &f, float2 *table, cudaStream_t st);
// the forward kernel's shared-memory attribute on the current device: once per layer
int rope_setup(int dtype, int D, int half, int norm);
int k_norm_rope(const RowArgs &a, int dtype, int D, int num_sms, cudaStream_t st);
// upper bound on ctas[0] + ctas[1] of k_norm_rope_back
int back_ctas(int num_sms);
int k_norm_rope_back(BackArgs &a, int dtype, int D, int num_sms, cudaStream_t st);

// ---- ac_cache_attn.cu
struct CacheAttnArgs {
    int seqs, tokens, max_q, max_kv, heads, kv_heads, group, D;
    int max_pages, num_pages, page_log2;
    int causal_block, window;
    float scale_log2;  // scale * log2(e)
    const int32_t *q_start, *kv_len, *block_table;
    View q, out;
    const void *kp, *vp;
    float *lse;
    int *status;
    int *counters;     // two words of the layer, 0 between calls
    void *ws;
};
// the kernel's attributes on the current device: once per layer
int cache_attn_setup(int D);
size_t cache_attn_ws(int num_sms, int D);
int k_cache_attn(const CacheAttnArgs &a, int num_sms, void *encode_fn, cudaStream_t st);

}  // namespace ac
