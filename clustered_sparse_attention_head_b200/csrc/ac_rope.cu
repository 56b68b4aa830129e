// Per-head norm and rotary position of queries and keys, their gradients, and
// the same on the way into a paged cache.
//
// Row of a head: x [d] -> n = (x - [mean]) r, r = 1 / sqrt(mean(.^2) + eps)
// -> n w + b -> pairs (a, b) turned by the token's angle:
//    (a cos - b sin, a sin + b cos).
// Bound by memory: each row is read once and written once, about 60
// instructions per 16 bytes.  A group of G lanes (16 bytes each) holds one row
// in registers, so the statistics are xor shuffles within the group; it keeps
// one token's cosines, sines and the weights and takes HC heads of that token,
// so the table's 8 bytes per pair are read once per HC rows and HC loads of 16
// bytes are in flight per lane.
#include "ac_layer.cuh"

namespace ac {
namespace {

constexpr int NT = 256;

// 16 bytes of a row as floats and back (round to nearest even).
template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void get(const uint4 &u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x);
        x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z);
        x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(const uint4 &u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<uint32_t *>(&b);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <int G> __device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// V elements of a weight vector from element e.
template <int V> __device__ __forceinline__ void load_w(const void *w, int f32, int e, float dflt, float (&x)[V]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < V; i++) x[i] = dflt;
    } else if (f32) {
#pragma unroll
        for (int i = 0; i < V; i++) x[i] = __ldg((const float *)w + e + i);
    } else {
#pragma unroll
        for (int i = 0; i < V; i++) x[i] = __bfloat162float(((const __nv_bfloat16 *)w)[e + i]);
    }
}

// Coordinates of a token.  `index` is its place in its sample or sequence, `at`
// its first element of explicit positions.  Returns false when it is not rotated.
__device__ __forceinline__ bool token_pos(const RopeArgs &r, long long at, int index, int (&p)[3], int *status) {
    p[0] = p[1] = p[2] = 0;
    if (r.axes == 0) return false;
    if (!r.pos) {
        if (index >= r.cells) return false;
        if (r.axes == 1) {
            p[0] = index;
        } else if (r.axes == 2) {
            p[0] = index / r.max[1];
            p[1] = index - p[0] * r.max[1];
        } else {
            const int ab = index / r.max[2];
            p[2] = index - ab * r.max[2];
            p[0] = ab / r.max[1];
            p[1] = ab - p[0] * r.max[1];
        }
        return true;
    }
    bool on = true;
#pragma unroll
    for (int a = 0; a < 3; a++)
        if (a < r.axes) {
            p[a] = __ldg(r.pos + at + a);
            on = on && p[a] >= 0;
        }
    if (on) {
#pragma unroll
        for (int a = 0; a < 3; a++)
            if (a < r.axes && p[a] >= r.max[a]) {
                p[a] = r.max[a] - 1;
                set_status(status, ST_INVALID);
            }
    }
    return on;
}

// Cosine and sine of this lane's pairs: V/2 pairs (2i, 2i + 1) when
// interleaved, one per element when half.  e is the lane's first element.
template <int V, bool HALF> struct Angles {
    static constexpr int N = HALF ? V : V / 2;
    float c[N], s[N];
    uint32_t on;  // bit i: pair i is rotated
    __device__ __forceinline__ void load(const RopeArgs &r, int e, bool rotated, const int (&p)[3]) {
        on = 0;
        const int first = HALF ? (e < r.pairs ? e : e - r.pairs) : e / 2;
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int q = first + i;
            c[i] = 1.f;
            s[i] = 0.f;
            if (rotated && q < r.pairs) {
                const int a = q < r.first[1] ? 0 : (q < r.first[2] ? 1 : 2);
                const int pa = a == 0 ? p[0] : (a == 1 ? p[1] : p[2]);
                const int fa = a == 0 ? 0 : (a == 1 ? r.first[1] : r.first[2]);
                const int na = a == 0 ? r.np[0] : (a == 1 ? r.np[1] : r.np[2]);
                const long long oa = a == 0 ? 0 : (a == 1 ? r.off[1] : r.off[2]);
                const float2 t = __ldg(r.table + oa + (long long)pa * na + (q - fa));
                c[i] = t.x;
                s[i] = t.y;
                on |= 1u << i;
            }
        }
    }
    // x turned by the angles, or back (sign = -1).  All lanes of the warp call
    // it; G lanes hold a row.  A pair that is not rotated keeps its elements
    // (not x * 1 - y * 0: y may be infinite).
    template <int G> __device__ __forceinline__ void turn(const RopeArgs &r, int e, float sign, float (&x)[V]) const {
        if (HALF) {
            // the partner element lies pairs / V lanes up (first half) or down
            const int step = r.pairs / V;
            const bool lower = e < r.pairs;
            const int lane = threadIdx.x & 31;
            const int src = lower ? lane + step : lane - step;
            const float sg = lower ? -sign : sign;
#pragma unroll
            for (int i = 0; i < V; i++) {
                const float y = __shfl_sync(0xffffffffu, x[i], src);
                if (on >> i & 1u) x[i] = x[i] * c[i] + sg * s[i] * y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; i++) {
                const float a = x[2 * i], b = x[2 * i + 1], si = sign * s[i];
                if (on >> i & 1u) {
                    x[2 * i] = a * c[i] - b * si;
                    x[2 * i + 1] = a * si + b * c[i];
                }
            }
        }
    }
};

// x -> (x - mean) r in place; returns r.
template <int V, int G> __device__ __forceinline__ float normalise(int norm, float eps, float (&x)[V]) {
    constexpr float inv_d = 1.f / (V * G);
    if (norm == NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < V; i++) s += x[i];
        const float mean = group_sum<G>(s) * inv_d;
#pragma unroll
        for (int i = 0; i < V; i++) x[i] -= mean;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; i++) s += x[i] * x[i];
    const float r = 1.f / sqrtf(group_sum<G>(s) * inv_d + eps);
#pragma unroll
    for (int i = 0; i < V; i++) x[i] *= r;
    return r;
}

// The sequence of a stacked row (binary search over q_start, every index within
// [0, seqs]) and its place in it; false for rows outside every sequence.
__device__ __forceinline__ bool find_seq(const PageArgs &g, int row, int &seq, int &place) {
    int lo = 0, hi = g.seqs;  // q_start[lo] <= row < q_start[hi], once checked
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(g.q_start + mid) <= row)
            lo = mid;
        else
            hi = mid;
    }
    const int a = __ldg(g.q_start + lo), b = __ldg(g.q_start + lo + 1);
    seq = lo;
    place = __ldg(g.kv_len + lo) - (b - a) + (row - a);
    return row >= a && row < b;
}

template <typename T, int D, bool HALF, int HC>
__global__ void __launch_bounds__(NT) norm_rope_kernel(const __grid_constant__ RowArgs a) {
    constexpr int V = Vec<T>::N, G = D / V, TOK = NT / G;
    // chunk = HC heads of one of the tensors
    int chunk = blockIdx.x, ti = 0;
    int total = 0;
#pragma unroll
    for (int i = 0; i < 3; i++)
        if (i < a.nt) total += (a.t[i].heads + HC - 1) / HC;
    const long long tile = chunk / total;
    chunk -= (int)tile * total;
    while (chunk >= (a.t[ti].heads + HC - 1) / HC) chunk -= (a.t[ti++].heads + HC - 1) / HC;
    const RowTensor &t = a.t[ti];
    const int h0 = chunk * HC, nh = min(HC, t.heads - h0);
    const int e = (threadIdx.x % G) * V;
    const long long tok = tile * TOK + threadIdx.x / G;
    bool live = tok < (long long)a.batch * a.n;
    const int b = live ? (int)(tok / a.n) : 0;
    const int i = live ? (int)(tok - (long long)b * a.n) : 0;

    int index = i;
    long long base = b * t.y.sb + i * t.y.sn;  // first element of the token's output rows
    bool store = live;
    if (a.page.seqs) {
        int seq = 0, place = 0;
        live = live && find_seq(a.page, i, seq, place);
        store = live;
        index = place;
        if (live && (place < 0 || (place >> a.page.page_log2) >= a.page.max_pages)) {
            set_status(a.status, ST_INVALID);
            store = !t.paged;
            index = place < 0 ? 0 : place;
        } else if (live && t.paged) {
            const int page = __ldg(a.page.block_table + (long long)seq * a.page.max_pages + (place >> a.page.page_log2));
            if (page < 0 || page >= a.page.num_pages) {
                set_status(a.status, ST_INVALID);
                store = false;
            } else {
                base = (((long long)page * a.page.kv_heads) << a.page.page_log2) * D +
                       (long long)(place & ((1 << a.page.page_log2) - 1)) * D;
            }
        }
    }
    const T *x = (const T *)t.x.p + b * t.x.sb + i * t.x.sn + h0 * t.x.sh + e;
    T *y = (T *)t.y.p + base + h0 * t.y.sh + e;
    uint4 u[HC];
#pragma unroll
    for (int h = 0; h < HC; h++) {
        u[h] = make_uint4(0u, 0u, 0u, 0u);
        if (live && h < nh) u[h] = __ldg((const uint4 *)(x + h * t.x.sh));
    }
    if (!t.copy) {
        int p[3];
        const bool rotated = live && token_pos(a.rope, b * a.rope.pos_batch + (long long)i * a.rope.axes, index, p, a.status);
        Angles<V, HALF> ang;
        ang.load(a.rope, e, rotated, p);
        float w[V], bias[V];
        if (a.norm != NORM_NONE) {
            load_w<V>(t.w, a.w_f32, e, 1.f, w);
            load_w<V>(t.b, a.w_f32, e, 0.f, bias);
        }
#pragma unroll
        for (int h = 0; h < HC; h++) {
            float v[V];
            Vec<T>::get(u[h], v);
            if (a.norm != NORM_NONE) {
                normalise<V, G>(a.norm, a.eps, v);
#pragma unroll
                for (int k = 0; k < V; k++) v[k] = v[k] * w[k] + bias[k];
            }
            if (a.rope.axes) ang.template turn<G>(a.rope, e, 1.f, v);
            u[h] = Vec<T>::put(v);
        }
    }
#pragma unroll
    for (int h = 0; h < HC; h++)
        if (store && h < nh) *(uint4 *)(y + h * t.y.sh) = u[h];
}

// Gradients.  A group takes HC heads of one token at a time, like the forward
// kernel, and the CTA walks its share of (token tile, head chunk) items, so
// that each lane sums its elements' dw and db over all of them in registers;
// the CTA's sums go to part[cta] and back_sum_kernel adds the CTAs in order.
template <typename T, int D, bool HALF, int HC>
__global__ void __launch_bounds__(NT) norm_rope_back_kernel(const __grid_constant__ BackArgs a) {
    constexpr int V = Vec<T>::N, G = D / V, TOK = NT / G;
    __shared__ float red[2][TOK][D];
    const int ti = (int)blockIdx.x < a.ctas[0] ? 0 : 1;
    const int cta = blockIdx.x - (ti ? a.ctas[0] : 0);
    const BackTensor &t = a.t[ti];
    const int grp = threadIdx.x / G, e = (threadIdx.x % G) * V;
    const long long tokens = (long long)a.batch * a.n;
    const int chunks = (t.heads + HC - 1) / HC;
    const long long items = (tokens + TOK - 1) / TOK * chunks;
    float w[V], dw[V], db[V];
    load_w<V>(t.w, a.w_f32, e, 1.f, w);
#pragma unroll
    for (int k = 0; k < V; k++) dw[k] = db[k] = 0.f;
    for (long long it = cta; it < items; it += a.ctas[ti]) {
        const long long tile = it / chunks;
        const int h0 = (int)(it - tile * chunks) * HC, nh = min(HC, t.heads - h0);
        const long long tok = tile * TOK + grp;
        const bool live = tok < tokens;
        const int b = live ? (int)(tok / a.n) : 0;
        const int i = live ? (int)(tok - (long long)b * a.n) : 0;
        const T *g = (const T *)t.g.p + b * t.g.sb + i * t.g.sn + h0 * t.g.sh + e;
        const T *x = (const T *)t.x.p + b * t.x.sb + i * t.x.sn + h0 * t.x.sh + e;
        T *dx = (T *)t.dx.p + b * t.dx.sb + i * t.dx.sn + h0 * t.dx.sh + e;
        uint4 ug[HC], ux[HC];
#pragma unroll
        for (int h = 0; h < HC; h++) {
            ug[h] = ux[h] = make_uint4(0u, 0u, 0u, 0u);
            if (live && h < nh) {
                ug[h] = __ldg((const uint4 *)(g + h * t.g.sh));
                if (a.norm != NORM_NONE) ux[h] = __ldg((const uint4 *)(x + h * t.x.sh));
            }
        }
        int p[3];
        const bool rotated = live && token_pos(a.rope, b * a.rope.pos_batch + (long long)i * a.rope.axes, i, p, a.status);
        Angles<V, HALF> ang;
        ang.load(a.rope, e, rotated, p);
#pragma unroll
        for (int h = 0; h < HC; h++) {
            float gv[V];
            Vec<T>::get(ug[h], gv);
            if (a.rope.axes) ang.template turn<G>(a.rope, e, -1.f, gv);
            if (a.norm != NORM_NONE) {
                float xv[V];
                Vec<T>::get(ux[h], xv);
                const float r = normalise<V, G>(a.norm, a.eps, xv);
                float m1 = 0.f, m2 = 0.f;
                const bool in = live && h < nh;
#pragma unroll
                for (int k = 0; k < V; k++) {
                    if (in) {
                        dw[k] += gv[k] * xv[k];
                        db[k] += gv[k];
                    }
                    gv[k] *= w[k];
                    m1 += gv[k];
                    m2 += gv[k] * xv[k];
                }
                m2 = group_sum<G>(m2) * (1.f / D);
                m1 = a.norm == NORM_LAYER ? group_sum<G>(m1) * (1.f / D) : 0.f;
#pragma unroll
                for (int k = 0; k < V; k++) gv[k] = r * (gv[k] - m1 - xv[k] * m2);
            }
            if (live && h < nh) *(uint4 *)(dx + h * t.dx.sh) = Vec<T>::put(gv);
        }
    }
    if (!a.part) return;
#pragma unroll
    for (int k = 0; k < V; k++) {
        red[0][grp][e + k] = dw[k];
        red[1][grp][e + k] = db[k];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * D; c += NT) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < TOK; k++) s += red[c / D][k][c % D];
        a.part[(size_t)blockIdx.x * 2 * D + c] = s;
    }
}

// Block (tensor, dw or db): the CTAs' partial sums in order, in double.
__global__ void __launch_bounds__(1024) back_sum_kernel(const __grid_constant__ BackArgs a, int D) {
    __shared__ double red[1024];
    const int ti = blockIdx.x >> 1, which = blockIdx.x & 1;
    const BackTensor &t = a.t[ti];
    void *out = which ? t.db : t.dw;
    if (!out) return;
    const int slices = 1024 / D, c = threadIdx.x % D, sl = threadIdx.x / D;
    const float *part = a.part + (size_t)(ti ? a.ctas[0] : 0) * 2 * D + which * D + c;
    double s = 0.0;
    for (int i = sl; i < a.ctas[ti]; i += slices) s += (double)part[(size_t)i * 2 * D];
    red[threadIdx.x] = s;
    __syncthreads();
    if (sl == 0) {
        for (int k = 1; k < slices; k++) s += red[k * D + c];
        if (a.w_f32)
            ((float *)out)[c] = (float)s;
        else
            ((__nv_bfloat16 *)out)[c] = __float2bfloat16((float)s);
    }
}

__global__ void rope_table_kernel(const __grid_constant__ RopeArgs r, const __grid_constant__ FreqArgs f, float2 *table,
                                  long long total) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= total) return;
    int a = 0;
    while (a + 1 < r.axes && i >= r.off[a + 1]) a++;
    const long long k = i - r.off[a];
    const int p = (int)(k / r.np[a]), j = (int)(k - (long long)p * r.np[a]);
    double s, c;
    sincos((double)p * f.f[r.first[a] + j], &s, &c);
    table[i] = make_float2((float)(c * f.mag), (float)(s * f.mag));
}

template <typename T, int D, bool HALF, int HC> int launch_rows(const RowArgs &a, cudaStream_t st) {
    constexpr int TOK = NT / (D / Vec<T>::N);
    long long chunks = 0;
    for (int i = 0; i < a.nt; i++) chunks += (a.t[i].heads + HC - 1) / HC;
    const long long grid = ((long long)a.batch * a.n + TOK - 1) / TOK * chunks;
    if (grid > 0x7fffffffLL) return -1;
    norm_rope_kernel<T, D, HALF, HC><<<(unsigned)grid, NT, 0, st>>>(a);
    note_launch();
    return 0;
}
// HC = 1 where HC = 8 would leave SMs without a CTA (few tokens): more groups
// at work on the same rows.
template <typename T, int D> int launch_rows_d(const RowArgs &a, int num_sms, cudaStream_t st) {
    constexpr int TOK = NT / (D / Vec<T>::N);
    long long chunks = 0;
    for (int i = 0; i < a.nt; i++) chunks += (a.t[i].heads + 7) / 8;
    const bool many = ((long long)a.batch * a.n + TOK - 1) / TOK * chunks >= 2 * num_sms;
    if (a.rope.half) return many ? launch_rows<T, D, true, 8>(a, st) : launch_rows<T, D, true, 1>(a, st);
    return many ? launch_rows<T, D, false, 8>(a, st) : launch_rows<T, D, false, 1>(a, st);
}

template <typename T, int D> void launch_back(const BackArgs &a, cudaStream_t st) {
    const int grid = a.ctas[0] + a.ctas[1];
    if (a.rope.half)
        norm_rope_back_kernel<T, D, true, 2><<<grid, NT, 0, st>>>(a);
    else
        norm_rope_back_kernel<T, D, false, 2><<<grid, NT, 0, st>>>(a);
    note_launch();
}

}  // namespace

void k_rope_table(const RopeArgs &r, const FreqArgs &f, float2 *table, cudaStream_t st) {
    const long long total = r.off[r.axes - 1] + (long long)r.max[r.axes - 1] * r.np[r.axes - 1];
    rope_table_kernel<<<(unsigned)((total + 255) / 256), 256, 0, st>>>(r, f, table, total);
    note_launch();
}

int k_norm_rope(const RowArgs &a, int dtype, int D, int num_sms, cudaStream_t st) {
    if (dtype == DT_BF16)
        return D == 64 ? launch_rows_d<__nv_bfloat16, 64>(a, num_sms, st)
                       : launch_rows_d<__nv_bfloat16, 128>(a, num_sms, st);
    return D == 64 ? launch_rows_d<float, 64>(a, num_sms, st) : launch_rows_d<float, 128>(a, num_sms, st);
}

int back_ctas(int num_sms) { return 2 * num_sms + 2; }

int k_norm_rope_back(BackArgs &a, int dtype, int D, int num_sms, cudaStream_t st) {
    // the tensors' CTAs in proportion to their heads
    const int total = 2 * num_sms, h0 = a.t[0].heads, h1 = a.t[1].heads;
    a.ctas[0] = h0 ? max(1, (int)((long long)total * h0 / (h0 + h1))) : 0;
    a.ctas[1] = h1 ? max(1, total - a.ctas[0]) : 0;
    if (dtype == DT_BF16) {
        if (D == 64) launch_back<__nv_bfloat16, 64>(a, st);
        else launch_back<__nv_bfloat16, 128>(a, st);
    } else {
        if (D == 64) launch_back<float, 64>(a, st);
        else launch_back<float, 128>(a, st);
    }
    if (a.part) {
        back_sum_kernel<<<4, 1024, 0, st>>>(a, D);
        note_launch();
    }
    return 0;
}

}  // namespace ac
