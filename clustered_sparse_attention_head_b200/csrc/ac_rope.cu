// Per-head norm and rotary position of queries and keys, their gradients, and
// the same on the way into a paged cache.
//
// Row of a head: x [d] -> n = (x - [mean]) r, r = 1 / sqrt(mean(.^2) + eps)
// -> n w + b -> pairs (a, b) turned by the token's angle:
//    (a cos - b sin, a sin + b cos).
// Bound by memory (each row is read once and written once) and, close behind it,
// by issue slots.  A group of G lanes (16 bytes each) holds one row in registers,
// so the statistics are xor shuffles within the group.  It takes one token at a
// time, with weight, bias, cosine and sine folded into coefficients once for a run
// of heads: y = r (x ca + x' cb) + rb with x' the pair's other element.
// 75,600 tokens x 40 heads of q and k, d = 128, bf16: 502 to 559 us on several B200s, 6.2 to
// 5.5 TB/s (0.94 to 0.84 of the measured copy rate; the faster end leaves the last of
// the output in L2); gradients of 2 x 17,776 tokens x 30 heads, d = 64: 153 to 168 us,
// 5.3 to 4.9 TB/s.
#include "ac_layer.cuh"
#include "ac_softmax.cuh"

namespace ac {
namespace {

constexpr int NT = 256;                  // threads of a CTA
constexpr int FWD_HC = 8, FWD_CTAS = 3;  // heads of a run, CTAs an SM
// heads of a step, steps of the ring, CTAs an SM, heads of a run at most
constexpr int BACK_HC = 4, BACK_STEPS = 3, BACK_CTAS = 2, BACK_MOST = 32;

// Packed pairs of fp32: one instruction for two elements.  The forward kernel runs
// at the memory's rate only with fewer than ~170 instructions per warp and 16
// bytes a lane; with layer norm the scalar form took 172, this one 140.
typedef uint64_t f2;
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2 dup2(float x) { return pack2(x, x); }
__device__ __forceinline__ float sum2(f2 a) {
    float x, y;
    unpack2(a, x, y);
    return x + y;
}

// A lane's 16 bytes of a row: N elements as packed pairs, first the even ones
// (0, 2), (4, 6), then the odd ones (1, 3), (5, 7), so that the interleaved
// layout's partner of pair k is pair k ^ (N / 4) as a whole.
template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void get(const uint4 &u, f2 (&x)[2]) {
        x[0] = pack2(__uint_as_float(u.x), __uint_as_float(u.z));
        x[1] = pack2(__uint_as_float(u.y), __uint_as_float(u.w));
    }
    static __device__ __forceinline__ uint4 put(const f2 (&x)[2]) {
        float a, b, c, d;
        unpack2(x[0], a, c);
        unpack2(x[1], b, d);
        return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
    static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
    static __device__ __forceinline__ void get(const uint4 &u, f2 (&x)[4]) {
        x[0] = pack2(lo(u.x), lo(u.y));
        x[1] = pack2(lo(u.z), lo(u.w));
        x[2] = pack2(hi(u.x), hi(u.y));
        x[3] = pack2(hi(u.z), hi(u.w));
    }
    static __device__ __forceinline__ uint32_t two(float a, float b) {
        __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&v);
    }
    static __device__ __forceinline__ uint4 put(const f2 (&x)[4]) {
        float e0, e1, e2, e3, o0, o1, o2, o3;
        unpack2(x[0], e0, e1);
        unpack2(x[1], e2, e3);
        unpack2(x[2], o0, o1);
        unpack2(x[3], o2, o3);
        return make_uint4(two(e0, o0), two(e1, o1), two(e2, o2), two(e3, o3));
    }
};
// element of half h of packed pair k
template <int V> __device__ __forceinline__ constexpr int elem(int k, int h) {
    return k < V / 4 ? 2 * (2 * k + h) : 2 * (2 * (k - V / 4) + h) + 1;
}

template <int G> __device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int P> __device__ __forceinline__ float total2(const f2 (&x)[P]) {
    f2 s = x[0];
#pragma unroll
    for (int k = 1; k < P; k++) s = fadd2(s, x[k]);
    return sum2(s);
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
        if (index >= r.cells) {
            if (r.line) set_status(status, ST_INVALID);
            return false;
        }
        if (r.axes == 1) {
            p[0] = index;
        } else if (r.axes == 2) {
            p[0] = r.by1.div(index);
            p[1] = index - p[0] * r.max[1];
        } else {
            const int ab = r.by2.div(index);
            p[2] = index - ab * r.max[2];
            p[0] = r.by1.div(ab);
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
    static constexpr uint32_t ALL = (1u << N) - 1u;
    float c[N], s[N];
    uint32_t on;  // bit i: pair i is rotated
    __device__ __forceinline__ void load(const RopeArgs &r, int e, bool rotated, const int (&p)[3]) {
        on = 0;
#pragma unroll
        for (int i = 0; i < N; i++) {
            c[i] = 1.f;
            s[i] = 0.f;
        }
        if (!rotated) return;
        // entry of pair q: the row of its axis plus q
        uint32_t row[3];
#pragma unroll
        for (int a = 0; a < 3; a++) row[a] = r.off[a] + (uint32_t)p[a] * r.np[a] - r.first[a];
        const int first = HALF ? (e < r.pairs ? e : e - r.pairs) : e / 2;
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int q = first + i;
            if (q < r.pairs) {
                const float2 t = __ldg(r.table + (q < r.first[1] ? row[0] : (q < r.first[2] ? row[1] : row[2])) + q);
                c[i] = t.x;
                s[i] = t.y;
                on |= 1u << i;
            }
        }
    }
    // the lane that holds the partners of this lane's elements (half layout)
    static __device__ __forceinline__ int partner(const RopeArgs &r, int e) {
        const int lane = threadIdx.x & 31, step = r.pairs / V;
        return e < r.pairs ? lane + step : lane - step;
    }
};

// Weight and bias folded into the rotation: turned_i = x_i ca_i + x'_i cb_i, with
// x' the pair's other element, and rb the turned bias.  BACK: the inverse turn.
template <int V, bool HALF> struct Coef {
    static constexpr int P = V / 2;
    f2 ca[P], cb[P], rb[P];
    // w, b: weight and bias in the order of the lanes' packed pairs, P a lane
    // (NULL: 1 and 0); lane: of the row's group.
    template <bool BACK>
    __device__ __forceinline__ void fold(const Angles<V, HALF> &g, const RopeArgs &r, int lane, const f2 *w,
                                         const f2 *b) {
        const int e = lane * V;
        const bool lower = e < r.pairs;
        // lanes at rest are their own partners
        const int mate = HALF && e < 2 * r.pairs ? (lower ? lane + r.pairs / V : lane - r.pairs / V) : lane;
#pragma unroll
        for (int k = 0; k < P; k++) {
            constexpr int d = HALF ? 1 : 2;
            const int i0 = elem<V>(k, 0) / d, i1 = elem<V>(k, 1) / d;
            const bool first = (HALF ? lower : k < V / 4) != BACK;
            const f2 c = pack2(g.c[i0], g.c[i1]);
            const f2 s = first ? pack2(-g.s[i0], -g.s[i1]) : pack2(g.s[i0], g.s[i1]);
            const int o = HALF ? mate * P + k : lane * P + (k ^ (V / 4));
            ca[k] = w ? mul2(w[lane * P + k], c) : c;
            cb[k] = w ? mul2(w[o], s) : s;
            rb[k] = b ? ffma2(b[o], s, mul2(b[lane * P + k], c)) : 0;
        }
    }
    // All lanes of the warp call it; src: the lane of the partners (half layout).
    // Pairs at rest (FULL: none) do not see their partner: it may be infinite.
    template <bool FULL> __device__ __forceinline__ void turn(uint32_t on, int src, f2 (&x)[P]) const {
        f2 y[P];
#pragma unroll
        for (int k = 0; k < P; k++) {
            const f2 o = HALF ? __shfl_sync(0xffffffffu, x[k], src) : x[k ^ (V / 4)];
            y[k] = mul2(x[k], ca[k]);
            const f2 t = ffma2(o, cb[k], y[k]);
            if (FULL) {
                y[k] = t;
            } else {
                float y0, y1, t0, t1;
                unpack2(y[k], y0, y1);
                unpack2(t, t0, t1);
                constexpr int d = HALF ? 1 : 2;
                y[k] = pack2(on >> (elem<V>(k, 0) / d) & 1u ? t0 : y0, on >> (elem<V>(k, 1) / d) & 1u ? t1 : y1);
            }
        }
#pragma unroll
        for (int k = 0; k < P; k++) x[k] = y[k];
    }
};

// LAYER: x - mean in place.  Returns r = 1 / sqrt(mean square + eps).
template <int P, int G> __device__ __forceinline__ float centre(int norm, float eps, f2 (&x)[P]) {
    constexpr float inv_d = 1.f / (2 * P * G);
    if (norm == NORM_LAYER) {
        const f2 m = dup2(group_sum<G>(total2(x)) * -inv_d);
#pragma unroll
        for (int k = 0; k < P; k++) x[k] = fadd2(x[k], m);
    }
    f2 s = mul2(x[0], x[0]);
#pragma unroll
    for (int k = 1; k < P; k++) s = ffma2(x[k], x[k], s);
    return rsqrtf(group_sum<G>(sum2(s)) * inv_d + eps);
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

// 16 bytes to shared memory, zeros where !ok (nothing is read then)
__device__ __forceinline__ void copy16(uint4 *dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(ok ? 16 : 0)
                 : "memory");
}

// Norm and rotation.  An item is a run of HC heads of one tensor for a tile of TT
// tokens: HC x 256 neighbouring bytes of each token in, TT x 256 of each head out
// (d = 128, bf16), which is what DRAM needs on both sides (two heads at a time
// ran at 5.4, 4 tokens x 32 heads at 5.1 instead of 6.1 TB/s).  CTAs take items in
// turn, tile by tile, so that those at work at one time share DRAM pages; each
// copies its next item's rows to shared memory (cp.async, a lane its own 16 bytes
// of each row) while it works on this one's, so loads are in flight all the time
// with few registers.
template <typename T, int D, bool HALF, bool STAT, int HC>
__global__ void __launch_bounds__(NT, FWD_CTAS) norm_rope_kernel(const __grid_constant__ RowArgs a, int runs,
                                                                 const FastDiv by_runs) {
    constexpr int V = Vec<T>::N, P = V / 2, G = D / V, TT = NT / G;
    extern __shared__ __align__(16) uint4 ring_raw[];
    uint4(*ring)[HC][NT] = reinterpret_cast<uint4(*)[HC][NT]>(ring_raw);  // [2]
    // weights and biases of q and k in the order of the lanes' packed pairs
    __shared__ f2 sw[2][2][STAT ? D / 2 : 1];
    const int lane = threadIdx.x % G, grp = threadIdx.x / G, e = lane * V;
    const int tokens = a.batch * a.n;
    // runs of heads of the first one and two tensors
    const int r0 = (a.t[0].heads + HC - 1) / HC, r1 = a.nt > 1 ? r0 + (a.t[1].heads + HC - 1) / HC : runs;
    const int items = ((tokens + TT - 1) / TT) * runs;  // the host checks the range
    const int src = Angles<V, HALF>::partner(a.rope, e);

    // Lanes past the last token walk its items too and store nothing.
    struct Item {
        int ti, tok, b, i, h0, nh;
    };
    auto item_of = [&](int it) {
        Item m;
        const int tile = by_runs.div(it), r = it - tile * runs;
        m.ti = r < r0 ? 0 : (r < r1 ? 1 : 2);
        m.h0 = (r - (m.ti == 0 ? 0 : (m.ti == 1 ? r0 : r1))) * HC;
        m.nh = min(HC, a.t[m.ti].heads - m.h0);
        m.tok = tile * TT + grp;
        const int tok = min(m.tok, tokens - 1);
        m.b = a.batch > 1 ? a.by_n.div(tok) : 0;
        m.i = tok - m.b * a.n;
        return m;
    };
    auto load = [&](const Item &m, int slot) {
        const View &x = a.t[m.ti].x;
        const T *p = (const T *)x.p + m.b * x.sb + (long long)m.i * x.sn + (long long)m.h0 * x.sh + e;
#pragma unroll
        for (int j = 0; j < HC; j++) {
            if (j >= m.nh) break;
            copy16(&ring[slot][j][threadIdx.x], p, true);
            p += x.sh;
        }
    };
    Item next = item_of(blockIdx.x);  // the grid has no more CTAs than items
    load(next, 0);
    asm volatile("cp.async.commit_group;" ::: "memory");

    if (STAT) {
        for (int i = threadIdx.x; i < 2 * D; i += NT) {
            const int ti = i / D, which = i / (D / 2) & 1, c = i % (D / 2);
            if (ti >= a.nt || a.t[ti].copy) continue;
            const void *p = which ? a.t[ti].b : a.t[ti].w;
            float v[2] = {which ? 0.f : 1.f, which ? 0.f : 1.f};
            if (p) {
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int x = c / P * V + elem<V>(c % P, h);
                    v[h] = a.w_f32 ? ((const float *)p)[x] : __bfloat162float(((const __nv_bfloat16 *)p)[x]);
                }
            }
            sw[ti][which][c] = pack2(v[0], v[1]);
        }
        __syncthreads();
    }
    int slot = 0;
    for (int it = blockIdx.x; it < items; it += gridDim.x, slot ^= 1) {
        const Item m = next;
        if (it + (int)gridDim.x < items) {
            next = item_of(it + gridDim.x);
            load(next, slot ^ 1);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        const RowTensor &t = a.t[m.ti];
        bool live = m.tok < tokens;
        int index = m.i;
        long long at_y = m.b * t.y.sb + (long long)m.i * t.y.sn;
        bool store = live;
        if (a.page.seqs) {
            int seq = 0, place = 0;
            live = find_seq(a.page, m.i, seq, place) && live;
            store = live;
            index = max(place, 0);
            if (live) {
                int page = -1;
                if (place >= 0 && (place >> a.page.page_log2) < a.page.max_pages)
                    page = __ldg(a.page.block_table + (long long)seq * a.page.max_pages + (place >> a.page.page_log2));
                const bool fits = page >= 0 && page < a.page.num_pages;
                if (!fits) set_status(a.status, ST_INVALID);
                if (t.paged) {
                    store = fits;
                    at_y = ((((long long)page * a.page.kv_heads) << a.page.page_log2) +
                            (place & ((1 << a.page.page_log2) - 1))) * D;
                }
            }
        }
        T *y = (T *)t.y.p + at_y + (long long)m.h0 * t.y.sh + e;
        if (t.copy) {
            asm volatile("cp.async.wait_group 1;" ::: "memory");
#pragma unroll
            for (int j = 0; j < HC; j++) {
                if (j >= m.nh) break;
                if (store) *(uint4 *)y = ring[slot][j][threadIdx.x];
                y += t.y.sh;
            }
            continue;
        }
        Coef<V, HALF> k;
        uint32_t on = 0;
        {
            int p[3];
            Angles<V, HALF> ang;
            const bool rotated =
                live && token_pos(a.rope, m.b * a.rope.pos_batch + (long long)m.i * a.rope.axes, index, p, a.status);
            ang.load(a.rope, e, rotated, p);
            on = ang.on;
            k.template fold<false>(ang, a.rope, lane, STAT && t.w ? sw[m.ti][0] : nullptr,
                                   STAT && t.b ? sw[m.ti][1] : nullptr);
        }
        const bool full = __all_sync(0xffffffffu, on == Angles<V, HALF>::ALL);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
#pragma unroll
        for (int j = 0; j < HC; j++) {
            if (j >= m.nh) break;
            f2 v[P];
            Vec<T>::get(ring[slot][j][threadIdx.x], v);
            f2 r = 0;
            if (STAT) r = dup2(centre<P, G>(a.norm, a.eps, v));
            if (full)
                k.template turn<true>(on, src, v);
            else
                k.template turn<false>(on, src, v);
            if (STAT) {
#pragma unroll
                for (int i = 0; i < P; i++) v[i] = ffma2(v[i], r, k.rb[i]);
            }
            if (store) *(uint4 *)y = Vec<T>::put(v);
            y += t.y.sh;
        }
    }
}

// Gradients.  With n = r x (x centred): e = g' w, c = r^3 mean(e x),
//   dx = r (e - [mean e]) - c x,  dw += (g' x) r,  db += g',
// both means in one round of shuffles.  The CTAs take items (token tile, run of
// heads) in turn, in steps of HC heads; a lane's own g and x come through a ring of
// STEPS steps of cp.async copies, two steps ahead (loads into registers held too
// few in flight: 39% of DRAM's peak against 60%).  Each lane sums its elements' dw
// and db over all its rows in registers; the CTA's sums go to part[cta] and
// back_sum_kernel adds the CTAs in order.
template <typename T, int D, bool HALF, bool STAT>
__global__ void __launch_bounds__(NT, BACK_CTAS) norm_rope_back_kernel(const __grid_constant__ BackArgs a) {
    constexpr int V = Vec<T>::N, P = V / 2, G = D / V, TT = NT / G, HC = BACK_HC, STEPS = BACK_STEPS;
    constexpr int PER = STAT ? 2 * HC : HC;  // pieces of 16 bytes a step
    extern __shared__ __align__(16) uint4 ring_raw[];
    uint4(*ring)[PER][NT] = reinterpret_cast<uint4(*)[PER][NT]>(ring_raw);
    static_assert(!STAT || STEPS * PER * NT * 16 >= 2 * TT * D * (int)sizeof(float), "the sums reuse the ring");
    const int ti = (int)blockIdx.x < a.ctas[0] ? 0 : 1;
    const int cta = blockIdx.x - (ti ? a.ctas[0] : 0);
    const BackTensor &t = a.t[ti];
    const int grp = threadIdx.x / G, e = (threadIdx.x % G) * V;
    const int tokens = a.batch * a.n;
    // an item: a.run heads of one tile of TT tokens; the CTAs take them in turn
    const int runs = (t.heads + a.run - 1) / a.run;
    const int items = ((tokens + TT - 1) / TT) * runs;  // the host checks the range
    const int src = Angles<V, HALF>::partner(a.rope, e);

    // Lanes past the last token walk its items too and store nothing.
    struct Item {
        int tok, b, i, h0, h1;
    };
    auto item_of = [&](int it) {
        Item m;
        const int tile = a.by_runs[ti].div(it);
        m.tok = tile * TT + grp;
        const int tok = min(m.tok, tokens - 1);
        m.b = a.batch > 1 ? a.by_n.div(tok) : 0;
        m.i = tok - m.b * a.n;
        m.h0 = (it - tile * runs) * a.run;
        m.h1 = min(m.h0 + a.run, t.heads);
        return m;
    };

    // the loading side: steps of all items in order, ahead of the computing side
    int lit = cta, lh = 0, lh1 = 0, slot = 0;
    bool llive = false;
    const T *lg = nullptr, *lx = nullptr;
    auto enter = [&]() {
        if (lit >= items) return;
        const Item m = item_of(lit);
        lh = m.h0;
        lh1 = m.h1;
        llive = m.tok < tokens;
        lg = (const T *)t.g.p + m.b * t.g.sb + (long long)m.i * t.g.sn + (long long)m.h0 * t.g.sh + e;
        lx = (const T *)t.x.p + m.b * t.x.sb + (long long)m.i * t.x.sn + (long long)m.h0 * t.x.sh + e;
    };
    auto load_step = [&]() {
        if (lit < items) {
#pragma unroll
            for (int j = 0; j < HC; j++) {
                const bool ok = llive && lh + j < lh1;
                copy16(&ring[slot][j][threadIdx.x], lg, ok);
                if (STAT) copy16(&ring[slot][(HC + j) % PER][threadIdx.x], lx, ok);
                lg += t.g.sh;
                lx += t.x.sh;
            }
            lh += HC;
            if (lh >= lh1) {
                lit += a.ctas[ti];
                enter();
            }
        }
        slot = slot == STEPS - 1 ? 0 : slot + 1;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    enter();
#pragma unroll
    for (int i = 0; i < STEPS - 1; i++) load_step();

    f2 w[P], dw[P], db[P];
    if (STAT) {
        float wv[V];
        load_w<V>(t.w, a.w_f32, e, 1.f, wv);
#pragma unroll
        for (int k = 0; k < P; k++) {
            w[k] = pack2(wv[elem<V>(k, 0)], wv[elem<V>(k, 1)]);
            dw[k] = db[k] = 0;
        }
    }
    int at = 0;
    for (int it = cta; it < items; it += a.ctas[ti]) {
        const Item m = item_of(it);
        const bool live = m.tok < tokens;
        T *dx = (T *)t.dx.p + m.b * t.dx.sb + (long long)m.i * t.dx.sn + (long long)m.h0 * t.dx.sh + e;
        Coef<V, HALF> turn;
        uint32_t on;
        {
            int p[3];
            Angles<V, HALF> ang;
            const bool rotated =
                token_pos(a.rope, m.b * a.rope.pos_batch + (long long)m.i * a.rope.axes, m.i, p, a.status);
            ang.load(a.rope, e, rotated, p);
            on = ang.on;
            turn.template fold<true>(ang, a.rope, e / V, nullptr, nullptr);
        }
        const bool full = __all_sync(0xffffffffu, on == Angles<V, HALF>::ALL);
        for (int h = m.h0; h < m.h1; h += HC) {
            load_step();
            asm volatile("cp.async.wait_group %0;" ::"n"(STEPS - 1) : "memory");
#pragma unroll
            for (int j = 0; j < HC; j++) {
                if (h + j >= m.h1) break;
                const bool in = live;  // else g and x are zeros
                f2 g[P];
                Vec<T>::get(ring[at][j][threadIdx.x], g);
                if (full)
                    turn.template turn<true>(on, src, g);
                else
                    turn.template turn<false>(on, src, g);
                if (STAT) {
                    f2 x[P], s1 = 0, s2 = 0;
                    Vec<T>::get(ring[at][(HC + j) % PER][threadIdx.x], x);
                    const float r = centre<P, G>(a.norm, a.eps, x);
                    const f2 rs = dup2(in ? r : 0.f);
#pragma unroll
                    for (int k = 0; k < P; k++) {
                        const f2 p = mul2(g[k], x[k]);
                        dw[k] = ffma2(p, rs, dw[k]);
                        db[k] = fadd2(db[k], g[k]);
                        s2 = ffma2(p, w[k], s2);
                        g[k] = mul2(g[k], w[k]);
                        s1 = fadd2(s1, g[k]);
                    }
                    const f2 c = dup2(group_sum<G>(sum2(s2)) * (-1.f / D) * r * r * r);
                    const f2 m1 = dup2(a.norm == NORM_LAYER ? group_sum<G>(sum2(s1)) * (-1.f / D) * r : 0.f);
                    const f2 r2 = dup2(r);
#pragma unroll
                    for (int k = 0; k < P; k++) g[k] = ffma2(g[k], r2, ffma2(x[k], c, m1));
                }
                if (in) *(uint4 *)dx = Vec<T>::put(g);
                dx += t.dx.sh;
            }
            at = at == STEPS - 1 ? 0 : at + 1;
        }
    }
    if (!STAT || !a.part) return;
    __syncthreads();  // every lane is through with its ring
    float *red = reinterpret_cast<float *>(ring);  // [2][TT][D]
#pragma unroll
    for (int k = 0; k < P; k++) {
        float x, y;
        unpack2(dw[k], x, y);
        red[grp * D + e + elem<V>(k, 0)] = x;
        red[grp * D + e + elem<V>(k, 1)] = y;
        unpack2(db[k], x, y);
        red[(TT + grp) * D + e + elem<V>(k, 0)] = x;
        red[(TT + grp) * D + e + elem<V>(k, 1)] = y;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * D; c += NT) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < TT; k++) s += red[((c / D) * TT + k) * D + c % D];
        a.part[(size_t)blockIdx.x * 2 * D + c] = s;
    }
}

// Block (tensor, dw or db): the CTAs' partial sums in order, in double.
__global__ void __launch_bounds__(1024) back_sum_kernel(const __grid_constant__ BackArgs a, int D) {
    __shared__ double red[1024];
    after_previous();
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

// One thread per (cos, sin) pair; once per layer.
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

typedef void (*FwdKernel)(const RowArgs, int, const FastDiv);
template <typename T, int D, int HC> FwdKernel fwd_kernel(bool half, bool stat) {
    if (stat) return half ? norm_rope_kernel<T, D, true, true, HC> : norm_rope_kernel<T, D, false, true, HC>;
    return half ? norm_rope_kernel<T, D, true, false, HC> : norm_rope_kernel<T, D, false, false, HC>;
}
constexpr int fwd_smem(int HC) { return 2 * HC * NT * 16; }

template <typename T, int D> constexpr int tile_tokens() { return NT / (D / Vec<T>::N); }

template <typename T, int D, int HC> int launch_rows(const RowArgs &a, int num_sms, cudaStream_t st) {
    long long runs = 0;
    for (int i = 0; i < a.nt; i++) runs += (a.t[i].heads + HC - 1) / HC;
    const int tt = tile_tokens<T, D>();
    const long long items = ((long long)a.batch * a.n + tt - 1) / tt * runs, ctas = (long long)FWD_CTAS * num_sms;
    if (items > 0x3fffffffLL) return -1;
    // as many rounds as the items need, and only as many CTAs as fill the rounds
    const long long rounds = (items + ctas - 1) / ctas;
    const unsigned grid = (unsigned)((items + rounds - 1) / rounds);
    fwd_kernel<T, D, HC>(a.rope.half, a.norm != NORM_NONE)<<<grid, NT, fwd_smem(HC), st>>>(a, (int)runs,
                                                                                        FastDiv((uint32_t)runs));
    note_launch();
    return 0;
}
// Runs of one head where runs of 8 would leave SMs without a CTA (few tokens): one
// token of 40 heads 2.5 instead of 4.1 us, 64 tokens 4.0 instead of 4.4; with 300
// both take 5.4.
template <typename T, int D> int launch_rows_d(const RowArgs &a, int num_sms, cudaStream_t st) {
    long long runs = 0;
    for (int i = 0; i < a.nt; i++) runs += (a.t[i].heads + FWD_HC - 1) / FWD_HC;
    const int tt = tile_tokens<T, D>();
    const bool many = ((long long)a.batch * a.n + tt - 1) / tt * runs >= num_sms;
    return many ? launch_rows<T, D, FWD_HC>(a, num_sms, st) : launch_rows<T, D, 1>(a, num_sms, st);
}

typedef void (*BackKernel)(const BackArgs);
template <typename T, int D> BackKernel back_kernel(bool half, bool stat) {
    if (stat) return half ? norm_rope_back_kernel<T, D, true, true> : norm_rope_back_kernel<T, D, false, true>;
    return half ? norm_rope_back_kernel<T, D, true, false> : norm_rope_back_kernel<T, D, false, false>;
}
constexpr int back_smem(bool stat) { return BACK_STEPS * (stat ? 2 : 1) * BACK_HC * NT * 16; }

template <typename T, int D> int setup(int half, bool stat) {
    auto raise = [](const void *fn, int smem) {
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess;
    };
    return raise((const void *)fwd_kernel<T, D, FWD_HC>(half, stat), fwd_smem(FWD_HC)) &&
                   raise((const void *)back_kernel<T, D>(half, stat), back_smem(stat))
               ? 0
               : -1;
}
}  // namespace
int rope_setup(int dtype, int D, int half, int norm) {
    const bool stat = norm != NORM_NONE;
    if (dtype == DT_BF16) return D == 64 ? setup<__nv_bfloat16, 64>(half, stat) : setup<__nv_bfloat16, 128>(half, stat);
    return D == 64 ? setup<float, 64>(half, stat) : setup<float, 128>(half, stat);
}

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

int back_ctas(int num_sms) { return BACK_CTAS * num_sms + 2; }

int k_norm_rope_back(BackArgs &a, int dtype, int D, int num_sms, cudaStream_t st) {
    // the tensors' CTAs in proportion to their heads
    const int total = BACK_CTAS * num_sms, h0 = a.t[0].heads, h1 = a.t[1].heads;
    a.ctas[0] = h0 ? max(1, (int)((long long)total * h0 / (h0 + h1))) : 0;
    a.ctas[1] = h1 ? max(1, total - a.ctas[0]) : 0;
    const long long tt = NT / (D / (dtype == DT_BF16 ? 8 : 4)), tiles = ((long long)a.batch * a.n + tt - 1) / tt;
    // Long runs spare the coefficients (all 30 heads 164, 8 heads 186 us on 2 x 17,776
    // tokens); few tokens: short ones, more CTAs at work (runs of 4 / 32 heads: 64 tokens
    // 6.6 / 17.3 us, 1,200 tokens 14.3 / 18.2).
    a.run = BACK_MOST;
    if (tiles * ((max(h0, h1) + a.run - 1) / a.run) < total) a.run = BACK_HC;
    for (int i = 0; i < 2; i++) {
        const int heads = a.t[i].heads;
        if (!heads) continue;
        const long long runs = (heads + a.run - 1) / a.run, items = tiles * runs;
        if (items > 0x3fffffffLL) return -1;
        a.by_runs[i] = FastDiv((uint32_t)runs);
        // as many rounds as the items need, and only as many CTAs as fill the rounds
        const long long rounds = (items + a.ctas[i] - 1) / a.ctas[i];
        a.ctas[i] = (int)((items + rounds - 1) / rounds);
    }
    const bool stat = a.norm != NORM_NONE;
    BackKernel fn = dtype == DT_BF16 ? (D == 64 ? back_kernel<__nv_bfloat16, 64>(a.rope.half, stat)
                                                : back_kernel<__nv_bfloat16, 128>(a.rope.half, stat))
                                     : (D == 64 ? back_kernel<float, 64>(a.rope.half, stat)
                                                : back_kernel<float, 128>(a.rope.half, stat));
    fn<<<a.ctas[0] + a.ctas[1], NT, back_smem(stat), st>>>(a);
    note_launch();
    if (a.part) launch_after(back_sum_kernel, 4, 1024, st, a, D);
    return 0;
}

}  // namespace ac
