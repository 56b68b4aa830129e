// Cache attention for up to 16 rows = (new token, head of the group) pairs of a
// sequence and key head: a step of a few tokens, bound by reading the cache.
//
// A cluster of CTAs takes one sequence and key head; its warps take the 16-key
// blocks in turn.  A warp streams its blocks through a ring of its own in shared
// memory (cp.async, STAGES - 1 blocks of K and V in flight), computes S = Q K^T and
// O += P V with m16n8k16 products (the 16 rows are one tile) and keeps its own
// running maximum and sum; the warps' sums are joined in shared memory and the
// CTAs' through the cluster's, so one launch does it all without a workspace.
// Rows of a block past the sequence's end are not read but filled with zeros, so
// what the cache holds there does not matter.
//
// 16 rows are the height of its one product tile; nothing taller was built, so that
// limit has one side only: 20 to 128 rows of those 16 sequences (5 to 32 tokens each) take
// 89 to 91 us in the tiles, 4.6 TB/s, where 16 rows take 71 us here.
// Tiles of 128 rows spend their time on empty rows here: 89 against 70 us (5.9
// TB/s) for 16 single tokens over up to 8,191 keys (32 / 8 heads, d = 128), and
// their TMEM set-up and second launch 11.5 against 7.0 us for one token over 777.
#include <algorithm>

#include "ac_cache.cuh"

namespace ac {
namespace {

constexpr int WARPS = 4, KEYS = 16, ROWS = 16;

template <int D> struct DCfg {
    static constexpr int STAGES = D == 128 ? 3 : 4, CTAS = D == 128 ? 2 : 3;
    static constexpr int HALF = KEYS * D * 2;                   // K or V of a block
    static constexpr int RING = STAGES * 2 * HALF;              // of a warp
    static constexpr int OFF_O = WARPS * RING;                  // the CTA's sums [ROWS, D] fp32
    static constexpr int OFF_ML = OFF_O + ROWS * D * 4;         // its (max, sum) per row
    static constexpr int OFF_WML = OFF_ML + ROWS * 8;           // each warp's (max, sum) per row
    static constexpr int SMEM = OFF_WML + WARPS * ROWS * 8;
    static_assert(RING >= ROWS * D * 4, "a warp's sums reuse its ring");
};

__device__ __forceinline__ void copy16z(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t bf2(float a, float b) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&v);
}
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 32-bit cluster address of a shared address in CTA `rank`
__device__ __forceinline__ uint32_t remote(uint32_t addr, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 ld_remote4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_remote2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

template <int D>
__global__ void __launch_bounds__(32 * WARPS, DCfg<D>::CTAS)
    cache_decode_kernel(const __grid_constant__ CacheAttnArgs a, int cs) {
    using C = DCfg<D>;
    constexpr int CH = D / 8;   // 16-byte pieces of a row
    extern __shared__ __align__(128) unsigned char sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = blockIdx.x / cs, rank = blockIdx.x - unit * cs;
    const int s = unit / a.kv_heads, kvh = unit - s * a.kv_heads;
    int row0, nq, p0, len;
    sequence(a, s, row0, nq, p0, len, rank == 0 && threadIdx.x == 0);
    const int R = nq * a.group;  // rows in use
    // the cluster's blocks [b0, b1)
    int b0 = 0, b1 = 0;
    if (nq) {
        int lo, hi, x;
        key_range(a, p0, len, lo, x);
        key_range(a, p0 + nq - 1, len, x, hi);
        if (hi > lo) {
            b0 = lo / KEYS;
            b1 = (hi + KEYS - 1) / KEYS;
        }
    }
    const int step = cs * WARPS;
    unsigned char *ring = sm + warp * C::RING;
    const uint32_t ring_a = smem_u32(ring);
    const int32_t *table = a.block_table + (long long)s * a.max_pages;
    const int in_page = (1 << a.page_log2) - 1;

    // the loading side: block `lb`, its page read one block ahead
    int lb = b0 + rank * WARPS + warp, lslot = 0;
    auto page_of = [&](int b) -> int {
        if (b >= b1) return 0;
        const int id = __ldg(table + ((b * KEYS) >> a.page_log2));
        if (id >= 0 && id < a.num_pages) return id;
        set_status(a.status, ST_INVALID);
        return id < 0 ? 0 : a.num_pages - 1;
    };
    int page = page_of(lb);
    auto load_block = [&]() {
        if (lb < b1) {
            const int id = page;
            page = page_of(lb + step);
            const long long at =
                ((((long long)id * a.kv_heads + kvh) << a.page_log2) + ((lb * KEYS) & in_page)) * D;
            const __nv_bfloat16 *k = (const __nv_bfloat16 *)a.kp + at, *v = (const __nv_bfloat16 *)a.vp + at;
            const uint32_t dst = ring_a + lslot * 2 * C::HALF;
#pragma unroll
            for (int i = 0; i < KEYS * CH / 32; i++) {
                const int x = i * 32 + lane, r = x / CH, c = x % CH;
                const uint32_t to = r * (D * 2) + ((c ^ (r & 7)) << 4);
                const bool ok = lb * KEYS + r < len;
                copy16z(dst + to, k + r * D + c * 8, ok);
                copy16z(dst + C::HALF + to, v + r * D + c * 8, ok);
            }
            lb += step;
        }
        lslot = lslot == C::STAGES - 1 ? 0 : lslot + 1;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < C::STAGES - 1; i++) load_block();

    // this thread's rows: lane / 4 and 8 further
    uint32_t q[D / 16][4];
    int lo[2], hi[2];
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const int r = lane / 4 + 8 * h;
        const bool in = r < R;
        const int tok = in ? r / a.group : 0;
        lo[h] = hi[h] = 0;
        if (in) key_range(a, p0 + tok, len, lo[h], hi[h]);
        const __nv_bfloat16 *src = (const __nv_bfloat16 *)a.q.p + (long long)(row0 + tok) * a.q.sn +
                                   (long long)(kvh * a.group + (in ? r - tok * a.group : 0)) * a.q.sh + (lane % 4) * 2;
#pragma unroll
        for (int k = 0; k < D / 16; k++) {
            q[k][h] = in ? __ldg((const uint32_t *)(src + k * 16)) : 0u;
            q[k][2 + h] = in ? __ldg((const uint32_t *)(src + k * 16 + 8)) : 0u;
        }
    }
    // blocks within [wlo, whi) need no mask (rows not in use: S = 0, never written)
    int wlo = max(lo[0], lo[1]), whi = 0x7fffffff;
#pragma unroll
    for (int h = 0; h < 2; h++)
        if (lane / 4 + 8 * h < R) whi = min(whi, hi[h]);
    wlo = __reduce_max_sync(0xffffffffu, wlo);
    whi = __reduce_min_sync(0xffffffffu, whi);

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; i++) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    const float sc = a.scale_log2;
    int slot = 0;
    for (int b = b0 + rank * WARPS + warp; b < b1; b += step) {
        asm volatile("cp.async.wait_group %0;" ::"n"(C::STAGES - 2) : "memory");
        __syncwarp();
        const uint32_t kb = ring_a + slot * 2 * C::HALF, vb = kb + C::HALF;
        float sv[2][4] = {};
        {
            const int key = (lane >> 4) * 8 + (lane & 7), odd = (lane >> 3) & 1;
            const uint32_t row = kb + key * (D * 2);
#pragma unroll
            for (int k = 0; k < D / 16; k++) {
                uint32_t f[4];
                ldm4(f, row + (((2 * k + odd) ^ (key & 7)) << 4));
                mma16816(sv[0], q[k], f[0], f[1]);
                mma16816(sv[1], q[k], f[2], f[3]);
            }
        }
        const int kbase = b * KEYS;
        if (kbase < wlo || kbase + KEYS > whi) {
#pragma unroll
            for (int t = 0; t < 2; t++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int key = kbase + t * 8 + (lane % 4) * 2 + (e & 1);
                    if (key < lo[e >> 1] || key >= hi[e >> 1]) sv[t][e] = -INFINITY;
                }
        }
        float mx[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            mx[h] = fmaxf(fmaxf(sv[0][2 * h], sv[0][2 * h + 1]), fmaxf(sv[1][2 * h], sv[1][2 * h + 1]));
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2)) * sc;
        }
        // the reference maximum moves only when the row's grew by more than 2^8
        if (__any_sync(0xffffffffu, mx[0] > m[0] + 8.f || mx[1] > m[1] + 8.f)) {
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const float to = fmaxf(m[h], mx[h]);
                const float f = to == -INFINITY ? 1.f : ex2_approx(m[h] - to);
                m[h] = to;
                l[h] *= f;
#pragma unroll
                for (int i = 0; i < D / 8; i++) {
                    o[i][2 * h] *= f;
                    o[i][2 * h + 1] *= f;
                }
            }
        }
        uint32_t p[4];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const float neg = m[h] == -INFINITY ? 0.f : -m[h];
            float e[4];
#pragma unroll
            for (int t = 0; t < 2; t++) {
                e[2 * t] = ex2_approx(fmaf(sv[t][2 * h], sc, neg));
                e[2 * t + 1] = ex2_approx(fmaf(sv[t][2 * h + 1], sc, neg));
            }
            l[h] += (e[0] + e[1]) + (e[2] + e[3]);
            p[h] = bf2(e[0], e[1]);
            p[2 + h] = bf2(e[2], e[3]);
        }
        {
            const int key = ((lane >> 3) & 1) * 8 + (lane & 7), up = lane >> 4;
            const uint32_t row = vb + key * (D * 2);
#pragma unroll
            for (int t = 0; t < D / 16; t++) {
                uint32_t f[4];
                ldm4t(f, row + (((2 * t + up) ^ (key & 7)) << 4));
                mma16816(o[2 * t], p, f[0], f[1]);
                mma16816(o[2 * t + 1], p, f[2], f[3]);
            }
        }
        __syncwarp();  // the slot is read; the next copies may overwrite it
        slot = slot == C::STAGES - 1 ? 0 : slot + 1;
        load_block();
    }
    // this warp's rows to shared memory
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
    float2 *wml = reinterpret_cast<float2 *>(sm + C::OFF_WML);
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const int r = lane / 4 + 8 * h;
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        if (lane % 4 == 0) wml[warp * ROWS + r] = make_float2(m[h], l[h]);
        if (r < R) {
            float *dst = reinterpret_cast<float *>(ring) + r * D + (lane % 4) * 2;
#pragma unroll
            for (int i = 0; i < D / 8; i++) *reinterpret_cast<float2 *>(dst + i * 8) = make_float2(o[i][2 * h], o[i][2 * h + 1]);
        }
    }
    __syncthreads();
    // the CTA's sums
    float *co = reinterpret_cast<float *>(sm + C::OFF_O);
    float2 *cml = reinterpret_cast<float2 *>(sm + C::OFF_ML);
    for (int x = threadIdx.x; x < R * (D / 4); x += 32 * WARPS) {
        const int r = x / (D / 4), c = x - r * (D / 4);
        float mm = -INFINITY, ll = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; w++) mm = fmaxf(mm, wml[w * ROWS + r].x);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < WARPS; w++) {
            const float f = weight(wml[w * ROWS + r].x, mm);
            const float4 v = reinterpret_cast<const float4 *>(sm + w * C::RING)[r * (D / 4) + c];
            ll += f * wml[w * ROWS + r].y;
            acc.x += f * v.x;
            acc.y += f * v.y;
            acc.z += f * v.z;
            acc.w += f * v.w;
        }
        reinterpret_cast<float4 *>(co)[x] = acc;
        if (c == 0) cml[r] = make_float2(mm, ll);
    }
    if (cs > 1)
        cluster_sync();
    else
        __syncthreads();
    // the cluster's: each CTA writes its share of the rows' elements
    const uint32_t co_a = smem_u32(co), cml_a = smem_u32(cml);
    for (int x = rank * 32 * WARPS + threadIdx.x; x < R * (D / 4); x += cs * 32 * WARPS) {
        const int r = x / (D / 4), c = x - r * (D / 4);
        float mm = -INFINITY, ll = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < cs; k++) mm = fmaxf(mm, ld_remote2(remote(cml_a + r * 8, k)).x);
        for (int k = 0; k < cs; k++) {
            const float2 ml = ld_remote2(remote(cml_a + r * 8, k));
            const float f = weight(ml.x, mm);
            const float4 v = ld_remote4(remote(co_a + x * 16, k));
            ll += f * ml.y;
            acc.x += f * v.x;
            acc.y += f * v.y;
            acc.z += f * v.z;
            acc.w += f * v.w;
        }
        const float inv = ll == 0.f ? 0.f : 1.f / ll;  // a row without keys: zeros
        const int tok = r / a.group, head = kvh * a.group + r - tok * a.group;
        __nv_bfloat16 *dst = (__nv_bfloat16 *)a.out.p + (long long)(row0 + tok) * a.out.sn +
                             (long long)head * a.out.sh + c * 4;
        *reinterpret_cast<uint2 *>(dst) = make_uint2(bf2(acc.x * inv, acc.y * inv), bf2(acc.z * inv, acc.w * inv));
        if (a.lse && c == 0)
            a.lse[(long long)(row0 + tok) * a.heads + head] =
                ll == 0.f ? -INFINITY : (mm + __log2f(ll)) * 0.69314718055994531f;
    }
    if (cs > 1) cluster_sync();  // no CTA leaves while others read its shared memory
}

constexpr int MOST_CLUSTER = 16;  // needs the non-portable attribute

template <int D> int launch(const CacheAttnArgs &a, int cs, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.gridDim = dim3((unsigned)(a.seqs * a.kv_heads * cs));
    cfg.blockDim = dim3(32 * WARPS);
    cfg.dynamicSmemBytes = DCfg<D>::SMEM;
    cfg.stream = st;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cs;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    // an error stays pending for the caller's check
    if (cudaLaunchKernelEx(&cfg, cache_decode_kernel<D>, a, cs) == cudaSuccess) note_launch();
    return 0;
}

}  // namespace

int cache_decode_setup(int D) {
    const void *fn = D == 64 ? (const void *)cache_decode_kernel<64> : (const void *)cache_decode_kernel<128>;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) return -1;
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                D == 64 ? DCfg<64>::SMEM : DCfg<128>::SMEM) == cudaSuccess
               ? 0
               : -1;
}

int decode_cluster(const CacheAttnArgs &a, int num_sms) {
    const long long units = (long long)a.seqs * a.kv_heads;
    if ((long long)a.max_q * a.group > ROWS || units * MOST_CLUSTER > 0x7fffffffLL) return 0;
    long long keys = a.max_kv;
    if (a.window) keys = std::min<long long>(keys, (long long)a.window + a.max_q + a.causal_block);
    const long long blocks = std::max<long long>(1, (keys + KEYS - 1) / KEYS);
    // CTAs for all SMs' places and some more (sequences differ in length: 16 of them, 8
    // key heads, clusters of 2 / 4 / 8 take 74 / 70 / 84 us), but two blocks a warp at
    // least
    const int places = num_sms * (a.D == 128 ? DCfg<128>::CTAS : DCfg<64>::CTAS);
    int cs = 1;
    while (cs < MOST_CLUSTER && units * cs < places + places / 2 && blocks >= 2LL * 2 * cs * WARPS) cs *= 2;
    // Too few units for the whole GPU and a long cache: the tiles' units are cut
    // along the keys as often as needed.  One token, d = 128, this kernel against
    // tiles: 8 key heads 29 / 37 us at 20,000 keys, 68 / 66 at 65,000; 2 key heads
    // 16 / 45 at 8,000, 70 / 53 at 65,000.
    if (units * cs < num_sms && blocks > 48LL * cs * WARPS) return 0;
    return cs;
}

int k_cache_decode(const CacheAttnArgs &a, int cs, cudaStream_t st) {
    return a.D == 64 ? launch<64>(a, cs, st) : launch<128>(a, cs, st);
}

}  // namespace ac
