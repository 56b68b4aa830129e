// Pieces of the tcgen05 softmax kernels (ac_attn3.cu, ac_cache_attn.cu): packed
// fp32 arithmetic, 2^x split between the special-function unit and the FMA pipe,
// register moves between warpgroups.
#pragma once
#include "ac_common.cuh"

namespace ac {
namespace {

__device__ __forceinline__ void drain3(uint64_t *bar, uint32_t parity) {
    const uint64_t t0 = gtimer();
    while (!mbar_try_wait(bar, parity) && gtimer() - t0 < 200000000ull) {
    }
}

template <int R> __device__ __forceinline__ void regs_dec3() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R> __device__ __forceinline__ void regs_inc3() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}

__device__ __forceinline__ void named_bar_sync(int id, int nthreads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float m;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// 2^x for a pair on the FMA pipe.  x is clamped to [-127, 2^22): with
// n = rint(x) (the 1.5 * 2^23 shift puts it in the low mantissa bits of t) and
// f = x - n in [-1/2, 1/2], 2^f = 1 + c1 f + c2 f^2 + c3 f^3 (relative error
// below 1.1e-4 on that interval: the minimax cubic with constant term 1,
// fitted by linear programming on 4001 points), and adding n << 23 to its bits
// scales it by 2^n.  x = -127 gives exactly +0 (f = 0, p = 1, exponent field 0),
// so masked scores (-inf) contribute nothing; x > -127 gives a normal number
// or, below -126, a nonnegative subnormal.
__device__ __forceinline__ void ex2_poly2(float x0, float x1, float &y0, float &y1) {
    constexpr float kShift = 12582912.0f;  // 1.5 * 2^23
    x0 = fmaxf(x0, -127.f);
    x1 = fmaxf(x1, -127.f);
    const uint64_t x = pack2(x0, x1);
    const uint64_t t = fadd2(x, pack2(kShift, kShift));
    const uint64_t n = fadd2(t, pack2(-kShift, -kShift));
    const uint64_t f = ffma2(n, pack2(-1.f, -1.f), x);
    uint64_t q = ffma2(pack2(0.0550091f, 0.0550091f), f, pack2(0.2422110f, 0.2422110f));
    q = ffma2(q, f, pack2(0.6932829f, 0.6932829f));
    q = ffma2(q, f, pack2(1.f, 1.f));
    float t0, t1, q0, q1;
    unpack2(t, t0, t1);
    unpack2(q, q0, q1);
    y0 = __uint_as_float(__float_as_uint(q0) + (__float_as_uint(t0) << 23));
    y1 = __uint_as_float(__float_as_uint(q1) + (__float_as_uint(t1) << 23));
}

// P for key pairs [P0, P0 + NP) of a row: x = s * scale - m (packed), 2^x on
// MUFU or, for EMU of every 8 pairs, on the FMA pipe; bf16 pairs into pk[pair
// - 32 * (pair / 32)], fp32 sums into la (alternating accumulators)
template <int EMU, int P0, int NP>
__device__ __forceinline__ void exp_pairs(const uint32_t (&s)[128], uint32_t (&pk)[32], uint64_t scale2, uint64_t neg2,
                                          uint64_t (&la)[2]) {
#pragma unroll
    for (int i = P0; i < P0 + NP; i++) {
        float x0, x1, e0, e1;
        unpack2(ffma2(pack2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), scale2, neg2), x0, x1);
        if ((i & 7) >= 8 - EMU) {
            ex2_poly2(x0, x1, e0, e1);
        } else {
            e0 = ex2_approx(x0);
            e1 = ex2_approx(x1);
        }
        la[i & 1] = fadd2(la[i & 1], pack2(e0, e1));
        __nv_bfloat162 b2 = __floats2bfloat162_rn(e0, e1);
        pk[i & 31] = *reinterpret_cast<uint32_t *>(&b2);
    }
}

}  // namespace
}  // namespace ac
