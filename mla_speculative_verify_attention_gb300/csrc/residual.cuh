// Sums of residuals max(p - A q, 0) as integers, two elements a step.  Everything here compiles for
// the host too, with the same roundings, so that the arithmetic can be compared with rational numbers.
#pragma once

#include <math.h>
#include <stdint.h>
#include <string.h>

namespace mla {

constexpr double UNIT = 1.0 / 17592186044416.0;      // 2^-44, the unit of the integer sums

// The residual's coefficient A in two fp32 parts, and which of three forms it takes.
enum { FROM_P, MINUS_Q, MINUS_AQ };                  // A = 0, A = 1, any A
struct Coef {
    float ah, al;
};

// Adding 1.5 * 2^23 rounds to an integer and leaves it in the low mantissa bits.
constexpr float MAGIC = 12582912.f;
constexpr unsigned MAGIC_BITS = 0x4B400000u;

__host__ __device__ __forceinline__ unsigned float_bits(float x) {
#ifdef __CUDA_ARCH__
    return __float_as_uint(x);
#else
    unsigned u;
    memcpy(&u, &x, 4);
    return u;
#endif
}

// Two elements a step: the fp32 operations on pairs (64 trees 43.2 -> 42.2 us).  On the host: one
// after the other (built with -ffp-contract=off, so that nothing is fused but mul_add).
struct Pair {
    unsigned long long v;
    __host__ __device__ __forceinline__ Pair() {}
    __host__ __device__ __forceinline__ Pair(float a, float b) {
#ifdef __CUDA_ARCH__
        asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
#else
        v = (unsigned long long)float_bits(b) << 32 | float_bits(a);
#endif
    }
    __host__ __device__ __forceinline__ explicit Pair(float a) : Pair(a, a) {}
    __host__ __device__ __forceinline__ void get(float& a, float& b) const {
#ifdef __CUDA_ARCH__
        asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
#else
        const unsigned lo = (unsigned)v, hi = (unsigned)(v >> 32);
        memcpy(&a, &lo, 4);
        memcpy(&b, &hi, 4);
#endif
    }
};
__host__ __device__ __forceinline__ Pair mul(Pair a, Pair b) {
#ifdef __CUDA_ARCH__
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
#else
    float a0, a1, b0, b1;
    a.get(a0, a1);
    b.get(b0, b1);
    return Pair(a0 * b0, a1 * b1);
#endif
}
__host__ __device__ __forceinline__ Pair add(Pair a, Pair b) {
#ifdef __CUDA_ARCH__
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
#else
    float a0, a1, b0, b1;
    a.get(a0, a1);
    b.get(b0, b1);
    return Pair(a0 + b0, a1 + b1);
#endif
}
__host__ __device__ __forceinline__ Pair mul_add(Pair a, Pair b, Pair c) {
#ifdef __CUDA_ARCH__
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
#else
    float a0, a1, b0, b1, c0, c1;
    a.get(a0, a1);
    b.get(b0, b1);
    c.get(c0, c1);
    return Pair(fmaf(a0, b0, c0), fmaf(a1, b1, c1));
#endif
}
__host__ __device__ __forceinline__ Pair minus(Pair a, Pair b) { return mul_add(b, Pair(-1.f), a); }

// A sum of up to 256 residuals in units of 2^-44: their leading parts, in units of 2^-22, and what
// is left of them, each at most 2^22 and taken up as the float's bits (one 32-bit addition).  What is
// left is the leading part's rounding, 2^-23 at most, and the errors of the operations before it: of
// the difference, of the product, and A's second part times q.  Where the residual is in (0, 1/2]
// these are at most 2^-26, 2^-25 and 2^-24, above 1/2 (so A q below 1/2) 2^-25, 2^-26 and 2^-25: less
// than 2^-23 together.  So both need the whole range of 2^-22, and a finer unit would leave the range
// in which the float's bits count its steps.
struct Few {
    unsigned hi, lo;
    __host__ __device__ __forceinline__ long long sum(int n) const {
        return (long long)(int)(hi - n * MAGIC_BITS) * 4194304ll + (int)(lo - n * MAGIC_BITS);
    }
};

// Adds max(p - A q, 0) of two elements.
template <int FORM>
__host__ __device__ __forceinline__ void add_residuals(float p0, float p1, float q0, float q1, const Coef& c, Few& few) {
    // p - A q = d + e, e the rounding errors of the product and of the difference (where d > 0)
    Pair d(p0, p1), e(0.f);
    if (FORM != FROM_P) {
        const Pair p = d, q(q0, q1);
        const Pair aq = mul(Pair(FORM == MINUS_Q ? -1.f : -c.ah), q);             // - A q, rounded
        d = add(p, aq);
        e = add(minus(p, d), aq);
        if (FORM == MINUS_AQ) e = minus(e, mul_add(Pair(c.al), q, mul_add(Pair(c.ah), q, aq)));
        float s0, s1, d0, d1, e0, e1;
        add(d, e).get(s0, s1);
        d.get(d0, d1);
        e.get(e0, e1);
        d = Pair(s0 > 0.f ? d0 : 0.f, s1 > 0.f ? d1 : 0.f);
        e = Pair(s0 > 0.f ? e0 : 0.f, s1 > 0.f ? e1 : 0.f);
    }
    const Pair th = mul_add(d, Pair(4194304.f), Pair(MAGIC));                     // d * 2^22
    const Pair hi = add(th, Pair(-MAGIC));
    Pair rem = mul_add(hi, Pair(-2.384185791015625e-07f), d);                     // |rem| <= 2^-23
    if (FORM != FROM_P) rem = add(rem, e);                                        // |rem| <= 2^-22
    const Pair tl = mul_add(rem, Pair(17592186044416.f), Pair(MAGIC));            // rem * 2^44
    float a0, a1, b0, b1;
    th.get(a0, a1);
    tl.get(b0, b1);
    few.hi += float_bits(a0) + float_bits(a1);
    few.lo += float_bits(b0) + float_bits(b1);
}

// Of one element.
template <int FORM>
__host__ __device__ __forceinline__ long long residual(float p, float q, const Coef& c) {
    Few few = {0, 0};
    add_residuals<FORM>(p, 0.f, q, 0.f, c, few);
    return few.sum(2);
}

}  // namespace mla
