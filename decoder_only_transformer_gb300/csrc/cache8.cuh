// cache8.cuh - the 8-bit key/value cache: codes, scales, and the rows of its sequences.
//
// Codes [B, Hkv, max_seq, dh], one byte each: int8, or e4m3 (the fp8 format of 4 exponent
// and 3 mantissa bits).  Scales [B, Hkv, ceil(max_seq / block)] fp32: a position's value is
// code * scale of its block of positions.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace tfm {

// Rows of sequence b among the packed new rows, n = 0 if they are not as they should be.
struct SeqRows {
    int row0;          // first row
    int n;             // rows
    int len;           // cached positions, the n new ones the last
    bool ok;
};

// Rows [first, end) and the length of a sequence.
__device__ __forceinline__ SeqRows seq_rows(int first, int end, int len, int T, int max_seq) {
    SeqRows s;
    const bool rows_ok = first >= 0 && end >= first && end <= T;
    s.row0 = first;
    s.n = rows_ok ? end - first : 0;
    s.len = len;
    s.ok = rows_ok && len >= 0 && len <= max_seq;
    return s;
}
__device__ __forceinline__ SeqRows seq_rows(const int32_t* __restrict__ cu, const int32_t* __restrict__ lens, int b,
                                            int per, int T, int max_seq) {
    const int len = __ldg(lens + b);
    return cu ? seq_rows(__ldg(cu + b), __ldg(cu + b + 1), len, T, max_seq) : seq_rows(b * per, (b + 1) * per, len, T, max_seq);
}

// ------------------------------------------------------------------ codes
// The code of x / s (s > 0), the nearest, ties to even, as 64 bits decide it: the quotient
// of two fp32 numbers is never within 2^-53 of a border between two codes unless it lies
// on it, so its rounding to fp64 decides as the quotient itself would.  NaN gives 0,
// infinities the largest code.  Slow: for extreme scales and
// units with such values only.
template <bool E4M3>
static __device__ __noinline__ uint32_t code_exact(float x, float s) {
    if (x != x) return 0;
    const double q = (double)x / (double)s;
    if constexpr (E4M3) {
        float f = __double2float_rz(q);
        if ((double)f != q) f = __uint_as_float(__float_as_uint(f) | 1u);       // to odd: no second rounding
        return (uint32_t)__nv_cvt_float_to_fp8(f, __NV_SATFINITE, __NV_E4M3);
    } else {
        return (uint32_t)__double2int_rn(fmin(fmax(q, -127.0), 127.0)) & 255u;
    }
}

template <bool E4M3>
__device__ __forceinline__ float code_top() { return E4M3 ? 448.0f : 127.0f; }

// x / s as fp32 on the right side of the one border between two codes in its cell: y = x r
// (r = 1 / s rounded) is within 2 ulp of the quotient, and the sign of x - s m, which a
// fused multiply-add gives exactly for scales between 2^-100 and 2^100, says on which side
// of the border m the quotient lies, or that it lies on it.
template <bool E4M3>
__device__ __forceinline__ float settled(float x, float s, float r) {
    float a = fabsf(x) * r;
    float m;
    if constexpr (E4M3) {
        m = a < 0.015625f ? (floorf(a * 512.0f) + 0.5f) * 0x1p-9f                       // subnormal codes: steps of 2^-9
                          : __uint_as_float((__float_as_uint(a) & 0xFFF00000u) | 0x80000u);
    } else {
        m = floorf(a) + 0.5f;
    }
    const float d = fmaf(-s, m, fabsf(x));
    if (d > 0.0f) a = fmaxf(a, __uint_as_float(__float_as_uint(m) + 1u));
    else if (d < 0.0f) a = fminf(a, __uint_as_float(__float_as_uint(m) - 1u));
    else a = m;
    return copysignf(a, x);
}

// One code of a quotient that fp32 holds on the right side of every border.
template <bool E4M3>
__device__ __forceinline__ uint32_t code_of(float y) {
    if constexpr (E4M3) return (uint32_t)__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
    else return (uint32_t)__float2int_rn(y) & 255u;
}

// The codes of x0 .. x3 in `w`, of which those in the bytes of `open` are still to be decided.
template <bool E4M3>
static __device__ __noinline__ uint32_t decide(uint32_t w, uint32_t open, float x0, float x1, float x2, float x3, float s,
                                               float r) {
    while (open) {
        const int at = (__ffs(open) - 1) & 24;
        const float x = at & 16 ? (at & 8 ? x3 : x2) : (at & 8 ? x1 : x0);
        const uint32_t byte = 255u << at;
        w = (w & ~byte) | code_of<E4M3>(settled<E4M3>(x, s, r)) << at;
        open &= ~byte;
    }
    return w;
}

// Four codes of x[0..4) r in a word, for the two reciprocals r1 and r2.
template <bool E4M3>
__device__ __forceinline__ uint2 codes4(const float* x, float r1, float r2) {
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float f = k ? r2 : r1;
        if constexpr (E4M3) {
            asm("{\n\t.reg .b16 a, b;\n\tcvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
                "mov.b32 %0, {a, b};\n\t}"
                : "=r"(w[k]) : "f"(x[0] * f), "f"(x[1] * f), "f"(x[2] * f), "f"(x[3] * f));
        } else {
            // the last bits of x r + 1.5 2^23, rounded once, are the integer
            uint32_t u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = __float_as_uint(fmaf(x[j], f, 12582912.0f));
            w[k] = __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
        }
    }
    return make_uint2(w[0], w[1]);
}

// How the codes of a unit's rows are decided, for scales s between 2^-100 and 2^100.  With r = 1 / s
// rounded, x / s lies between x r (1 - 2^-22) and x r (1 + 2^-22).
//
// bf16 rows, s = A / top rounded to fp32 for a bf16 number A (which every scale is that bf16 rows
// made): x top / A is a quotient of integers below 2^17 times a power of two, so that it lies on a border between
// two codes or more than 2^-17 of itself away from it, and borders are frequent.  x / s is x top / A times
// (1 + d), d the rounding of s (below 2^-23): quotients on a border are moved all to one side of it,
// which d's sign gives, the others to none.  So x r (1 -+ 2^-22) rounds to the code; and if d = 0 the
// two differ exactly where x / s lies on a border, and the even one is the code.
// Otherwise (fp32 rows, foreign scales) `sure` is 0, and codes that differ are looked at (decide).
struct Recip {
    float s, r, r1, r2;
    bool sure;
};
template <bool E4M3>
__device__ __forceinline__ Recip recip(float s, bool bf16_rows) {
    Recip c;
    c.s = s;
    c.r = __frcp_rn(s);
    c.r1 = c.r * (1.0f - 0x1p-22f);
    c.r2 = c.r * (1.0f + 0x1p-22f);
    const float top = code_top<E4M3>();
    const float A = __bfloat162float(__float2bfloat16_rn(s * top));
    c.sure = bf16_rows && __fdiv_rn(A, top) == s;
    if (c.sure) {
        const float d = fmaf(s, top, -A);
        if (d > 0.0f) c.r2 = c.r1;
        if (d < 0.0f) c.r1 = c.r2;
    }
    return c;
}
template <bool E4M3, bool SURE>
__device__ __forceinline__ uint32_t codes_of4(const float* x, const Recip& c) {
    const uint2 w = codes4<E4M3>(x, c.r1, c.r2);
    if (SURE) return w.x ^ ((w.x ^ w.y) & ((w.x & 0x01010101u) * 255u));  // where they differ, the even one
    if (w.x != w.y) return decide<E4M3>(w.x, w.x ^ w.y, x[0], x[1], x[2], x[3], c.s, c.r);
    return w.x;
}

template <bool E4M3>
__device__ __forceinline__ float code_value(uint32_t c) {      // the low byte
    if constexpr (E4M3) {
        const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)(c & 255u), __NV_E4M3);
        return __half2float(__half(h));
    } else {
        return (float)(int8_t)(c & 255u);
    }
}

}  // namespace tfm
