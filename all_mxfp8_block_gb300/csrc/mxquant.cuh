// Device helpers shared by the mixture-of-experts and linear-layer kernels:
// typed loads as fp32, the MX scale of a 32-element block, E4M3 / E5M2
// encoding, and the place of a scale byte in the MMA's scale tiles.
//
// MX block (OCP MX, as the library's input quantiser): the block's shared
// exponent is X = floor(log2 amax) - emax (emax 8 for E4M3, 15 for E5M2),
// clamped to >= -127; a code is the value / 2^X saturated to the format's
// largest value and rounded to nearest even.  An all-zero block has scale
// byte 0 and zero codes; a block holding an infinity or a NaN has scale 0xFF
// (the E8M0 NaN) and NaN codes, so it cannot pass for numbers.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>
#include <type_traits>

#include "kernels.cuh"
#include "ptx.cuh"

namespace mxa2a {

// element types (the C ABI's numbers)
constexpr int kTypeBf16 = 0, kTypeF16 = 1, kTypeF32 = 2, kTypeE4M3 = 3, kTypeE5M2 = 4;
constexpr uint32_t kLanes = 0xffffffffu;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// V consecutive elements of type T at p, as fp32 (V * sizeof(T) a multiple of
// 16 and p aligned to 16 bytes, or V = 1)
template <typename T, int V>
struct Vec {
    static_assert(V == 1 || (V * sizeof(T)) % 16 == 0, "vector width");
    static constexpr int kWords = V * (int)sizeof(T) / 16;
    // as loaded: half the registers of the fp32 values for 16-bit types
    struct Raw {
        uint4 w[V == 1 ? 1 : kWords];
    };
    __device__ static __forceinline__ Raw raw(const T* p) {
        Raw r;
        if constexpr (V == 1) {
            r.w[0].x = sizeof(T) == 4 ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p);
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) r.w[i] = ptx::ld_nc_v4(reinterpret_cast<const uint4*>(p) + i);
        }
        return r;
    }
    __device__ static __forceinline__ void values(const Raw& r, float (&f)[V]) {
        if constexpr (V > 1) {
            unpack(r.w, f);
        } else if constexpr (sizeof(T) == 4) {
            f[0] = __uint_as_float(r.w[0].x);
        } else {
            const uint16_t h = (uint16_t)r.w[0].x;
            f[0] = (float)*reinterpret_cast<const T*>(&h);
        }
    }
    __device__ static __forceinline__ void load(const T* p, float (&f)[V]) { values(raw(p), f); }
    __device__ static __forceinline__ void unpack(const uint4* w, float (&f)[V]) {
        const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = __uint_as_float(u[i]);
        } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                f[2 * i] = bf16_lo(u[i]);
                f[2 * i + 1] = bf16_hi(u[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
                f[2 * i] = t.x;
                f[2 * i + 1] = t.y;
            }
        }
    }
    __device__ static __forceinline__ void store(T* p, const float (&f)[V]) {
        if constexpr (V == 1) {
            *p = (T)f[0];
        } else {
            uint32_t u[kWords * 4];
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int i = 0; i < V; ++i) u[i] = __float_as_uint(f[i]);
            } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
                for (int i = 0; i < V / 2; ++i) u[i] = bf16x2_bits(f[2 * i], f[2 * i + 1]);
            } else {
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                    u[i] = *reinterpret_cast<const uint32_t*>(&h);
                }
            }
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                reinterpret_cast<uint4*>(p)[i] = make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
        }
    }
};

// scale byte of a block whose largest |value| has these fp32 bits (taken as an
// unsigned maximum of the bit patterns, which orders NaN above infinity)
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits, int emax) {
    const int e = (int)(amax_bits >> 23);   // 0 for zero and for subnormals, which clamp to -127 as well
    return e == 255 ? 255u : (uint32_t)max(e - emax, 0);
}
// 2^-X of a scale byte X + 127: a normal number (X >= -127, X <= 119), NaN for byte 255
__device__ __forceinline__ float mx_inv_scale(uint32_t byte) {
    return __uint_as_float(byte == 255 ? 0x7fffffffu : (254u - byte) << 23);
}

// max(m, |a|, |b|), keeping a NaN: one instruction
__device__ __forceinline__ float abs_max(float m, float a, float b) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
    return r;
}
// two fp32 operations in one instruction, each rounded as the single one
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(r))
        : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(r))
        : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(r))
        : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)),
          "l"(reinterpret_cast<const uint64_t&>(c)));
    return r;
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// two codes, lo in the low byte (saturating, nearest even)
template <bool kE5m2>
__device__ __forceinline__ uint32_t fp8x2(float lo, float hi) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, kE5m2 ? __NV_E5M2 : __NV_E4M3);
}
// four codes of v / 2^X (inv = 2^-X; a block with a NaN scale passes inv = NaN,
// which makes all its codes NaN, 0x7f in both formats)
template <bool kE5m2>
__device__ __forceinline__ uint32_t mx_codes4(float2 a, float2 b, float inv) {
    a = mul2(a, both(inv));
    b = mul2(b, both(inv));
    return __byte_perm(fp8x2<kE5m2>(a.x, a.y), fp8x2<kE5m2>(b.x, b.y), 0x5410);
}
template <bool kE5m2>
__device__ constexpr int mx_emax() { return kE5m2 ? 15 : 8; }

// byte offset of the scale word (4 scales: 128 elements along the contraction)
// of row r, contraction block kb of 128, among rt row tiles of 128 rows
__device__ __forceinline__ size_t scale_word(int kb, long long r, int rt) {
    return ((size_t)kb * rt + (size_t)(r >> 7)) * 512 + (size_t)((r & 31) * 16 + ((r & 127) >> 5) * 4);
}

__device__ __forceinline__ float exp2f_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// maxima and minima that keep a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Activations and their derivatives in fp32 (ids as in the C ABI), through
// s = logistic(x) = 1 / (1 + e), e = exp(-x), and 1 - s = s e.  Relative errors,
// in units of 2^-24: e's exponent is rounded before the power is taken, 1.25 |x|
// (silu, x = z) or 6 |x| (gelu, x = 2 u); ex2, the reciprocal and the products 8
// more.  So a value is off by 8 near 0 and above it, by some tens where it is far
// below its argument (at most 83 for silu at -60, 304 for gelu at -8).  A slope's
// second term has twice that, and its two cancel at the curve's lowest point.
//   gelu(z) = 0.5 z (1 + tanh u) = z logistic(2 u), u = sqrt(2/pi) (z + 0.044715 z^3)
// The logistic's argument is kept where e is finite, i.e. z >= -87 (silu) or
// |z| <= 10 (gelu); past it the values are the saturated ones to 1e-35.  The
// slopes' z is kept at or below 87 (silu) or 10 as well, where they are 1: they
// multiply z by e, and at +inf that would be inf * 0.
constexpr int kActNone = 0, kActRelu = 1, kActGelu = 2, kActSilu = 3;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluA = 2.f * 0.7978845608028654f, kGeluB = 0.044715f;   // 2 sqrt(2 / pi)
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float logistic_e(float e) { return rcp_approx(1.f + e); }
template <int kAct>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (kAct == kActRelu) {
        return max_nan(z, 0.f);
    } else if constexpr (kAct == kActSilu) {
        const float l = max_nan(z, -87.f);
        return l * logistic_e(exp2f_approx(-kLog2e * l));
    } else if constexpr (kAct == kActGelu) {
        const float l = max_nan(z, -10.f), m = min_nan(l, 10.f);
        const float u = m * fmaf(kGeluA * kGeluB * -kLog2e, m * m, kGeluA * -kLog2e);
        return l * logistic_e(exp2f_approx(u));
    }
    return z;
}
// g * act'(z) for two values at a time
template <int kAct>
__device__ __forceinline__ float2 act_back2(float2 g, float2 z) {
    if constexpr (kAct == kActRelu) {
        return make_float2(z.x > 0.f ? g.x : (z.x != z.x ? z.x : 0.f), z.y > 0.f ? g.y : (z.y != z.y ? z.y : 0.f));
    } else if constexpr (kAct == kActSilu) {
        const float2 m = make_float2(min_nan(max_nan(z.x, -87.f), 87.f), min_nan(max_nan(z.y, -87.f), 87.f)), x = mul2(m, both(-kLog2e));
        const float2 e = make_float2(exp2f_approx(x.x), exp2f_approx(x.y)), d = add2(e, both(1.f));
        const float2 s = make_float2(rcp_approx(d.x), rcp_approx(d.y));
        return mul2(g, fma2(mul2(m, s), mul2(s, e), s));
    } else if constexpr (kAct == kActGelu) {
        const float2 m = make_float2(min_nan(max_nan(z.x, -10.f), 10.f), min_nan(max_nan(z.y, -10.f), 10.f)), m2 = mul2(m, m);
        const float2 x = mul2(m, fma2(m2, both(kGeluA * kGeluB * -kLog2e), both(kGeluA * -kLog2e)));
        const float2 e = make_float2(exp2f_approx(x.x), exp2f_approx(x.y)), d = add2(e, both(1.f));
        const float2 s = make_float2(rcp_approx(d.x), rcp_approx(d.y));
        const float2 w = fma2(m2, both(3.f * kGeluA * kGeluB), both(kGeluA));
        return mul2(g, fma2(mul2(mul2(m, s), mul2(s, e)), w, s));
    }
    return g;
}

}  // namespace mxa2a
