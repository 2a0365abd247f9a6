// linear_common.h -- device and host pieces shared by the layer products
// (linear.hip) and the dropout (dropout.hip): the counter-based mask, the
// activations, 16-bit conversions, argument checks.  Internal.
#ifndef ZERO_SHARD_LINEAR_COMMON_H
#define ZERO_SHARD_LINEAR_COMMON_H

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "host_common.h"
#include "zero_linear.h"

namespace zero_linear_impl {

using f32x4 = float __attribute__((ext_vector_type(4)));
using u32x4 = uint32_t __attribute__((ext_vector_type(4)));
using u16x4 = uint16_t __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// 16-bit element types

struct BF16 {
    static __device__ __forceinline__ float up(uint16_t h) {
        return __builtin_bit_cast(float, static_cast<uint32_t>(h) << 16);
    }
    static __device__ __forceinline__ uint16_t down(float f) {
        return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
    }
};
struct FP16 {
    static __device__ __forceinline__ float up(uint16_t h) {
        return static_cast<float>(__builtin_bit_cast(_Float16, h));
    }
    static __device__ __forceinline__ uint16_t down(float f) {
        return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
    }
};

// Four elements as fp32, and back; n < 4 touches the first n only.  Whole
// quads are one access whatever their alignment, which global memory takes.
template <class T>
__device__ __forceinline__ f32x4 load16(const uint16_t *p, int n) {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (n == 4) {
        u16x4 h;
        __builtin_memcpy(&h, p, 8);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = T::up(h[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < n) v[e] = T::up(p[e]);
    }
    return v;
}

template <class T>
__device__ __forceinline__ void store16(uint16_t *p, f32x4 v, int n) {
    u16x4 h;
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = T::down(v[e]);
    if (n == 4) {
        __builtin_memcpy(p, &h, 8);
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < n) p[e] = h[e];
    }
}

__device__ __forceinline__ f32x4 load32(const float *p, int n) {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (n == 4) {
        __builtin_memcpy(&v, p, 16);
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < n) v[e] = p[e];
    }
    return v;
}

__device__ __forceinline__ void store32(float *p, f32x4 v, int n) {
    if (n == 4) {
        __builtin_memcpy(p, &v, 16);
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < n) p[e] = v[e];
    }
}

// eight elements at once
using u16x8 = uint16_t __attribute__((ext_vector_type(8)));

template <class T>
__device__ __forceinline__ void load16x8(const uint16_t *p, f32x4 &a, f32x4 &b) {
    u16x8 h;
    __builtin_memcpy(&h, p, 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        a[e] = T::up(h[e]);
        b[e] = T::up(h[e + 4]);
    }
}

template <class T>
__device__ __forceinline__ void store16x8(uint16_t *p, f32x4 a, f32x4 b) {
    u16x8 h;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        h[e] = T::down(a[e]);
        h[e + 4] = T::down(b[e]);
    }
    __builtin_memcpy(p, &h, 16);
}

// The same, past the caches' usual order (the tiles' outputs: 8192 x 6400 x
// 1600 with GELU and z 242 -> 224 us when it came in).  The dropout's own
// stores lose by it, and so do fp32 outputs: the weight gradient 4096 x 4096
// over 512 rows would take 44 us for 28, 333 x 50257 x 1600 133 for 98.
using u16x8_any = u16x8 __attribute__((aligned(2)));

template <class T>
__device__ __forceinline__ void stream16x8(uint16_t *p, f32x4 a, f32x4 b) {
    u16x8 h;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        h[e] = T::down(a[e]);
        h[e + 4] = T::down(b[e]);
    }
    __builtin_nontemporal_store(h, reinterpret_cast<u16x8_any *>(p));
}

// ---------------------------------------------------------------------------
// dropout

struct Drop {
    uint32_t on, threshold, k0, k1, row0;
    float scale;
    uint64_t offset;
    const int64_t *step;
};

// a ^ b ^ c in one instruction (0x96: the truth table of the three)
__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
    return static_cast<uint32_t>(__builtin_amdgcn_bitop3_b32(
        static_cast<int>(a), static_cast<int>(b), static_cast<int>(c), 0x96));
}

// Philox4x32-10 (the generator of Salmon et al., 2011): ten rounds of two
// 32 x 32 -> 64 bit products.  Integer work of about 20 full products for
// eight mask elements.
__device__ __forceinline__ u32x4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                        uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c0;
        const uint64_t p1 = static_cast<uint64_t>(0xCD9E8D57u) * c2;
        c0 = xor3(static_cast<uint32_t>(p1 >> 32), c1, k0);
        c1 = static_cast<uint32_t>(p1);
        c2 = xor3(static_cast<uint32_t>(p0 >> 32), c3, k1);
        c3 = static_cast<uint32_t>(p0);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u32x4{c0, c1, c2, c3};
}

__device__ __forceinline__ uint64_t drop_stream(const Drop &d) {
    return d.offset + (d.step != nullptr ? static_cast<uint64_t>(*d.step) : 0u);
}

// The words of (row, block).  One call serves the columns 4b..4b+3 (low
// halves) and 16+4b..16+4b+3 (high halves) of a 32-column group, which is
// what a lane of the products holds of two neighbouring 16 x 16 tiles: no
// random bit is drawn twice or thrown away in either kernel.
__device__ __forceinline__ u32x4 drop_words(const Drop &d, uint64_t stream, uint32_t row,
                                            uint32_t block) {
    return philox(block, d.row0 + row, static_cast<uint32_t>(stream),
                  static_cast<uint32_t>(stream >> 32), d.k0, d.k1);
}

__device__ __forceinline__ f32x4 drop_apply(const Drop &d, u32x4 w, int half, f32x4 v) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t u = half ? w[e] >> 16 : w[e] & 0xFFFFu;
        v[e] = u >= d.threshold ? v[e] * d.scale : 0.0f;
    }
    return v;
}

// ---------------------------------------------------------------------------
// activations (fp32).  Sigmoids are 1 / (1 + 2^(-u log2 e)) by the hardware's
// exp2 and reciprocal, each good to about an ulp.  The argument's own
// roundings weigh |u| in the falling tail: a relative error of
// (6 |u| + 8) 2^-24 at most, 2^-17 at u = -20, below the half step 2^-11 of
// the finest 16-bit output; with an fp32 output it is the largest error of
// the call.  The erf GELU takes erfc, which keeps its relative error there
// (1 + erf cancels: 4 % off at v = -5); its argument's roundings weigh v^2, a
// relative error of (2 v^2 + 14) 2^-24.  A sigmoid below 2^-126 may be 0.

// A 256 x 256 tile's workgroup has its CU alone, so nothing runs beside these
// instructions: the constants are folded and multiply-adds fused.

// 1 / (1 + 2^w)
__device__ __forceinline__ float logistic(float w) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(w));
}
constexpr float kLog2e = 1.44269504088896341f;
// GELU_TANH: (1 + tanh(u / 2)) / 2 = logistic(-u log2 e) with
// u = v (kTanh1 + kTanh3 v^2), and du/dv = kTanh1 + 3 kTanh3 v^2
constexpr float kTanh1 = 1.5957691216057308f, kTanh3 = kTanh1 * 0.044715f;

__device__ __forceinline__ float act_value(float v, int act) {
    switch (act) {
        case ZERO_ACT_RELU: return v > 0.0f ? v : (v != v ? v : 0.0f);
        case ZERO_ACT_GELU: return 0.5f * v * erfcf(v * -0.70710678118654752f);
        case ZERO_ACT_GELU_TANH:
            return v * logistic(v * __builtin_fmaf(-kLog2e * kTanh3, v * v, -kLog2e * kTanh1));
        case ZERO_ACT_SILU: return v * logistic(-kLog2e * v);
        default: return v;
    }
}

// The two activations v logistic(v (c3 v^2 + c1)) without a choice in the
// code, for the straight epilogues: value, and the slope as below.
struct Logistic {
    float c3, c1, d3, d1;
};
__device__ __forceinline__ Logistic logistic_of(int act) {
    return act == ZERO_ACT_SILU
               ? Logistic{0.0f, -kLog2e, 0.0f, 1.0f}
               : Logistic{-kLog2e * kTanh3, -kLog2e * kTanh1, 3.0f * kTanh3, kTanh1};
}
// v^2, kept finite: 0 * Inf would spoil SILU
__device__ __forceinline__ float square(float v) { return fminf(v * v, 3e38f); }
__device__ __forceinline__ float logistic_value(float v, const Logistic &l) {
    return v * logistic(v * __builtin_fmaf(l.c3, square(v), l.c1));
}
__device__ __forceinline__ float logistic_slope(float v, const Logistic &l) {
    const float q = square(v);
    const float s = logistic(v * __builtin_fmaf(l.c3, q, l.c1)), t = __builtin_fmaf(-s, s, s);
    return t == 0.0f ? s : __builtin_fmaf(t, v * __builtin_fmaf(l.d3, q, l.d1), s);
}

// Where the bell factor t of a derivative has vanished its product with v is
// 0 (0 * Inf would not be).
__device__ __forceinline__ float act_slope(float v, int act) {
    float s, t, d;
    switch (act) {
        case ZERO_ACT_GELU:
            s = 0.5f * erfcf(v * -0.70710678118654752f);
            t = __builtin_amdgcn_exp2f(v * v * (-0.5f * kLog2e));
            d = v * 0.39894228040143268f;
            break;
        case ZERO_ACT_GELU_TANH: {
            const float q = v * v;
            s = logistic(v * __builtin_fmaf(-kLog2e * kTanh3, q, -kLog2e * kTanh1));
            t = __builtin_fmaf(-s, s, s);
            d = v * __builtin_fmaf(3.0f * kTanh3, q, kTanh1);
            break;
        }
        default:  // SILU
            s = logistic(-kLog2e * v);
            t = __builtin_fmaf(-s, s, s);
            d = v;
            break;
    }
    return t == 0.0f ? s : __builtin_fmaf(t, d, s);
}

// ---------------------------------------------------------------------------
// host: arguments

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1024;
constexpr int64_t kMaxSpan = int64_t(1) << 60;

inline bool is16(zero_dtype t) { return t == ZERO_BF16 || t == ZERO_FP16; }
inline int64_t size_of(zero_dtype t) { return t == ZERO_FP32 ? 4 : 2; }

// one matrix argument: its checks and its span in memory
struct Mat {
    const void *p;
    int64_t rows, cols, ld, elem;
    bool empty() const { return rows == 0 || cols == 0; }
    // elements from the first to one past the last
    int64_t extent() const { return empty() ? 0 : (rows - 1) * ld + cols; }
    bool ok() const {
        if (ld < cols) return false;
        if (empty()) return true;
        if (p == nullptr || reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(elem) != 0)
            return false;
        return rows == 1 || ld <= (kMaxSpan - cols) / (rows - 1);
    }
    zero_host::Span span() const {
        return p == nullptr ? zero_host::Span{0, 0} : zero_host::span_of(p, extent(), elem);
    }
    bool same_place(const Mat &o) const {
        return p == o.p && (ld == o.ld || rows <= 1) && elem == o.elem;
    }
};

inline bool dim_ok(int64_t d) { return d >= 0 && d <= kMaxDim; }

// EINVAL for parameters out of their domain; fills *out (off for a NULL
// struct or a threshold of zero)
inline bool make_drop(const zero_dropout_params *d, int64_t rows, Drop *out) {
    *out = Drop{};
    if (d == nullptr) return true;
    if (!(d->p >= 0.0 && d->p < 1.0) || d->row0 < 0 || d->row0 > (int64_t(1) << 32) - rows ||
        (reinterpret_cast<uintptr_t>(d->step) & 7u) != 0)
        return false;
    const double t = std::rint(d->p * 65536.0);
    out->threshold = t > 65535.0 ? 65535u : static_cast<uint32_t>(t);
    out->on = out->threshold != 0;
    out->scale = static_cast<float>(65536.0 / (65536.0 - out->threshold));
    out->k0 = static_cast<uint32_t>(d->seed);
    out->k1 = static_cast<uint32_t>(d->seed >> 32);
    out->row0 = static_cast<uint32_t>(d->row0);
    out->offset = d->offset;
    out->step = out->on ? d->step : nullptr;
    return true;
}

}  // namespace zero_linear_impl

#endif
