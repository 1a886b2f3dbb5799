// ffn_act.cuh -- activations of the gated feed-forward, their slopes, and stores of 16-bit results.
#pragma once

#include "block_common.cuh"

namespace gdr {

enum FfnActivation { FFN_SILU = 0, FFN_SIGMOID = 1, FFN_GELU_TANH = 2 };

// 1 / (1 + exp(-x)) by the approximate exponential (2 + 1.2 |x| units in the last place) and quotient (2 of them): off by 2^-20
// of itself around 0, by up to 2^-16 where x comes near -87, and 0 from -87.4 down, where it is below 2^-126.  Results round to
// 2^-8 or 2^-11.
__device__ __forceinline__ float fast_sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

constexpr float GELU_C = 0.79788456f, GELU_B = 0.044715f;  // sqrt(2 / pi)

// gelu with tanh: g (1 + tanh(y)) / 2 = g sigmoid(2 y), y = C (g + B g^3), which keeps its digits where tanh comes near -1.
template <int ACT> __device__ __forceinline__ float activate(float g) {
    if constexpr (ACT == FFN_SIGMOID) return fast_sigmoid(g);
    if constexpr (ACT == FFN_SILU) return g * fast_sigmoid(g);
    return g * fast_sigmoid(2.f * GELU_C * g * fmaf(GELU_B * g, g, 1.f));
}
// s = sigmoid(x) and t = s (1 - s), neither of them by a difference.
__device__ __forceinline__ void sigmoid_slope(float x, float &s, float &t) {
    const float e = __expf(-fabsf(x)), r = __fdividef(1.f, 1.f + e), er = e * r;
    s = x < 0.f ? er : r;
    t = er * r;
}
template <int ACT> __device__ __forceinline__ void activate_slope(float g, float &a, float &da) {
    float s, t;
    if constexpr (ACT == FFN_GELU_TANH) {
        sigmoid_slope(2.f * GELU_C * g * fmaf(GELU_B * g, g, 1.f), s, t);
        a = g * s;
        const float slope = 2.f * GELU_C * g * fmaf(3.f * GELU_B * g, g, 1.f);  // g times the slope of 2 y
        da = t == 0.f ? s : fmaf(slope, t, s);  // (far out the slope passes fp32 where t is 0)
    } else {
        sigmoid_slope(g, s, t);
        a = ACT == FFN_SILU ? g * s : s;
        da = ACT == FFN_SILU ? fmaf(g, t, s) : t;
    }
}

// ---- 32 values of a result's row, the first `n` of which lie inside it, rounded and stored in pieces of 32 or 16 bytes.
template <typename T> __device__ __forceinline__ void store_row32(T *to, const float (&v)[32], int n, int piece) {
    constexpr int WORDS = 8 * sizeof(T), PER = 32 / (int)sizeof(T);  // words of the row, elements of 32 bytes
    uint32_t w[WORDS];
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
        if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v[i]);
        else w[i] = Pair<T>::of(v[2 * i], v[2 * i + 1]);
    }
    if (piece >= 32) {
#pragma unroll
        for (int i = 0; i < WORDS / 8; ++i)
            if (PER * i < n)
                asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to + PER * i), "r"(w[8 * i]),
                             "r"(w[8 * i + 1]), "r"(w[8 * i + 2]), "r"(w[8 * i + 3]), "r"(w[8 * i + 4]), "r"(w[8 * i + 5]),
                             "r"(w[8 * i + 6]), "r"(w[8 * i + 7])
                             : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < WORDS / 4; ++i)
            if (PER / 2 * i < n)
                *reinterpret_cast<uint4 *>(to + PER / 2 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
}
__device__ __forceinline__ void store_part32(float *to, const float (&v)[32]) {  // of a partial result
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to + 8 * i), "f"(v[8 * i]), "f"(v[8 * i + 1]),
                     "f"(v[8 * i + 2]), "f"(v[8 * i + 3]), "f"(v[8 * i + 4]), "f"(v[8 * i + 5]), "f"(v[8 * i + 6]), "f"(v[8 * i + 7])
                     : "memory");
}

}  // namespace gdr
