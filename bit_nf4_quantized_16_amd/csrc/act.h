// Activations of the linear layer's epilogue and their slopes (gfx950), in fp32
// for results that are rounded to bf16.
#pragma once

#include "common.h"

namespace qlnf4 {

// 1 / (1 + 2^-x): v_exp_f32 and v_rcp_f32, 1 ulp each.
__device__ __forceinline__ float logistic2(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-x));
}

// The normal distribution function of -a, a >= 0: e^(-a^2 / 2) t P(t), t = 1 /
// (1 + k a), P the polynomial with the least largest relative error over [0,
// 40] (a linear program over 2100 points). For values, which are rounded to
// bf16, degree 5: 1.1e-5, 2^-7.5 of the half step (degree 4: 6e-5; a polynomial
// in a for the logarithm of the odds 3e-4 up to a = 8 for as many operations).
// Formed in fp32 it is 1.2e-5 up to a = 6 and 1.8e-5 up to 13, where the result
// leaves fp32: the exponent, up to 122, is rounded twice.
// For slopes, whose sums over rows stay fp32, degree 8: 1.2e-7 with the
// coefficients as fp32 holds them, before fp32's own roundings (with degree 5 a
// bias's gradient was off by 2.2e-6 of its norm, with 8 by 4e-7).
template <bool FINE>
__device__ __forceinline__ float normal_tail(float a) {
    constexpr float kFine[9] = {0.14361748099327087f,   0.14368759095668793f, 0.12394635379314423f,
                                0.09638447314500809f,   -0.0014430495211854577f, 0.1092388704419136f,
                                -0.22550803422927856f,  0.14054939150810242f, -0.030473075807094574f};
    constexpr float kCoarse[6] = {0.12768974900245667f, 0.12682759761810303f, 0.12305349111557007f,
                                  0.04961111769080162f, 0.13958674669265747f, -0.06677417457103729f};
    constexpr int n = FINE ? 9 : 6;
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(FINE ? 0.36f : 0.32f, a, 1.0f));
    float p = FINE ? kFine[n - 1] : kCoarse[5];
#pragma unroll
    for (int i = n - 2; i >= 0; --i) p = __builtin_fmaf(p, t, FINE ? kFine[i] : kCoarse[i < 6 ? i : 0]);
    return p * t * __builtin_amdgcn_exp2f(a * a * -0.721347520f);
}
template <bool FINE>
__device__ __forceinline__ float normal_cdf(float z) {
    const float h = normal_tail<FINE>(fabsf(z));
    return z < 0.0f ? h : 1.0f - h;
}

// 2 sqrt(2 / pi) log2 e
constexpr float kGeluTanh = 2.30220819f, kGeluCube = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == QL_ACT_SILU) return z * logistic2(1.44269504f * z);
    if constexpr (ACT == QL_ACT_GELU) return z * normal_cdf<false>(z);
    if constexpr (ACT == QL_ACT_GELU_TANH)  // z (1 + tanh(y)) / 2 = z / (1 + e^-2y)
        return z * logistic2(kGeluTanh * z * __builtin_fmaf(kGeluCube * z, z, 1.0f));
    return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == QL_ACT_SILU) {
        const float p = logistic2(1.44269504f * z);
        return p * __builtin_fmaf(z, 1.0f - p, 1.0f);
    }
    if constexpr (ACT == QL_ACT_GELU)
        return __builtin_fmaf(0.398942280f * z, __builtin_amdgcn_exp2f(z * z * -0.721347520f), normal_cdf<true>(z));
    if constexpr (ACT == QL_ACT_GELU_TANH) {
        const float p = logistic2(kGeluTanh * z * __builtin_fmaf(kGeluCube * z, z, 1.0f));
        // 2 y' z, y' = sqrt(2 / pi) (1 + 3 c z^2); past 16, where p is 0 or 1, any finite value
        const float c = __builtin_amdgcn_fmed3f(z, -16.0f, 16.0f);
        const float d = 1.59576912f * c * __builtin_fmaf(3.0f * kGeluCube * c, c, 1.0f);
        return p * __builtin_fmaf(d, 1.0f - p, 1.0f);
    }
    return 1.0f;
}

// f with the activation as a compile-time number.
template <typename F>
__host__ __device__ __forceinline__ void with_act(int act, F f) {
    switch (act) {
        case QL_ACT_SILU: f(std::integral_constant<int, QL_ACT_SILU>{}); break;
        case QL_ACT_GELU: f(std::integral_constant<int, QL_ACT_GELU>{}); break;
        case QL_ACT_GELU_TANH: f(std::integral_constant<int, QL_ACT_GELU_TANH>{}); break;
        default: f(std::integral_constant<int, QL_ACT_NONE>{}); break;
    }
}

// What follows a product's sum: act(z) + residual with z = sum + bias, in fp32;
// z is kept for the backward where asked, in fp32 or rounded to bf16.
struct Epilogue {
    const uint16_t* bias;  // [N], null: none
    const uint16_t* res;   // as the output, null: none
    void* z;               // as the output, null: not kept
    int z_f32;
    int act;

    __device__ __forceinline__ void keep(int64_t at, float v) const {
        if (z == nullptr) return;
        if (z_f32)
            static_cast<float*>(z)[at] = v;
        else
            static_cast<uint16_t*>(z)[at] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
    }
    // eight values at a multiple of eight
    __device__ __forceinline__ void keep8(int64_t at, const float (&v)[8]) const {
        if (z == nullptr) return;
        if (z_f32) {
            float4* const o = reinterpret_cast<float4*>(static_cast<float*>(z) + at);
            o[0] = make_float4(v[0], v[1], v[2], v[3]);
            o[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(z) + at) =
                make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        }
    }
    // four values at a multiple of four
    __device__ __forceinline__ void keep4(int64_t at, float a, float b, float c, float d) const {
        if (z == nullptr) return;
        if (z_f32)
            *reinterpret_cast<float4*>(static_cast<float*>(z) + at) = make_float4(a, b, c, d);
        else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(z) + at) = make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
    }
};

}  // namespace qlnf4
