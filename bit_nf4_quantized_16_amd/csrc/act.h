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
// (1 + 0.32 a). P is the polynomial of degree 5 with the least largest relative
// error over [0, 40] (a linear program over 2100 points): 1.1e-5, 2^-7.5 of
// bf16's half step. With degree 4 it is 6e-5, with a polynomial in a for the
// logarithm of the odds 3e-4 up to a = 8 for as many operations.
__device__ __forceinline__ float normal_tail(float a) {
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.32f, a, 1.0f));
    float p = -0.06677417457103729f;
    p = __builtin_fmaf(p, t, 0.13958674669265747f);
    p = __builtin_fmaf(p, t, 0.04961111769080162f);
    p = __builtin_fmaf(p, t, 0.12305349111557007f);
    p = __builtin_fmaf(p, t, 0.12682759761810303f);
    p = __builtin_fmaf(p, t, 0.12768974900245667f);
    return p * t * __builtin_amdgcn_exp2f(a * a * -0.721347520f);
}
__device__ __forceinline__ float normal_cdf(float z) {
    const float h = normal_tail(fabsf(z));
    return z < 0.0f ? h : 1.0f - h;
}

// 2 sqrt(2 / pi) log2 e
constexpr float kGeluTanh = 2.30220819f, kGeluCube = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == QL_ACT_SILU) return z * logistic2(1.44269504f * z);
    if constexpr (ACT == QL_ACT_GELU) return z * normal_cdf(z);
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
        return __builtin_fmaf(0.398942280f * z, __builtin_amdgcn_exp2f(z * z * -0.721347520f), normal_cdf(z));
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

// What follows a product's sum z, output n of a row with its residual at i:
// act(z + bias) + residual in fp32; z + bias is kept for the backward where
// asked.
struct Epilogue {
    const uint16_t* bias;  // [N], null: none
    const uint16_t* res;   // as the output, null: none
    uint16_t* z;           // as the output, null: not kept
    int act;
};

}  // namespace qlnf4
