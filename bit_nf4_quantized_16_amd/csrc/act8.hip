// 8-bit activation checkpoints and the gated activation that uses them
// (gfx950): elementwise kernels over a row-major [rows, cols] activation,
// cols a multiple of 32. The format is in act8.h. Every kernel gives a lane
// eight consecutive values (one 16-byte bf16 access, one 8-byte code access);
// a block of 32 is an aligned quad of lanes, so its maximum takes two DPP
// steps and no LDS, and a wave's accesses are whole lines. All are bound by
// HBM (a large copy: 5.2 TB/s): 4096 x 11008 stored in 24.2 us (5.7 TB/s) and
// restored in 21.0 (6.5, part of it from the last-level cache), the gated
// activation at 4096 x 22016 in 123.8 us forward and 123.8 backward (5.9 TB/s);
// at 77 x 11008 by the launch itself (3.4 us, an empty one takes 3.6 back to
// back).
#include "act8.h"
#include "common.h"
#include "internal.h"

namespace qlnf4 {

namespace {

constexpr int kThreads = 256;

__global__ __launch_bounds__(kThreads) void act8_quantize_kernel(const uint16_t* __restrict__ X, int64_t n8,
                                                                 uint8_t* __restrict__ codes,
                                                                 uint8_t* __restrict__ scale) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= n8) return;  // n8 is a multiple of 4: a quad stays whole
    const uint4 v = *reinterpret_cast<const uint4*>(X + 8 * i);
    const uint32_t b = act8_scale_byte(v);
    *reinterpret_cast<uint2*>(codes + 8 * i) = act8_encode8(v, b);
    if ((i & 3) == 0) scale[i >> 2] = static_cast<uint8_t>(b);
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void act8_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                   const uint8_t* __restrict__ scale, int64_t n8,
                                                                   void* __restrict__ out) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= n8) return;
    const uint4 v = act8_decode8(*reinterpret_cast<const uint2*>(codes + 8 * i), scale[i >> 2]);
    if constexpr (BF16) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + 8 * i) = v;
    } else {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + 8 * i);
        o[0] = make_float4(bf16_to_f32(v.x & 0xFFFFu), __uint_as_float(v.x & 0xFFFF0000u), bf16_to_f32(v.y & 0xFFFFu),
                           __uint_as_float(v.y & 0xFFFF0000u));
        o[1] = make_float4(bf16_to_f32(v.z & 0xFFFFu), __uint_as_float(v.z & 0xFFFF0000u), bf16_to_f32(v.w & 0xFFFFu),
                           __uint_as_float(v.w & 0xFFFF0000u));
    }
}

// 1 / (1 + e^-g): v_exp_f32 and v_rcp_f32 (1 ulp each; the result is rounded
// to bf16 by its users; v_rcp_f32 gives zero for results under 2^-126, g under
// -87.33, where h is under 1e-36 |u|). e^-g = 0 gives 1.
__device__ __forceinline__ float sigmoid(float g) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * g));
}

// h = g sigmoid(g) u in fp32, rounded to bf16 once; checkpoints of g, u and
// of the rounded h, each where its codes pointer is given.
__global__ __launch_bounds__(kThreads) void swiglu_fwd_kernel(const uint16_t* __restrict__ gate,
                                                              const uint16_t* __restrict__ up, int64_t n8,
                                                              uint16_t* __restrict__ H, Act8Dev g8, Act8Dev u8,
                                                              Act8Dev h8) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= n8) return;
    const uint4 gv = *reinterpret_cast<const uint4*>(gate + 8 * i);
    const uint4 uv = *reinterpret_cast<const uint4*>(up + 8 * i);
    const uint32_t gw[4] = {gv.x, gv.y, gv.z, gv.w}, uw[4] = {uv.x, uv.y, uv.z, uv.w};
    uint32_t hw[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float g0 = __uint_as_float(gw[q] << 16), g1 = __uint_as_float(gw[q] & 0xFFFF0000u);
        const float u0 = __uint_as_float(uw[q] << 16), u1 = __uint_as_float(uw[q] & 0xFFFF0000u);
        hw[q] = pack_bf16x2(g0 * sigmoid(g0) * u0, g1 * sigmoid(g1) * u1);
    }
    const uint4 hv = make_uint4(hw[0], hw[1], hw[2], hw[3]);
    *reinterpret_cast<uint4*>(H + 8 * i) = hv;
    auto keep = [&](const Act8Dev& a, const uint4& v) {
        if (a.codes == nullptr) return;
        const uint32_t b = act8_scale_byte(v);
        *reinterpret_cast<uint2*>(a.codes + 8 * i) = act8_encode8(v, b);
        if ((i & 3) == 0) a.scale[i >> 2] = static_cast<uint8_t>(b);
    };
    keep(g8, gv);
    keep(u8, uv);
    keep(h8, hv);
}

// From the restored g and u, with p = sigmoid(g):
//   du = dh g p,   dg = dh u p (1 + g (1 - p))
__global__ __launch_bounds__(kThreads) void swiglu_bwd_kernel(Act8Dev g8, Act8Dev u8, const uint16_t* __restrict__ dH,
                                                              int64_t n8, uint16_t* __restrict__ dgate,
                                                              uint16_t* __restrict__ dup) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= n8) return;
    const uint4 gv = act8_decode8(*reinterpret_cast<const uint2*>(g8.codes + 8 * i), g8.scale[i >> 2]);
    const uint4 uv = act8_decode8(*reinterpret_cast<const uint2*>(u8.codes + 8 * i), u8.scale[i >> 2]);
    const uint4 dv = *reinterpret_cast<const uint4*>(dH + 8 * i);
    const uint32_t gw[4] = {gv.x, gv.y, gv.z, gv.w}, uw[4] = {uv.x, uv.y, uv.z, uv.w}, dw[4] = {dv.x, dv.y, dv.z, dv.w};
    uint32_t og[4], ou[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float rg[2], ru[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float g = __uint_as_float(h ? gw[q] & 0xFFFF0000u : gw[q] << 16);
            const float u = __uint_as_float(h ? uw[q] & 0xFFFF0000u : uw[q] << 16);
            const float d = __uint_as_float(h ? dw[q] & 0xFFFF0000u : dw[q] << 16);
            const float p = sigmoid(g), dp = d * p;
            ru[h] = dp * g;
            rg[h] = dp * u * (1.0f + g * (1.0f - p));
        }
        og[q] = pack_bf16x2(rg[0], rg[1]);
        ou[q] = pack_bf16x2(ru[0], ru[1]);
    }
    *reinterpret_cast<uint4*>(dgate + 8 * i) = make_uint4(og[0], og[1], og[2], og[3]);
    *reinterpret_cast<uint4*>(dup + 8 * i) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
}

dim3 grid_of(int64_t n8) { return dim3(static_cast<uint32_t>(ceil_div(n8, kThreads))); }

}  // namespace

int launch_act8_quantize(const uint16_t* X, int64_t n, Act8Dev out, hipStream_t stream) {
    timer_begin(QL_KERNEL_ACT8, stream);
    hipLaunchKernelGGL(act8_quantize_kernel, grid_of(n / 8), dim3(kThreads), 0, stream, X, n / 8, out.codes, out.scale);
    timer_end(QL_KERNEL_ACT8, stream);
    return check_launch("8-bit activation quantize");
}

int launch_act8_dequantize(Act8Dev a, int64_t n, void* out, bool bf16_out, hipStream_t stream) {
    timer_begin(QL_KERNEL_ACT8, stream);
    if (bf16_out)
        hipLaunchKernelGGL(act8_dequantize_kernel<true>, grid_of(n / 8), dim3(kThreads), 0, stream, a.codes, a.scale,
                           n / 8, out);
    else
        hipLaunchKernelGGL(act8_dequantize_kernel<false>, grid_of(n / 8), dim3(kThreads), 0, stream, a.codes, a.scale,
                           n / 8, out);
    timer_end(QL_KERNEL_ACT8, stream);
    return check_launch("8-bit activation dequantize");
}

int launch_swiglu_fwd(const uint16_t* gate, const uint16_t* up, int64_t n, uint16_t* H, Act8Dev g8, Act8Dev u8,
                      Act8Dev h8, hipStream_t stream) {
    timer_begin(QL_KERNEL_SWIGLU, stream);
    hipLaunchKernelGGL(swiglu_fwd_kernel, grid_of(n / 8), dim3(kThreads), 0, stream, gate, up, n / 8, H, g8, u8, h8);
    timer_end(QL_KERNEL_SWIGLU, stream);
    return check_launch("gated activation forward");
}

int launch_swiglu_bwd(Act8Dev g8, Act8Dev u8, const uint16_t* dH, int64_t n, uint16_t* dgate, uint16_t* dup,
                      hipStream_t stream) {
    timer_begin(QL_KERNEL_SWIGLU, stream);
    hipLaunchKernelGGL(swiglu_bwd_kernel, grid_of(n / 8), dim3(kThreads), 0, stream, g8, u8, dH, n / 8, dgate, dup);
    timer_end(QL_KERNEL_SWIGLU, stream);
    return check_launch("gated activation backward");
}

}  // namespace qlnf4
