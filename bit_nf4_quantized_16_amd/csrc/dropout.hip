// LoRA dropout on the adapter input, with the keep mask given (gfx950).
//
// ai-reference-codex "QLoRA 与 PEFT 全家", §3.4: dropout on the adapters
// (0.05-0.1 for small data); aivaro.ru "Как работает QLoRA", §11:
// lora_dropout = 0.05. Inverted dropout of the adapter branch's input only:
//
//   U  = (X * keep) A^T / (1 - p),   H = X W'^T + s U B^T
//   dX = dY W' + (G A) * keep / (1 - p),   dA = G^T (X * keep) / (1 - p)
//
// The mask is bit-packed: row t of the [T, K] keep mask is K / 8 bytes,
// element 8i + j in bit j of byte i (1 = kept). One kernel serves the layer
// before the unchanged projection, GEMM and gradient kernels, keep_apply_kernel:
// X_d = X * keep (bf16, exact: entries kept or zeroed). The mask of dX's
// adapter term is applied inside the dX GEMM (gemm_tiles.hip).
#include <algorithm>

#include "common.h"
#include "internal.h"

namespace qlnf4 {

namespace {

// 16-bit lane masks of eight elements from their eight keep bits: word q of
// the result covers elements 2q (low half) and 2q + 1 (high half).
__device__ __forceinline__ uint4 keep_lanes(uint32_t bits) {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
        w[q] = ((bits >> (2 * q)) & 1u ? 0x0000FFFFu : 0u) | ((bits >> (2 * q + 1)) & 1u ? 0xFFFF0000u : 0u);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Thread i: elements 8i .. 8i + 7 of the row-major [T, K] input (K % 8 == 0,
// so they share keep byte i), 16 bytes in and out.
__global__ __launch_bounds__(256) void keep_apply_kernel(const uint16_t* __restrict__ X,
                                                         const uint8_t* __restrict__ keep, int64_t n8,
                                                         uint16_t* __restrict__ Xd) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n8) return;
    const uint4 x = *reinterpret_cast<const uint4*>(X + 8 * i);
    const uint4 m = keep_lanes(keep[i]);
    *reinterpret_cast<uint4*>(Xd + 8 * i) = make_uint4(x.x & m.x, x.y & m.y, x.z & m.z, x.w & m.w);
}

}  // namespace

int launch_keep_apply(const uint16_t* X, const uint8_t* keep, int64_t T, int64_t K, uint16_t* Xd, hipStream_t stream) {
    const int64_t n8 = T * K / 8;
    timer_begin(QL_KERNEL_KEEP_APPLY, stream);
    hipLaunchKernelGGL(keep_apply_kernel, dim3(static_cast<uint32_t>(ceil_div(n8, 256))), dim3(256), 0, stream, X,
                       keep, n8, Xd);
    timer_end(QL_KERNEL_KEEP_APPLY, stream);
    return check_launch("dropout: keep mask on the adapter input");
}

}  // namespace qlnf4
