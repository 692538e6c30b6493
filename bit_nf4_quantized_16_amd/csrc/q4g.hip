// 4-bit weights with group scales (gfx950): quantize, expand and multiply.
//
// W [N, K] row-major is cut along its rows into groups of G = 32, 64 or 128
// values (the last of a row may be shorter). A group has a scale s and a zero
// point z in 0..15 (8 throughout when no zero points are kept); a value is
// held as a code q in 0..15 and stands for w' = s (q - z). Row n's codes are
// ceil(K / 32) x 16 bytes, element e in byte e/2, high nibble for even e (the
// order of the NF4 codes); its scales and zero points are rows of ceil(K / G).
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "internal.h"
#include "mm_common.h"

namespace qlnf4 {

namespace {

constexpr int kThreads = 256;

template <bool F32>
__device__ __forceinline__ float load_scale(const void* p, int64_t i) {
    return F32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

// ---------------------------------------------------------------------------
// Quantize. A lane holds eight consecutive values, so a group is 4, 8 or 16
// lanes and its range takes DPP maxima only. w / s is the correctly rounded
// fp32 quotient: the product with the correctly rounded 1 / s, corrected
// once by its exact remainder (Markstein's theorem), three operations a value
// instead of a division's ten. HBM-bound.
// ---------------------------------------------------------------------------
template <int G>
__device__ __forceinline__ float group_max(float v) {
    if constexpr (G == 128) return max16(v);
    if constexpr (G == 64) return max8(v);
    v = fmaxf(v, dpp_f<0x4E>(v));
    return fmaxf(v, dpp_f<0xB1>(v));
}

template <bool WF32, int G, bool SF32>
__global__ __launch_bounds__(kThreads) void q4g_quantize_kernel(const void* __restrict__ W, int64_t N, int64_t K,
                                                                uint8_t* __restrict__ packed,
                                                                void* __restrict__ scale, uint8_t* __restrict__ zero) {
    const int64_t ng = ceil_div(K, G);
    const int64_t lpr = ng * (G / 8);  // lanes of a row: whole groups
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kThreads;
    const int64_t row0 = base / lpr;
    const uint32_t off = static_cast<uint32_t>(base - row0 * lpr) + threadIdx.x;
    const uint32_t rows = off / static_cast<uint32_t>(lpr);
    const int64_t row = row0 + rows;
    const int64_t u = off - rows * static_cast<uint32_t>(lpr);  // eight-value unit of the row
    const bool in = row < N && 8 * u < K;
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 0.0f;
    if (in) {
        if constexpr (WF32) {
            const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(W) + row * K + 8 * u);
            const float4 a = p[0], b = p[1];
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
        } else {
            const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(W) + row * K + 8 * u);
            const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w[2 * e] = __uint_as_float(vw[e] << 16);
                w[2 * e + 1] = __uint_as_float(vw[e] & 0xFFFF0000u);
            }
        }
    }
    float hi = 0.0f, lo = 0.0f;  // lo: of -w
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        hi = fmaxf(hi, w[e]);
        lo = fmaxf(lo, -w[e]);
    }
    hi = group_max<G>(hi);
    lo = group_max<G>(lo);
    const bool sym = zero == nullptr;
    float s = sym ? fmaxf(hi, lo) / 7.0f : (hi + lo) / 15.0f;
    if constexpr (!SF32) s = __uint_as_float(pack_bf16x2(s, 0.0f) << 16);
    const bool live = s >= 0x1p-126f;  // below: the group is held as zeros
    if (!live) s = 0.0f;
    const float inv = 1.0f / s;
    auto quotient = [&](float a) {
        const float x = a * inv;
        return __builtin_fmaf(__builtin_fmaf(-x, s, a), inv, x);
    };
    const float z = (sym || !live) ? 8.0f : fminf(__builtin_rintf(quotient(lo)), 15.0f);
    uint32_t c = 0;
    if (in) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float q = live ? fminf(fmaxf(__builtin_rintf(quotient(w[e])) + z, 0.0f), 15.0f) : 8.0f;
            c |= static_cast<uint32_t>(q) << (8 * (e / 2) + (e % 2 ? 0 : 4));
        }
    }
    const int64_t upr = ceil_div(K, 32) * 4;  // units a row has room for
    if (row < N) {
        if (u < upr) reinterpret_cast<uint32_t*>(packed)[row * upr + u] = c;
        if (u % (G / 8) == 0) {
            const int64_t gi = row * ng + u / (G / 8);
            if constexpr (SF32)
                static_cast<float*>(scale)[gi] = s;
            else
                static_cast<uint16_t*>(scale)[gi] = static_cast<uint16_t>(__float_as_uint(s) >> 16);
            if (!sym) zero[gi] = static_cast<uint8_t>(z);
        }
    }
}

// ---------------------------------------------------------------------------
// Expand: w' = s (q - z) in fp32 (one rounding), rounded to bf16 for the bf16
// output. A lane expands eight values. HBM-bound.
// ---------------------------------------------------------------------------
template <bool BF16, bool SF32>
__global__ __launch_bounds__(kThreads) void q4g_dequantize_kernel(Q4GDev w, int64_t N, int64_t K,
                                                                  void* __restrict__ out) {
    const int64_t k8 = K / 8;
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kThreads;
    const int64_t row0 = base / k8;
    const uint32_t off = static_cast<uint32_t>(base - row0 * k8) + threadIdx.x;
    const uint32_t rows = off / static_cast<uint32_t>(k8);
    const int64_t row = row0 + rows;
    const int64_t u = off - rows * static_cast<uint32_t>(k8);
    if (row >= N) return;
    const uint32_t c = reinterpret_cast<const uint32_t*>(w.packed)[row * (ceil_div(K, 32) * 4) + u];
    const int64_t gi = row * ceil_div(K, w.group) + 8 * u / w.group;
    const float s = load_scale<SF32>(w.scale, gi);
    const int z = w.zero != nullptr ? w.zero[gi] : 8;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] = static_cast<float>(static_cast<int>((c >> (8 * (e / 2) + (e % 2 ? 0 : 4))) & 15u) - z) * s;
    if constexpr (BF16) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + row * K + 8 * u) =
            make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + row * K + 8 * u);
        o[0] = make_float4(v[0], v[1], v[2], v[3]);
        o[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

// ---------------------------------------------------------------------------
// Y[t][n] = sum over groups of s (sum_k x q - z sum_k x), bf16 MFMA.
//
// The codes 0..15 are exact in bf16, so the products run on the codes
// themselves and the scale comes in once per group, in fp32: nothing of the
// weight is rounded. A nibble as a byte is the E4M3 value q 2^-9 (subnormal
// and first binade are one linear range), which the scaled conversion brings
// to bf16 q, two values an instruction.
//
// A workgroup of eight waves owns 16 RT rows and 16 TT tokens; wave w takes
// the 128-wide chunks w, w + 8, ... of K. In a chunk, lane (i = l % 16,
// g = l / 16) loads 16 bytes of row i's codes (32 values at 32 g) and the
// matching pieces of token i; x is the MFMA's first operand (its rows the
// tokens), the codes the second (its columns the weight's rows), so a lane's
// four sums are tokens 4 g .. 4 g + 3 of row i, and row i's scale is the
// lane's own. For groups under 128 the 16 bytes are transposed over the four
// lane groups (four lane swaps), so that MFMA m covers values 32 m .. + 31.
// sum_k x comes from one more MFMA with ones, shared by the row tiles. The
// waves' sums are added in order through LDS.
//
// Where a result is not finite (an infinite or NaN x, or sums that overflow
// only because q and z are apart), it is formed again value by value as
// x s (q - z): the formula's infinities, not the difference of two.
// ---------------------------------------------------------------------------
constexpr int kWaves = 8;

template <bool SF32>
__device__ __attribute__((noinline)) float q4g_dot(const Q4GDev& w, const uint16_t* x, int64_t n, int64_t K) {
    float y = 0.0f;
    const int64_t ng = ceil_div(K, w.group), rowbytes = ceil_div(K, 32) * 16;
    for (int64_t k = 0; k < K; ++k) {
        const uint32_t b = w.packed[n * rowbytes + k / 2];
        const int64_t gi = n * ng + k / w.group;
        const int q = static_cast<int>(k % 2 ? b & 15u : b >> 4);
        const int z = w.zero != nullptr ? w.zero[gi] : 8;
        y = __builtin_fmaf(bf16_to_f32(x[k]), static_cast<float>(q - z) * load_scale<SF32>(w.scale, gi), y);
    }
    return y;
}

// Eight codes (one packed word) -> eight bf16 integers in the order of k.
__device__ __forceinline__ bf16x8_t q4g_operand(uint32_t c) {
    const uint32_t hi = (c >> 4) & 0x0F0F0F0Fu, lo = c & 0x0F0F0F0Fu;
    const uint32_t a = __builtin_amdgcn_perm(lo, hi, 0x05010400u);  // e0 e1 e2 e3
    const uint32_t b = __builtin_amdgcn_perm(lo, hi, 0x07030602u);  // e4 e5 e6 e7
    uint4 r;
    r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 512.0f, false));
    r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 512.0f, true));
    r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.0f, false));
    r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.0f, true));
    return as_bf16x8(r);
}

struct Q4GLinearArgs {
    Q4GDev w;
    const uint16_t* X;
    int64_t T, N, K;
    uint16_t* Y;
};

// One chunk's operands of a lane.
template <int RT, int TT>
struct Q4GStage {
    uint4 c[RT];
    uint4 x[TT][4];
    float s[RT];
    uint32_t z[RT];
};

template <int RT, int TT, int GL, bool SF32>
__global__ __launch_bounds__(64 * kWaves) void q4g_linear_kernel(Q4GLinearArgs p) {
    constexpr int D = 2;             // chunks in flight
    constexpr int NG = 128 >> GL;    // groups of a chunk
    constexpr int MG = 4 / NG;       // MFMA steps of a group
    __shared__ float red[kWaves][TT][16][16];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, g = lane >> 4;
    const int64_t N = p.N, K = p.K, T = p.T;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16 * RT, t0 = static_cast<int64_t>(blockIdx.y) * 16 * TT;
    const int64_t nch = ceil_div(K, 128), rowbytes = ceil_div(K, 32) * 16, ng = ceil_div(K, int64_t{1} << GL);
    const bool has_zero = p.w.zero != nullptr;

    auto piece = [&](int m) { return GL == 7 ? 4 * g + m : 4 * m + g; };  // eight values of x
    auto issue = [&](Q4GStage<RT, TT>& st, int64_t ch) {
        ch = std::min(ch, nch - 1);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int64_t row = std::min<int64_t>(n0 + 16 * rt + li, N - 1);
            st.c[rt] = *reinterpret_cast<const uint4*>(p.w.packed + row * rowbytes +
                                                       std::min<int64_t>(64 * ch + 16 * g, rowbytes - 16));
            const int64_t gi = row * ng + std::min<int64_t>(ch * NG + (g * NG) / 4, ng - 1);
            st.s[rt] = load_scale<SF32>(p.w.scale, gi);
            st.z[rt] = has_zero ? p.w.zero[gi] : 8;
        }
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
            const uint16_t* xr = p.X + std::min<int64_t>(t0 + 16 * tt + li, T - 1) * K;
#pragma unroll
            for (int m = 0; m < 4; ++m)
                st.x[tt][m] = *reinterpret_cast<const uint4*>(xr + std::min<int64_t>(128 * ch + 8 * piece(m), K - 8));
        }
    };

    const bf16x8_t ones = as_bf16x8(make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u));
    f32x4 tot[RT][TT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) tot[rt][tt] = f32x4{0.f, 0.f, 0.f, 0.f};

    auto consume = [&](Q4GStage<RT, TT>& st, int64_t ch) {
        if (128 * ch + 128 > K) {  // the last chunk: nothing past K
#pragma unroll
            for (int m = 0; m < 4; ++m)
                if (128 * ch + 8 * piece(m) >= K) {
#pragma unroll
                    for (int tt = 0; tt < TT; ++tt) st.x[tt][m] = make_uint4(0, 0, 0, 0);
                }
        }
        uint32_t cw[RT][4];
        float s[RT][NG], z[RT][NG];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            cw[rt][0] = st.c[rt].x, cw[rt][1] = st.c[rt].y, cw[rt][2] = st.c[rt].z, cw[rt][3] = st.c[rt].w;
            if constexpr (GL == 7) {
                s[rt][0] = st.s[rt];
                z[rt][0] = static_cast<float>(st.z[rt]);
            } else {
                // word m of lane group g <-> word g of lane group m
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const auto sw = __builtin_amdgcn_permlane32_swap(cw[rt][q], cw[rt][q + 2], false, false);
                    cw[rt][q] = sw[0], cw[rt][q + 2] = sw[1];
                }
#pragma unroll
                for (int q = 0; q < 4; q += 2) {
                    const auto sw = __builtin_amdgcn_permlane16_swap(cw[rt][q], cw[rt][q + 1], false, false);
                    cw[rt][q] = sw[0], cw[rt][q + 1] = sw[1];
                }
                // lane group g holds the constants of group g NG / 4: hand each to all
                const uint32_t sb = __float_as_uint(st.s[rt]), zb = st.z[rt];
                const auto s2 = __builtin_amdgcn_permlane32_swap(sb, sb, false, false);
                const auto z2 = __builtin_amdgcn_permlane32_swap(zb, zb, false, false);
                if constexpr (NG == 2) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        s[rt][q] = __uint_as_float(s2[q]);
                        z[rt][q] = static_cast<float>(z2[q]);
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const auto s4 = __builtin_amdgcn_permlane16_swap(s2[q], s2[q], false, false);
                        const auto z4 = __builtin_amdgcn_permlane16_swap(z2[q], z2[q], false, false);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            s[rt][2 * q + h] = __uint_as_float(s4[h]);
                            z[rt][2 * q + h] = static_cast<float>(z4[h]);
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int q = 0; q < NG; ++q) {
            f32x4 acc[RT][TT], xs[TT];
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) {
                xs[tt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) acc[rt][tt] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
#pragma unroll
            for (int mm = 0; mm < MG; ++mm) {
                const int m = q * MG + mm;
#pragma unroll
                for (int tt = 0; tt < TT; ++tt)
                    xs[tt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(st.x[tt][m]), ones, xs[tt], 0, 0, 0);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const bf16x8_t wv = q4g_operand(cw[rt][m]);
#pragma unroll
                    for (int tt = 0; tt < TT; ++tt)
                        acc[rt][tt] =
                            __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(st.x[tt][m]), wv, acc[rt][tt], 0, 0, 0);
                }
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                    for (int rr = 0; rr < 4; ++rr)
                        tot[rt][tt][rr] = __builtin_fmaf(s[rt][q], __builtin_fmaf(-z[rt][q], xs[tt][rr], acc[rt][tt][rr]),
                                                         tot[rt][tt][rr]);
        }
    };

    const int64_t mine = wave < nch ? (nch - 1 - wave) / kWaves + 1 : 0;  // chunks of this wave
    Q4GStage<RT, TT> ring[D];
#pragma unroll
    for (int q = 0; q < D; ++q) issue(ring[q], wave + kWaves * q);
    for (int64_t k0 = 0; k0 < mine; k0 += D) {
#pragma unroll
        for (int q = 0; q < D; ++q) {
            if (k0 + q < mine) consume(ring[q], wave + kWaves * (k0 + q));
            issue(ring[q], wave + kWaves * (k0 + q + D));
        }
    }

#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        if (rt > 0) __syncthreads();
#pragma unroll
        for (int tt = 0; tt < TT; ++tt)
#pragma unroll
            for (int rr = 0; rr < 4; ++rr) red[wave][tt][4 * g + rr][li] = tot[rt][tt][rr];
        __syncthreads();
        for (int e = tid; e < TT * 256; e += 64 * kWaves) {
            const int tt = e >> 8, tl = (e >> 4) & 15, nl = e & 15;
            const int64_t t = t0 + 16 * tt + tl, n = n0 + 16 * rt + nl;
            if (t >= T || n >= N) continue;
            float y = 0.0f;
#pragma unroll
            for (int ww = 0; ww < kWaves; ++ww) y += red[ww][tt][tl][nl];
            if (!(fabsf(y) < __builtin_inff())) y = q4g_dot<SF32>(p.w, p.X + t * K, n, K);
            p.Y[t * N + n] = to_bf16_bits(y);
        }
    }
}

template <int RT, int TT, bool SF32>
void launch_linear(const Q4GLinearArgs& a, hipStream_t stream) {
    const dim3 grid(static_cast<uint32_t>(ceil_div(a.N, 16 * RT)), static_cast<uint32_t>(ceil_div(a.T, 16 * TT)));
    const dim3 block(64 * kWaves);
    switch (a.w.group) {
        case 32: hipLaunchKernelGGL((q4g_linear_kernel<RT, TT, 5, SF32>), grid, block, 0, stream, a); break;
        case 64: hipLaunchKernelGGL((q4g_linear_kernel<RT, TT, 6, SF32>), grid, block, 0, stream, a); break;
        default: hipLaunchKernelGGL((q4g_linear_kernel<RT, TT, 7, SF32>), grid, block, 0, stream, a); break;
    }
}

template <bool WF32, bool SF32>
void launch_quantize_g(const void* W, int64_t N, int64_t K, int group, uint8_t* packed, void* scale, uint8_t* zero,
                       hipStream_t stream) {
    const dim3 grid(static_cast<uint32_t>(ceil_div(N * ceil_div(K, group) * (group / 8), kThreads))), block(kThreads);
    switch (group) {
        case 32:
            hipLaunchKernelGGL((q4g_quantize_kernel<WF32, 32, SF32>), grid, block, 0, stream, W, N, K, packed, scale, zero);
            break;
        case 64:
            hipLaunchKernelGGL((q4g_quantize_kernel<WF32, 64, SF32>), grid, block, 0, stream, W, N, K, packed, scale, zero);
            break;
        default:
            hipLaunchKernelGGL((q4g_quantize_kernel<WF32, 128, SF32>), grid, block, 0, stream, W, N, K, packed, scale,
                               zero);
            break;
    }
}

}  // namespace

// f(a, b) with a and b as compile-time truth values
template <typename F>
void with_flags(bool a, bool b, F f) {
    if (a)
        b ? f(std::true_type{}, std::true_type{}) : f(std::true_type{}, std::false_type{});
    else
        b ? f(std::false_type{}, std::true_type{}) : f(std::false_type{}, std::false_type{});
}

int launch_q4g_quantize(const void* W, bool w_f32, int64_t N, int64_t K, int group, uint8_t* packed, void* scale,
                        bool scale_f32, uint8_t* zero, hipStream_t stream) {
    timer_begin(QL_KERNEL_Q4G_QUANTIZE, stream);
    with_flags(w_f32, scale_f32, [&](auto wf, auto sf) {
        launch_quantize_g<decltype(wf)::value, decltype(sf)::value>(W, N, K, group, packed, scale, zero, stream);
    });
    timer_end(QL_KERNEL_Q4G_QUANTIZE, stream);
    return check_launch("4-bit group quantize");
}

int launch_q4g_dequantize(const Q4GDev& w, int64_t N, int64_t K, void* out, bool bf16_out, hipStream_t stream) {
    const dim3 grid(static_cast<uint32_t>(ceil_div(N * (K / 8), kThreads))), block(kThreads);
    timer_begin(QL_KERNEL_Q4G_DEQUANTIZE, stream);
    with_flags(bf16_out, w.scale_f32 != 0, [&](auto bf, auto sf) {
        hipLaunchKernelGGL((q4g_dequantize_kernel<decltype(bf)::value, decltype(sf)::value>), grid, block, 0, stream, w,
                           N, K, out);
    });
    timer_end(QL_KERNEL_Q4G_DEQUANTIZE, stream);
    return check_launch("4-bit group dequantize");
}

int launch_q4g_linear(const Q4GDev& w, const uint16_t* X, int64_t T, int64_t N, int64_t K, uint16_t* Y,
                      hipStream_t stream) {
    const Q4GLinearArgs a{w, X, T, N, K, Y};
    timer_begin(QL_KERNEL_Q4G_LINEAR, stream);
    with_flags(w.scale_f32 != 0, false, [&](auto sf, auto) {
        constexpr bool SF32 = decltype(sf)::value;
        if (T <= 16)
            launch_linear<1, 1, SF32>(a, stream);
        else if (T <= 32)
            launch_linear<1, 2, SF32>(a, stream);
        else
            launch_linear<1, 4, SF32>(a, stream);
    });
    timer_end(QL_KERNEL_Q4G_LINEAR, stream);
    return check_launch("4-bit group linear");
}

}  // namespace qlnf4
