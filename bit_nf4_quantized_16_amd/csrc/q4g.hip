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
#include "proj_dma.h"

namespace qlnf4 {

namespace {

constexpr int kThreads = 256;

template <bool F32>
__device__ __forceinline__ float load_scale(const void* p, int64_t i) {
    return F32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

// Division of a thread index under 2^31 by a row's length, for a kernel whose
// threads run through rows of units: n / d = (n m) >> (31 + s), s = ceil(log2 d),
// m = floor(2^(31 + s) / d) + 1 < 2^32 (exact for n < 2^31).
struct RowDivisor {
    uint32_t d, m;
    int s;
};

RowDivisor row_divisor(int64_t d) {
    RowDivisor r{static_cast<uint32_t>(d), 0, 0};
    while ((int64_t{1} << r.s) < d) ++r.s;
    r.m = static_cast<uint32_t>((uint64_t{1} << (31 + r.s)) / static_cast<uint64_t>(d) + 1);
    return r;
}

// row and unit within it of thread n
__device__ __forceinline__ uint32_t row_of(uint32_t n, const RowDivisor& r, uint32_t& unit) {
    const uint32_t row = r.d == 1 ? n : static_cast<uint32_t>((static_cast<uint64_t>(n) * r.m) >> (31 + r.s));
    unit = n - row * r.d;
    return row;
}

// ---------------------------------------------------------------------------
// Quantize. A lane holds eight consecutive values, so a group is 4, 8 or 16
// lanes and its range takes DPP maxima only. The range is found on the bits:
// as signed integers positive floats order like their values (and above the
// negative ones), as unsigned integers the negative ones like their magnitudes
// (and above the positive), so two integer maxima, packed for bf16, give both
// ends. Quotients are correctly rounded fp32: the product with the correctly
// rounded reciprocal, corrected once by its exact remainder (Markstein's
// theorem), three operations instead of a division's ten; adding 1.5 2^23
// rounds to an integer, ties to even, in the low bits. 11008 x 4096 from bf16
// takes 24.4 us (114 MB, 4.7 TB/s: HBM), 4096 x 4096 from fp32 13.7; with
// divisions, float maxima and a 64-bit index division the arithmetic bounds it
// (34 us).
// ---------------------------------------------------------------------------
__device__ __forceinline__ int imax_(int a, int b) { return a > b ? a : b; }

// Maxima over a group's lanes, everywhere: hi as signed, lo as unsigned.
template <int G>
__device__ __forceinline__ void group_range(int& hi, uint32_t& lo) {
    auto step = [&](auto ctrl) {
        constexpr int C = decltype(ctrl)::value;
        hi = imax_(hi, static_cast<int>(dpp_u<C>(static_cast<uint32_t>(hi))));
        lo = umax_(lo, dpp_u<C>(lo));
    };
    if constexpr (G == 128) {
        step(std::integral_constant<int, 0x128>{});  // row_ror:8
        step(std::integral_constant<int, 0x124>{});  // row_ror:4
    } else if constexpr (G == 64) {
        step(std::integral_constant<int, 0x141>{});  // row_half_mirror
    }
    step(std::integral_constant<int, 0x4E>{});  // quad_perm [2,3,0,1]
    step(std::integral_constant<int, 0xB1>{});  // quad_perm [1,0,3,2]
}

// a / b, correctly rounded, from inv = fl32(1 / b).
__device__ __forceinline__ float quotient(float a, float b, float inv) {
    const float x = a * inv;
    return __builtin_fmaf(__builtin_fmaf(-x, b, a), inv, x);
}

template <bool WF32, int G, bool SF32>
__global__ __launch_bounds__(kThreads) void q4g_quantize_kernel(const void* __restrict__ W, uint32_t N, uint32_t K,
                                                                RowDivisor lanes, uint8_t* __restrict__ packed,
                                                                void* __restrict__ scale, uint8_t* __restrict__ zero) {
    uint32_t u;  // eight-value unit of the row
    const uint32_t row = row_of(blockIdx.x * kThreads + threadIdx.x, lanes, u);
    const bool in = row < N && 8 * u < K;
    uint32_t w[8];  // the values as fp32 bits
    int hi = 0;
    uint32_t lo = 0;
    if constexpr (WF32) {
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        if (in) {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(W) + static_cast<int64_t>(row) * K + 8 * u);
            a = p[0], b = p[1];
        }
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            hi = imax_(hi, static_cast<int>(w[e]));
            lo = umax_(lo, w[e]);
        }
    } else {
        typedef short i16x2 __attribute__((ext_vector_type(2)));
        typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
        uint4 v = make_uint4(0, 0, 0, 0);
        if (in) v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(W) + static_cast<int64_t>(row) * K + 8 * u);
        const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
        i16x2 h2 = {0, 0};
        u16x2 l2 = {0, 0};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            h2 = __builtin_elementwise_max(h2, __builtin_bit_cast(i16x2, vw[e]));
            l2 = __builtin_elementwise_max(l2, __builtin_bit_cast(u16x2, vw[e]));
            w[2 * e] = vw[e] << 16;
            w[2 * e + 1] = vw[e] & 0xFFFF0000u;
        }
        hi = imax_(h2[0], h2[1]) << 16;
        lo = umax_(l2[0], l2[1]) << 16;
    }
    group_range<G>(hi, lo);
    const float top = __int_as_float(hi);
    float bottom = static_cast<int>(lo) < 0 ? __uint_as_float(lo & 0x7FFFFFFFu) : 0.0f;
    const bool sym = zero == nullptr;
    float s = sym ? quotient(fmaxf(top, bottom), 7.0f, 1.0f / 7.0f) : quotient(top + bottom, 15.0f, 1.0f / 15.0f);
    if constexpr (!SF32) s = __uint_as_float(pack_bf16x2(s, 0.0f) << 16);
    const bool live = s >= 0x1p-126f;  // below: the group is held as zeros
    if (!live) s = 0.0f;
    // the remainder of a quotient by a scale under about 2^-102 may have places under
    // fp32's last: small scales and their values come up by 2^64 first, exactly (by a
    // branch of the wave: products for all took 11008 x 4096 from 23.6 to 25.2 us)
    float su = s;
    if (__builtin_expect(__any(s < 0x1p-64f), 0)) {
        const float up = s < 0x1p-64f ? 0x1p64f : 1.0f;
        su *= up;
        bottom *= up;
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * up);
    }
    const float inv = 1.0f / su;
    constexpr float kRound = 12582912.0f;  // 1.5 2^23
    constexpr int kRoundBits = 0x4B400000;
    auto nearest = [&](float a) { return __float_as_int(quotient(a, su, inv) + kRound) - kRoundBits; };
    const int z = (sym || !live) ? 8 : std::min(nearest(bottom), 15);
    uint32_t c = 0x88888888u;
    if (live) {
        c = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int q = std::min(std::max(nearest(__uint_as_float(w[e])) + z, 0), 15);
            c |= static_cast<uint32_t>(q) << (8 * (e / 2) + (e % 2 ? 0 : 4));
        }
    }
    const uint32_t upr = (K + 31) / 32 * 4, ng = (K + G - 1) / G;  // units a row has room for, groups of a row
    if (row < N) {
        if (u < upr) reinterpret_cast<uint32_t*>(packed)[static_cast<int64_t>(row) * upr + u] = in ? c : 0u;
        if (u % (G / 8) == 0) {
            const int64_t gi = static_cast<int64_t>(row) * ng + u / (G / 8);
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
// output. A lane expands eight values. HBM-bound: 11008 x 4096 in 18.5 us
// (114 MB, 6.2 TB/s, the codes from the last-level cache).
// ---------------------------------------------------------------------------
template <bool BF16, bool SF32>
__global__ __launch_bounds__(kThreads) void q4g_dequantize_kernel(Q4GDev w, uint32_t N, uint32_t K, RowDivisor units,
                                                                  void* __restrict__ out) {
    uint32_t u;
    const uint32_t row = row_of(blockIdx.x * kThreads + threadIdx.x, units, u);
    if (row >= N) return;
    const uint32_t shift = __builtin_ctz(w.group);
    const int64_t gi = static_cast<int64_t>(row) * ((K + w.group - 1) >> shift) + (8 * u >> shift);
    const uint32_t c = reinterpret_cast<const uint32_t*>(w.packed)[static_cast<int64_t>(row) * ((K + 31) / 32 * 4) + u];
    const float s = load_scale<SF32>(w.scale, gi);
    const int z = w.zero != nullptr ? w.zero[gi] : 8;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] = static_cast<float>(static_cast<int>((c >> (8 * (e / 2) + (e % 2 ? 0 : 4))) & 15u) - z) * s;
    const int64_t at = static_cast<int64_t>(row) * K + 8 * u;
    if constexpr (BF16) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) =
            make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
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
// A workgroup owns 16 RT rows; its waves split K (each a contiguous run of
// 128-wide chunks), so that every wave streams codes of its own. In a chunk,
// lane (i = l % 16, g = l / 16) loads 16 bytes of row i's codes (values
// 32 g .. 32 g + 31), which four lane swaps transpose over the lane groups: MFMA
// m then covers values 32 m .. 32 m + 31, never more than one group of any
// size. x is the MFMA's first operand (its rows the tokens), the codes the
// second (its columns the weight's rows): a lane's sums are tokens of row i,
// whose scale is the lane's own. sum_k x comes from one more MFMA with ones.
// The waves' sums are added in order through LDS.
//
// What bounds it: at one token HBM and the time from launch to the last
// wave's first bytes. Loads that touch one line per row cost as much as the
// row's 64 bytes of codes, so nothing but the codes is loaded that way: scales
// and zero points come in once, row by row, and stay in LDS (loaded per chunk
// they took 4096 x 4096 from 4.9 to 6.0 us and 22016 x 8192 from 25 to 46 us),
// and x comes in whole lines, to the operands through LDS. Straight-line code
// costs fetches: four chunks in flight measured slower than two.
//
// Where a result is not finite (an infinite or NaN x, or sums that overflow
// only because q and z are apart), it is formed again value by value as
// x s (q - z): the formula's infinities, not the difference of two. The wave
// does so together, 512 values a step, and stops at a NaN: rows of a padded
// batch may hold anything.
// ---------------------------------------------------------------------------
template <bool SF32>
__device__ float q4g_dot(const Q4GDev& w, const uint16_t* x, int64_t n, int64_t K, int lane) {
    float y = 0.0f;
    const int64_t ng = ceil_div(K, w.group), rowbytes = ceil_div(K, 32) * 16;
    const int gl = __builtin_ctz(w.group);
    for (int64_t k0 = 0; k0 < K; k0 += 512) {
        const int64_t k = k0 + 8 * lane;
        if (k < K) {
            const uint32_t c = *reinterpret_cast<const uint32_t*>(w.packed + n * rowbytes + k / 2);
            const uint4 xv = *reinterpret_cast<const uint4*>(x + k);
            const int64_t gi = n * ng + (k >> gl);
            const float sc = load_scale<SF32>(w.scale, gi);
            const int z = w.zero != nullptr ? w.zero[gi] : 8;
            const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int q = static_cast<int>(c >> (8 * (j / 2) + (j % 2 ? 0 : 4)) & 15u);
                const uint32_t xb = j % 2 ? xw[j / 2] >> 16 : xw[j / 2] & 0xFFFFu;
                y = __builtin_fmaf(bf16_to_f32(xb), static_cast<float>(q - z) * sc, y);
            }
        }
        if (__any(y != y)) return __builtin_nanf("");
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) y += __shfl_xor(y, d);
    return y;
}

// The wave's results y (of token tl and row nl behind X and n0, where live),
// those that are not finite formed again, one after the other.
template <bool SF32>
__device__ __forceinline__ float q4g_finite(float y, bool live, const Q4GDev& w, const uint16_t* X, int tl, int64_t n0,
                                            int nl, int64_t K, int lane) {
    for (uint64_t bad = __ballot(live && !(fabsf(y) < __builtin_inff())); bad != 0; bad &= bad - 1) {
        const int l = __builtin_ctzll(bad);
        const float v = q4g_dot<SF32>(w, X + __builtin_amdgcn_readlane(tl, l) * K, n0 + __builtin_amdgcn_readlane(nl, l), K, lane);
        if (lane == l) y = v;
    }
    return y;
}

// Eight codes (one packed word) -> eight bf16 integers, even elements before
// odd ones (x_slot_order puts x in the same order).
__device__ __forceinline__ bf16x8_t q4g_operand(uint32_t c) {
    const uint32_t hi = (c >> 4) & 0x0F0F0F0Fu, lo = c & 0x0F0F0F0Fu;
    uint4 r;
    r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false));
    r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true));
    r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false));
    r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true));
    return as_bf16x8(r);
}

// The same in the order of k.
__device__ __forceinline__ bf16x8_t q4g_operand_ordered(uint32_t c) {
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

// s_waitcnt lgkmcnt(0): the wave's LDS reads have returned.
__device__ __forceinline__ void wait_lgkmcnt0() { __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4) | (0 << 8)); }

// 16 bytes a lane straight to LDS: lane l's land at dst + 16 l (dst the same
// for the wave).
__device__ __forceinline__ void load_lds16(const uint8_t* src, uint8_t* dst) {
    __builtin_amdgcn_global_load_lds(src, (QL_LDS_AS void*)dst, 16, 0, 0);
}

struct Q4GLinearArgs {
    Q4GDev w;
    const uint16_t* X;
    int64_t T, N, K;
    uint16_t* Y;
    int64_t slice;     // set by the launcher: values of a row whose constants are in LDS at a time
    int slice_groups;  // their groups
    Epilogue ep;       // where epilogue is set
    int epilogue;
};

// act(y + bias) + residual for output n of a row, at i of Y. The loads come last
// (issued ahead of the weight they gained nothing): bias and residual add 0.4 us
// to 14.3 at 4096 x 11008, T = 24, and 0.25 to 4.9 at 4096 x 4096, T = 1.
__device__ __forceinline__ float q4g_epilogue(const Epilogue& ep, float y, int64_t n, int64_t i) {
    if (ep.bias != nullptr) y += bf16_to_f32(ep.bias[n]);
    with_act(ep.act, [&](auto act) { y = act_value<decltype(act)::value>(y); });
    if (ep.res != nullptr) y += bf16_to_f32(ep.res[i]);
    return y;
}

// One chunk's operands of a lane, as loaded.
template <int RT, int TX>
struct Q4GStage {
    uint4 c[RT];
    uint4 x[TX];
};

// Words of LDS that a row's scales and zero points take: an odd number, so
// that 16 rows of a column fall into different banks.
__host__ __device__ inline int q4g_row_words(int groups, bool scale_f32) { return (scale_f32 ? 2 * groups : groups) | 1; }

// Scales and zero points of a slice (groups g0 .. of the workgroup's rows)
// into LDS, a row's at szrow words from the last row's: bf16 scales and zero
// points as one word, fp32 scales as two. A wave takes rows wave, wave + NW,
// ... and 64 groups at a time; the loads of eight such pieces are issued
// together, since each round trip to memory costs about as long as the
// product itself.
template <int RPW, int NW, bool SF32>
__device__ __forceinline__ void q4g_stage_constants(const Q4GLinearArgs& p, uint32_t* sz, int szrow, int64_t n0, int nrows,
                                                    int g0, int ng, int wave, int lane) {
    using Scale = std::conditional_t<SF32, uint32_t, uint16_t>;
    constexpr int U = 8;
    const bool has_zero = p.w.zero != nullptr;
    const Scale* const sp = static_cast<const Scale*>(p.w.scale) + n0 * ng + g0;
    const uint8_t* const zp = (has_zero ? p.w.zero : p.w.packed) + n0 * ng + g0;  // without: a byte read and not used
    const int gcnt = std::min(p.slice_groups, ng - g0);
    const int pieces = RPW * ((p.slice_groups + 63) / 64);
    for (int i = 0; i < pieces; i += U) {
        uint32_t s[U], z[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = wave + NW * ((i + u) % RPW), c = lane + 64 * ((i + u) / RPW);
            const uint32_t at = static_cast<uint32_t>(std::min(row, nrows - 1)) * static_cast<uint32_t>(ng) +
                                static_cast<uint32_t>(std::min(c, gcnt - 1));
            s[u] = sp[at];
            z[u] = zp[at];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = wave + NW * ((i + u) % RPW), c = lane + 64 * ((i + u) / RPW);
            if (i + u < pieces && c < p.slice_groups) {
                const uint32_t zz = has_zero ? z[u] : 8u;
                if constexpr (SF32) {
                    sz[row * szrow + 2 * c] = s[u];
                    sz[row * szrow + 2 * c + 1] = zz;
                } else {
                    sz[row * szrow + c] = s[u] << 16 | zz;
                }
            }
        }
    }
}

template <int RT, int TX, int D, int GL, bool SF32>
__global__ __launch_bounds__(512) void q4g_linear_kernel(Q4GLinearArgs p) {
    constexpr int NG = 128 >> GL;  // groups of a chunk
    constexpr int MG = 4 / NG;     // MFMA steps of a group
    constexpr int NW = 8;
    constexpr int kSlot = 1024 * TX;  // x of a chunk; the wave's sums take its place at the end
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, g = lane >> 4;
    const int64_t N = p.N, K = p.K;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16 * RT;
    const int rowbytes = static_cast<int>(ceil_div(K, 32)) * 16, ng = static_cast<int>(ceil_div(K, int64_t{1} << GL));
    const int nrows = static_cast<int>(std::min<int64_t>(16 * RT, N - n0)), ntok = static_cast<int>(p.T);
    uint4* const slot = reinterpret_cast<uint4*>(lds + wave * kSlot);
    uint32_t* const sz = reinterpret_cast<uint32_t*>(lds + NW * kSlot);
    const int szrow = q4g_row_words(p.slice_groups, SF32);

    // Addresses: a base that is the same for the wave and a 32-bit offset of
    // the lane. Rows past N and tokens past T read the last one.
    const uint8_t* const cbase = p.w.packed + n0 * rowbytes;
    const uint8_t* const xbase = reinterpret_cast<const uint8_t*>(p.X);
    // The chunk that K ends in reads back from the end of a row instead.
    const int last = static_cast<int>(ceil_div(K, 128)) - 1;
    const bool ragged = K % 128 != 0;
    const int cback = std::max(0, 64 * last + 16 * g + 16 - rowbytes);
    const int xback = std::max(0, 256 * last + 16 * li + 16 - static_cast<int>(2 * K));
    uint32_t coff[RT], xoff[TX];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
        coff[rt] = static_cast<uint32_t>(std::min(16 * rt + li, nrows - 1)) * static_cast<uint32_t>(rowbytes) + 16 * g;
#pragma unroll
    for (int u = 0; u < TX; ++u)
        xoff[u] = static_cast<uint32_t>(std::min(4 * u + g, ntok - 1)) * static_cast<uint32_t>(2 * K) + 16 * li;

    auto issue = [&](Q4GStage<RT, TX>& st, int ch) {
        const uint8_t* const cp = cbase + 64 * ch;
        const uint8_t* const xp = xbase + 256 * ch;
        const uint32_t cb = ch == last ? cback : 0, xb = ch == last ? xback : 0;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) st.c[rt] = *reinterpret_cast<const uint4*>(cp + (coff[rt] - cb));
#pragma unroll
        for (int u = 0; u < TX; ++u) st.x[u] = *reinterpret_cast<const uint4*>(xp + (xoff[u] - xb));
    };

    const bf16x8_t ones = as_bf16x8(make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u));
    float tot[RT][TX];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int rr = 0; rr < TX; ++rr) tot[rt][rr] = 0.0f;

    // piece c of token j in the wave's slot: at j 16 + (c ^ j % 16), so the 16
    // lanes that read one piece of 16 tokens hit distinct banks
    auto put_x = [&](Q4GStage<RT, TX>& st, int ch) {
        if (ragged && ch == last && xback > 0) {  // nothing of x past K
#pragma unroll
            for (int u = 0; u < TX; ++u) st.x[u] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < TX; ++u) {
            const int j = 4 * u + g;
            slot[16 * j + (li ^ (j & 15))] = x_slot_order(st.x[u]);
        }
    };
    auto xin = [&](int m) {
        const int j = std::min((li >> 2) * TX + std::min(li & 3, TX - 1), ntok - 1);
        return as_bf16x8(slot[16 * j + ((4 * m + g) ^ (j & 15))]);
    };

    auto consume = [&](Q4GStage<RT, TX>& st, int ch, int ch0) {
        put_x(st, ch);
        wave_lds_sync();
        uint32_t cw[RT][4];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            cw[rt][0] = st.c[rt].x, cw[rt][1] = st.c[rt].y, cw[rt][2] = st.c[rt].z, cw[rt][3] = st.c[rt].w;
            // word m of lane group g <-> word g of lane group m: MFMA m then
            // covers values 32 m .. 32 m + 31 of the chunk
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
        }
#pragma unroll
        for (int q = 0; q < NG; ++q) {
            f32x4 acc[RT], xs = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) acc[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int mm = 0; mm < MG; ++mm) {
                const int m = q * MG + mm;
                const bf16x8_t xv = xin(m);
                xs = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, ones, xs, 0, 0, 0);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
                    acc[rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, q4g_operand(cw[rt][m]), acc[rt], 0, 0, 0);
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                // the row's scale and zero point (past the last group x is zero)
                const uint32_t* const e =
                    sz + (16 * rt + li) * szrow + (SF32 ? 2 : 1) * std::min((ch - ch0) * NG + q, p.slice_groups - 1);
                const float s = __uint_as_float(SF32 ? e[0] : e[0] & 0xFFFF0000u);
                const float z = static_cast<float>((SF32 ? e[1] : e[0]) & 0xFFu);
#pragma unroll
                for (int rr = 0; rr < TX; ++rr)
                    tot[rt][rr] = __builtin_fmaf(s, __builtin_fmaf(-z, xs[rr], acc[rt][rr]), tot[rt][rr]);
            }
        }
        wave_lds_sync();  // the slot has been read
    };

    Q4GStage<RT, TX> ring[D];
    const int nch = static_cast<int>(ceil_div(K, 128)), sch = static_cast<int>(p.slice / 128);
    for (int ch0 = 0; ch0 < nch; ch0 += sch) {
        // this slice's chunks, a contiguous run of them per wave
        const int cnt = std::min(sch, nch - ch0);
        const int first = ch0 + cnt * wave / NW, mine = ch0 + cnt * (wave + 1) / NW - first;
        auto at = [&](int k) { return first + std::min(k, std::max(mine - 1, 0)); };
#pragma unroll
        for (int q = 0; q < D; ++q) issue(ring[q], at(q));
        __builtin_amdgcn_sched_barrier(0);
        // scales and zero points of the slice, row by row
        if (ch0 > 0) __syncthreads();
        q4g_stage_constants<16 * RT / NW, NW, SF32>(p, sz, szrow, n0, nrows, ch0 << (7 - GL), ng, wave, lane);
        __syncthreads();
        for (int k0 = 0; k0 < mine; k0 += D) {
#pragma unroll
            for (int q = 0; q < D; ++q) {
                if (k0 + q < mine) consume(ring[q], first + k0 + q, ch0);
                __builtin_amdgcn_sched_barrier(0);
                issue(ring[q], at(k0 + q + D));
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }

    // the waves' sums through LDS, added in order
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        __syncthreads();
        float* const red = reinterpret_cast<float*>(slot);
#pragma unroll
        for (int rr = 0; rr < TX; ++rr) red[16 * (TX * g + rr) + li] = tot[rt][rr];
        __syncthreads();
        for (int e = tid; e < 64 * TX; e += 64 * NW) {
            const int tl = e >> 4, nl = 16 * rt + (e & 15);
            const bool live = tl < ntok && nl < nrows;
            float y = 0.0f;
#pragma unroll
            for (int ww = 0; ww < NW; ++ww) y += reinterpret_cast<const float*>(lds + ww * kSlot)[e];
            y = q4g_finite<SF32>(y, live, p.w, p.X, tl, n0, nl, K, lane);
            if (live) {
                const int64_t i = tl * N + n0 + nl;
                if (p.epilogue) y = q4g_epilogue(p.ep, y, n0 + nl, i);
                p.Y[i] = to_bf16_bits(y);
            }
        }
    }
}

// The same product for more tokens: x, 4 KiB per 16 tokens and chunk, goes
// straight from memory to the wave's LDS slot (global_load_lds), so that it
// takes no registers on the way, and every x operand serves RT row tiles. The
// next chunk's codes load while a chunk is multiplied, its x once the slot has
// been read; the SIMD's other wave works meanwhile.
//
// What bounds it: vector instructions on the CU with the most row tiles
// (unpacking, constants and the ends of groups; two row tiles and three of
// tokens with groups of 32 take 250 a chunk, 1000 cycles against 768 of MFMA),
// and a workgroup's way in and out, as many again over a wave's few chunks. So
// the tiles are dealt out evenly (launch_wide_variant; T = 37 at 11008 x 4096,
// groups of 32: 23.1 -> 19.7 us). Measured and not kept: x in two halves, one on
// its way while the other is used, codes a chunk ahead (within 3 %, so the loads
// are not what is waited for); waves side by side on one chunk's x (a quarter of
// x's way from L2, but a barrier a step lines the waves up: 25.4 us, and 15.8
// for 9.2 at 4096 x 4096).
template <int RT, int TT, int NW, int GL, bool SF32>
__global__ __launch_bounds__(64 * NW) void q4g_linear_wide_kernel(Q4GLinearArgs p) {
    constexpr int NG = 128 >> GL, MG = 4 / NG;
    constexpr int kSlot = 4096 * TT;
    // z sum_k x: a multiply-add per sum and group on the sums of x (one MFMA
    // with ones a step, shared by the row tiles), or, where groups are short,
    // one more MFMA per row tile with -z as the operand
    constexpr bool kZeroOperand = NG > 1;
    const bool has_zero = p.w.zero != nullptr;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, g = lane >> 4;
    const int64_t N = p.N, K = p.K, T = p.T;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16 * RT, t0 = static_cast<int64_t>(blockIdx.y) * 16 * TT;
    const int rowbytes = static_cast<int>(ceil_div(K, 32)) * 16, ng = static_cast<int>(ceil_div(K, int64_t{1} << GL));
    const int nrows = static_cast<int>(std::min<int64_t>(16 * RT, N - n0)), ntok = static_cast<int>(std::min<int64_t>(16 * TT, T - t0));
    uint8_t* const slot = lds + wave * kSlot;
    uint32_t* const sz = reinterpret_cast<uint32_t*>(lds + NW * kSlot);
    const int szrow = q4g_row_words(p.slice_groups, SF32);

    const uint8_t* const cbase = p.w.packed + n0 * rowbytes;
    const uint8_t* const xbase = reinterpret_cast<const uint8_t*>(p.X + t0 * K);
    const int last = static_cast<int>(ceil_div(K, 128)) - 1;
    const bool ragged = K % 128 != 0;
    const int cback = std::max(0, 64 * last + 16 * g + 16 - rowbytes);
    uint32_t coff[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
        coff[rt] = static_cast<uint32_t>(std::min(16 * rt + li, nrows - 1)) * static_cast<uint32_t>(rowbytes) + 16 * g;

    auto load_codes = [&](uint4 (&c)[RT], int ch) {
        const uint8_t* const cp = cbase + 64 * ch;
        const uint32_t cb = ch == last ? cback : 0;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) c[rt] = *reinterpret_cast<const uint4*>(cp + (coff[rt] - cb));
    };
    // load u takes tokens 4 u .. 4 u + 3; the lane's 16 bytes land at its own
    // place, so it fetches the piece that belongs there: position c of token j
    // holds piece c ^ j % 16
    uint32_t xoff[4 * TT];
#pragma unroll
    for (int u = 0; u < 4 * TT; ++u)
        xoff[u] = static_cast<uint32_t>(std::min(4 * u + g, ntok - 1)) * static_cast<uint32_t>(2 * K) + 16 * (li ^ ((4 * u + g) & 15));
    auto load_x = [&](int ch) {
        const uint8_t* const xp = xbase + 256 * ch;
        if (ragged && ch == last) {
            const int most = static_cast<int>(2 * K) - 256 * ch - 16;  // the last piece that a row has
#pragma unroll
            for (int u = 0; u < 4 * TT; ++u)
                load_lds16(xp + (xoff[u] - std::max(16 * (li ^ ((4 * u + g) & 15)) - most, 0)), slot + 1024 * u);
        } else {
#pragma unroll
            for (int u = 0; u < 4 * TT; ++u) load_lds16(xp + xoff[u], slot + 1024 * u);
        }
    };
    // the chunk that K ends in: x from K on is zero
    auto clear_past = [&]() {
#pragma unroll
        for (int u = 0; u < 4 * TT; ++u) {
            const int j = 4 * u + g;
            if (128 * static_cast<int64_t>(last) + 8 * (li ^ (j & 15)) >= K)
                *reinterpret_cast<uint4*>(slot + 1024 * u + 16 * lane) = make_uint4(0, 0, 0, 0);
        }
    };
    auto xin = [&](int tt, int m) {
        const int j = 16 * tt + li;
        return as_bf16x8(*reinterpret_cast<const uint4*>(slot + 256 * j + 16 * ((4 * m + g) ^ li)));
    };

    const bf16x8_t ones = as_bf16x8(make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u));
    f32x4 tot[RT][TT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) tot[rt][tt] = f32x4{0.f, 0.f, 0.f, 0.f};

    auto multiply = [&](const uint4 (&c)[RT], int gi0) {
        uint32_t cw[RT][4];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            cw[rt][0] = c[rt].x, cw[rt][1] = c[rt].y, cw[rt][2] = c[rt].z, cw[rt][3] = c[rt].w;
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
        }
        // a tile's sums of a group, times the scale, to the totals. Left alone the
        // compiler puts this off to the chunk's end and holds the sums of all groups
        // till then: a little faster where there are registers (1 to 5 %), but three
        // row tiles spill (T = 64 at 11008 x 4096, groups of 32: 62 us, pinned 23)
        auto add_part = [&](const f32x4 (&acc)[TT], float sc, int rt) {
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) {
#pragma unroll
                for (int rr = 0; rr < 4; ++rr) tot[rt][tt][rr] = __builtin_fmaf(sc, acc[tt][rr], tot[rt][tt][rr]);
                if constexpr (RT > 2 || RT * TT > 6) asm volatile("" : "+v"(tot[rt][tt]));
            }
        };
        f32x4 part[2][TT];
        float spart = 0.0f;
#pragma unroll
        for (int q = 0; q < NG; ++q) {
            // the rows' scales and zero points (past the last group x is zero)
            float sv[RT];
            uint32_t zv[RT];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const uint32_t* const e = sz + (16 * rt + li) * szrow + (SF32 ? 2 : 1) * std::min(gi0 + q, p.slice_groups - 1);
                sv[rt] = __uint_as_float(SF32 ? e[0] : e[0] & 0xFFFF0000u);
                zv[rt] = (SF32 ? e[1] : e[0]) & 0xFFu;
            }
            if constexpr (kZeroOperand) {
                // -z as an operand: 8 for all, or the row's; a row tile's sums at a time
                bf16x8_t xv[MG][TT];
#pragma unroll
                for (int mm = 0; mm < MG; ++mm)
#pragma unroll
                    for (int tt = 0; tt < TT; ++tt) xv[mm][tt] = xin(tt, q * MG + mm);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    uint32_t zz = 0xC100C100u;
                    if (has_zero) {
                        zz = __float_as_uint(-static_cast<float>(zv[rt]));
                        zz = __builtin_amdgcn_perm(zz, zz, 0x07060302u);
                    }
                    const bf16x8_t zop = as_bf16x8(make_uint4(zz, zz, zz, zz));
                    f32x4 (&acc)[TT] = part[(q * RT + rt) & 1];
#pragma unroll
                    for (int tt = 0; tt < TT; ++tt) acc[tt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int mm = 0; mm < MG; ++mm) {
                        const bf16x8_t wv = q4g_operand_ordered(cw[rt][q * MG + mm]);
#pragma unroll
                        for (int tt = 0; tt < TT; ++tt) {
                            acc[tt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[mm][tt], zop, acc[tt], 0, 0, 0);
                            acc[tt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[mm][tt], wv, acc[tt], 0, 0, 0);
                        }
                    }
                    // the tile before, whose products are done by now
                    if (q * RT + rt > 0) add_part(part[(q * RT + rt + 1) & 1], spart, (rt + RT - 1) % RT);
                    spart = sv[rt];
                }
            } else {
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
                    bf16x8_t xv[TT];
#pragma unroll
                    for (int tt = 0; tt < TT; ++tt) {
                        xv[tt] = xin(tt, m);
                        xs[tt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[tt], ones, xs[tt], 0, 0, 0);
                    }
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        const bf16x8_t wv = q4g_operand_ordered(cw[rt][m]);
#pragma unroll
                        for (int tt = 0; tt < TT; ++tt)
                            acc[rt][tt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[tt], wv, acc[rt][tt], 0, 0, 0);
                    }
                }
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                        for (int rr = 0; rr < 4; ++rr) {
                            const float d = __builtin_fmaf(-static_cast<float>(zv[rt]), xs[tt][rr], acc[rt][tt][rr]);
                            tot[rt][tt][rr] = __builtin_fmaf(sv[rt], d, tot[rt][tt][rr]);
                        }
            }
        }
        if constexpr (kZeroOperand) add_part(part[(NG * RT + 1) & 1], spart, RT - 1);
    };

    const int nch = last + 1, sch = static_cast<int>(p.slice / 128);
    for (int ch0 = 0; ch0 < nch; ch0 += sch) {
        const int cnt = std::min(sch, nch - ch0);
        const int first = ch0 + cnt * wave / NW, end = ch0 + cnt * (wave + 1) / NW;
        if (ch0 > 0) __syncthreads();  // the previous slice's constants have been read
        q4g_stage_constants<16 * RT / NW, NW, SF32>(p, sz, szrow, n0, nrows, ch0 << (7 - GL), ng, wave, lane);
        uint4 cur[RT], nxt[RT];
        if (first < end) {
            load_codes(cur, first);
            load_x(first);
        }
        __syncthreads();
        for (int ch = first; ch < end; ++ch) {
            wait_vmcnt<0>();  // x and the codes of this chunk are here
            wave_lds_sync();
            load_codes(nxt, std::min(ch + 1, end - 1));
            __builtin_amdgcn_sched_barrier(0);
            if (ragged && ch == last) {
                clear_past();
                wave_lds_sync();
            }
            multiply(cur, (ch - ch0) * NG);
            wave_lds_sync();
            if (ch + 1 < end) {
                wait_lgkmcnt0();  // the slot has been read
                load_x(ch + 1);
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) cur[rt] = nxt[rt];
        }
    }

#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        __syncthreads();
        float* const red = reinterpret_cast<float*>(slot);
#pragma unroll
        for (int tt = 0; tt < TT; ++tt)
#pragma unroll
            for (int rr = 0; rr < 4; ++rr) red[256 * tt + 16 * (4 * g + rr) + li] = tot[rt][tt][rr];
        __syncthreads();
        for (int e = tid; e < TT * 256; e += 64 * NW) {
            const int tl = e >> 4, nl = 16 * rt + (e & 15);
            const bool live = tl < ntok && nl < nrows;
            float y = 0.0f;
#pragma unroll
            for (int ww = 0; ww < NW; ++ww) y += reinterpret_cast<const float*>(lds + ww * kSlot)[e];
            y = q4g_finite<SF32>(y, live, p.w, p.X + t0 * K, tl, n0, nl, K, lane);
            if (live) {
                const int64_t i = (t0 + tl) * N + n0 + nl;
                if (p.epilogue) y = q4g_epilogue(p.ep, y, n0 + nl, i);
                p.Y[i] = to_bf16_bits(y);
            }
        }
    }
}

// Values of a row whose constants a workgroup keeps in LDS at a time: the
// whole row where 16 RT rows of them fit the budget, else a slice of whole
// chunks that does.
void set_slice(Q4GLinearArgs& a, int rows, bool sf32, size_t budget) {
    const int64_t words = static_cast<int64_t>(budget / sizeof(uint32_t)) / rows - 1;
    const int64_t most = std::max<int64_t>((sf32 ? words / 2 : words) * a.w.group / 128 * 128, 128);
    a.slice = std::min(ceil_div(a.K, 128) * 128, most);
    a.slice_groups = static_cast<int>(a.slice / a.w.group);
}

// LDS may pass the 64 KiB that a launch gets unasked.
template <typename Kernel>
int launch_lds(Kernel kern, dim3 grid, int threads, size_t lds, const Q4GLinearArgs& a, hipStream_t stream) {
    if (lds > 65536 && hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(lds)) != hipSuccess)
        return set_error(QL_ERR_HIP, "4-bit group linear: %zu bytes of LDS refused", lds);
    hipLaunchKernelGGL(kern, grid, dim3(threads), static_cast<uint32_t>(lds), stream, a);
    return QL_OK;
}

constexpr size_t kLdsBytes = 163840, kConstBytes = 32768;

template <int RT, int TX, int D, int GL, bool SF32>
int launch_narrow(Q4GLinearArgs a, hipStream_t stream) {
    set_slice(a, 16 * RT, SF32, kConstBytes);
    const size_t lds = 8 * 1024 * TX + 16 * RT * sizeof(uint32_t) * q4g_row_words(a.slice_groups, SF32);
    return launch_lds(q4g_linear_kernel<RT, TX, D, GL, SF32>, dim3(static_cast<uint32_t>(ceil_div(a.N, 16 * RT))), 512, lds,
                      a, stream);
}

template <int RT, int TT, int NW, int GL, bool SF32>
int launch_wide(Q4GLinearArgs a, hipStream_t stream) {
    constexpr size_t slots = NW * 4096 * TT;
    set_slice(a, 16 * RT, SF32, std::min(kConstBytes, kLdsBytes - slots));
    const size_t lds = slots + 16 * RT * sizeof(uint32_t) * q4g_row_words(a.slice_groups, SF32);
    const dim3 grid(static_cast<uint32_t>(ceil_div(a.N, 16 * RT)), static_cast<uint32_t>(ceil_div(a.T, 16 * TT)));
    return launch_lds(q4g_linear_wide_kernel<RT, TT, NW, GL, SF32>, grid, 64 * NW, lds, a, stream);
}

// The variant of the wide kernel. A CU's work is its share of the row tiles,
// so the tiles a workgroup takes (RT) are those with the least of them on the
// fullest CU, RT ceil(workgroups / 256); of equals the most, which read x (and
// fetch instructions) least often. Measured (us; 16 x RT rows by NW waves
// 1x8 | 2x8 | 2x4 | 3x8 | 3x4, groups of 128 unless said):
//   256 tiles   T = 37 4096 x 4096 9.3 | 10.9 | 12.8, T = 64 4096 x 11008 23.8 | 25.3 | 31.3 | 30.5 | 38.1
//   512         T = 128 4096 x 4096 20.0 | 13.7 | 16.2, T = 37 8192 x 8192 - | 19.1 | - | 22.1 | 25.5
//   640         T = 37 10240 x 8192 - | - | 28.4 | 22.6 | 26.2, (32) 43.6 | 37.4 | 46.1 for the last three
//   688         T = 37 11008 x 4096 (32) 28.4 | 24.7 | 23.1 | 19.8 | 22.4, T = 64 29.2 | 25.2 | 21.4 | 18.0 | 20.5
//   1024        T = 200 4096 x 4096 38.4 | 25.6 | 23.5
//   1376        T = 64 22016 x 8192 101 | 65.4 | 62.4 | 54.8 | 52.5, (64) 107 | 71.6 | 84 | 65 | 75,
//               (32) - | 87 | - | 86 | 105, T = 37 - | - | 56.5 | 45.5 | 42.7
// Eight waves where each CU gets one workgroup; beyond, four (and two of them)
// but for short groups with many tokens, whose registers leave no room for two
// (T = 200 4096 x 4096 (32) 31 | 37 with eight and four; T = 40 13824 x 5120 (32)
// 31.4 | 29.5).
template <int TT, int GL, bool SF32>
int launch_wide_variant(const Q4GLinearArgs& a, hipStream_t stream) {
    auto blocks = [&](int rt) { return ceil_div(a.N, 16 * rt) * ceil_div(a.T, 16 * TT); };
    auto most = [&](int rt) { return rt * ceil_div(blocks(rt), 256); };
    constexpr int kWaves3 = TT == 4 && GL < 7 ? 8 : 4, kWaves2 = TT == 4 && GL == 5 ? 8 : 4;
    if (most(3) <= std::min(most(1), most(2)))
        return blocks(3) <= 256 ? launch_wide<3, TT, 8, GL, SF32>(a, stream) : launch_wide<3, TT, kWaves3, GL, SF32>(a, stream);
    if (most(2) <= most(1))
        return blocks(2) <= 256 ? launch_wide<2, TT, 8, GL, SF32>(a, stream) : launch_wide<2, TT, kWaves2, GL, SF32>(a, stream);
    return launch_wide<1, TT, 8, GL, SF32>(a, stream);
}

// The variant by tokens. Up to 8 of them (16 with short groups) two row tiles
// from four workgroups a CU on (1024), one before (us, one | two):
//   T = 1   4096 x 4096 5.0 | 6.5, 11008 x 4096 (32) 9.5 | 11.0, 22016 x 8192 26.8 | 24.4
//   T = 8   4096 x 4096 5.3 | 7.0, 22016 x 8192 36.9 | 28.0
//   T = 16  11008 x 4096 (64) 11.6 | 13.2, (32) 12.4 | 15.2, 22016 x 8192 (32) 44.6 | 42.6
// At 16 tokens the wide kernel's rule gains with groups of 128 (10240 x 8192
// 18.2 -> 16.2, 22016 x 8192 31.1 -> 29.2) and loses with groups of 32 (19.3 ->
// 25.9, 41.8 -> 47.1); with groups of 64 it is even but for the largest (4096 x
// 4096 6.4 | 6.5, 11008 x 4096 11.4 | 10.9, 10240 x 8192 19.0 | 19.1, 22016 x 8192
// 29.0 | 32.6), so they go with those of 32.
template <int GL, bool SF32>
int launch_linear_variant(const Q4GLinearArgs& a, hipStream_t stream) {
    const bool two = ceil_div(a.N, 16) > 1024;
    if (a.T <= 4) return two ? launch_narrow<2, 1, 1, GL, SF32>(a, stream) : launch_narrow<1, 1, 2, GL, SF32>(a, stream);
    if (a.T <= 8) return two ? launch_narrow<2, 2, 1, GL, SF32>(a, stream) : launch_narrow<1, 2, 2, GL, SF32>(a, stream);
    if (a.T <= 16) {
        if constexpr (GL == 7)
            return launch_wide_variant<1, GL, SF32>(a, stream);
        else
            return two ? launch_wide<2, 1, 4, GL, SF32>(a, stream) : launch_wide<1, 1, 8, GL, SF32>(a, stream);
    }
    if (a.T <= 32) return launch_wide_variant<2, GL, SF32>(a, stream);
    if (a.T <= 48) return launch_wide_variant<3, GL, SF32>(a, stream);
    return launch_wide_variant<4, GL, SF32>(a, stream);
}

template <bool WF32, int G, bool SF32>
void launch_quantize_g(const void* W, int64_t N, int64_t K, uint8_t* packed, void* scale, uint8_t* zero,
                       hipStream_t stream) {
    const int64_t lanes = ceil_div(K, G) * (G / 8);  // of a row: whole groups
    hipLaunchKernelGGL((q4g_quantize_kernel<WF32, G, SF32>), dim3(static_cast<uint32_t>(ceil_div(N * lanes, kThreads))),
                       dim3(kThreads), 0, stream, W, static_cast<uint32_t>(N), static_cast<uint32_t>(K), row_divisor(lanes),
                       packed, scale, zero);
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
        constexpr bool WF32 = decltype(wf)::value, SF32 = decltype(sf)::value;
        switch (group) {
            case 32: launch_quantize_g<WF32, 32, SF32>(W, N, K, packed, scale, zero, stream); break;
            case 64: launch_quantize_g<WF32, 64, SF32>(W, N, K, packed, scale, zero, stream); break;
            default: launch_quantize_g<WF32, 128, SF32>(W, N, K, packed, scale, zero, stream); break;
        }
    });
    timer_end(QL_KERNEL_Q4G_QUANTIZE, stream);
    return check_launch("4-bit group quantize");
}

int launch_q4g_dequantize(const Q4GDev& w, int64_t N, int64_t K, void* out, bool bf16_out, hipStream_t stream) {
    const dim3 grid(static_cast<uint32_t>(ceil_div(N * (K / 8), kThreads))), block(kThreads);
    timer_begin(QL_KERNEL_Q4G_DEQUANTIZE, stream);
    with_flags(bf16_out, w.scale_f32 != 0, [&](auto bf, auto sf) {
        hipLaunchKernelGGL((q4g_dequantize_kernel<decltype(bf)::value, decltype(sf)::value>), grid, block, 0, stream, w,
                           static_cast<uint32_t>(N), static_cast<uint32_t>(K), row_divisor(K / 8), out);
    });
    timer_end(QL_KERNEL_Q4G_DEQUANTIZE, stream);
    return check_launch("4-bit group dequantize");
}

int launch_q4g_linear(const Q4GDev& w, const uint16_t* X, int64_t T, int64_t N, int64_t K, uint16_t* Y,
                      hipStream_t stream, const Epilogue* ep) {
    const Q4GLinearArgs a{w, X, T, N, K, Y, 0, 0, ep != nullptr ? *ep : Epilogue{}, ep != nullptr};
    timer_begin(QL_KERNEL_Q4G_LINEAR, stream);
    int s;
    switch (w.group) {
        case 32: s = w.scale_f32 ? launch_linear_variant<5, true>(a, stream) : launch_linear_variant<5, false>(a, stream); break;
        case 64: s = w.scale_f32 ? launch_linear_variant<6, true>(a, stream) : launch_linear_variant<6, false>(a, stream); break;
        default: s = w.scale_f32 ? launch_linear_variant<7, true>(a, stream) : launch_linear_variant<7, false>(a, stream); break;
    }
    timer_end(QL_KERNEL_Q4G_LINEAR, stream);
    if (s != QL_OK) return s;
    return check_launch("4-bit group linear");
}

}  // namespace qlnf4
