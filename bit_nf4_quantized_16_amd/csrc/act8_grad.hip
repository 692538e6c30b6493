// Adapter gradients from an 8-bit checkpoint of the layer's input (gfx950,
// bf16 MFMA): reductions over the tokens
//
//   out[j][c] (dA) or out[c][j] (dB) = scale * sum_t V[t][j] M[t][c]
//
// with M = X (8-bit checkpoint, the dropout mask applied where there is one)
// and V = G = s dY B for dA; M = dY (bf16) and V = U for dB. V comes as fp32
// and is not rounded: it is split into three bf16 terms v = h + m + l (8
// significant bits each, 24 in all), multiplied by the exact bf16 values of M
// and summed in fp32, so dA and dB carry fp32 rounding only. An infinite M
// times a term that is zero would be NaN where v M is infinite: a wave whose
// sums are not finite takes its tokens again with M's infinities (and NaN) in
// the products of the leading term h alone. One grid holds
// both problems: workgroups [0, nblk0) take column blocks of the first, the
// rest those of the second.
//
// The waves of a workgroup take 32-token chunks in turn. A wave expands its
// chunk of M to bf16 in a private LDS tile and reads it back column-wise
// (eight consecutive tokens of one column per lane: the MFMA B operand). The
// next chunk's loads are issued before a chunk is multiplied and kept as they
// come (codes, not values), so nothing waits for them until they are used.
// V up to rank 16 is split by every workgroup for itself, through a second
// tile, one term at a time (read like M: the A operand). Larger ranks would
// spend most of their instructions on that (rank 64, T = 4096: 102 us), so
// their terms are written once, by a small kernel before, in the order of the
// A operand: 1 KiB per 32 tokens, 16 ranks and term, read in one load.
// With one token split the workgroup writes the gradient itself (fixed-order
// sum of the waves); with several, fp32 partials in the output's layout go to
// the workspace and a second kernel adds them in order.
//
// What bounds it: the instructions that expand M and carry it through LDS to
// the transposed operand, each wave's chunk after chunk. N = K = 4096, rank 16,
// T = 1024: 9.7 us replayed (12.7 MB, 1.3 TB/s). N = 4096, K = 11008, rank 64,
// T = 4096: 5.0 us for the terms, 53.1 here (79 MB, 1.5 TB/s; 24 GFLOP of term
// products), 5.1 for the partials. Eight 16-column tiles a wave there: 122 us
// for the whole (few workgroups), two waves' loads more in flight at 128
// registers: 107.
#include <algorithm>
#include <type_traits>

#include "act8.h"
#include "common.h"
#include "internal.h"
#include "mm_common.h"

namespace qlnf4 {

namespace {

constexpr int kRows = 32;  // tokens per MFMA step

// 16-bit lane masks of eight elements from their eight keep bits.
__device__ __forceinline__ uint4 keep_mask(uint32_t bits) {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
        w[q] = ((bits >> (2 * q)) & 1u ? 0x0000FFFFu : 0u) | ((bits >> (2 * q + 1)) & 1u ? 0xFFFF0000u : 0u);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// What v's leading 8 significant bits (its top half) leave, exactly. Infinity
// less itself would be NaN: with check it leaves nothing.
__device__ __forceinline__ float split_rest(float v, bool check) {
    const float rest = v - __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
    return check && fabsf(v) == __builtin_inff() ? 0.0f : rest;
}

// The operand with its infinities and NaN as zeros.
__device__ __forceinline__ bf16x8_t finite_only(bf16x8_t v) {
    uint4 x = __builtin_bit_cast(uint4, v);
    uint32_t* const w[4] = {&x.x, &x.y, &x.z, &x.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        // a magnitude of 0x7F80 or more carries into its half's sign bit, which then fills the half
        const u16x2_act c = __builtin_bit_cast(u16x2_act, *w[q] & 0x7FFF7FFFu) + u16x2_act{0x80, 0x80};
        *w[q] &= ~__builtin_bit_cast(uint32_t, __builtin_bit_cast(i16x2_act, c) >> i16x2_act{15, 15});
    }
    return as_bf16x8(x);
}

// Tiles of a rank of RT x 16: the columns a workgroup takes (16 CB), its
// waves, and whether V's terms come prepared.
template <int RT, int CB_>
struct GradTile {
    static constexpr int CB = CB_;
    static constexpr bool kTerms = RT > 1;
    static constexpr int NW = 8;
    static constexpr int LdM = 16 * CB + 8, LdV = kTerms ? 0 : 16 * RT + 8;
    static constexpr int kTile = kRows * (LdM + LdV);  // 16-bit words of one wave
};

// A wave's chunk of M as loaded: MI pieces of eight columns a lane (codes or
// bf16 values); of a checkpoint also the scale byte and the keep bits of one
// block of 32, block b of token t in lane t CB / 2 + b.
template <int MI, bool ACT8>
struct GradStage {
    uint4 m[ACT8 ? 1 : MI];
    uint2 c[ACT8 ? MI : 1];
    uint32_t s, k;
};

template <int RT, int CB_, bool ACT8>
__device__ __forceinline__ void grads_block(const Act8GradArgs& a, const Act8GradProblem& pb, int64_t c0, uint16_t* sm) {
    using G = GradTile<RT, CB_>;
    constexpr bool kTerms = G::kTerms;
    constexpr int CB = G::CB, NW = G::NW, LdM = G::LdM, LdV = G::LdV;
    constexpr int PR = 2 * CB;        // pieces of a token's row
    constexpr int MI = kRows * PR / 64;
    using Stage = GradStage<MI, ACT8>;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, g = lane >> 4;
    const int64_t C = pb.C;
    const int r = a.r;
    const int64_t tb = blockIdx.y * a.t_per;
    const int64_t te = std::min<int64_t>(tb + a.t_per, a.T);
    f32x4 acc[RT][CB];
    uint16_t* const tm = sm + wave * G::kTile;
    uint16_t* const tv = tm + kRows * LdM;
    const bool masked = ACT8 && pb.keep != nullptr;
    const bool quads = (r & 3) == 0;
    constexpr int RI = 64 / PR;  // tokens of a load

    // A base that is the same for the wave and an offset of the lane. Out of
    // range (tokens from te on, columns from C on, ranks from r on) the nearest
    // element in range is read, and zeroed or left out when it is used.
    const int64_t col = std::min<int64_t>(c0 + 8 * (lane % PR), C - 8), moff = (lane / PR) * C + col;
    constexpr int BPR = CB / 2;  // blocks of a token's row
    static_assert(kRows * BPR <= 64, "a lane per block");
    const int brow = std::min(lane / BPR, kRows - 1);
    const int64_t bcol = std::min<int64_t>(c0 / kAct8Block + lane % BPR, C / kAct8Block - 1);
    auto load_m = [&](Stage& st, int64_t t) {
        const bool tail = t + kRows > te;
        if constexpr (ACT8) {
            // one load for the chunk's scales (and one for its mask): a byte per
            // piece would touch a line per token again and again
            const int64_t at = std::min<int64_t>(t + brow, te - 1) * (C / kAct8Block) + bcol;
            if (masked) st.k = reinterpret_cast<const uint32_t*>(pb.keep)[at];
            st.s = pb.scale8[at];
        }
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            int64_t at = (t + RI * i) * C + moff;
            if (tail) at = std::min<int64_t>(t + RI * i + lane / PR, te - 1) * C + col;
            if constexpr (ACT8)
                st.c[i] = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(pb.M) + at);
            else
                st.m[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(pb.M) + at);
        }
    };
    // V of the chunk: quads of ranks, 4 RT a token
    auto load_v = [&](float (&v)[2 * RT][4], int64_t t) {
        const int left = static_cast<int>(std::min<int64_t>(te - t, kRows)) - 1;
        const float* const base = pb.V + t * r;
#pragma unroll
        for (int i = 0; i < 2 * RT; ++i) {
            const int q = lane + 64 * i, j = 4 * (q % (4 * RT));
            const float* const p = base + std::min(q / (4 * RT), left) * r;
            if (quads) {
                const float4 f = *reinterpret_cast<const float4*>(p + std::min(j, r - 4));
                v[i][0] = f.x, v[i][1] = f.y, v[i][2] = f.z, v[i][3] = f.w;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i][e] = p[std::min(j + e, r - 1)];
            }
        }
    };
    // M of a chunk to the wave's tile
    auto put_m = [&](const Stage& st, int64_t t) {
        const bool tail = t + kRows > te;
        wave_lds_sync();  // the previous chunk's reads are done
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int e = lane + 64 * i;
            uint4 x;
            if constexpr (ACT8) {
                const int from = (e / PR) * BPR + (e % PR) / 4;  // the lane with the piece's block
                x = act8_decode8(st.c[i], __shfl(st.s, from, 64));
                if (masked) {
                    const uint4 k = keep_mask(__shfl(st.k, from, 64) >> (8 * (e % 4)));
                    x = make_uint4(x.x & k.x, x.y & k.y, x.z & k.z, x.w & k.w);
                }
            } else {
                x = st.m[i];
            }
            if (tail && t + e / PR >= te) x = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(tm + (e / PR) * LdM + 8 * (e % PR)) = x;
        }
    };
    bf16x8_t bv[CB];
    auto get_m = [&]() {
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) bv[cb] = lds_col8(tm, LdM, 8 * g, 16 * cb, li);
    };
    auto drop_infinities = [&]() {
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) bv[cb] = finite_only(bv[cb]);
    };
    // the chunk's products with V's terms as prepared. Loads return in order:
    // the terms (from L2) are asked for before the next chunk of M (from HBM),
    // or every chunk would wait for that as well (rank 64, T = 4096,
    // 4096 + 11008 columns: 63 against 57 us).
    constexpr int RS = RT <= 4 ? RT : (RT + 1) / 2;  // rank tiles whose operands are in registers together
    // careful (a constant): M's infinities meet the leading terms alone, and no
    // loads ahead.
    auto multiply_terms = [&](auto careful, const Stage& st, Stage& next, int64_t t, int64_t tn) {
        const uint4* const vop = reinterpret_cast<const uint4*>(pb.terms) + (t / kRows) * (3 * RT * 64) + lane;
#pragma unroll
        for (int r0 = 0; r0 < RT; r0 += RS) {
            uint4 av[RS][3];
#pragma unroll
            for (int rt = 0; rt < RS; ++rt)
#pragma unroll
                for (int term = 0; term < 3; ++term)
                    if (r0 + rt < RT) av[rt][term] = vop[((r0 + rt) * 3 + term) * 64];
            __builtin_amdgcn_sched_barrier(0);
            if (!careful && r0 + RS >= RT) load_m(next, tn);
            __builtin_amdgcn_sched_barrier(0);
            if (r0 == 0) {
                put_m(st, t);
                wave_lds_sync();
                get_m();
            } else if (careful) {
                get_m();
            }
#pragma unroll
            for (int i = 0; i < RS * 3; ++i) {
                // a rank tile's terms one after the other, or (careful) all leading terms first
                const int rt = careful ? i % RS : i / 3, term = careful ? i / RS : i % 3;
                if (careful && i == RS) drop_infinities();
                if (r0 + rt < RT) {
#pragma unroll
                    for (int cb = 0; cb < CB; ++cb)
                        acc[r0 + rt][cb] =
                            __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(av[rt][term]), bv[cb], acc[r0 + rt][cb], 0, 0, 0);
                }
            }
        }
    };
    // the same with V split here
    auto multiply_split = [&](auto careful, const Stage& st, float (&v)[2 * RT][4], int64_t t) {
        put_m(st, t);
        if (t + kRows > te || (r & 15) != 0) {  // nothing past the tokens and the rank
#pragma unroll
            for (int i = 0; i < 2 * RT; ++i) {
                const int q = lane + 64 * i, j = 4 * (q % (4 * RT));
                const bool out = t + q / (4 * RT) >= te;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (out || j + e >= r) v[i][e] = 0.0f;
            }
        }
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < 2 * RT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) most = fmaxf(most, fabsf(v[i][e]));
        const bool inf = __any(most == __builtin_inff());
#pragma unroll
        for (int term = 0; term < 3; ++term) {
            if (term > 0) wave_lds_sync();
#pragma unroll
            for (int i = 0; i < 2 * RT; ++i) {
                const int q = lane + 64 * i;
                uint32_t h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    h[e] = __float_as_uint(v[i][e]);
                    if (term < 2) v[i][e] = split_rest(v[i][e], inf);
                }
                *reinterpret_cast<uint2*>(tv + (q / (4 * RT)) * LdV + 4 * (q % (4 * RT))) =
                    make_uint2(__builtin_amdgcn_perm(h[1], h[0], 0x07060302u), __builtin_amdgcn_perm(h[3], h[2], 0x07060302u));
            }
            wave_lds_sync();
            if (term == 0) get_m();
            if (term == 1 && careful) drop_infinities();
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const bf16x8_t av = lds_col8(tv, LdV, 8 * g, 16 * rt, li);
#pragma unroll
                for (int cb = 0; cb < CB; ++cb)
                    acc[rt][cb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, bv[cb], acc[rt][cb], 0, 0, 0);
            }
        }
    };

    auto clear = [&]() {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int cb = 0; cb < CB; ++cb) acc[rt][cb] = f32x4{0.f, 0.f, 0.f, 0.f};
    };
    Stage cur, nxt;
    constexpr std::false_type kPlain{};
    constexpr std::true_type kCareful{};
    clear();
    int64_t t = tb + kRows * wave;
    if (t < te) {
        load_m(cur, t);
        if constexpr (kTerms) {
            for (; t < te; t += NW * kRows) {
                multiply_terms(kPlain, cur, nxt, t, std::min<int64_t>(t + NW * kRows, te - 1));
                cur = nxt;
            }
        } else {
            float vcur[2 * RT][4], vnxt[2 * RT][4];
            load_v(vcur, t);
            for (; t < te; t += NW * kRows) {
                const int64_t tn = std::min<int64_t>(t + NW * kRows, te - 1);
                load_m(nxt, tn);
                load_v(vnxt, tn);
                __builtin_amdgcn_sched_barrier(0);
                multiply_split(kPlain, cur, vcur, t);
                cur = nxt;
#pragma unroll
                for (int i = 0; i < 2 * RT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) vcur[i][e] = vnxt[i][e];
            }
        }
    }
    bool finite = true;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
            for (int q = 0; q < 4; ++q) finite = finite && fabsf(acc[rt][cb][q]) < __builtin_inff();
    if (__builtin_expect(!__all(finite), 0)) {
        clear();
#pragma unroll 1
        for (t = tb + kRows * wave; t < te; t += NW * kRows) {
            load_m(cur, t);
            if constexpr (kTerms) {
                multiply_terms(kCareful, cur, cur, t, t);
            } else {
                float v[2 * RT][4];
                load_v(v, t);
                multiply_split(kCareful, cur, v, t);
            }
        }
    }

    // D[j = 4 g + q][column li] of each tile, rank tile by rank tile: the upper
    // half of the waves hand theirs to the lower half through LDS, whose sums
    // are then added in order
    float* const red = reinterpret_cast<float*>(sm);
    constexpr int W2 = NW / 2, kRed = 16 * 16 * CB;
    static_assert(W2 * kRed * 2 <= NW * G::kTile, "the sums fit the tiles");
    const bool direct = gridDim.y == 1;
    float* const out = direct ? pb.out : pb.part + static_cast<int64_t>(blockIdx.y) * r * C;
    const float scale = direct ? pb.scale : 1.0f;
    for (int rt = 0; rt < RT; ++rt) {
        __syncthreads();
#pragma unroll
        for (int half = 1; half >= 0; --half) {
            if ((wave >= W2) == (half == 1)) {
                float* const rw = red + (wave % W2) * kRed;
#pragma unroll
                for (int cb = 0; cb < CB; ++cb)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float& d = rw[(4 * g + q) * 16 * CB + 16 * cb + li];
                        float v = acc[0][cb][q];
#pragma unroll
                        for (int x = 1; x < RT; ++x) v = x == rt ? acc[x][cb][q] : v;
                        d = half == 1 ? v : v + d;
                    }
            }
            __syncthreads();
        }
        for (int e = tid; e < kRed; e += 64 * NW) {
            // consecutive threads along the output's contiguous direction
            const int jl = pb.layout_jc ? e / (16 * CB) : e % 16, cl = pb.layout_jc ? e % (16 * CB) : e / 16;
            const int j = 16 * rt + jl;
            const int64_t c = c0 + cl;
            if (c >= C || j >= r) continue;
            float v = 0.0f;
#pragma unroll
            for (int ww = 0; ww < W2; ++ww) v += red[ww * kRed + jl * 16 * CB + cl];
            const int64_t idx = pb.layout_jc ? j * C + c : c * r + j;
            v *= scale;
            out[idx] = direct && a.accumulate ? out[idx] + v : v;
        }
    }
}

template <int RT, int CB>
__global__ __launch_bounds__((64 * GradTile<RT, CB>::NW), RT <= 2 ? 4 : 2) void act8_grads_kernel(Act8GradArgs a) {
    using G = GradTile<RT, CB>;
    __shared__ __attribute__((aligned(16))) uint16_t sm[G::NW * G::kTile];
    const bool second = static_cast<int>(blockIdx.x) >= a.nblk0;
    const Act8GradProblem& pb = second ? a.pb[1] : a.pb[0];
    const int64_t c0 = static_cast<int64_t>(second ? blockIdx.x - a.nblk0 : blockIdx.x) * 16 * CB;
    if (pb.scale8 != nullptr)
        grads_block<RT, CB, true>(a, pb, c0, sm);
    else
        grads_block<RT, CB, false>(a, pb, c0, sm);
}

// V's terms in the order of the A operand: for 32 tokens, 16 ranks and term
// the 64 lanes' 16 bytes, lane (li, g) holding rank li at tokens 8 g .. 8 g + 7;
// zero past the tokens and the rank. One wave per 32 tokens and 16 ranks.
__global__ __launch_bounds__(256) void act8_terms_kernel(Act8GradArgs a, int rt_all, int64_t units) {
    const int lane = threadIdx.x & 63, li = lane & 15, g = lane >> 4;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    const Act8GradProblem& pb = a.pb[blockIdx.y];
    if (unit >= units || pb.out == nullptr) return;
    const int64_t t0 = unit / rt_all * kRows + 8 * g;
    const int j = static_cast<int>(unit % rt_all) * 16 + li;
    uint32_t h[3][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float v = t0 + e < a.T && j < a.r ? pb.V[(t0 + e) * a.r + j] : 0.0f;
#pragma unroll
        for (int term = 0; term < 3; ++term) {
            h[term][e] = __float_as_uint(v);
            v = split_rest(v, true);
        }
    }
    uint4* const out = reinterpret_cast<uint4*>(pb.terms) + unit * (3 * 64) + lane;
#pragma unroll
    for (int term = 0; term < 3; ++term) {
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = __builtin_amdgcn_perm(h[term][2 * q + 1], h[term][2 * q], 0x07060302u);
        out[term * 64] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Sum of the token splits of both problems, in split order.
__global__ __launch_bounds__(256) void act8_grads_final_kernel(Act8GradArgs a, int splits) {
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t n0 = static_cast<int64_t>(a.r) * a.pb[0].C;
    const int64_t n1 = static_cast<int64_t>(a.r) * a.pb[1].C;
    if (idx >= n0 + n1) return;
    const bool second = idx >= n0;
    const Act8GradProblem& pb = second ? a.pb[1] : a.pb[0];
    const int64_t e = second ? idx - n0 : idx, n = second ? n1 : n0;
    float s = 0.0f;
    for (int ts = 0; ts < splits; ++ts) s += pb.part[ts * n + e];
    const float v = pb.scale * s;
    pb.out[e] = a.accumulate ? pb.out[e] + v : v;
}

constexpr int kCols = 64;  // columns a workgroup takes, but for the narrow tile below
constexpr int kWaves = 8;

// Token splits: one (no second kernel) while a wave's loop stays short; else
// about one workgroup a CU, each wave keeping two chunks at least.
int splits_of(int64_t T, int64_t C0, int64_t C1, int r) {
    if (T <= 2048 || C0 + C1 <= 0) return 1;
    const int64_t blocks = ceil_div(C0, kCols) + ceil_div(C1, kCols);
    const int64_t s = std::min<int64_t>(ceil_div(256, blocks), T / (2 * kWaves * kRows));
    return static_cast<int>(std::max<int64_t>(s, 1));
}

// Bytes of one V's terms (ranks over 16).
size_t terms_bytes(int64_t T, int r) {
    return r <= 16 ? 0 : static_cast<size_t>(ceil_div(T, kRows)) * (lora_grad_rp(r) / 16) * 3 * 1024;
}

template <int RT, int CB>
void launch_grads(const Act8GradArgs& a, dim3 grid, hipStream_t stream) {
    hipLaunchKernelGGL((act8_grads_kernel<RT, CB>), grid, dim3(64 * GradTile<RT, CB>::NW), 0, stream, a);
}

}  // namespace

size_t act8_grads_part_bytes(int64_t T, int64_t C0, int64_t C1, int r) {
    const int sp = splits_of(T, C0, C1, r);
    const size_t part = sp == 1 ? 0 : static_cast<size_t>(sp) * r * (C0 + C1) * sizeof(float);
    return (part + 255) / 256 * 256 + terms_bytes(T, r) * ((C0 > 0) + (C1 > 0));
}

int launch_act8_grads(Act8GradArgs a, float* part, hipStream_t stream) {
    if (a.pb[0].out == nullptr) {  // only the second problem: move it first
        a.pb[0] = a.pb[1];
        a.pb[1] = Act8GradProblem{};
    }
    if (a.pb[0].out == nullptr) return QL_OK;
    if (a.r < 1 || a.r > QL_MAX_RANK) return set_error(QL_ERR_SHAPE, "adapter gradients: rank %d out of range", a.r);
    if (a.pb[1].out == nullptr) a.pb[1].C = 0;
    const int64_t c0 = a.pb[0].C, c1 = a.pb[1].C;
    const int per = kWaves * kRows;
    int splits = splits_of(a.T, c0, c1, a.r);
    if (act8_grads_part_bytes(a.T, c0, c1, a.r) > 0 && part == nullptr)
        return set_error(QL_ERR_WORKSPACE, "adapter gradients: workspace missing");
    if (a.r > 16) {  // the terms sit behind the partials
        const size_t pbytes = splits == 1 ? 0 : static_cast<size_t>(splits) * a.r * (c0 + c1) * sizeof(float);
        char* at = reinterpret_cast<char*>(part) + (pbytes + 255) / 256 * 256;
        a.pb[0].terms = reinterpret_cast<uint16_t*>(at);
        a.pb[1].terms = reinterpret_cast<uint16_t*>(at + terms_bytes(a.T, a.r));
    }
    a.pb[0].part = part;
    a.pb[1].part = splits == 1 ? part : part + static_cast<size_t>(splits) * a.r * c0;
    a.t_per = ceil_div(ceil_div(a.T, splits), per) * per;
    const int want = splits;
    splits = static_cast<int>(ceil_div(a.T, a.t_per));  // none without a token
    if (want > 1 && splits == 1) a.t_per = a.T;
    timer_begin(QL_KERNEL_ACT8_GRAD, stream);
    const int rt = lora_grad_rp(a.r) / 16;
    if (a.r > 16) {
        const int64_t units = ceil_div(a.T, kRows) * rt;
        hipLaunchKernelGGL(act8_terms_kernel, dim3(static_cast<uint32_t>(ceil_div(units, 4)), c1 > 0 ? 2 : 1), dim3(256), 0,
                           stream, a, rt, units);
    }
    // Ranks to 64 and few columns: tiles half as wide, for workgroups on all CUs.
    const bool narrow = rt <= 4 && ceil_div(c0, kCols) + ceil_div(c1, kCols) <= 128;
    const int cols = narrow ? 32 : kCols;
    a.nblk0 = static_cast<int>(ceil_div(c0, cols));
    const dim3 grid(static_cast<uint32_t>(a.nblk0 + ceil_div(c1, cols)), static_cast<uint32_t>(splits));
    switch (rt) {
        case 1: narrow ? launch_grads<1, 2>(a, grid, stream) : launch_grads<1, 4>(a, grid, stream); break;
        case 2: narrow ? launch_grads<2, 2>(a, grid, stream) : launch_grads<2, 4>(a, grid, stream); break;
        case 3: narrow ? launch_grads<3, 2>(a, grid, stream) : launch_grads<3, 4>(a, grid, stream); break;
        case 4: narrow ? launch_grads<4, 2>(a, grid, stream) : launch_grads<4, 4>(a, grid, stream); break;
        case 5: launch_grads<5, 4>(a, grid, stream); break;
        case 6: launch_grads<6, 4>(a, grid, stream); break;
        case 7: launch_grads<7, 4>(a, grid, stream); break;
        default: launch_grads<8, 4>(a, grid, stream); break;
    }
    if (splits > 1)
        hipLaunchKernelGGL(act8_grads_final_kernel,
                           dim3(static_cast<uint32_t>(ceil_div(static_cast<int64_t>(a.r) * (c0 + c1), 256))),
                           dim3(256), 0, stream, a, splits);
    timer_end(QL_KERNEL_ACT8_GRAD, stream);
    return check_launch("adapter gradients from an 8-bit checkpoint");
}

}  // namespace qlnf4
