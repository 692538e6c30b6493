// Host-only exercise of the entry points for 8-bit activation checkpoints and
// 4-bit weights with group scales, for the sanitizer build: rejected
// arguments, and valid shapes with fake (aligned, never dereferenced on the
// host) device pointers, which run the validation, the host-side planning and
// the workspace carving and stop at their first launch (no GPU here). Prints
// "driver ok" and exits 0 when every status is one of those expected.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "qlora_nf4.h"

namespace {
int failures = 0;

void expect(bool ok, const char* what, int line) {
    if (!ok) {
        std::fprintf(stderr, "line %d: %s (last error: %s)\n", line, what, qlora_last_error());
        ++failures;
    }
}
#define EXPECT(c) expect((c), #c, __LINE__)

void* fake(uintptr_t v) { return reinterpret_cast<void*>(v); }

ql_nf4_weight weight(int64_t rows, int64_t cols, int dq) {
    ql_nf4_weight w{};
    w.rows = rows;
    w.cols = cols;
    w.blocksize = 64;
    w.dq_blocksize = dq ? 256 : 0;
    w.packed = static_cast<const uint8_t*>(fake(0x100000));
    w.absmax = static_cast<const float*>(fake(0x200000));
    w.c8 = static_cast<const uint8_t*>(fake(0x300000));
    w.dq_scale = static_cast<const float*>(fake(0x400000));
    w.dq_mean = static_cast<const float*>(fake(0x500000));
    return w;
}

bool stop(int s) { return s == QL_OK || s == QL_ERR_HIP; }
}  // namespace

int main() {
    uint16_t* P = static_cast<uint16_t*>(fake(0x1000000));
    float* F = static_cast<float*>(fake(0x2000000));
    uint8_t* B8 = static_cast<uint8_t*>(fake(0x3000000));
    void* WS = fake(0x4000000);
    uint8_t* MIS = static_cast<uint8_t*>(fake(0x4000004));
    const int64_t big = int64_t{1} << 62;

    // checkpoints
    auto act = [&](int64_t rows, int64_t cols) { return ql_act8{rows, cols, B8, B8}; };
    for (int64_t rows : {int64_t{0}, int64_t{1}, int64_t{77}, int64_t{65536}})
        for (int64_t cols : {32, 64, 11008}) {
            ql_act8 a = act(rows, cols);
            EXPECT(stop(act8_quantize(P, &a, nullptr)));
            EXPECT(stop(act8_dequantize(&a, F, QL_F32, nullptr)));
            EXPECT(stop(act8_dequantize(&a, P, QL_BF16, nullptr)));
            EXPECT(stop(qlora_swiglu_fwd(P, P, rows, cols, P, &a, &a, &a, nullptr)));
            EXPECT(stop(qlora_swiglu_fwd(P, P, rows, cols, P, nullptr, nullptr, nullptr, nullptr)));
            EXPECT(stop(qlora_swiglu_bwd(&a, &a, P, P, P, nullptr)));
        }
    for (int64_t rows : {int64_t{-1}, big, -big})
        for (int64_t cols : {int64_t{32}, int64_t{0}, int64_t{33}, int64_t{-32}, big}) {
            ql_act8 a = act(rows, cols);
            EXPECT(act8_quantize(P, &a, nullptr) == QL_ERR_SHAPE);
            EXPECT(act8_dequantize(&a, F, QL_F32, nullptr) == QL_ERR_SHAPE);
            EXPECT(qlora_swiglu_fwd(P, P, rows, cols, P, nullptr, nullptr, nullptr, nullptr) == QL_ERR_SHAPE);
            EXPECT(qlora_swiglu_bwd(&a, &a, P, P, P, nullptr) == QL_ERR_SHAPE);
        }
    {
        ql_act8 a = act(8, 64), other = act(8, 32), none = act(8, 64), off = act(8, 64);
        none.scale = nullptr;
        off.codes = MIS;
        EXPECT(act8_quantize(P, nullptr, nullptr) == QL_ERR_NULL);
        EXPECT(act8_quantize(nullptr, &a, nullptr) == QL_ERR_NULL);
        EXPECT(act8_quantize(P, &none, nullptr) == QL_ERR_NULL);
        EXPECT(act8_quantize(P, &off, nullptr) == QL_ERR_ALIGN);
        EXPECT(act8_dequantize(&a, P, 7, nullptr) == QL_ERR_UNSUPPORTED);
        EXPECT(qlora_swiglu_fwd(P, P, 8, 64, P, &other, nullptr, nullptr, nullptr) == QL_ERR_SHAPE);
        EXPECT(qlora_swiglu_fwd(P, nullptr, 8, 64, P, &a, &a, nullptr, nullptr) == QL_ERR_NULL);
        EXPECT(qlora_swiglu_bwd(&a, &other, P, P, P, nullptr) == QL_ERR_SHAPE);
        EXPECT(qlora_swiglu_bwd(&a, nullptr, P, P, P, nullptr) == QL_ERR_NULL);
        EXPECT(qlora_swiglu_bwd(&a, &a, P, P, nullptr, nullptr) == QL_ERR_NULL);
    }

    // the layer's backward: each output alone and all, with the workspace it
    // asks for, with one byte less, without any
    for (int dq : {0, 1})
        for (int64_t N : {8, 72, 4096})
            for (int64_t K : {64, 4096, 11008})
                for (int64_t T : {1, 5, 64, 1000, 4096, 16384})
                    for (int32_t r : {0, 1, 16, 40, 128})
                        for (int want = 0; want < 8; ++want)
                            for (int drop : {0, 1}) {
                                if (r == 0 && (want & 6)) continue;
                                ql_nf4_weight w = weight(N, K, dq);
                                ql_act8 x = act(T, K);
                                const size_t need = qlora_linear_bwd_act8_workspace(N, K, T, r, drop);
                                auto run = [&](void* ws, size_t bytes) {
                                    return qlora_linear_bwd_act8(&w, &x, P, T, P, P, r, 0.5f, drop ? B8 : nullptr,
                                                                 drop ? 0.25f : 0.0f, F, want & 1 ? P : nullptr,
                                                                 want & 2 ? F : nullptr, want & 4 ? F : nullptr, 0, ws,
                                                                 bytes, nullptr);
                                };
                                EXPECT(stop(run(WS, need)));
                                if (want == 7 && need > 0) {
                                    EXPECT(run(WS, need - 1) == QL_ERR_WORKSPACE);
                                    EXPECT(run(nullptr, need) == QL_ERR_WORKSPACE);
                                    EXPECT(run(MIS, need) == QL_ERR_ALIGN);
                                }
                            }
    {
        ql_nf4_weight w = weight(72, 128, 1);
        ql_act8 x = act(40, 128), few = act(39, 128);
        auto run = [&](const ql_act8* x8, int32_t r, float p, const uint8_t* keep, const float* U, int acc, int64_t T) {
            return qlora_linear_bwd_act8(&w, x8, P, T, P, P, r, 1.0f, keep, p, U, P, F, F, acc, WS, size_t{1} << 40, nullptr);
        };
        EXPECT(run(&few, 8, 0.0f, nullptr, F, 0, 40) == QL_ERR_SHAPE);
        EXPECT(run(nullptr, 8, 0.0f, nullptr, F, 0, 40) == QL_ERR_NULL);
        EXPECT(run(&x, 8, 0.0f, nullptr, nullptr, 0, 40) == QL_ERR_NULL);
        EXPECT(run(&x, 0, 0.0f, nullptr, F, 0, 40) == QL_ERR_SHAPE);
        EXPECT(run(&x, QL_MAX_RANK + 1, 0.0f, nullptr, F, 0, 40) != QL_OK);
        EXPECT(run(&x, -1, 0.0f, nullptr, F, 0, 40) != QL_OK);
        EXPECT(run(&x, 8, 0.5f, nullptr, F, 0, 40) == QL_ERR_UNSUPPORTED);
        EXPECT(run(&x, 8, 1.0f, B8, F, 0, 40) != QL_OK);
        EXPECT(run(&x, 8, 0.0f, nullptr, F, 2, 40) == QL_ERR_UNSUPPORTED);
        EXPECT(run(&x, 8, 0.0f, nullptr, F, 0, -1) != QL_OK);
        EXPECT(qlora_linear_bwd_act8_workspace(-1, 64, 1, 8, 0) == 0);
        EXPECT(qlora_linear_bwd_act8_workspace(64, 64, 1, QL_MAX_RANK + 1, 0) == 0);
    }

    // layers that share their input
    for (int32_t nw = 0; nw <= 5; ++nw)
        for (int64_t T : {1, 70, 2048})
            for (int32_t r : {0, 4, 128}) {
                std::vector<ql_nf4_weight> ws;
                std::vector<int64_t> rows;
                for (int i = 0; i < nw; ++i) {
                    rows.push_back(i == 0 ? 4096 : 1024 * i);
                    ws.push_back(weight(rows.back(), 4096, 1));
                }
                std::vector<const ql_nf4_weight*> wp;
                for (auto& w : ws) wp.push_back(&w);
                std::vector<const uint16_t*> in(nw, P);
                std::vector<const float*> U(nw, F);
                std::vector<float*> g(nw, F);
                ql_act8 x = act(T, 4096);
                const size_t need = qlora_linear_bwd_group_act8_workspace(rows.data(), nw, 4096, T, r);
                auto run = [&](size_t bytes) {
                    return qlora_linear_bwd_group_act8(wp.data(), nw, &x, in.data(), T, in.data(), in.data(), r, 0.5f,
                                                       r ? U.data() : nullptr, P, r ? g.data() : nullptr,
                                                       r ? g.data() : nullptr, 1, WS, bytes, nullptr);
                };
                if (nw < 1 || nw > 4) {
                    EXPECT(need == 0 && run(size_t{1} << 40) == QL_ERR_SHAPE);
                } else {
                    EXPECT(stop(run(need)));
                    if (need > 0) EXPECT(run(need - 1) == QL_ERR_WORKSPACE);
                    if (r > 0) {  // one layer's gradients only
                        for (int i = 1; i < nw; ++i) g[i] = nullptr;
                        EXPECT(stop(run(need)));
                    }
                }
            }
    EXPECT(qlora_linear_bwd_group_act8_workspace(nullptr, 2, 64, 1, 8) == 0);

    // 4-bit weights with group scales
    auto q4 = [&](int64_t rows, int64_t cols, int group, int sd) {
        ql_q4g_weight w{};
        w.rows = rows;
        w.cols = cols;
        w.group = group;
        w.scale_dtype = sd;
        w.packed = B8;
        w.scale = F;
        w.zero = B8;
        return w;
    };
    for (int group : {32, 64, 128})
        for (int sd : {QL_F32, QL_BF16})
            for (int64_t rows : {1, 17, 8200, 22016})
                for (int64_t cols : {int64_t{8}, int64_t{1000}, int64_t{8192}, int64_t{34000}, int64_t{1} << 18}) {
                    ql_q4g_weight w = q4(rows, cols, group, sd);
                    if (rows == 1) w.zero = nullptr;
                    EXPECT(q4g_packed_bytes(rows, cols) == static_cast<size_t>(rows) * ((cols + 31) / 32) * 16);
                    EXPECT(q4g_num_groups(rows, cols, group) == rows * ((cols + group - 1) / group));
                    EXPECT(stop(q4g_quantize(F, QL_F32, rows, cols, group, B8, F, sd, B8, nullptr)));
                    EXPECT(stop(q4g_quantize(P, QL_BF16, rows, cols, group, B8, F, sd, nullptr, nullptr)));
                    EXPECT(stop(q4g_dequantize(&w, P, QL_BF16, nullptr)));
                    EXPECT(stop(q4g_dequantize(&w, F, QL_F32, nullptr)));
                    for (int64_t T : {0, 1, 4, 5, 8, 9, 16, 17, 33, 49, 64, 65, 1000})
                        EXPECT(stop(q4g_linear_fwd(&w, P, T, P, nullptr)));
                }
    for (int64_t rows : {int64_t{0}, int64_t{-5}, big}) {
        ql_q4g_weight w = q4(rows, 64, 32, QL_F32);
        EXPECT(q4g_packed_bytes(rows, 64) == 0 && q4g_num_groups(rows, 64, 32) == 0);
        EXPECT(q4g_quantize(F, QL_F32, rows, 64, 32, B8, F, QL_F32, B8, nullptr) == QL_ERR_SHAPE);
        EXPECT(q4g_dequantize(&w, F, QL_F32, nullptr) == QL_ERR_SHAPE);
        EXPECT(q4g_linear_fwd(&w, P, 1, P, nullptr) == QL_ERR_SHAPE);
    }
    for (int64_t cols : {int64_t{0}, int64_t{-8}, int64_t{12}, (int64_t{1} << 24) + 8, big})
        EXPECT(q4g_quantize(F, QL_F32, 4, cols, 32, B8, F, QL_F32, B8, nullptr) == QL_ERR_SHAPE);
    {
        ql_q4g_weight w = q4(16, 64, 48, QL_F32), f16 = q4(16, 64, 32, 9), off = q4(16, 64, 32, QL_BF16), ok = off;
        off.scale = MIS;
        EXPECT(q4g_linear_fwd(&w, P, 1, P, nullptr) == QL_ERR_UNSUPPORTED);
        EXPECT(q4g_linear_fwd(&f16, P, 1, P, nullptr) == QL_ERR_UNSUPPORTED);
        EXPECT(q4g_linear_fwd(&off, P, 1, P, nullptr) == QL_ERR_ALIGN);
        EXPECT(q4g_linear_fwd(nullptr, P, 1, P, nullptr) == QL_ERR_NULL);
        EXPECT(q4g_linear_fwd(&ok, nullptr, 1, P, nullptr) == QL_ERR_NULL);
        EXPECT(q4g_linear_fwd(&ok, P, -1, P, nullptr) == QL_ERR_SHAPE);
        EXPECT(q4g_linear_fwd(&ok, P, big, P, nullptr) == QL_ERR_SHAPE);
        EXPECT(q4g_dequantize(&ok, P, 5, nullptr) == QL_ERR_UNSUPPORTED);
        EXPECT(q4g_quantize(P, 3, 16, 64, 32, B8, F, QL_F32, B8, nullptr) == QL_ERR_UNSUPPORTED);
    }
    for (int k = QL_KERNEL_GEMM_FWD; k < QL_KERNEL_COUNT; ++k) EXPECT(qlora_timer_disarm(k) == QL_OK);

    if (failures) {
        std::fprintf(stderr, "%d failures\n", failures);
        return 1;
    }
    std::printf("driver ok\n");
    return 0;
}
