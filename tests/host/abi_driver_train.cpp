// Host-only exercise of the entry points for norms, linear epilogues and the
// losses on logits, for the sanitizer build: rejected arguments, and valid
// shapes with fake (aligned, never dereferenced on the host) device pointers,
// which run the validation, the host-side planning and the workspace carving
// and stop at their first launch (no GPU here). Prints "driver ok" and exits 0
// when every status is one of those expected.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <utility>

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
bool stop(int s) { return s == QL_OK || s == QL_ERR_HIP; }

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
}  // namespace

int main() {
    uint16_t* P = static_cast<uint16_t*>(fake(0x1000000));
    float* F = static_cast<float*>(fake(0x2000000));
    int64_t* I = static_cast<int64_t*>(fake(0x3000000));
    uint8_t* B8 = static_cast<uint8_t*>(fake(0x3800000));
    void* WS = fake(0x4000000);
    const size_t all = ~size_t{0};
    const int64_t big = int64_t{1} << 62;
    const int64_t sizes[] = {1, 2, 7, 77, 1001, 70000, (int64_t{1} << 22) - 1};

    // norms
    for (int64_t rows : sizes)
        for (int64_t cols : {8, 264, 4096, 8192, 16384})
            for (int xd : {QL_F32, QL_BF16})
                for (int wd : {QL_F32, QL_BF16}) {
                    EXPECT(stop(qlora_norm_fwd(P, xd, rows, cols, P, P, wd, 1e-5f, 0, P, F, F, nullptr)));
                    EXPECT(stop(qlora_norm_fwd(P, xd, rows, cols, P, nullptr, wd, 0.0f, 1, P, nullptr, nullptr, nullptr)));
                    EXPECT(qlora_norm_bwd_workspace(rows, cols) > 0);
                    EXPECT(stop(qlora_norm_bwd(P, xd, rows, cols, P, wd, P, F, F, P, F, F, 1, WS, all, nullptr)));
                    EXPECT(stop(qlora_norm_bwd(P, xd, rows, cols, P, wd, P, nullptr, F, P, nullptr, nullptr, 0, nullptr, 0, nullptr)));
                }
    EXPECT(stop(qlora_norm_bwd(nullptr, QL_F32, 0, 64, nullptr, QL_F32, nullptr, nullptr, nullptr, nullptr, F, F, 0, nullptr, 0, nullptr)));
    for (int64_t rows : {int64_t{-1}, int64_t{1} << 22, big, -big}) {
        EXPECT(qlora_norm_fwd(P, QL_F32, rows, 64, P, P, QL_F32, 0.0f, 0, P, F, F, nullptr) == QL_ERR_SHAPE);
        EXPECT(qlora_norm_bwd_workspace(rows, 64) == 0);
    }
    for (int64_t cols : {int64_t{0}, int64_t{-8}, int64_t{12}, int64_t{16392}, big, -big}) {
        EXPECT(qlora_norm_fwd(P, QL_F32, 4, cols, P, P, QL_F32, 0.0f, 0, P, F, F, nullptr) == QL_ERR_SHAPE);
        EXPECT(qlora_norm_bwd(P, QL_F32, 4, cols, P, QL_F32, P, F, F, P, F, F, 0, WS, all, nullptr) == QL_ERR_SHAPE);
    }
    EXPECT(qlora_norm_fwd(P, QL_F32, 4, 64, P, P, QL_F32, std::nanf(""), 0, P, F, F, nullptr) == QL_ERR_UNSUPPORTED);

    // epilogues
    ql_epilogue e{P, QL_ACT_GELU, P, F, QL_F32}, none{nullptr, QL_ACT_NONE, nullptr, nullptr, QL_BF16};
    for (int64_t T : {1, 16, 17, 300, 1024, 4096})
        for (int r : {0, 3, 8, 16, 64, QL_MAX_RANK})
            for (int dq : {0, 1}) {
                for (const auto& s : {std::pair<int64_t, int64_t>{4096, 4096}, {264, 192}, {11008, 4096}, {4096, 11008}}) {
                    ql_nf4_weight w = weight(s.first, s.second, dq);
                    for (const ql_epilogue* ep : {&e, &none}) {
                        const size_t need = qlora_linear_fwd_epilogue_workspace(s.first, s.second, T, r, 0);
                        EXPECT(stop(qlora_linear_fwd_epilogue(&w, P, T, P, P, r, 0.5f, nullptr, 0.0f, ep, P, F, WS, need, nullptr)));
                        EXPECT(need == 0 || qlora_linear_fwd_epilogue(&w, P, T, P, P, r, 0.5f, nullptr, 0.0f, ep, P, F, WS, need - 1,
                                                                      nullptr) == QL_ERR_WORKSPACE);
                        EXPECT(stop(qlora_linear_fwd_epilogue(&w, P, T, P, P, r, 0.5f, B8, 0.1f, ep, P, nullptr, WS,
                                                              qlora_linear_fwd_epilogue_workspace(s.first, s.second, T, r, 1), nullptr)));
                    }
                }
            }
    {
        ql_nf4_weight w = weight(264, 192, 1);
        EXPECT(qlora_linear_fwd_epilogue(&w, P, 4, P, P, 8, 1.0f, nullptr, 0.0f, nullptr, P, F, WS, all, nullptr) == QL_ERR_NULL);
        EXPECT(qlora_linear_fwd_epilogue_workspace(264, 192, 0, 8, 0) == 0);
        EXPECT(qlora_linear_fwd_epilogue_workspace(-1, 192, 4, 8, 0) == 0);
        ql_q4g_weight q{264, 200, 32, QL_BF16, B8, P, B8};
        ql_epilogue kept = none, act = none;
        kept.Z = F;
        act.act = 77;
        for (int64_t T : {0, 1, 8, 16, 64, 1000}) EXPECT(stop(q4g_linear_fwd_epilogue(&q, P, T, &none, P, nullptr)));
        EXPECT(q4g_linear_fwd_epilogue(&q, P, 4, &kept, P, nullptr) == QL_ERR_UNSUPPORTED);
        EXPECT(q4g_linear_fwd_epilogue(&q, P, 4, &act, P, nullptr) == QL_ERR_UNSUPPORTED);
        EXPECT(q4g_linear_fwd_epilogue(&q, P, big, &none, P, nullptr) == QL_ERR_SHAPE);
    }
    for (int64_t rows : {int64_t{1}, int64_t{1000}, int64_t{1} << 31})
        for (int64_t cols : {8, 24, 512, 11008})
            for (int act = QL_ACT_NONE; act <= QL_ACT_GELU_TANH; ++act) {
                if (rows > (int64_t{1} << 30) && cols > 512) continue;
                EXPECT(stop(qlora_epilogue_bwd(P, F, QL_F32, rows, cols, act, P, F, 0, WS, all, nullptr)));
                EXPECT(stop(qlora_epilogue_bwd(P, P, QL_BF16, rows, cols, act, P, nullptr, 0, nullptr, 0, nullptr)));
            }
    for (int64_t n : {int64_t{-1}, big, -big}) {
        EXPECT(qlora_epilogue_bwd(P, P, QL_BF16, n, 64, 1, P, F, 0, WS, all, nullptr) == QL_ERR_SHAPE);
        EXPECT(qlora_epilogue_bwd(P, P, QL_BF16, 4, n, 1, P, F, 0, WS, all, nullptr) == QL_ERR_SHAPE);
        EXPECT(qlora_epilogue_bwd_workspace(n, 64) == 0 && qlora_epilogue_bwd_workspace(4, n) == 0);
    }

    // losses on logits
    for (int64_t T : {int64_t{0}, int64_t{1}, int64_t{777}, int64_t{1} << 22})
        for (int64_t V : {int64_t{1}, int64_t{9}, int64_t{8192}, int64_t{50257}, int64_t{300000}, (int64_t{1} << 30) - 1})
            for (int dt : {QL_F32, QL_BF16}) {
                const bool fits = T == 0 || V <= (int64_t{1} << 35) / T;
                auto ok = [&](int s) { return fits ? stop(s) : s == QL_ERR_SHAPE; };
                EXPECT((qlora_token_logp_workspace(T, V, dt) > 0) == (fits && T > 0));
                EXPECT(ok(qlora_token_logp(P, dt, T, V, V + 3, I, F, WS, all, nullptr)));
                EXPECT(ok(qlora_preference_loss_fwd(P, dt, T, V, V, I, I, 3, F, 0.1f, 0.1f, QL_PREF_SIGMOID, 1, F, F, F, WS, all, nullptr)));
                EXPECT(ok(qlora_preference_loss_bwd(P, dt, T, V, V, I, F, F, 3, P, nullptr)));
                for (int64_t K : {1, 255, 256}) {
                    EXPECT(ok(qlora_distill_loss(P, dt, T, V, V, I, F, QL_F32, K, I, 2.0f, 0.5f, F, F, P, nullptr)));
                    EXPECT(ok(qlora_distill_loss(P, dt, T, V, V, I, P, QL_BF16, K, nullptr, 1.0f, 0.0f, nullptr, F, nullptr, nullptr)));
                }
            }
    for (int64_t n : {int64_t{-1}, big, -big}) {
        EXPECT(qlora_token_logp(P, QL_BF16, n, 64, 64, I, F, WS, all, nullptr) == QL_ERR_SHAPE);
        EXPECT(qlora_token_logp(P, QL_BF16, 4, n, 64, I, F, WS, all, nullptr) == QL_ERR_SHAPE);
        EXPECT(qlora_token_logp(P, QL_BF16, 4, 64, n, I, F, WS, all, nullptr) == QL_ERR_SHAPE);
        EXPECT(qlora_token_logp_workspace(n, 64, QL_BF16) == 0 && qlora_token_logp_workspace(4, n, QL_BF16) == 0);
        EXPECT(qlora_distill_loss(P, QL_BF16, 4, 64, 64, I, F, QL_F32, n, I, 1.0f, 0.0f, F, F, P, nullptr) == QL_ERR_SHAPE);
        EXPECT(qlora_preference_loss_fwd(P, QL_BF16, 4, 64, 64, I, I, n, F, 0.1f, 0.0f, 0, 0, F, F, F, WS, all, nullptr) == QL_ERR_SHAPE);
    }
    EXPECT(stop(qlora_preference_loss_fwd(P, QL_BF16, 4, 64, 64, I, I, 0, nullptr, 0.1f, 0.0f, 0, 0, nullptr, nullptr, F, WS, all, nullptr)));

    if (failures) {
        std::fprintf(stderr, "%d failures\n", failures);
        return 1;
    }
    std::printf("driver ok\n");
    return 0;
}
