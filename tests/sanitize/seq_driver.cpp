// Host-side checks of libmhla's sequence entry points (gated attention, query/key
// norm with rotation): validation, workspace arithmetic and refusals, built with
// AddressSanitizer and UndefinedBehaviorSanitizer on the host code
// (tests/test_seq_sanitized.py).  No GPU is used: every call here returns before any
// HIP call.
#include <mhla.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>

static int failures = 0;
#define CHECK(cond)                                                            \
    do {                                                                       \
        if (!(cond)) {                                                         \
            std::fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #cond); \
            ++failures;                                                        \
        }                                                                      \
    } while (0)

int main() {
    const uintptr_t BIG = (uintptr_t)1 << 42;   // fake, aligned, never dereferenced
    auto P = [&](int k) { return reinterpret_cast<void*>(BIG * (uintptr_t)k); };
    auto F = [&](int k) { return reinterpret_cast<float*>(P(k)); };
    auto I = [&](int k) { return reinterpret_cast<const int32_t*>(P(k)); };
    const int32_t top = INT32_MAX, low = INT32_MIN;
    const int32_t batches[] = {0, 1, 7, 65536, top, -1, low};
    const int32_t tokens[] = {0, 1, 64, 65, 1023, 1 << 20, 1 << 30, (1 << 30) + 1, top, low};
    const int32_t heads[] = {0, 1, 3, 12, 65536, 65537, top, -5};
    const int32_t dims[] = {32, 64, 128, 16, 0, low};
    const int64_t strides[] = {0, 1, 512, 8388608, 8388616, -16, INT64_MAX, INT64_MIN};
    long ok = 0;
    mhla_rope rope;
    std::memset(&rope, 0, sizeof(rope));
    rope.axes = 1;
    rope.section[0] = 8;
    rope.eps = 1e-6f;
    for (int32_t B : batches)
        for (int32_t T : tokens)
            for (int32_t H : heads)
                for (int32_t HK : heads)
                    for (int32_t d : dims)
                        for (int dt = 0; dt < 3; ++dt)
                            for (int64_t st : strides) {
                                mhla_seq s;
                                std::memset(&s, 0, sizeof(s));
                                s.batch = B; s.tokens = T; s.heads = H; s.kv_heads = HK; s.head_dim = d; s.dtype = dt;
                                s.q_stride = st; s.k_stride = st; s.scale = 0.5f;
                                const mhla_status c = mhla_check_seq(&s);
                                const size_t f = mhla_gated_workspace_bytes(&s), b = mhla_gated_backward_workspace_bytes(&s);
                                (void)mhla_qk_norm_rope_backward_workspace_bytes(&s);
                                if (c != MHLA_OK) {
                                    CHECK(f == 0 && b == 0);
                                    CHECK(mhla_gated_forward(P(1), P(2), P(3), F(4), nullptr, nullptr, &s, P(5), nullptr,
                                                             nullptr, 0, nullptr) == c);
                                    continue;
                                }
                                ++ok;
                                if (B == 0 || H == 0 || T == 0) continue;
                                // every span of a valid problem is formed; an output on an input is refused
                                CHECK(mhla_gated_forward(P(1), P(2), P(3), F(4), nullptr, F(6), &s, P(1), nullptr, P(7), ~(size_t)0,
                                                         nullptr) == MHLA_ERR_INVALID_ARG);
                                CHECK(mhla_gated_backward(P(1), P(2), P(3), F(4), nullptr, F(6), P(8), F(9), &s, P(10), P(11), P(12),
                                                          F(4), F(13), P(7), ~(size_t)0, nullptr) == MHLA_ERR_INVALID_ARG);
                                if (T == 1)
                                    CHECK(mhla_gated_step(P(1), P(2), P(3), F(4), I(5), &s, F(6), top, P(1), nullptr) ==
                                          MHLA_ERR_INVALID_ARG);
                            }
    CHECK(ok > 100);
    mhla_seq s;
    std::memset(&s, 0, sizeof(s));
    s.batch = 2; s.tokens = 100; s.heads = 4; s.kv_heads = 2; s.head_dim = 64; s.dtype = MHLA_BF16; s.scale = 1.f;
    const int32_t secs[] = {0, 1, 8, 16, 32, 40, -8, top, low};
    for (int32_t a : secs)
        for (int32_t b : secs)
            for (int32_t c : secs)
                for (int32_t ax = -1; ax < 5; ++ax)
                    for (int32_t style = -1; style < 4; ++style) {
                        rope.style = style; rope.axes = ax;
                        rope.section[0] = a; rope.section[1] = b; rope.section[2] = c;
                        // the output lies on the positions: refused for one reason or the other
                        CHECK(mhla_qk_norm_rope(P(1), P(2), F(3), F(4), I(5), F(6), &rope, &s, P(5), P(7), nullptr) ==
                              MHLA_ERR_INVALID_ARG);
                    }
    s.scale = NAN;
    CHECK(mhla_check_seq(&s) == MHLA_ERR_INVALID_ARG);
    if (failures) return 1;
    std::printf("OK %ld valid problems\n", ok);
    return 0;
}
