// Host ABI of the operators between the projections under sanitizers, with stub
// launchers: every refusal, and random calls whose accepted sizes keep the
// launches' index arithmetic in range. No HIP runtime call is made.
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "../../weight_only_bit_block_amd/csrc/wq_internal.h"

static int launches = 0, failures = 0;

namespace wq {
uint64_t prompt_ws_bytes(int64_t T, int64_t B, int64_t, int64_t kv, int64_t d) { return (uint64_t)(T / 32 + B) * kv * d * 256; }
uint64_t decode_ws_bytes(int64_t B, int64_t, int64_t, int64_t, int64_t pages) { return B <= 512 && pages > 16 ? 4096 : 0; }
hipError_t launch_attn_prefill(const PromptArgs &a, hipStream_t)
{
    ++launches;
    if ((a.T / 32 + a.B) * (int64_t)a.heads >= (1 << 24) || a.heads % a.kv_heads) ++failures;
    return hipSuccess;
}
hipError_t launch_kv_append(const AppendArgs &a, hipStream_t)
{
    ++launches;
    if (a.T * a.cache.kv_heads >= (1 << 27) || a.max_pages == 0 || a.cache.n_pages == 0) ++failures;
    return hipSuccess;
}
hipError_t launch_attn_decode(const DecodeArgs &a, hipStream_t)
{
    ++launches;
    if ((int64_t)a.B * a.heads >= (1 << 24) || a.heads % a.cache.kv_heads) ++failures;
    return hipErrorUnknown;
}
hipError_t launch_residual_norm(const NormArgs &a, hipStream_t)
{
    ++launches;
    if (a.M <= 0 || a.N <= 0) ++failures;
    return hipSuccess;
}
}  // namespace wq

#define EXPECT(c)                                                       \
    do {                                                                \
        if (!(c)) {                                                     \
            std::fprintf(stderr, "%s:%d: %s\n", __FILE__, __LINE__, #c); \
            ++failures;                                                 \
        }                                                               \
    } while (0)

static uint64_t state = 88172645463325252ull;
static uint64_t rnd()
{
    state ^= state << 13;
    state ^= state >> 7;
    state ^= state << 17;
    return state;
}
// Sizes around every limit: small, powers of two and their neighbours, negative.
static int64_t size()
{
    switch (rnd() % 4) {
    case 0: return (int64_t)(rnd() % 70) - 3;
    case 1: return ((int64_t)1 << (rnd() % 63)) + (int64_t)(rnd() % 3) - 1;
    case 2: return 64 * (int64_t)(1 + rnd() % 40);
    default: return (int64_t)rnd();
    }
}

int main()
{
    float *const F = reinterpret_cast<float *>(0x10000);
    float *const MIS = reinterpret_cast<float *>(0x10004);
    const int32_t *I = reinterpret_cast<const int32_t *>(F);
    wq_kv_cache c = {F, reinterpret_cast<uint16_t *>(F), F, reinterpret_cast<uint16_t *>(F), 10, 8, 128};

    EXPECT(wq_attn_prefill(F, 2048, F, 1024, F, 1024, 8, I, 2, 16, 8, 128, 1.0f, F, 2048, F, 1u << 30, nullptr) == WQ_OK);
    EXPECT(wq_attn_prefill(MIS, 2048, F, 1024, F, 1024, 8, I, 2, 16, 8, 128, 1.0f, F, 2048, F, 1u << 30, nullptr) == WQ_ERR_ALIGN);
    EXPECT(wq_attn_prefill(F, 2048, F, 1024, F, 1024, 8, I, 2, 16, 8, 128, 1.0f, F, 2048, F, 5, nullptr) == WQ_ERR_SHAPE);
    EXPECT(wq_kv_append(&c, F, 1024, F, 1024, 8, I, nullptr, 2, I, 4, nullptr) == WQ_OK);
    EXPECT(wq_attn_decode(&c, F, 2048, 16, I, 2, I, 4, 1.0f, F, 2048, nullptr, 0, nullptr) == WQ_ERR_HIP);   // the launch's error
    EXPECT(wq_residual_norm(F, nullptr, nullptr, nullptr, 0, 1.0f, nullptr, 0.0f, 3, 5, nullptr, F, nullptr) == WQ_OK);
    EXPECT(launches == 4);

    for (int i = 0; i < 300000; ++i) {
        const int64_t T = size(), B = size(), H = size(), K = size(), D = rnd() % 3 ? (rnd() % 2 ? 64 : 128) : size(), W = size(),
                      s1 = size(), s2 = size();
        (void)wq_attn_prefill_ws(T, B, H, K, D);
        (void)wq_attn_decode_ws(B, H, K, D, W);
        (void)wq_attn_prefill(F, s1, F, s2, F, s2, T, I, B, H, K, D, 1.0f, F, s1, F, ~0ull, nullptr);
        c.n_pages = size();
        c.kv_heads = (int32_t)K;
        c.head_dim = (int32_t)D;
        (void)wq_kv_append(&c, F, s1, F, s2, T, I, I, B, I, W, nullptr);
        (void)wq_attn_decode(&c, F, s1, H, I, B, I, W, 1.0f, F, s2, F, ~0ull, nullptr);
        (void)wq_residual_norm(F, F, F, F, s1, 1.0f, F, 0.0f, T, B, F, F, nullptr);
    }
    if (failures) {
        std::fprintf(stderr, "%d expectations failed\n", failures);
        return 1;
    }
    std::printf("layer abi sanitize run: all checks passed, %d launches\n", launches);
    return 0;
}
