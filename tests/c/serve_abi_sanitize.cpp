// Host ABI of the operators of a serving step under sanitizers, with stub
// launchers: random calls whose accepted sizes keep the launches' index
// arithmetic in range. No HIP runtime call is made.
#include <cstdint>
#include <cstdio>

#include "../../weight_only_bit_block_amd/csrc/wq_internal.h"

static int launches = 0, failures = 0;

namespace wq {
uint64_t prompt_ws_bytes(int64_t T, int64_t B, int64_t, int64_t kv, int64_t d) { return (uint64_t)(T / 32 + B) * kv * d * 256; }
uint64_t decode_window_ws_bytes(int64_t B, int64_t, int64_t, int64_t, int64_t pages, int64_t window, int64_t) { return B <= 512 && pages > 16 && window > 1000 ? 4096 : 0; }
uint64_t shared_ws_bytes(int64_t B, int64_t heads, int64_t, int64_t d, int64_t, int64_t) { return (uint64_t)B * heads * d; }
hipError_t launch_attn_prefill(const PromptArgs &a, hipStream_t)
{
    ++launches;
    if ((a.T / 32 + a.B) * (int64_t)a.heads >= (1 << 24) || a.heads % a.kv_heads || a.window < 1 || a.window > a.T || a.sinks < 0 || a.sinks > a.T) ++failures;
    return hipSuccess;
}
hipError_t launch_kv_append(const AppendArgs &a, hipStream_t)
{
    ++launches;
    if (a.T * a.cache.kv_heads >= (1 << 27) || a.cache.n_pages == 0 || !a.slots) ++failures;
    return hipSuccess;
}
hipError_t launch_attn_decode(const DecodeArgs &a, hipStream_t)
{
    ++launches;
    if ((int64_t)a.B * a.heads >= (1 << 24) || a.heads % a.cache.kv_heads || a.window < 0 || a.window > a.max_pages * 64 || a.sinks > a.max_pages * 64) ++failures;
    return hipErrorUnknown;
}
hipError_t launch_attn_decode_shared(const SharedArgs &a, hipStream_t)
{
    ++launches;
    if ((int64_t)a.own.B * a.own.heads >= (1 << 24) || a.own.heads % a.own.cache.kv_heads || a.prefix_pages >= (1 << 25)) ++failures;
    return hipSuccess;
}
hipError_t launch_qk_norm_rope(const RopeArgs &a, bool, bool, hipStream_t)
{
    ++launches;
    if (a.T <= 0 || a.T >= (1 << 24) || a.pairs * 2 > a.head_dim || a.heads + a.kv_heads < 1) ++failures;
    return hipSuccess;
}
hipError_t launch_kv_plan(const PlanArgs &a, hipStream_t)
{
    ++launches;
    if (a.B >= (1 << 24) || a.max_pages >= (1 << 25) || a.T >= (1 << 30)) ++failures;
    return hipSuccess;
}
}  // namespace wq

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
static int64_t pick(int64_t usual) { return rnd() % 4 ? usual : size(); }

int main()
{
    float *const F = reinterpret_cast<float *>(0x10000);
    int32_t *I = reinterpret_cast<int32_t *>(F);
    int64_t *L = reinterpret_cast<int64_t *>(F);
    for (int i = 0; i < 400000; ++i) {
        const int64_t d = rnd() % 8 ? (rnd() % 2 ? 64 : 128) : size(), kv = pick(2), h = pick(8), B = pick(3), W = pick(40), T = pick(500);
        const int64_t window = pick(100), sinks = pick(4), st = pick(4096);
        wq_kv_cache c = {F, reinterpret_cast<uint16_t *>(F), F, reinterpret_cast<uint16_t *>(F), pick(10), (int32_t)kv, (int32_t)d};
        const uint64_t ws = 1ull << 62;
        wq_attn_prefill_window(F, st, F, st, F, st, T, I, B, h, kv, d, 1.0f, window, sinks, F, st, F, ws, nullptr);
        wq_attn_decode_window_ws(B, h, kv, d, W, window, sinks);
        wq_attn_decode_window(&c, F, st, h, I, B, I, W, 1.0f, window, sinks, F, st, F, ws, nullptr);
        wq_attn_decode_shared_ws(B, h, kv, d, W, window);
        wq_attn_decode_shared(&c, F, st, h, I, window, I, I, B, I, W, 1.0f, F, st, F, ws, nullptr);
        wq_kv_append_slots(&c, F, st, F, st, T, L, nullptr);
        wq_qk_norm_rope(F, st, h, F, st, kv, d, T, I, F, pick(32), 0, 1.0f, 1, F, F, 1e-6f, F, st, F, st, nullptr);
        wq_kv_plan(I, I, B, I, W, I, pick(9), I, T, I, I, I, L, I + 64, nullptr);
        // (memory of their own, 2^52 bytes apart, which no size reaches)
        const auto far = [](int n) { return (uintptr_t)0x10000 + ((uintptr_t)n << 52); };
        const auto ints = [&](int n) { return reinterpret_cast<int32_t *>(far(n)); };
        wq_kv_plan(ints(1), ints(2), B, ints(3), W, ints(4), pick(9), ints(5), T, ints(6), ints(7), ints(8), reinterpret_cast<int64_t *>(far(9)), ints(10), nullptr);
    }
    if (launches < 100000) {
        std::fprintf(stderr, "only %d launches\n", launches);
        ++failures;
    }
    if (failures) {
        std::fprintf(stderr, "%d failures\n", failures);
        return 1;
    }
    std::puts("all checks passed");
    return 0;
}
