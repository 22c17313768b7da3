// wq_shared.hip -- attention of single tokens whose sequences share a prefix in
// the int4 cache: the prefix is read once for all of them.
//
//   out[b, j] = sum_u p_u v_u,  softmax over the prefix's tokens and b's own
//
// One launch takes the sequences' own tokens (decode_job, wq_kv_decode.h) and runs
// of the prefix's pages, a second one joins the parts. Own tokens and prefix apart
// cost a launch more and wait for one another's last workgroups (5 requests
// behind 777 tokens 22.5 us apart, 15.4 together; 64 behind 32768 85 and 76).
//
// For one key/value head the prefix meets R = B * group query rows, so that its
// scores are a matrix product of R x L x D. Few rows (kFewRows) run as one sequence
// of the attention of single tokens with 8 heads a workgroup, near HBM's rate.
// More, on prefix_job:
//   A workgroup takes 64 or 128 rows and a run of pages. A page's 64 keys are two
// tiles of 32, one for each of the two wavefronts that share 32 rows and meet at the
// end in LDS. All threads turn the page's codes into operands in LDS, once for all rows:
//   k   the codes themselves, exact in binary16. q is split in two parts (22
//       bits) after a power of two, so a block's sum is two products; it is scaled
//       in fp32, one multiplication a key and block: exact for every scale.
//   v   code times scale (15 bits) in two binary16 parts that hold it exactly:
//       hi = c s rounded, lo = fma(c, s, -hi), packed instructions. The scales are
//       brought below 2^kScaleTop by the power of two of the largest seen, v_exp.
// Scores come out transposed, S' = K Q' (a lane holds one query and 16 of the 32
// keys), so the softmax runs within a lane but for one exchange between the
// halves, and the weights, split in two parts, are already the second operand of
// O' = V' P', three products. v lies in LDS by rows; ds_read_b64_tr_b16 turns it.
//
// Bound: the rate of binary16 products and the vector instructions beside them. 64
// sequences of 16/8 heads of 128: 1.3 us for 1024 tokens of prefix, 1030 TFLOP/s of
// products where a large library product reaches 1153; a wavefront's instructions
// for a tile are 40 products and 350 others, which two wavefronts on a SIMD hide
// from one another by half (without the scaling 1.03, without making operands 1.04).
// k in two parts with a factor per key instead of scaled sums is 8 products more
// and 48 other instructions fewer: 81 us instead of 77 for 32768 tokens. Beside that
// stand 35 us that do not grow with the prefix: own tokens 10, first pages 8, parts
// written and joined 12, launches.
#include "wq_internal.h"
#include "wq_device.h"
#include "wq_kv_decode.h"

#include <type_traits>

namespace wq {
namespace {

typedef float f2 __attribute__((ext_vector_type(2)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

constexpr int kKeys = 32;                    // of a wavefront's tile; a page has two
constexpr float kBig = 3.4028235e38f;
constexpr int kScaleTop = 12;                // |code| <= 8: values stay below 2^15

__device__ __forceinline__ f16v mfma(h8 a, h8 b, f16v c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32); }

// Place of 16 bytes (8 values, `piece` of the row's D / 8) of a key's v in LDS, in
// bytes: written by 16 keys at once and read by 4 keys and 4 pieces, on different banks.
template <int D>
__device__ __forceinline__ int v_at(int key, int piece)
{
    if constexpr (D == 128) return key * 256 + (piece ^ ((key & 3) * 4 + (key >> 2 & 3))) * 16;
    return key * 128 + (piece ^ ((key >> 1 & 1) * 4 + (key >> 2 & 3))) * 16;
}

// RW x 32 rows, two wavefronts for 32 of them. Two buffers of operands where a compute
// unit holds one workgroup (128 rows), one where it holds two (heads of 64: three), which take turns.
constexpr int operand_bytes(int D) { return 3 * kTile * D * 2 + D / 32 * kTile * 2; }
constexpr int at_least(int a, int b) { return a > b ? a : b; }
constexpr int prefix_lds_bytes(int D, int RW) { return at_least((RW == 4 ? 2 : 1) * operand_bytes(D), 32 * RW * (D + kPartialExtra) * 4); }

template <int D, int RW>
__device__ __forceinline__ void prefix_job(const SharedArgs &a, float *parts, int chunks, float c_man, int c_exp, uint8_t *lds, unsigned job)
{
    constexpr int NB = D / 32, F = D / 16, W = 2 * RW;
    constexpr bool kTwo = RW == 4;
    constexpr int kMine = F / W;                                          // pieces of 16 values of a key's k and v, of a thread
    static_assert(F % W == 0, "pieces");
    constexpr int kRowBytes = D * 2, kPitch = D + kPartialExtra, kOperands = operand_bytes(D);
    typedef _Float16 hb __attribute__((ext_vector_type(NB)));
    const DecodeArgs &own = a.own;
    const int kv = own.cache.kv_heads, group = own.heads / kv;
    const int64_t rows = (int64_t)own.B * group;
    // key/value heads next to each other: ids go round the 8 XCDs
    const int kh = job % kv, run = job / kv % chunks;
    const int64_t block = job / kv / chunks;
    const PrefixRuns runs = prefix_runs(a.prefix_len, a.prefix_pages, chunks, 1);
    if (run >= runs.count) return;
    const int page0 = run * runs.per, page_end = page0 + runs.per < runs.pages ? page0 + runs.per : runs.pages;
    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), rw = wave % RW, kw = wave / RW;
    const int64_t row = (block * RW + rw) * 32 + (lane & 31);
    const bool live = row < rows, any = (block * RW + rw) * 32 < rows;

    // ---- pages come into registers one ahead: codes of this thread's pieces, scales of the lane's key
    u2 kc[kMine], vc[kMine];
    hb ks, vs;
    bool bad = false;
    if (own.cache.n_pages <= 0) {            // no page to read at all
        if (live && kw == 0 && half == 0) {
            float *dst = prefix_part(parts, run, kv, kh, rows, row, D);
            for (int i = 0; i < D; ++i) dst[i] = 0.0f;
            dst[D] = -3.0e38f;
            dst[D + 1] = __builtin_nanf("");
        }
        return;
    }
    int ids = page0 + lane < page_end ? a.prefix[page0 + lane] : 0;       // numbers of the run's next 64 pages
    // (past the run's end: its last page again. No branch around the loads: it would wait for them)
    const auto fetch = [&](int next) __attribute__((always_inline)) {
        const int page = next < page_end ? next : page_end - 1;
        if (next < page_end && page != page0 && (page - page0) % 64 == 0) ids = page + lane < page_end ? a.prefix[page + lane] : 0;
        int id = __builtin_amdgcn_readlane(ids, (page - page0) & 63);
        const bool out = id < 0 || id >= own.cache.n_pages;
        bad |= out;
        id = out ? 0 : id;
        const int64_t at = ((int64_t)id * kv + kh) * kTile;
        const uint8_t *kq = reinterpret_cast<const uint8_t *>(own.cache.kq) + at * (D / 2), *vq = reinterpret_cast<const uint8_t *>(own.cache.vq) + at * (D / 2);
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int o = lane * (D / 2) + (wave + W * i) % F * 8;
            kc[i] = *reinterpret_cast<const u2 *>(kq + o);
            vc[i] = *reinterpret_cast<const u2 *>(vq + o);
        }
        ks = *reinterpret_cast<const hb *>(own.cache.ks + (at + lane) * NB);
        vs = *reinterpret_cast<const hb *>(own.cache.vs + (at + lane) * NB);
    };
    int v_exp = kMinScaleExp;
    uint32_t v_limit = kRankZero + 2;        // rank of 2^v_exp
    // The page in the registers becomes operands. Returns the power of two that the output's units change by.
    const auto put = [&](int page) __attribute__((always_inline)) -> int {
        uint8_t *const kb = lds + (kTwo ? page & 1 : 0) * kOperands, *const vb = kb + kTile * kRowBytes;      // v: high parts, low parts
        _Float16 *const ksb = reinterpret_cast<_Float16 *>(kb + 3 * kTile * kRowBytes);                       // k's scales, [block][key]
        // magnitudes of the lane's scales of v in their order, what is not finite below zero
        if ((int64_t)page * kTile + lane >= runs.len) vs = hb{};
        typedef uint16_t ub __attribute__((ext_vector_type(NB)));
        const ub rank = scale_rank(__builtin_bit_cast(ub, vs));
        uint16_t top = rank[0];
        int by = 0;
#pragma unroll
        for (int i = 1; i < NB; ++i) top = top > rank[i] ? top : rank[i];
        if (__any(top > v_limit)) {          // (the same in every wavefront)
            float vmax = top > kRankZero ? (float)__builtin_bit_cast(_Float16, (uint16_t)((top - kRankZero) >> 1)) : 0.0f;
#pragma unroll
            for (int s = 1; s < 64; s <<= 1) vmax = fmaxf(vmax, __shfl_xor(vmax, s));
            const int e = vmax > ldexpf(1.0f, v_exp) ? __builtin_amdgcn_frexp_expf(vmax) : v_exp;
            by = __builtin_amdgcn_readfirstlane(v_exp - e);
            v_exp = e;
            v_limit = kRankZero + 2 * (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)ldexpf(1.0f, e));
        }
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int piece = (wave + W * i) % F, b = piece >> 1;                         // 16 values, half a block
            _Float16 s = ks[0], s1 = vs[0];
#pragma unroll
            for (int n = 1; n < NB; ++n) {
                s = b == n ? ks[n] : s;
                s1 = b == n ? vs[n] : s1;
            }
            if ((piece & 1) == 0) ksb[b * kTile + lane] = s;
            // fragment `piece` of the key's tile, lane (key, half)
            h8 *kd = reinterpret_cast<h8 *>(kb) + (lane >> 5) * (F * 64) + piece * 64 + (lane & 31);
            kd[0] = codes8(kc[i].x);
            kd[32] = codes8(kc[i].y);
            s1 = (_Float16)ldexpf((float)s1, kScaleTop - v_exp);
            const h8 s8 = {s1, s1, s1, s1, s1, s1, s1, s1};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const h8 c = codes8(vc[i][j]);
                h8 hi = c * s8;
                asm("" : "+v"(hi));
                const h8 lo = __builtin_elementwise_fma(c, s8, -hi);
                const int at = v_at<D>(lane, 2 * piece + j);
                *reinterpret_cast<h8 *>(vb + at) = hi;
                *reinterpret_cast<h8 *>(vb + kTile * kRowBytes + at) = lo;
            }
        }
        return by;
    };
    fetch(page0);

    // ---- the query: values 16 f + 8 half + nibble_of(e) of the lane's row
    h8 q1[F], q2[F];
    float f;                                 // scores in powers of two = sums times this
    {
        const float *src = own.q + (live ? row / group : 0) * own.q_stride + (kh * group + (live ? (int)(row % group) : 0)) * D + 8 * half;
        float x[F][8], top = 0.0f;
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const f4 y = *reinterpret_cast<const f4 *>(src + 16 * i + 4 * j);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[i][4 * j + e] = y[e];
                    const float m = fabsf(y[e]);
                    if (m <= kBig) top = fmaxf(top, m);
                }
            }
        top = fmaxf(top, other_half(top));
        const int e2 = top > 0.0f ? 14 - __builtin_amdgcn_frexp_expf(top) : 0;
        // (never 0: times a masked key's -inf that is no number. Sums are below 2^42, so such scores are as good as equal)
        f = ldexpf(1.0f, c_exp - e2 > 127 ? 127 : c_exp - e2 < -126 ? -126 : c_exp - e2);
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                half2_t hi, lo;
                split2(ldexpf(x[i][nibble_of(e)], e2) * c_man, ldexpf(x[i][nibble_of(e + 1)], e2) * c_man, hi, lo);
                q1[i][e] = hi.x;
                q1[i][e + 1] = hi.y;
                q2[i][e] = lo.x;
                q2[i][e + 1] = lo.y;
            }
    }

    f16v o[NB];                              // value positions 32 n + 8 (i / 4) + 4 half + i % 4
#pragma unroll
    for (int n = 0; n < NB; ++n) o[n] = f16v{};
    float m = -3.0e38f, l = 0.0f;
    // The wavefront's tile of a page.
    const auto attend = [&](int page) __attribute__((always_inline)) {
        const uint8_t *const kb = lds + (kTwo ? page & 1 : 0) * kOperands, *const vb = kb + kTile * kRowBytes;
        const h8 *const kf = reinterpret_cast<const h8 *>(kb) + kw * (F * 64) + lane;
        const _Float16 *const sb = reinterpret_cast<const _Float16 *>(kb + 3 * kTile * kRowBytes) + kw * kKeys + 4 * half;
        // (matrix instructions before the SIMD's other wavefront's vector instructions: 131072 tokens 190 -> 186 us)
        __builtin_amdgcn_s_setprio(1);
        f16v x = {};
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            f16v z = {};
#pragma unroll
            for (int i = 2 * b; i < 2 * b + 2; ++i) {
                const h8 k = kf[64 * i];
                z = mfma(k, q2[i], z);
                z = mfma(k, q1[i], z);
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const h4 s = *reinterpret_cast<const h4 *>(sb + b * kTile + 8 * g);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[4 * g + i] = fmaf(z[4 * g + i], (float)s[i], x[4 * g + i]);
            }
        }
        __builtin_amdgcn_s_setprio(0);
        const int64_t left = runs.len - (int64_t)page * kTile - kw * kKeys;
        if (left < kKeys) {
            const int end = (int)left - 4 * half;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (8 * (i >> 2) + (i & 3) >= end) x[i] = -__builtin_inff();
        }
        float high = fmaxf(x[0], x[1]);
#pragma unroll
        for (int i = 2; i < 16; ++i) high = fmaxf(high, x[i]);
        high = fmaxf(high, other_half(high)) * f;
        if (__any(high > m + kSlack)) {
            const float mn = fmaxf(m, high), by = __builtin_amdgcn_exp2f(m - mn);
            l *= by;
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[n][i] *= by;
            m = mn;
        }
        const float up = (float)kWeightBits - m;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            x[i] = __builtin_amdgcn_exp2f(fmaf(x[i], f, up));
            sum += x[i];
        }
        l += sum;
        __builtin_amdgcn_s_setprio(1);
        // output: 16 keys at a time; a lane reads 4 keys of 16 values and gets its value of them
        const int c = lane & 15;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            h8 p1, p2;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                half2_t hi, lo;
                split2(x[8 * t + i], x[8 * t + i + 1], hi, lo);
                p1[i] = hi.x;
                p1[i + 1] = hi.y;
                p2[i] = lo.x;
                p2[i + 1] = lo.y;
            }
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                h8 v[2];
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    h4 r[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int key = kw * kKeys + 16 * t + 8 * e + 4 * half + (c >> 2), d = 32 * n + (lane & 16) + 4 * (c & 3);
                        r[e] = __builtin_bit_cast(h4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4 *)(
                            vb + w * kTile * kRowBytes + v_at<D>(key, d >> 3) + (d & 7) * 2)));
                    }
                    v[w] = __builtin_shufflevector(r[0], r[1], 0, 1, 2, 3, 4, 5, 6, 7);
                }
                o[n] = mfma(v[1], p1, o[n]);
                o[n] = mfma(v[0], p2, o[n]);
                o[n] = mfma(v[0], p1, o[n]);
            }
        }
        __builtin_amdgcn_s_setprio(0);
    };
    const auto rescale = [&](int by) __attribute__((always_inline)) {
        if (by == 0) return;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[n][i] = ldexpf(o[n][i], by);
    };

    put(page0);                              // (the output is zero: its units change for nothing)
    fetch(page0 + 1);
    for (int page = page0; page < page_end; ++page) {
        lds_barrier();                       // the page's operands are there; with two buffers, those before have been read
        if constexpr (kTwo) {
            // wavefronts of a SIMD take turns: one's matrix instructions beside the other's operands
            int by = 0;
            if (any) attend(page);
            by = put(page + 1);              // (past the run's end: into a buffer that is not read)
            fetch(page + 2);
            rescale(by);
        } else {
            if (any) attend(page);
            if (page + 1 < page_end) {
                lds_barrier();               // read
                rescale(put(page + 1));
                fetch(page + 2);
            }
        }
    }

    // ---- the two wavefronts of the same rows meet in LDS; row position j of a block is value (j & ~7) + nibble_of(j & 7)
    l += other_half(l);
    const auto place = [&](int n, int g, int k) { return 32 * n + 8 * g + 2 * half + 4 * k; };       // of values i = 4 g + k and 4 g + k + 2
    float *const res = reinterpret_cast<float *>(lds) + (rw * 32 + (lane & 31)) * kPitch;
    __syncthreads();
    if (kw == 1) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int k = 0; k < 2; ++k) *reinterpret_cast<f2 *>(res + place(n, g, k)) = f2{o[n][4 * g + k], o[n][4 * g + k + 2]};
        if (half == 0) {
            res[D] = m;
            res[D + 1] = l;
        }
    }
    __syncthreads();
    if (kw == 1 || !live) return;
    const float m1 = res[D], l1 = res[D + 1], mm = fmaxf(m, m1);
    const float by0 = __builtin_amdgcn_exp2f(m - mm), by1 = __builtin_amdgcn_exp2f(m1 - mm);
    const int e = v_exp - kScaleTop - kWeightBits;
    float *dst = prefix_part(parts, run, kv, kh, rows, row, D);
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const f2 y = *reinterpret_cast<const f2 *>(res + place(n, g, k));
                const f2 z = {ldexpf(fmaf(by1, y.x, by0 * o[n][4 * g + k]), e), ldexpf(fmaf(by1, y.y, by0 * o[n][4 * g + k + 2]), e)};
                *reinterpret_cast<f2 *>(dst + place(n, g, k)) = z;
            }
    if (half == 0) {
        dst[D] = mm;
        dst[D + 1] = bad ? __builtin_nanf("") : ldexpf(fmaf(by1, l1, by0 * l), -kWeightBits);
    }
}

// A step: workgroups of the sequences' own tokens, RW / 2 jobs each, then those of
// the prefix. Apart, either would wait for the other's last. Heads of 64 leave room for a
// third workgroup of 64 rows on a compute unit if registers are held to a third (one fewer than
// the compiler takes): all workgroups of a call begin at once. 64 requests of 16/8 heads behind 8000
// tokens 32.8 -> 27.0 us, 75 of 14/2 behind 8191 30.7 -> 27.7 (behind 2000 18.4 -> 19.6).
template <int D, int RW, int H>
__global__ __launch_bounds__(128 * RW, D == 64 ? 3 : 2) void shared_kernel(SharedArgs a, float *parts, int chunks, float c_man, int c_exp, int groups, int cut, unsigned own_jobs)
{
    constexpr int kJobs = RW / 2, kJobBytes = (decode_lds_bytes(D, H) + 15) / 16 * 16;
    __shared__ __attribute__((aligned(16))) uint8_t lds[at_least(prefix_lds_bytes(D, RW), kJobs * kJobBytes)];
    const unsigned own_groups = (own_jobs + kJobs - 1) / kJobs;
    if (blockIdx.x < own_groups) {
        const int which = kJobs == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
        const unsigned job = blockIdx.x * kJobs + which;             // (two meet at unequal barriers: decode_job)
        if (job < own_jobs) decode_job<D, H, Form::sums>(a.own, groups, cut, c_man, c_exp, lds + which * kJobBytes, job, threadIdx.x & 255);
        return;
    }
    prefix_job<D, RW>(a, parts, chunks, c_man, c_exp, lds, blockIdx.x - own_groups);
}

// The same for few rows: the prefix as one sequence of the attention of single
// tokens, whose heads are the rows, 8 a workgroup.
template <int D, int H>
__global__ __launch_bounds__(64 * kDecodeWaves, 2) void shared_few_kernel(SharedArgs a, float *parts, int chunks, float c_man, int c_exp, int groups, int cut, unsigned own_jobs)
{
    __shared__ __attribute__((aligned(16))) uint8_t lds[at_least(decode_lds_bytes(D, H), decode_lds_bytes(D, kMaxGroup))];
    if (blockIdx.x < own_jobs) {
        decode_job<D, H, Form::sums>(a.own, groups, cut, c_man, c_exp, lds, blockIdx.x, threadIdx.x);
        return;
    }
    DecodeArgs p = a.own;
    p.query_heads = p.heads / p.cache.kv_heads;
    p.heads = p.cache.kv_heads * p.B * p.query_heads;
    p.B = 1;
    p.lens = a.prefix_len;
    p.table = a.prefix;
    p.max_pages = a.prefix_pages;
    p.ws = parts;
    decode_job<D, kMaxGroup, Form::prefix>(p, head_groups(p.heads, p.cache.kv_heads), chunks, c_man, c_exp, lds, blockIdx.x - own_jobs, threadIdx.x);
}

// Joins a head's parts: those of the prefix's runs, then its own tokens', each in a
// fixed order. As wq_kv.hip's join: a thread takes 4 values of every kJoinParts-th part and
// asks for kJoinAhead of them at once; for the prefix's before it is known how many there are.
constexpr int kJoinParts = 8, kJoinAhead = 4;

template <int D>
__global__ __launch_bounds__(D / 4 * kJoinParts) void shared_join_kernel(SharedArgs a, float *parts, int chunks, int unit, int groups, int cut)
{
    constexpr int V = D / 4;
    __shared__ f4 red[kJoinParts][V];
    __shared__ float ml[kJoinParts][2];
    const DecodeArgs &own = a.own;
    const int b = blockIdx.x / own.heads, j = blockIdx.x % own.heads, c = threadIdx.x % V, part = threadIdx.x / V;
    const int kv = own.cache.kv_heads, group = own.heads / kv, per_step = kv * groups, per = (group + groups - 1) / groups;
    const int kh = j / group, hg = j % group / per, hh = j % group % per;
    const int64_t rows = (int64_t)own.B * group, row = (int64_t)b * group + j % group;
    f4 *out = (f4 *)(own.out + (int64_t)b * own.out_stride + j * D) + c;
    float m = -3.0e38f, l = 0.0f;
    f4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    float pm[kJoinAhead], pl[kJoinAhead];
    f4 po[kJoinAhead];
    // (an entry of an empty sequence, and a part that no run wrote, may hold anything: they are not used)
    const auto ask = [&](int k, const float *p) __attribute__((always_inline)) {
        pm[k] = p[D];
        pl[k] = p[D + 1];
        po[k] = ((const f4 *)p)[c];
    };
    const auto add = [&](int i0, int count) __attribute__((always_inline)) {
        float mn = m;
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k) {
            if (i0 + k * kJoinParts >= count) {
                pm[k] = -3.0e38f;
                pl[k] = 0.0f;
                po[k] = f4{0.0f, 0.0f, 0.0f, 0.0f};
            }
            mn = fmaxf(mn, pm[k]);
        }
        const float by = __builtin_amdgcn_exp2f(m - mn);
        l *= by;
        o *= by;
        m = mn;
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k) {
            const float f = __builtin_amdgcn_exp2f(pm[k] - m);
            l = fmaf(f, pl[k], l);
            o += f * po[k];
        }
    };
    const auto ask_prefix = [&](int i0) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k) {
            const int i = i0 + k * kJoinParts;
            if (i < chunks) ask(k, prefix_part(parts, i, kv, kh, rows, row, D));
        }
    };
    ask_prefix(part);
    Pieces at = {0, 1, 0, 0};
    if (cut) at = ((const Pieces *)own.ws)[b];
    const int64_t len = own.lens[b];
    const PrefixRuns runs = prefix_runs(a.prefix_len, a.prefix_pages, chunks, unit);
    if (runs.bad || len < 0 || len > own.max_pages * kTile || (len == 0 && runs.len == 0)) {
        const float y = runs.bad || len != 0 ? __builtin_nanf("") : 0.0f;
        if (part == 0) *out = f4{y, y, y, y};
        return;
    }
    add(part, runs.count);
    for (int i0 = part + kJoinAhead * kJoinParts; i0 < runs.count; i0 += kJoinAhead * kJoinParts) {
        ask_prefix(i0);
        add(i0, runs.count);
    }
    const int mine = len > 0 ? at.count : 0;
    if (mine == 1) {                             // one piece: divided already
        if (part == 0) {
            const float *s = own.sums + ((int64_t)b * own.heads + j) * 2;
            pm[0] = s[0];
            pl[0] = s[1];
            po[0] = *out * pl[0];
            add(0, 1);
        }
    } else {
        for (int i0 = part; i0 < mine; i0 += kJoinAhead * kJoinParts) {
#pragma unroll
            for (int k = 0; k < kJoinAhead; ++k) {
                const int i = i0 + k * kJoinParts;
                if (i < mine) ask(k, partial<D>(own, (int64_t)(at.first + i) * per_step + hg * kv + kh, i == 0 ? at.slot : 0, hh));
            }
            add(i0, mine);
        }
    }
    red[part][c] = o;
    if (c == 0) {
        ml[part][0] = m;
        ml[part][1] = l;
    }
    __syncthreads();
    if (part == 0) {
        float mn = ml[0][0];
#pragma unroll
        for (int w = 1; w < kJoinParts; ++w) mn = fmaxf(mn, ml[w][0]);
        float ll = 0.0f;
        f4 oo = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < kJoinParts; ++w) {
            const float f = __builtin_amdgcn_exp2f(ml[w][0] - mn);
            ll = fmaf(f, ml[w][1], ll);
            oo += f * red[w][c];
        }
        *out = oo / ll;
    }
}

// ---- how the prefix is cut
// Workgroups of 8 rows (up to kFewRows), of 64, two or three on each compute unit, or of 128, one. us a call, prefixes in
// tokens, 8 / 64 rows: heads of 128, 8 key/value heads, 32768 tokens: 8 rows 30.8 / 41.9, 16 35.5 / 43.1, 24 43.5
// / 44.7, 32 47.0 / 45.8; heads of 64, 4 key/value heads, 16000: 16 rows 13.8 / 15.0, 24 14.7
// / 15.2, 32 15.6 / 15.3; 8, 8000: 24 16.4 / 14.6; 2, 4000: 28 11.5 / 13.0; 2048 tokens the same within 1 us.
// 64 / 128 rows, 16/8 heads of 128: 64 rows, 32768 tokens 52 / 62; 128 rows, 2048 26.8 / 33.8, 8192 46.5 / 46.6, 16000
// 55.8 / 55.4, 32768 79 / 77. Heads of 64 take 64 always: 14/2, 525 rows, 16000 tokens 34 / 41, 32000 45 / 52, 131000 129
// / 137, 262000 241 / 249; 16/8, 128 rows, 65000 67 / 71, 131000 118 / 118.
// Two places on each compute unit: the third of heads of 64 takes what comes beside them (filled with runs of its own, 768
// places: 16/8 heads, 64 requests behind 4000 tokens 21 -> 26, behind 16000 33 -> 39).
constexpr int kSharedFill = 512;
constexpr int64_t kFewRows = 24;
inline int row_waves(int64_t rows, int64_t head_dim, int64_t prefix_pages)
{
    return head_dim == 64 || rows <= 64 || prefix_pages <= 128 ? 2 : 4;
}
inline int run_unit(int64_t rows) { return rows <= kFewRows ? kDecodeWaves : 1; }        // pages
// A sequence's own tokens are cut whenever that makes parts, since there is a join anyway, into no more
// runs than there can be steps; the prefix into as many as fill what is left of the card, half of it at
// least, and all of it where its runs are longer than kRunPages. Own tokens leave it a place from the start (but
// beside workgroups of 128 rows: 64 sequences behind 16000 tokens 55.4 us, 58.2 with a place): half of the card (64
// behind 4096 37.7 -> 31.1), or, where it has little to do beside them, its share of the work. That is counted
// in steps of own tokens, as the table's width allows them: a page of the prefix takes as long as one (with 8 rows:
// four pages), and a part of it kStartSteps to begin. us, half / share, with the prefix's part of the work: 16/8 heads
// of 128, 1 request of 131072 own tokens behind 64 (0.01) 39.7 / 38.6, behind 4096 (0.16) 40.1 / 41.2; 4 requests,
// 120000, behind 1024 (0.02) 35.5 / 32.5, behind 4096 (0.07) 35.5 / 37.5; 32, 24864, behind 1024 (0.02) 25.4 / 23.2, behind 4096
// (0.09) 28.6 / 31.8; 32/8 heads, 64, 524288, behind 64 (0.001) 143 / 127, behind 4096 (0.03) 159 / 149. Few steps gain nothing
// by more runs: 14/2 heads of 64, 16 requests, 65536 in 87 steps at most, behind 256 17.0 / 17.6; 64, 262144 in 155, 28.5 / 25.2.
constexpr int kRunPages = 4, kStartSteps = 4;
constexpr int kLittle = 16, kShortRuns = 12;
struct SharedCut {
    int groups, per_step;                        // of the sequences' own heads
    int own, chunks;                             // runs of own tokens (0: whole sequences), of the prefix
    int waves, together;                         // row_waves (0: few rows), own jobs of a workgroup
    unsigned own_jobs;
    int64_t blocks;                              // of rows and key/value heads
};
inline SharedCut shared_cut(int64_t B, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t max_pages, int64_t prefix_pages)
{
    SharedCut c;
    const int64_t rows = B * (heads / kv_heads), steps = (max_pages + kDecodeWaves - 1) / kDecodeWaves;
    c.groups = head_groups((int)heads, (int)kv_heads);
    c.per_step = (int)kv_heads * c.groups;
    int64_t most = runs_per_head(c.per_step);
    c.waves = rows <= kFewRows ? 0 : row_waves(rows, head_dim, prefix_pages);
    c.together = c.waves == 4 ? 2 : 1;
    const int64_t each = c.waves ? 32 * c.waves : kMaxGroup;
    c.blocks = (rows + each - 1) / each * kv_heads;
    const int64_t unit = run_unit(rows), units = (prefix_pages + unit - 1) / unit;
    if (c.waves != 4) {                          // beside the prefix, not before it
        const int64_t parts = c.blocks * ((prefix_pages + kRunPages - 1) / kRunPages);
        const int64_t there = c.blocks * units + parts * kStartSteps, work = c.per_step * B * (steps + kChangeSteps);
        if (kLittle * there >= work || c.per_step * B * steps <= kShortRuns * (kSharedFill / 2)) most = (most + 1) / 2;
        else most = (kSharedFill - (there * (kSharedFill / 2) + there + work - 1) / (there + work)) / c.per_step;
        if (most < 1) most = 1;
    }
    c.own = B > kCutMaxSeqs || steps <= 1 ? 0 : (int)(B * steps < most ? B * steps : most);
    c.own_jobs = (unsigned)((int64_t)c.per_step * (c.own ? c.own : B));
    const int64_t slots = c.waves == 4 ? kSharedFill / 2 : kSharedFill, taken = (c.own_jobs + c.together - 1) / c.together;
    const int64_t left = (taken > slots / 2 ? slots / 2 : slots - taken) / c.blocks, all = slots / c.blocks;
    int64_t n = prefix_pages / kRunPages < all ? prefix_pages / kRunPages : all;
    if (n < left) n = left;
    c.chunks = (int)(n > units ? units : n < 1 ? (units > 0) : n);
    return c;
}
inline uint64_t round256(uint64_t x) { return (x + 255) / 256 * 256; }
inline uint64_t sums_bytes(int64_t B, int64_t heads) { return round256((uint64_t)B * heads * 8); }
inline uint64_t own_bytes(const SharedCut &c, int64_t head_dim) { return c.own ? round256(pieces_bytes(c.per_step, c.own, head_dim)) : 0; }

}  // namespace

uint64_t shared_ws_bytes(int64_t B, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t max_pages, int64_t prefix_pages)
{
    const SharedCut c = shared_cut(B, heads, kv_heads, head_dim, max_pages, prefix_pages);
    // (own tokens behind a short prefix may be cut into more runs: more pages never ask for less)
    const SharedCut alone = shared_cut(B, heads, kv_heads, head_dim, max_pages, 0);
    return own_bytes(alone.own > c.own ? alone : c, head_dim) + sums_bytes(B, heads) + (uint64_t)c.chunks * B * heads * (uint64_t)(head_dim + kPartialExtra) * 4;
}

hipError_t launch_attn_decode_shared(const SharedArgs &args, hipStream_t stream)
{
    SharedArgs a = args;
    DecodeArgs &own = a.own;
    const int D = own.cache.head_dim, group = own.heads / own.cache.kv_heads;
    const SharedCut cut = shared_cut(own.B, own.heads, own.cache.kv_heads, D, own.max_pages, a.prefix_pages);
    const int per = (group + cut.groups - 1) / cut.groups;
    char *ws = (char *)own.ws + own_bytes(cut, D);
    own.sums = (float *)ws;
    float *parts = (float *)(ws + sums_bytes(own.B, own.heads));
    int c_exp = 0;
    const double c = frexp((double)own.scale * 1.4426950408889634, &c_exp);    // softmax in powers of two
    const unsigned grid = (cut.own_jobs + cut.together - 1) / cut.together + (unsigned)(cut.blocks * cut.chunks);
    const auto start = [&](auto kernel) {
        kernel<<<grid, cut.waves == 4 ? 512 : 256, 0, stream>>>(a, parts, cut.chunks, (float)(2.0 * c), c_exp - 1, cut.groups, cut.own, cut.own_jobs);
    };
    const auto pick = [&](auto dim, auto heads) {
        constexpr int DIM = decltype(dim)::value, H = decltype(heads)::value;
        if (cut.waves == 0) start(shared_few_kernel<DIM, H>);
        else if (DIM == 64 || cut.waves == 2) start(shared_kernel<DIM, 2, H>);
        else if constexpr (DIM == 128) start(shared_kernel<DIM, 4, H>);
    };
    using std::integral_constant;
    if (D == 128) {
        if (per <= 2) pick(integral_constant<int, 128>{}, integral_constant<int, 2>{});
        else if (per <= 4) pick(integral_constant<int, 128>{}, integral_constant<int, 4>{});
        else pick(integral_constant<int, 128>{}, integral_constant<int, 8>{});
    } else {
        if (per <= 4) pick(integral_constant<int, 64>{}, integral_constant<int, 4>{});
        else pick(integral_constant<int, 64>{}, integral_constant<int, 8>{});
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const unsigned jobs = (unsigned)((int64_t)own.B * own.heads);
    const int unit = run_unit((int64_t)own.B * group);
    if (D == 128) shared_join_kernel<128><<<jobs, 128 / 4 * kJoinParts, 0, stream>>>(a, parts, cut.chunks, unit, cut.groups, cut.own);
    else shared_join_kernel<64><<<jobs, 64 / 4 * kJoinParts, 0, stream>>>(a, parts, cut.chunks, unit, cut.groups, cut.own);
    return hipGetLastError();
}

}  // namespace wq
