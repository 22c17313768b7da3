// wq_prompt.hip -- causal attention over packed prompts (fp32, grouped heads).
//
//   out[t, j] = sum_u p_u v[u] / sum_u p_u,  p_u = exp(scale <q, k_u> - max),
//   u <= t in t's own sequence.
//
// fp32 products on the fp16 matrix cores: every operand is normalised by a
// power of two and split into two binary16 parts, x = x1 + x2 (22 bits), and a
// product is three matrix products, x1 y1 + x1 y2 + x2 y1. That is a third of
// the fp16 rate, 2.6 times the rate of the fp32 matrix instructions.
//
// Two kernels:
//   prepare_kernel  splits k and v once per call into a workspace, in tiles of
//     32 keys per key/value head that begin at the sequence's first token, in
//     the order the matrix instructions take their operands (a fragment is
//     64 lanes x 16 bytes of consecutive memory), so that the attention kernel
//     copies and reads them without any shuffling.
//   attend_kernel   one wavefront per 32 query rows of a head. Scores come out
//     transposed, S' = K Q' (a lane holds one query and 16 of the 32 keys), so
//     the softmax runs within a lane but for one exchange between the wave's
//     halves, and the weights, split in place, are already the second operand
//     of O' = V' P': no trip through LDS.
//
// Normalisation. Query rows have a factor each. k and v have one per tile, which
// is exact enough (22 bits for every row) while no row of the tile is 2^14
// smaller than the largest; a "wild" tile (rows further apart) takes a factor
// per row: on the scores for k, on the weights for v. Sums, maxima and weights
// are fp32. The output of a query is kept in units of the largest tile (wild:
// visible row) of v seen so far; tiles are walked first to last, so that its
// precision never depends on values it does not see by more than the 2^14 of
// one tile.
#include "wq_internal.h"
#include "wq_device.h"
#include "wq_seq.h"

#include <math.h>

namespace wq {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr int kTileKeys = 32;
constexpr float kBig = 3.4028235e38f;
constexpr int kWildBits = 14;        // rows of a tile further apart than this are not normalised together
constexpr int kWeightBits = 12;      // a weight of 1 is 2^12 as a binary16 operand
constexpr float kSlack = 3.0f;       // log2 a score may pass the running maximum by before rescaling: 2^15 at most

// What the attention kernel needs to know of a tile.
struct TileMeta {
    int k_exp;                       // k was multiplied by 2^k_exp (wild: by 2^k_row[u] row by row)
    int v_exp;                       // v is its operands times 2^v_exp (wild: 2^v_row[u])
    int flags;
    int pad;
    int k_row[kTileKeys];
    int v_row[kTileKeys];
};
enum { kWildK = 1, kWildV = 2, kOddV = 4 };      // kOddV: v holds values that are not finite (0 in the operands)
constexpr int kNoExp = -100000;      // of a row of zeros

__host__ __device__ inline int64_t tile_slots(int64_t T, int64_t B, int rows) { return T / rows + B; }
constexpr int tile_halves(int D) { return 4 * D * kTileKeys; }      // binary16 values of a tile: k1 k2 v1 v2

// First slot of a sequence's tiles: slots of different sequences never meet,
// since floor((c + L) / r) + 1 >= floor(c / r) + ceil(L / r).
__device__ __forceinline__ int first_slot(int begin, int b, int rows) { return begin / rows + b; }

// The sequence that a slot belongs to, if any: the last b whose first slot is
// not behind it.
__device__ __forceinline__ int seq_of_slot(const int32_t *cu, int T, int B, int rows, int slot)
{
    if (!cu) return 0;
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first_slot(clamp_token(cu[mid], T), mid, rows) <= slot) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ float finite_abs(float x)
{
    const float y = fabsf(x);
    return y <= kBig ? y : 0.0f;
}

// Power of two that brings a (>= 0) into [2^(top-1), 2^top); 0 for a == 0.
__device__ __forceinline__ int normaliser(float a, int top) { return a > 0.0f ? top - __builtin_amdgcn_frexp_expf(a) : 0; }

// x = hi + lo to 22 bits (hi rounded to nearest, the remainder exact in fp32).
// x is made opaque first: contracted with the product that made it, the hi
// that is subtracted could be rounded differently from the hi that is kept.
__device__ __forceinline__ void split(float x, _Float16 &hi, _Float16 &lo)
{
    asm("" : "+v"(x));
    hi = (_Float16)x;
    lo = (_Float16)(x - (float)hi);
}

// ---------------------------------------------------------------- prepare
// One workgroup per (tile, key/value head); 8 threads share a row of D values.
template <int D>
__global__ __launch_bounds__(256) void prepare_kernel(PromptArgs a, _Float16 *__restrict__ tiles, TileMeta *__restrict__ metas)
{
    constexpr int E = D / 8;                     // values a thread holds of its row
    __shared__ float vt[kTileKeys][D + 1];
    __shared__ float red[4][4];
    __shared__ int v_factor[kTileKeys];
    const int slot = blockIdx.x, head = blockIdx.y, tid = threadIdx.x;
    const int b = seq_of_slot(a.cu, (int)a.T, a.B, kTileKeys, slot);
    const SeqRange r = seq_range(a.cu, (int)a.T, b);
    const int len = r.end - r.begin, tile = slot - first_slot(r.begin, b, kTileKeys);
    if (tile < 0 || tile * kTileKeys >= len) return;
    const int row = tid >> 3, seg = tid & 7, key = tile * kTileKeys + row;
    const bool live = key < len;
    float k[E], v[E];
    float kmax = 0.0f, vmax = 0.0f;
    int odd = 0;                                 // v not finite
    const float *ks = a.k + (int64_t)(r.begin + key) * a.k_stride + head * D + seg * E;
    const float *vs = a.v + (int64_t)(r.begin + key) * a.v_stride + head * D + seg * E;
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
        f4 x = {0.0f, 0.0f, 0.0f, 0.0f}, y = x;
        if (live) {
            x = reinterpret_cast<const f4 *>(ks)[i];
            y = reinterpret_cast<const f4 *>(vs)[i];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            k[4 * i + j] = x[j];
            v[4 * i + j] = y[j];
            kmax = fmaxf(kmax, finite_abs(x[j]));
            vmax = fmaxf(vmax, finite_abs(y[j]));
            odd |= !(fabsf(y[j]) <= kBig);
        }
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {            // the row's maxima
        kmax = fmaxf(kmax, __shfl_xor(kmax, o));
        vmax = fmaxf(vmax, __shfl_xor(vmax, o));
    }
    // tile maxima and smallest rows that are not zero
    float kt = kmax, vt_max = vmax, kl = kmax > 0.0f ? kmax : kBig, vl = vmax > 0.0f ? vmax : kBig;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        kt = fmaxf(kt, __shfl_xor(kt, o));
        vt_max = fmaxf(vt_max, __shfl_xor(vt_max, o));
        kl = fminf(kl, __shfl_xor(kl, o));
        vl = fminf(vl, __shfl_xor(vl, o));
        odd |= __shfl_xor(odd, o);
    }
    if ((tid & 63) == 0) {
        float *w = red[tid >> 6];
        w[0] = kt;
        w[1] = odd ? -vt_max - 1e-45f : vt_max;  // a sign marks data that is not finite
        w[2] = kl;
        w[3] = vl;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) vt[row][seg * E + i] = v[i];
    __syncthreads();
    odd = 0;
    kt = vt_max = 0.0f;
    kl = vl = kBig;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        kt = fmaxf(kt, red[w][0]);
        odd |= red[w][1] < 0.0f;
        vt_max = fmaxf(vt_max, fabsf(red[w][1]));
        kl = fminf(kl, red[w][2]);
        vl = fminf(vl, red[w][3]);
    }
    const int ke = normaliser(kt, 15), ve = normaliser(vt_max, 15);
    const bool wild_k = kt > 0.0f && normaliser(kl, 15) - ke > kWildBits;
    const bool wild_v = vt_max > 0.0f && normaliser(vl, 15) - ve > kWildBits;
    const int kr = wild_k ? normaliser(kmax, 15) : ke;
    const int64_t at = (int64_t)slot * a.kv_heads + head;
    TileMeta *m = metas + at;
    if (tid == 0) {
        m->k_exp = ke;
        m->v_exp = -ve;
        m->flags = (wild_k ? kWildK : 0) | (wild_v ? kWildV : 0) | (odd ? kOddV : 0);
    }
    const int vr = wild_v ? normaliser(vmax, 15) : ve;
    if (seg == 0) {
        m->k_row[row] = kr;
        m->v_row[row] = vmax > 0.0f ? -vr : kNoExp;
        v_factor[row] = vr;
    }
    __syncthreads();
    _Float16 *dst = tiles + at * tile_halves(D);
    // k: fragment f covers values 16 f .. 16 f + 15; lane (key, half) holds 8 of them
#pragma unroll
    for (int c = 0; c < E / 8; ++c) {
        const int d0 = seg * E + 8 * c, f = d0 >> 4, half = (d0 >> 3) & 1;
        h8 hi, lo;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            _Float16 x, y;
            split(ldexpf(k[8 * c + j], kr), x, y);
            hi[j] = x;
            lo[j] = y;
        }
        const int o = f * 512 + (half * 32 + row) * 8;
        *reinterpret_cast<h8 *>(dst + o) = hi;
        *reinterpret_cast<h8 *>(dst + D * kTileKeys + o) = lo;
    }
    // v': fragment (db, s) covers values 32 db .. + 31 and 16 keys; lane (d, half)
    // holds the keys that the scores' lane of that half holds: 16 s + 8 (e / 4) + 4 half + e % 4
#pragma unroll
    for (int i = 0; i < D * kTileKeys / 8 / 256; ++i) {
        const int c = tid + 256 * i, lane = c & 63, f = c >> 6;
        const int d = (f >> 1) * 32 + (lane & 31), k0 = (f & 1) * 16 + 4 * (lane >> 5);
        h8 hi, lo;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int u = k0 + 8 * (e >> 2) + (e & 3);
            const float y = vt[u][d];
            _Float16 x, z;
            split(fabsf(y) <= kBig ? ldexpf(y, v_factor[u]) : 0.0f, x, z);
            hi[e] = x;
            lo[e] = z;
        }
        *reinterpret_cast<h8 *>(dst + 2 * D * kTileKeys + c * 8) = hi;
        *reinterpret_cast<h8 *>(dst + 3 * D * kTileKeys + c * 8) = lo;
    }
}

// ---------------------------------------------------------------- attend
__device__ __forceinline__ f16v mfma(h8 a, h8 b, f16v c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }

// Both halves of the wave's value: {this lane's or its partner's, the other}.
__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32); }

// Running state of 32 query rows: a lane holds query lane % 32; its half of the
// wave holds half of the output's values and half of the keys of each tile.
template <int D>
struct Rows {
    h8 q1[D / 16], q2[D / 16];
    f16v o[D / 32];                  // value 32 db + 8 (i / 4) + 4 half + i % 4
    float m, l;                      // running maximum (log2), sum of weights of this lane's keys
    int q_exp;                       // scores are 2^(q_exp - k_exp) times the products
    int v_exp;                       // o is in units of 2^(v_exp - kWeightBits)
};

template <int D>
__device__ __forceinline__ void load_query(Rows<D> &s, const float *q, bool live, float c_man, int c_exp, int half)
{
    constexpr int F = D / 16;
    float x[F][8];
    float top = 0.0f;
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
            if (live) v = *reinterpret_cast<const f4 *>(q + 16 * f + 8 * half + 4 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[f][4 * i + j] = v[j];
                top = fmaxf(top, finite_abs(v[j]));
            }
        }
    top = fmaxf(top, other_half(top));
    const int e = normaliser(top, 14);           // |c_man| < 2 keeps the product below 2^15
    s.q_exp = c_exp - e;
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            _Float16 hi, lo;
            split(ldexpf(x[f][j], e) * c_man, hi, lo);
            s.q1[f][j] = hi;
            s.q2[f][j] = lo;
        }
#pragma unroll
    for (int db = 0; db < D / 32; ++db) s.o[db] = f16v{};
    s.m = -3.0e38f;
    s.l = 0.0f;
    s.v_exp = kNoExp;
}

// One tile of 32 keys. `tile` (LDS or global memory) holds its operands.
// `first`: position of its first key minus that of this lane's query (keys
// with first + u > 0 are masked), looked at where `edge`.
template <int D>
__device__ __forceinline__ void tile_step(Rows<D> &s, const _Float16 *tile, const TileMeta *meta, bool edge, int first,
                                          const float *v_rows, int64_t v_stride, int live_keys, int lane)
{
    constexpr int F = D / 16;
    const int half = lane >> 5;
    const h8 *k1 = reinterpret_cast<const h8 *>(tile) + lane;
    const h8 *k2 = k1 + D * kTileKeys / 8;
    f16v x = {};
#pragma unroll
    for (int f = 0; f < F; ++f) {
        const h8 a1 = k1[64 * f], a2 = k2[64 * f];
        x = mfma(a2, s.q1[f], x);
        x = mfma(a1, s.q2[f], x);
        x = mfma(a1, s.q1[f], x);
    }
    const int flags = meta->flags;
    int e = s.q_exp - meta->k_exp;
    if (flags & kWildK) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = ldexpf(x[i], s.q_exp - meta->k_row[8 * (i >> 2) + 4 * half + (i & 3)]);
        e = 0;
    }
    if (edge) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (first + 8 * (i >> 2) + 4 * half + (i & 3) > 0) x[i] = -__builtin_inff();
    }
    const float f = ldexpf(1.0f, e > 127 ? 127 : e);
    float top = fmaxf(x[0], x[1]);
#pragma unroll
    for (int i = 2; i < 16; ++i) top = fmaxf(top, x[i]);
    top = fmaxf(top, other_half(top)) * f;
    int ve = meta->v_exp;
    if (flags & kWildV) {                        // the largest row this query sees
        ve = kNoExp;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int u = 8 * (i >> 2) + 4 * half + (i & 3), r = meta->v_row[u];
            if (!(edge && first + u > 0) && r > ve) ve = r;
        }
        const int o = __shfl_xor(ve, 32);
        ve = ve > o ? ve : o;
    }
    if (__any(top > s.m + kSlack || ve > s.v_exp)) {
        const float m = fmaxf(s.m, top);
        const int vn = ve > s.v_exp ? ve : s.v_exp;
        const float r = __builtin_amdgcn_exp2f(s.m - m);
        const float ro = ldexpf(r, s.v_exp - vn);
        s.l *= r;
#pragma unroll
        for (int db = 0; db < D / 32; ++db)
#pragma unroll
            for (int i = 0; i < 16; ++i) s.o[db][i] *= ro;
        s.m = m;
        s.v_exp = vn;
    }
    // weights in units of 2^-(kWeightBits + d), d <= 0 the distance of this tile's values below the largest
    const int d = (flags & kWildV) ? 0 : ve - s.v_exp < -60 ? -60 : ve - s.v_exp;
    const float up = (float)(kWeightBits + d) - s.m;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        x[i] = __builtin_amdgcn_exp2f(fmaf(x[i], f, up));
        sum += x[i];
    }
    s.l = fmaf(sum, ldexpf(1.0f, -kWeightBits - d), s.l);
    if (flags & kWildV) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int r = meta->v_row[8 * (i >> 2) + 4 * half + (i & 3)] - s.v_exp;
            x[i] = ldexpf(x[i], r < 0 ? r : 0);
        }
    }
    const h8 *v1 = reinterpret_cast<const h8 *>(tile) + 2 * D * kTileKeys / 8 + lane;
    const h8 *v2 = v1 + D * kTileKeys / 8;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        h8 p1, p2;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            _Float16 hi, lo;
            split(x[8 * t + i], hi, lo);
            p1[i] = hi;
            p2[i] = lo;
        }
#pragma unroll
        for (int db = 0; db < D / 32; ++db) {
            const h8 a1 = v1[64 * (2 * db + t)], a2 = v2[64 * (2 * db + t)];
            s.o[db] = mfma(a2, p1, s.o[db]);
            s.o[db] = mfma(a1, p2, s.o[db]);
            s.o[db] = mfma(a1, p1, s.o[db]);
        }
    }
    if (flags & kOddV) {
        // count, for each output, the visible values that are not finite: a product of two masks
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
            h8 seen;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                seen[e] = !edge || first + 16 * t + 8 * (e >> 2) + 4 * half + (e & 3) <= 0 ? (_Float16)1.0f : (_Float16)0.0f;
#pragma unroll
            for (int db = 0; db < D / 32; ++db) {
                h8 odd;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int u = 16 * t + 8 * (e >> 2) + 4 * half + (e & 3);
                    const float y = v_rows[(u < live_keys ? u : 0) * v_stride + 32 * db + (lane & 31)];
                    odd[e] = u < live_keys && !(fabsf(y) <= kBig) ? (_Float16)1.0f : (_Float16)0.0f;
                }
                const f16v n = mfma(odd, seen, f16v{});
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (n[i] > 0.0f) s.o[db][i] = __builtin_nanf("");
            }
        }
    }
}

template <int D>
__device__ __forceinline__ void store_rows(const Rows<D> &s, float *out, int half)
{
    const float l = s.l + other_half(s.l), inv = 1.0f / l;
#pragma unroll
    for (int db = 0; db < D / 32; ++db)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            f4 y;
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = ldexpf(s.o[db][4 * g + j] * inv, s.v_exp - kWeightBits);
            if (out) *reinterpret_cast<f4 *>(out + 32 * db + 8 * g + 4 * half) = y;
        }
}

// W wavefronts of consecutive 32-row blocks of one query head share the tiles
// through a double buffer in LDS, filled by direct-to-LDS copies one tile ahead.
template <int D, int W>
__global__ __launch_bounds__(64 * W, 2) void attend_kernel(PromptArgs a, const _Float16 *__restrict__ tiles,
                                                          const TileMeta *__restrict__ metas, float c_man, int c_exp,
                                                          int slots)
{
    constexpr int kRows = 32 * W, kBytes = tile_halves(D) * 2;
    __shared__ __attribute__((aligned(16))) _Float16 buf[2][tile_halves(D)];
    const int id = blockIdx.x, group = a.heads / a.kv_heads;
    // heads of one key/value head run next to each other on one XCD (ids go round the 8 XCDs), later
    // (longer) row blocks first
    const int hp = id % a.heads, kvh = hp % a.kv_heads, head = kvh * group + hp / a.kv_heads;
    const int slot = slots - 1 - id / a.heads;
    const int b = seq_of_slot(a.cu, (int)a.T, a.B, kRows, slot);
    const SeqRange r = seq_range(a.cu, (int)a.T, b);
    const int len = r.end - r.begin, row0 = (slot - first_slot(r.begin, b, kRows)) * kRows;
    if (row0 < 0 || row0 >= len) return;
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wrow = row0 + 32 * wave, pos = wrow + (lane & 31);
    const bool live = pos < len;
    Rows<D> s;
    load_query<D>(s, a.q + (int64_t)(r.begin + pos) * a.q_stride + head * D, live, c_man, c_exp, half);
    const int last = (len - 1 < row0 + kRows - 1 ? len - 1 : row0 + kRows - 1) / kTileKeys;      // last tile of the block
    const int64_t step = a.kv_heads;
    const int64_t at0 = (int64_t)first_slot(r.begin, b, kTileKeys) * step + kvh;
    auto copy = [&](int tile) {
        const char *src = reinterpret_cast<const char *>(tiles + (at0 + tile * step) * tile_halves(D)) + wave * 1024 + lane * 16;
        char *dst = reinterpret_cast<char *>(buf[tile & 1]) + wave * 1024;
#pragma unroll
        for (int i = 0; i < kBytes / 1024 / W; ++i)
            __builtin_amdgcn_global_load_lds(
                (const __attribute__((address_space(1))) void *)(src + i * 1024 * W),
                (__attribute__((address_space(3))) void *)(dst + i * 1024 * W), 16, 0, 0);
    };
    copy(0);
    for (int t = 0; t <= last; ++t) {
        __builtin_amdgcn_s_waitcnt(0x0070);      // this wave's copies of tile t have arrived; its reads of t - 1 are done
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (t < last) copy(t + 1);
        if (t * kTileKeys <= wrow + 31 && wrow < len)
            tile_step<D>(s, buf[t & 1], metas + at0 + t * step, t * kTileKeys + 31 > wrow, t * kTileKeys - pos,
                         a.v + (int64_t)(r.begin + t * kTileKeys) * a.v_stride + kvh * D, a.v_stride,
                         len - t * kTileKeys, lane);
    }
    if (wrow < len)
        store_rows<D>(s, live ? a.out + (int64_t)(r.begin + pos) * a.out_stride + head * D : nullptr, half);
}

inline uint64_t round256(uint64_t x) { return (x + 255) / 256 * 256; }
inline uint64_t meta_bytes(int64_t slots, int64_t kv_heads) { return round256((uint64_t)slots * kv_heads * sizeof(TileMeta)); }

template <int D>
hipError_t launch(const PromptArgs &a, hipStream_t stream)
{
    constexpr int W = 4;
    const int64_t slots = tile_slots(a.T, a.B, kTileKeys);
    TileMeta *metas = reinterpret_cast<TileMeta *>(a.ws);
    _Float16 *tiles = reinterpret_cast<_Float16 *>((char *)a.ws + meta_bytes(slots, a.kv_heads));
    prepare_kernel<D><<<dim3((unsigned)slots, (unsigned)a.kv_heads), 256, 0, stream>>>(a, tiles, metas);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    int c_exp = 0;
    const double c = frexp((double)a.scale * 1.4426950408889634, &c_exp);      // softmax in powers of two
    const int64_t rows = tile_slots(a.T, a.B, 32 * W);
    attend_kernel<D, W><<<(unsigned)(rows * a.heads), 64 * W, 0, stream>>>(a, tiles, metas, (float)(2.0 * c), c_exp - 1, (int)rows);
    return hipGetLastError();
}

}  // namespace

uint64_t prompt_ws_bytes(int64_t T, int64_t B, int64_t, int64_t kv_heads, int64_t head_dim)
{
    const int64_t slots = tile_slots(T, B, kTileKeys);
    return meta_bytes(slots, kv_heads) + (uint64_t)slots * kv_heads * tile_halves((int)head_dim) * 2;
}

hipError_t launch_attn_prefill(const PromptArgs &a, hipStream_t stream)
{
    return a.head_dim == 128 ? launch<128>(a, stream) : launch<64>(a, stream);
}

}  // namespace wq
