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
// Two kernels, and one for very short prompts that does without the first (attend_direct_kernel):
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
// visible row) of v seen so far, which values of zero leave alone; tiles are
// walked first to last, so that its precision never depends on values it does
// not see by more than the 2^14 of one tile.
//
// Bound: in long prompts the rate of binary16 products (8192 tokens, 16 heads of 128: 815 us,
// 1012 TFLOP/s where a large library product reaches 1205 of nominal 2500), the
// latency of a launch or two in short ones (128 tokens: 10.6 us), in between the L2's
// k and v and the issue of matrix and vector instructions in turns (1024 tokens: 30 us).
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
    int k_exp, k_flags;              // k was multiplied by 2^k_exp (wild: by 2^k_row[u] row by row)
    int v_exp, v_flags;              // v is its operands times 2^v_exp (wild: 2^v_row[u]; kNoExp: all are zero)
    int k_row[kTileKeys];
    int v_row[kTileKeys];
};
typedef int i4 __attribute__((ext_vector_type(4)));

// The first four numbers, by a scalar load: asked for a tile ahead, since each is a miss.
struct TileHead {
    int k_exp, v_exp, flags;
};
__device__ __forceinline__ TileHead head_of(const TileMeta *m)
{
    const i4 x = *(const __attribute__((address_space(4))) i4 *)(uintptr_t)m;
    return {x.x, x.z, x.y | x.w};
}
enum { kWildK = 1, kWildV = 2, kOddV = 4 };      // kOddV: v holds values that are not finite (0 in the operands)
constexpr int kNoExp = -100000;      // of zeros: below every other, so that they never set the units of the output

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
// One workgroup per (tile, key/value head, k or v); 8 threads share a row of D
// values. All latency at short prompts; at long ones 4 D bytes in and as many out for a
// row (8192 tokens, 8 heads of 128: 134 MB, 36 us).
template <int CTRL>
__device__ __forceinline__ float max_dpp(float x)
{
    return fmaxf(x, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true)));
}

// Stores that leave the L2 at once: what is still dirty there when a kernel ends
// delays the next one's start (1024 tokens: 32.4 us without, 30.8 with them). `at`
// in values from the tile's k or v on.
template <int D>
__device__ __forceinline__ void store_through(_Float16 *dst, int at, h8 x)
{
    constexpr int kSc0Sc1 = 17;
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, x), make_rsrc(dst, tile_halves(D)), at * 2, 0, kSc0Sc1);
}

template <int D>
__global__ __launch_bounds__(256) void prepare_kernel(PromptArgs a, _Float16 *__restrict__ tiles, TileMeta *__restrict__ metas)
{
    constexpr int E = D / 8;                     // values a thread holds of its row
    __shared__ float rows[kTileKeys][D + 1];
    __shared__ float red[4][2];
    __shared__ int factor[kTileKeys], any_odd;
    const int slot = blockIdx.x, head = blockIdx.y, tid = threadIdx.x;
    const bool values = blockIdx.z != 0;
    const int b = seq_of_slot(a.cu, (int)a.T, a.B, kTileKeys, slot);
    const SeqRange r = seq_range(a.cu, (int)a.T, b);
    const int len = r.end - r.begin, tile = slot - first_slot(r.begin, b, kTileKeys);
    if (tile < 0 || tile * kTileKeys >= len) return;
    const int row = tid >> 3, seg = tid & 7, key = tile * kTileKeys + row;
    const float *src = (values ? a.v + (int64_t)(r.begin + key) * a.v_stride : a.k + (int64_t)(r.begin + key) * a.k_stride) +
                       head * D + seg * E;
    float x[E], top = 0.0f;
    bool odd = false;                            // not finite
    if (tid == 0) any_odd = 0;
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
        f4 y = {0.0f, 0.0f, 0.0f, 0.0f};
        if (key < len) y = reinterpret_cast<const f4 *>(src)[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[4 * i + j] = y[j];
            top = fmaxf(top, finite_abs(y[j]));
            odd |= !(fabsf(y[j]) <= kBig);
        }
    }
    top = max_dpp<0xB1>(top);                    // the row's 8 lanes: quad_perm 1 0 3 2, 2 3 0 1, row_half_mirror
    top = max_dpp<0x4E>(top);
    top = max_dpp<0x141>(top);
    // the tile's largest row and smallest one that is not zero
    float most = top, least = top > 0.0f ? -top : -kBig;
    most = max_dpp<0x128>(most);                 // row_ror:8
    least = max_dpp<0x128>(least);
#pragma unroll
    for (int o = 16; o < 64; o <<= 1) {
        most = fmaxf(most, __shfl_xor(most, o));
        least = fmaxf(least, __shfl_xor(least, o));
    }
    if ((tid & 63) == 0) {
        red[tid >> 6][0] = most;
        red[tid >> 6][1] = least;
    }
    if (values) {
#pragma unroll
        for (int i = 0; i < E; ++i) rows[row][seg * E + i] = x[i];
    }
    __syncthreads();
    if (odd) any_odd = 1;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        most = fmaxf(most, red[w][0]);
        least = fmaxf(least, red[w][1]);
    }
    const int e = normaliser(most, 15);
    const bool wild = most > 0.0f && normaliser(-least, 15) - e > kWildBits;
    const int er = wild ? normaliser(top, 15) : e;
    const int64_t at = (int64_t)slot * a.kv_heads + head;
    TileMeta *m = metas + at;
    _Float16 *dst = tiles + at * tile_halves(D);
    if (!values) {
        if (tid == 0) {
            m->k_exp = e;
            m->k_flags = wild ? kWildK : 0;
        }
        if (seg == 0) m->k_row[row] = er;
        // fragment f covers values 16 f .. 16 f + 15; lane (key, half) holds 8 of them
#pragma unroll
        for (int c = 0; c < E / 8; ++c) {
            const int d0 = seg * E + 8 * c, f = d0 >> 4, half = (d0 >> 3) & 1;
            h8 hi, lo;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                _Float16 y, z;
                split(ldexpf(x[8 * c + j], er), y, z);
                hi[j] = y;
                lo[j] = z;
            }
            const int o = f * 512 + (half * 32 + row) * 8;
            store_through<D>(dst, o, hi);
            store_through<D>(dst, D * kTileKeys + o, lo);
        }
        return;
    }
    if (seg == 0) {
        m->v_row[row] = top > 0.0f ? -er : kNoExp;
        factor[row] = er;
    }
    __syncthreads();
    if (tid == 0) {
        m->v_exp = most > 0.0f ? -e : kNoExp;
        m->v_flags = (wild ? kWildV : 0) | (any_odd ? kOddV : 0);
    }
    // fragment (db, s) covers values 32 db .. + 31 and 16 keys; lane (d, half) holds the keys that the scores' lane
    // of that half holds: 16 s + 8 (e / 4) + 4 half + e % 4
    dst += 2 * D * kTileKeys;
#pragma unroll
    for (int i = 0; i < D * kTileKeys / 8 / 256; ++i) {
        const int c = tid + 256 * i, lane = c & 63, f = c >> 6;
        const int d = (f >> 1) * 32 + (lane & 31), k0 = (f & 1) * 16 + 4 * (lane >> 5);
        h8 hi, lo;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int u = k0 + 8 * (j >> 2) + (j & 3);
            const float y = rows[u][d];
            _Float16 p, z;
            split(fabsf(y) <= kBig ? ldexpf(y, factor[u]) : 0.0f, p, z);
            hi[j] = p;
            lo[j] = z;
        }
        store_through<D>(dst, c * 8, hi);
        store_through<D>(dst, D * kTileKeys + c * 8, lo);
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
    f16v o[D / 32];                  // value 32 db + 8 (i / 4) + 4 half + i % 4
    float m, l;                      // running maximum (log2), sum of weights of this lane's keys
    int q_exp;                       // scores are 2^(q_exp - k_exp) times the products
    int v_exp;                       // o is in units of 2^(v_exp - kWeightBits)
    float f, up, unit;               // of the tile at hand: weight = 2^(f score + up), worth `unit` of 1
};

template <int D>
struct Query {
    h8 q1[D / 16], q2[D / 16];
};

// The lane's half of 16 F values of a query, and the largest of both halves.
template <int F>
__device__ __forceinline__ float load_query(float (&x)[F][8], const float *q, bool live, int half)
{
    float top = 0.0f;
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
            if (live) v = *reinterpret_cast<const f4 *>(q + 16 * f + 8 * half + 4 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[f][4 * i + j] = v[j];
        }
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, finite_abs(x[f][j]));
    return fmaxf(top, other_half(top));
}

// Starts the rows' state; the power of two that brings the query, `top` its
// largest value, below 2^14.
template <int D>
__device__ __forceinline__ int start_rows(Rows<D> &s, float top, int c_exp)
{
    const int e = normaliser(top, 14);
    s.q_exp = c_exp - e;
#pragma unroll
    for (int db = 0; db < D / 32; ++db) s.o[db] = f16v{};
    s.m = -3.0e38f;
    s.l = 0.0f;
    s.v_exp = kNoExp;
    return e;
}

// Operands of 16 values of the query: |c_man| < 2 keeps the products below 2^15.
__device__ __forceinline__ void split_query(const float (&x)[8], int e, float c_man, h8 &q1, h8 &q2)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        _Float16 hi, lo;
        split(ldexpf(x[j], e) * c_man, hi, lo);
        q1[j] = hi;
        q2[j] = lo;
    }
}

// Scores of a tile: k' operands in LDS or global memory.
template <int D>
__device__ __forceinline__ f16v scores(const Query<D> &s, const h8 *k1)
{
    const h8 *k2 = k1 + D * kTileKeys / 8;
    f16v x = {};
#pragma unroll
    for (int f = 0; f < D / 16; ++f) {
        const h8 a1 = k1[64 * f], a2 = k2[64 * f];
        x = mfma(a2, s.q1[f], x);
        x = mfma(a1, s.q2[f], x);
        x = mfma(a1, s.q1[f], x);
    }
    return x;
}

// The same from k in registers (k1 then k2) and queries in LDS (q1 then q2).
template <int D>
__device__ __forceinline__ f16v scores(const h8 *q, const h8 (&k)[D / 8])
{
    f16v x = {};
#pragma unroll
    for (int f = 0; f < D / 16; ++f) {
        const h8 b1 = q[64 * f], b2 = q[64 * (D / 16 + f)];
        x = mfma(k[D / 16 + f], b1, x);
        x = mfma(k[f], b2, x);
        x = mfma(k[f], b1, x);
    }
    return x;
}

// A tile's scores made ready: rows of wild k scaled, keys this query does not
// see masked (where `edge`; `first`: position of the tile's first key minus
// that of this lane's query), the running maximum and the units of the output
// moved where they have to be. Leaves in s.f and s.up what turns a score into a
// weight.
template <int D>
__device__ __forceinline__ void settle(Rows<D> &s, f16v &x, TileHead h, const TileMeta *meta, bool edge, int first, int half)
{
    const int flags = h.flags;
    int e = s.q_exp - h.k_exp, ve = h.v_exp;
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
    // (never 0: times a masked key's -inf that is no number. Products are below 2^38, so such scores are as good as equal)
    const float f = ldexpf(1.0f, e > 127 ? 127 : e < -126 ? -126 : e);
    float top = fmaxf(x[0], x[1]);
#pragma unroll
    for (int i = 2; i < 16; ++i) top = fmaxf(top, x[i]);
    top = fmaxf(top, other_half(top)) * f;
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
    // weights in units of 2^-(kWeightBits + d), d <= 0 the distance of this tile's values below the largest (none for
    // values of zero, whose weights only count in the sum)
    const int d = (flags & kWildV) || ve == kNoExp ? 0 : ve - s.v_exp < -60 ? -60 : ve - s.v_exp;
    s.f = f;
    s.up = (float)(kWeightBits + d) - s.m;
    s.unit = ldexpf(1.0f, -kWeightBits - d);
}

// Scores become weights, and their sum is taken.
template <int D>
__device__ __forceinline__ void weigh(Rows<D> &s, f16v &x)
{
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        x[i] = __builtin_amdgcn_exp2f(fmaf(x[i], s.f, s.up));
        sum += x[i];
    }
    s.l = fmaf(sum, s.unit, s.l);
}

__device__ __forceinline__ void split8(const f16v &x, int t, h8 &p1, h8 &p2)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        _Float16 hi, lo;
        split(x[8 * t + i], hi, lo);
        p1[i] = hi;
        p2[i] = lo;
    }
}

// Adds the weighted values of a tile, 16 keys at a time.
template <int D>
__device__ __forceinline__ void accumulate(Rows<D> &s, const h8 *v1, int t, h8 p1, h8 p2)
{
    const h8 *v2 = v1 + D * kTileKeys / 8;
#pragma unroll
    for (int db = 0; db < D / 32; ++db) {
        const h8 a1 = v1[64 * (2 * db + t)], a2 = v2[64 * (2 * db + t)];
        s.o[db] = mfma(a2, p1, s.o[db]);
        s.o[db] = mfma(a1, p2, s.o[db]);
        s.o[db] = mfma(a1, p1, s.o[db]);
    }
}

// The same from v in registers (v1 then v2), all 32 keys.
template <int D>
__device__ __forceinline__ void accumulate_held(Rows<D> &s, const h8 (&v)[D / 8], const f16v &x)
{
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        h8 p1, p2;
        split8(x, t, p1, p2);
#pragma unroll
        for (int db = 0; db < D / 32; ++db) {
            s.o[db] = mfma(v[D / 16 + 2 * db + t], p1, s.o[db]);
            s.o[db] = mfma(v[2 * db + t], p2, s.o[db]);
            s.o[db] = mfma(v[2 * db + t], p1, s.o[db]);
        }
    }
}

// Weights of a tile with wild v, whose rows have a factor each.
template <int D>
__device__ __forceinline__ void weigh_rows(const Rows<D> &s, f16v &x, const TileMeta *meta, int half)
{
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int r = meta->v_row[8 * (i >> 2) + 4 * half + (i & 3)] - s.v_exp;
        x[i] = ldexpf(x[i], r < 0 ? r : 0);
    }
}

// Values that are not finite (0 in the operands): counts, for each output, the
// visible ones as a product of two masks.
template <int D>
__device__ __forceinline__ void odd_values(Rows<D> &s, bool edge, int first, const float *v_rows, int64_t v_stride,
                                           int live_keys, int lane)
{
    const int half = lane >> 5;
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
    Query<D> q;
    {
        float x[D / 16][8];
        const int e = start_rows<D>(s, load_query(x, a.q + (int64_t)(r.begin + pos) * a.q_stride + head * D, live, half), c_exp);
#pragma unroll
        for (int f = 0; f < D / 16; ++f) split_query(x[f], e, c_man, q.q1[f], q.q2[f]);
    }
    // last tile of the block
    const int last = __builtin_amdgcn_readfirstlane((len - 1 < row0 + kRows - 1 ? len - 1 : row0 + kRows - 1) / kTileKeys);
    const int step = a.kv_heads, at0 = __builtin_amdgcn_readfirstlane(first_slot(r.begin, b, kTileKeys) * step + kvh);
    // k of tile t is wanted one step before v of tile t: two buffers of each, t & 1
    auto copy = [&](int tile, int values) {
        const char *src = reinterpret_cast<const char *>(tiles + (int64_t)(at0 + tile * step) * tile_halves(D)) + values * (kBytes / 2) +
                          wave * 1024 + lane * 16;
        char *dst = reinterpret_cast<char *>(buf[tile & 1]) + values * (kBytes / 2) + wave * 1024;
#pragma unroll
        for (int i = 0; i < kBytes / 2048 / W; ++i)
            __builtin_amdgcn_global_load_lds(
                (const __attribute__((address_space(1))) void *)(src + i * 1024 * W),
                (__attribute__((address_space(3))) void *)(dst + i * 1024 * W), 16, 0, 0);
    };
    auto meet = [&]() {                          // this wave's copies have arrived, its reads are done; so have all waves'
        __builtin_amdgcn_s_waitcnt(0x0070);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    const int mine = wrow < len ? wrow / kTileKeys : -1;         // this wave's last tile
    int odd = 0;
    copy(0, 0);
    TileHead now = head_of(metas + at0), next = head_of(metas + at0 + (last > 0 ? step : 0));
    meet();
    copy(0, 1);
    if (last > 0) copy(1, 0);
    f16v x = {};
    if (mine >= 0) {
        x = scores<D>(q, reinterpret_cast<const h8 *>(buf[0]) + lane);
        settle<D>(s, x, now, metas + at0, mine == 0, -pos, half);
    }
    for (int t = 0; t <= last; ++t) {
        const TileHead after = head_of(metas + at0 + (t + 2 <= last ? t + 2 : last) * step);
        meet();                                  // v of tile t and k of tile t + 1
        if (t < last) copy(t + 1, 1);
        if (t + 1 < last) copy(t + 2, 0);
        if (t <= mine) {
            const TileMeta *meta = metas + at0 + t * step;
            const int flags = now.flags;
            const h8 *v1 = reinterpret_cast<const h8 *>(buf[t & 1]) + 2 * D * kTileKeys / 8 + lane;
            const h8 *k1 = reinterpret_cast<const h8 *>(buf[(t + 1) & 1]) + lane;
            // the next tile's scores are computed while this one's become weights (after the last tile: of
            // whatever the buffer holds, to no use)
            f16v y;
            h8 p1[2], p2[2];
            if (flags == 0) {
                y = scores<D>(q, k1);
                weigh<D>(s, x);
                split8(x, 0, p1[0], p2[0]);
                split8(x, 1, p1[1], p2[1]);
                // one matrix instruction, the vector instructions that fit beside it, and the reads of a later one
                __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
                for (int i = 0; i < 3 * D / 16; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x402, 128 / (3 * D / 16), 0);
                    if (i % 3 != 2) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                }
            } else {
                weigh<D>(s, x);
                if (flags & kWildV) weigh_rows<D>(s, x, meta, half);
                split8(x, 0, p1[0], p2[0]);
                split8(x, 1, p1[1], p2[1]);
                y = scores<D>(q, k1);
            }
            accumulate<D>(s, v1, 0, p1[0], p2[0]);
            accumulate<D>(s, v1, 1, p1[1], p2[1]);
            odd |= flags & kOddV;
            if (t < mine) {
                x = y;
                settle<D>(s, x, next, meta + step, t + 1 == mine, (t + 1) * kTileKeys - pos, half);
            }
        }
        now = next;
        next = after;
    }
    if (odd)                                     // (apart from the loop, whose registers it would take)
        for (int t = 0; t <= mine; ++t)
            if (metas[at0 + t * step].v_flags & kOddV)
                odd_values<D>(s, t == mine, t * kTileKeys - pos,
                              a.v + (int64_t)(r.begin + t * kTileKeys) * a.v_stride + kvh * D, a.v_stride,
                              len - t * kTileKeys, lane);
    if (wrow < len)
        store_rows<D>(s, live ? a.out + (int64_t)(r.begin + pos) * a.out_stride + head * D : nullptr, half);
}

// Few rows: the 4 wavefronts of a workgroup share 32 rows and take every fourth
// tile each, so that short prompts fill the card and no wavefront walks far; what
// they found is joined through LDS, where the queries, the same for all, stay
// until then.
constexpr int kShare = 4;

constexpr int result_pitch(int D) { return D + 4; }             // floats between rows of results
struct RowSums {
    float top[kShare][32], sum[kShare][32];
};

// Where a workgroup's rows are.
struct Block {
    int head, kvh, b, last;                      // last: block of 32 rows within sequence b, and its last tile
    SeqRange r;
    int len, row0;
};

__device__ __forceinline__ Block find_block(const PromptArgs &a, int slots)
{
    Block x;
    const int id = blockIdx.x, group = a.heads / a.kv_heads, hp = id % a.heads;
    x.kvh = hp % a.kv_heads;
    x.head = x.kvh * group + hp / a.kv_heads;
    // long blocks first, then short ones: a compute unit that begins with a long one gets a short one beside it
    const int rank = id / a.heads, slot = rank < (slots + 1) / 2 ? slots - 1 - rank : rank - (slots + 1) / 2;
    x.b = seq_of_slot(a.cu, (int)a.T, a.B, 32, slot);
    x.r = seq_range(a.cu, (int)a.T, x.b);
    x.len = x.r.end - x.r.begin;
    x.last = __builtin_amdgcn_readfirstlane(slot - first_slot(x.r.begin, x.b, 32));
    x.row0 = x.last * 32;
    return x;
}

// Each wavefront brings its share of every row's values, D / 4 side by side, into
// LDS (q1 then q2; qs: this lane's part); `between` runs while they are under way. The caller lets all waves meet.
template <int D, typename F>
__device__ __forceinline__ void share_queries(Rows<D> &s, h8 *qs, RowSums &sh, const float *q, bool live, float c_man, int c_exp,
                                              int lane, int wave, F between)
{
    constexpr int P = D / 16 / kShare;
    const int half = lane >> 5;
    float x[P][8];
    float most = load_query<P>(x, q + wave * (D / kShare), live, half);
    between();
    if (half == 0) sh.top[wave][lane] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kShare; ++w) most = fmaxf(most, sh.top[w][lane & 31]);
    const int e = start_rows<D>(s, most, c_exp);
#pragma unroll
    for (int f = 0; f < P; ++f) split_query(x[f], e, c_man, qs[64 * (wave * P + f)], qs[64 * (D / 16 + wave * P + f)]);
}

// Results in units of the largest maximum (the queries have been read when all meet).
template <int D>
__device__ __forceinline__ void join_rows(const PromptArgs &a, const Block &x, const Rows<D> &s, float *res, RowSums &sh, int lane, int wave)
{
    constexpr int kPitch = result_pitch(D);
    const int half = lane >> 5;
    if (half == 0) sh.top[wave][lane] = s.m;
    __syncthreads();
    float m = sh.top[0][lane & 31];
#pragma unroll
    for (int w = 1; w < kShare; ++w) m = fmaxf(m, sh.top[w][lane & 31]);
    const float by = __builtin_amdgcn_exp2f(s.m - m), l = (s.l + other_half(s.l)) * by;
    if (half == 0) sh.sum[wave][lane] = l;
    float *mine = res + (wave * 32 + (lane & 31)) * kPitch + 4 * half;
#pragma unroll
    for (int db = 0; db < D / 32; ++db)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            f4 y;
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = ldexpf(s.o[db][4 * g + j] * by, s.v_exp - kWeightBits);
            *reinterpret_cast<f4 *>(mine + 32 * db + 8 * g) = y;
        }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < 32 * D / 4 / (64 * kShare); ++n) {
        const int i = threadIdx.x + n * 64 * kShare, row = i / (D / 4), d = i % (D / 4) * 4;
        f4 y = *reinterpret_cast<const f4 *>(res + row * kPitch + d);
        float total = sh.sum[0][row];
#pragma unroll
        for (int w = 1; w < kShare; ++w) {
            y += *reinterpret_cast<const f4 *>(res + (w * 32 + row) * kPitch + d);
            total += sh.sum[w][row];
        }
        if (x.row0 + row < x.len)
            *reinterpret_cast<f4 *>(a.out + (int64_t)(x.r.begin + x.row0 + row) * a.out_stride + x.head * D + d) = y * (1.0f / total);
    }
}

// Prepared k and v come from L2 straight into registers, a tile ahead.
template <int D>
__global__ __launch_bounds__(64 * kShare, 2) void attend_shared_kernel(PromptArgs a, const _Float16 *__restrict__ tiles,
                                                                      const TileMeta *__restrict__ metas, float c_man,
                                                                      int c_exp, int slots)
{
    constexpr int F = D / 8;                     // operands of k or v (both parts)
    __shared__ __attribute__((aligned(16))) float res[kShare * 32 * result_pitch(D)];           // until the join: queries
    __shared__ RowSums sh;
    const Block x = find_block(a, slots);
    if (x.row0 < 0 || x.row0 >= x.len) return;
    const int lane = threadIdx.x & 63, half = lane >> 5, last = x.last;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int pos = x.row0 + (lane & 31);
    const int step = a.kv_heads, at0 = __builtin_amdgcn_readfirstlane(first_slot(x.r.begin, x.b, kTileKeys) * step + x.kvh);
    auto load = [&](int tile, int values, h8 (&y)[F]) {
        const h8 *src = reinterpret_cast<const h8 *>(tiles + (int64_t)(at0 + tile * step) * tile_halves(D)) + values * (2 * D * kTileKeys / 8);
#pragma unroll
        for (int f = 0; f < F; ++f) y[f] = (src + 64 * f)[lane];
    };
    const auto head_at = [&](int t) { return head_of(metas + at0 + (t <= last ? t : last) * step); };
    h8 k[F], v[F];
    TileHead now = head_at(wave);
    int odd = 0;
    Rows<D> s;
    h8 *const qs = reinterpret_cast<h8 *>(res) + lane;
    share_queries<D>(s, qs, sh, a.q + (int64_t)(x.r.begin + pos) * a.q_stride + x.head * D, pos < x.len, c_man, c_exp, lane, wave,
                     [&]() { if (wave <= last) load(wave, 0, k); });
    if (wave <= last) load(wave, 1, v);
    __syncthreads();
    for (int t = wave; t <= last; t += kShare) {
        const TileMeta *meta = metas + at0 + t * step;
        const TileHead next = head_at(t + kShare);
        const bool edge = t == last;
        const int first = t * kTileKeys - pos;
        __builtin_amdgcn_sched_barrier(0);
        f16v y = scores<D>(qs, k);
        // two reads of queries ahead, not all of them: registers are what is short
        __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
        for (int f = 0; f < D / 16; ++f) {
            __builtin_amdgcn_sched_group_barrier(0x008, 3, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        }
        __builtin_amdgcn_sched_barrier(0);       // (moved up, the loads would need registers of their own)
        if (t + kShare <= last) load(t + kShare, 0, k);
        settle<D>(s, y, now, meta, edge, first, half);
        weigh<D>(s, y);
        if (now.flags & kWildV) weigh_rows<D>(s, y, meta, half);
        accumulate_held<D>(s, v, y);
        __builtin_amdgcn_sched_barrier(0);
        if (t + kShare <= last) load(t + kShare, 1, v);
        odd |= now.flags & kOddV;
        now = next;
    }
    if (odd)                                     // (apart from the loop, whose registers it would take)
        for (int t = wave; t <= last; t += kShare)
            if (metas[at0 + t * step].v_flags & kOddV)
                odd_values<D>(s, t == last, t * kTileKeys - pos,
                              a.v + (int64_t)(x.r.begin + t * kTileKeys) * a.v_stride + x.kvh * D, a.v_stride,
                              x.len - t * kTileKeys, lane);
    join_rows<D>(a, x, s, res, sh, lane, wave);
}

// ---------------------------------------------------------------- attend, without prepare
// Very few rows: a launch costs more than splitting k and v where they are used.
// As attend_shared_kernel, but every wavefront copies its own tiles as they are
// into LDS and splits them on the way to the operands: rows for k and for the
// maxima of v, columns for v. 16-byte pieces of a row are swizzled by row.
__device__ __forceinline__ float wave_max(float x)             // over 32 lanes; both halves hold the same
{
    x = max_dpp<0xB1>(x);                        // quad_perm 1 0 3 2, 2 3 0 1, row_half_mirror, row_ror:8
    x = max_dpp<0x4E>(x);
    x = max_dpp<0x141>(x);
    x = max_dpp<0x128>(x);
    return fmaxf(x, __shfl_xor(x, 16));
}

// Largest magnitude of a row, half of it per lane, what is not finite left out; `odd`: there was some.
template <int D>
__device__ __forceinline__ float row_top(const float (&x)[D / 16][8], bool &odd)
{
    float top = 0.0f;
#pragma unroll
    for (int f = 0; f < D / 16; ++f)
#pragma unroll
        for (int j = 0; j < 8; ++j) top = __builtin_elementwise_maximum(top, fabsf(x[f][j]));       // (a NaN stays)
    odd = !(top <= kBig);
    if (__any(odd)) {
        top = 0.0f;
#pragma unroll
        for (int f = 0; f < D / 16; ++f)
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fmaxf(top, finite_abs(x[f][j]));
    }
    return fmaxf(top, other_half(top));
}

// Values times a power of two that is no number by itself; by: 1 from then on.
template <int F>
__device__ __forceinline__ void scale_row(float (&x)[F][8], int e, float &by)
{
    by = 1.0f;
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[f][j] = ldexpf(x[f][j], e);
}

__device__ __forceinline__ void split_by(const float (&x)[8], float by, h8 &y1, h8 &y2)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        _Float16 hi, lo;
        split(x[j] * by, hi, lo);
        y1[j] = hi;
        y2[j] = lo;
    }
}

struct Factors {
    int tile, row;                               // powers of two of the tile, and of this lane's row
    bool wild, zero;                             // zero: the whole tile
};

__device__ __forceinline__ Factors factors(float top)
{
    const float most = wave_max(top), least = wave_max(top > 0.0f ? -top : -kBig);
    Factors f;
    f.tile = __builtin_amdgcn_readfirstlane(normaliser(most, 15));
    f.zero = !__builtin_amdgcn_readfirstlane(most > 0.0f);
    f.wild = most > 0.0f && __builtin_amdgcn_readfirstlane(normaliser(-least, 15)) - f.tile > kWildBits;
    f.row = f.wild ? normaliser(top, 15) : f.tile;
    return f;
}

template <int D>
__global__ __launch_bounds__(64 * kShare, 1) void attend_direct_kernel(PromptArgs a, float c_man, int c_exp, int slots)
{
    constexpr int C = D / 4, kTileFloats = kTileKeys * D;        // pieces of a row
    static_assert(2 * kTileFloats >= 32 * result_pitch(D), "the results fit the buffers");
    __shared__ __attribute__((aligned(16))) float buf[kShare][2][kTileFloats];      // k and v; after the last tile: results
    __shared__ __attribute__((aligned(16))) h8 queries[D / 8 * 64];
    __shared__ RowSums sh;
    __shared__ TileMeta metas[kShare];
    const Block x = find_block(a, slots);
    if (x.row0 < 0 || x.row0 >= x.len) return;
    const int lane = threadIdx.x & 63, half = lane >> 5, last = x.last;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int pos = x.row0 + (lane & 31);
    TileMeta *const meta = &metas[wave];
    const float *const ks = a.k + (int64_t)x.r.begin * a.k_stride + x.kvh * D, *const vs = a.v + (int64_t)x.r.begin * a.v_stride + x.kvh * D;
    // (keys past the end: the last one's values, whose weights are 0)
    auto copy = [&](const float *p, int64_t stride, int tile, float *dst) {
        const float *const end = p + (x.len - 1) * stride, *at = p + (int64_t)(tile * kTileKeys + lane / C) * stride;
#pragma unroll
        for (int i = 0; i < C / 2; ++i) {
            const int piece = (lane % C ^ ((i * (64 / C) + lane / C) & (C - 1))) * 4;
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)((at < end ? at : end) + piece),
                                             (__attribute__((address_space(3))) void *)(dst + i * 256), 16, 0, 0);
            at += 64 / C * stride;
        }
    };
    auto load = [&](int tile) {
        copy(ks, a.k_stride, tile, buf[wave][0]);
        copy(vs, a.v_stride, tile, buf[wave][1]);
    };
    // half of row lane % 32, 8 values in turns
    auto read_row = [&](const float *src, float (&y)[D / 16][8]) {
        const int row = lane & 31;
#pragma unroll
        for (int f = 0; f < D / 16; ++f)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const f4 z = *reinterpret_cast<const f4 *>(src + row * D + ((4 * f + 2 * half + i) ^ (row & (C - 1))) * 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) y[f][4 * i + j] = z[j];
            }
    };
    // as prepare_kernel's fragment f: values 32 (f / 2) + lane % 32 of keys 16 (f % 2) + 8 (j / 4) + 4 half + j % 4
    auto read_column = [&](const float *src, int f, float (&y)[8]) {
        const int piece = ((lane & 31) >> 2) ^ (half << 2);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int u = 16 * (f & 1) + 8 * (j >> 2) + (j & 3);               // and 4 half
            y[j] = src[(u + 4 * half) * D + (piece ^ (j & 3)) * 4 + (lane & 3) + ((8 * (f >> 1)) ^ (u & (C - 8))) * 4];
        }
    };
    bool any_odd = false;
    Rows<D> s;
    h8 *const qs = queries + lane;
    share_queries<D>(s, qs, sh, a.q + (int64_t)(x.r.begin + pos) * a.q_stride + x.head * D, pos < x.len, c_man, c_exp, lane, wave,
                     [&]() { if (wave <= last) load(wave); });
    __syncthreads();
    for (int t = wave; t <= last; t += kShare) {
        const bool edge = t == last;
        const int first = t * kTileKeys - pos;
        __builtin_amdgcn_s_waitcnt(0x0F70);      // vmcnt(0): the tile has arrived
        asm volatile("" ::: "memory");
        float x8[D / 16][8];                     // k's rows, then v's
        bool odd;
        read_row(buf[wave][0], x8);
        const Factors fk = factors(row_top<D>(x8, odd));
        if (half == 0) meta->k_row[lane] = fk.row;
        f16v y = {};
        {
            float by = ldexpf(1.0f, fk.row);
            if (__any(fk.row > 127 || fk.row < -126)) scale_row(x8, fk.row, by);
#pragma unroll
            for (int f = 0; f < D / 16; ++f) {
                h8 k1, k2;
                split_by(x8[f], by, k1, k2);
                const h8 q1 = qs[64 * f], q2 = qs[64 * (D / 16 + f)];
                y = mfma(k2, q1, y);
                y = mfma(k1, q2, y);
                y = mfma(k1, q1, y);
            }
        }
        read_row(buf[wave][1], x8);
        const float top = row_top<D>(x8, odd);
        odd = __any(odd);
        any_odd |= odd;
        const Factors fv = factors(top);
        if (half == 0) meta->v_row[lane] = top > 0.0f ? -fv.row : kNoExp;
        float by = ldexpf(1.0f, fv.tile);
        if (odd || fv.wild || fv.tile > 127 || fv.tile < -126) {
            // v is made what its operands are split of, in place
#pragma unroll
            for (int f = 0; f < D / 16; ++f)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    f4 z;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float w = x8[f][4 * i + j];
                        z[j] = fabsf(w) <= kBig ? ldexpf(w, fv.row) : 0.0f;
                    }
                    *reinterpret_cast<f4 *>(buf[wave][1] + (lane & 31) * D + ((4 * f + 2 * half + i) ^ (lane & (C - 1))) * 4) = z;
                }
            by = 1.0f;
        }
        asm volatile("" ::: "memory");
        const TileHead now = {fk.tile, fv.zero ? kNoExp : -fv.tile, (fk.wild ? kWildK : 0) | (fv.wild ? kWildV : 0)};
        settle<D>(s, y, now, meta, edge, first, half);
        weigh<D>(s, y);
        if (now.flags & kWildV) weigh_rows<D>(s, y, meta, half);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            h8 p1, p2;
            split8(y, h, p1, p2);
#pragma unroll
            for (int db = 0; db < D / 32; ++db) {
                float z[8];
                h8 v1, v2;
                read_column(buf[wave][1], 2 * db + h, z);
                split_by(z, by, v1, v2);
                s.o[db] = mfma(v2, p1, s.o[db]);
                s.o[db] = mfma(v1, p2, s.o[db]);
                s.o[db] = mfma(v1, p1, s.o[db]);
            }
        }
        if (t + kShare <= last) {
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): read, the buffers may be filled again
            load(t + kShare);
        }
    }
    if (any_odd)
        for (int t = wave; t <= last; t += kShare)
            odd_values<D>(s, t == last, t * kTileKeys - pos, vs + (int64_t)(t * kTileKeys) * a.v_stride, a.v_stride,
                          x.len - t * kTileKeys, lane);
    join_rows<D>(a, x, s, buf[0][0], sh, lane, wave);
}

inline uint64_t round256(uint64_t x) { return (x + 255) / 256 * 256; }
inline uint64_t meta_bytes(int64_t slots, int64_t kv_heads) { return round256((uint64_t)slots * kv_heads * sizeof(TileMeta)); }

// Up to so many workgroups of 128 rows, prompts run on the kernel whose wavefronts
// share 32 rows; of several prompts, whose lengths will differ, more, since a long one's
// last rows would be walked by few wavefronts. Measured, both kernels (us, shared / other): 16
// heads of 128, one prompt of 1024 (144 groups) 32 / 64, 2048 (272) 85 / 117, 3000 (384)
// 154 / 173, 4096 (528) 264 / 266; 64 heads, 1024 tokens (576) 85 / 78; 8 prompts of 256 (384)
// 33 / 36, 12 (576) 44 / 43; of different lengths, 4 of 4094 in all (560) 139 / 156, 13 of
// 4997 (832) 102 / 105, 24 of 4085 (880) 68 / 80, 24 of 7990 (1376) 134 / 125; 12 heads, 8 of
// 3998 (468) 70 / 101. Heads of 64: one prompt of 4096 (528) 141 / 170, 8 of 1024 (1152) 97 / 96, 16
// of 7991 (1248) 85 / 106, 24 of 7989 (1204) 64 / 67, 8 of 15995 (2112) 1012 / 932. The limit of
// 1200 lies between what many prompts and one would have: 24 of 7977 (1204) 60 / 68, 16 of 7982
// (1248) 104 / 118, but one of 9700 (1216) 690 / 658, of 11300 (1246) 812 / 789. The number of
// prompts stands for how their lengths differ, which only the device knows: one long prompt
// beside empty ones counts as several.
inline int64_t few_groups(int D, int64_t B) { return D == 64 ? 1200 : B >= 4 ? 880 : 528; }

// Prompts so short are not prepared: no wavefront has more than one tile of 128 values (two of
// 64), and the workgroups, whose k and v fill a compute unit's LDS (half of it), run at
// once. Measured (us on the device, without / with; from the host a call costs 9 / 14 at least): 16
// heads of 128, 128 tokens (80 workgroups) 10.9 / 11.4, 192 (112) 15.9 / 13.1, 4 x 32 (128)
// 10.6 / 11.4; 64 heads, 128 tokens (320) 11.5 / 11.7; 14 heads of 64, 128 tokens (70)
// 7.4 / 8.6, 256 (126) 10.3 / 9.9; 16 heads of 128, 16 x 32 (512) 20 / 13.
inline bool direct(int64_t T, int64_t B, int64_t heads, int64_t head_dim)
{
    return T * head_dim <= 16384 && tile_slots(T, B, 32) * heads * head_dim <= 40960;
}

template <int D>
hipError_t launch(const PromptArgs &a, hipStream_t stream)
{
    constexpr int W = 4;
    int c_exp = 0;
    const double c = frexp((double)a.scale * 1.4426950408889634, &c_exp);      // softmax in powers of two
    const int64_t slots = tile_slots(a.T, a.B, kTileKeys);
    if (direct(a.T, a.B, a.heads, D)) {
        attend_direct_kernel<D><<<(unsigned)(slots * a.heads), 64 * kShare, 0, stream>>>(a, (float)(2.0 * c), c_exp - 1, (int)slots);
        return hipGetLastError();
    }
    TileMeta *metas = reinterpret_cast<TileMeta *>(a.ws);
    _Float16 *tiles = reinterpret_cast<_Float16 *>((char *)a.ws + meta_bytes(slots, a.kv_heads));
    prepare_kernel<D><<<dim3((unsigned)slots, (unsigned)a.kv_heads, 2), 256, 0, stream>>>(a, tiles, metas);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t rows = tile_slots(a.T, a.B, 32 * W);
    if (rows * a.heads <= few_groups(D, a.B)) {
        const int64_t blocks = tile_slots(a.T, a.B, 32);
        attend_shared_kernel<D><<<(unsigned)(blocks * a.heads), 64 * kShare, 0, stream>>>(a, tiles, metas, (float)(2.0 * c),
                                                                                          c_exp - 1, (int)blocks);
        return hipGetLastError();
    }
    attend_kernel<D, W><<<(unsigned)(rows * a.heads), 64 * W, 0, stream>>>(a, tiles, metas, (float)(2.0 * c), c_exp - 1, (int)rows);
    return hipGetLastError();
}

}  // namespace

uint64_t prompt_ws_bytes(int64_t T, int64_t B, int64_t heads, int64_t kv_heads, int64_t head_dim)
{
    if (direct(T, B, heads, head_dim)) return 0;
    const int64_t slots = tile_slots(T, B, kTileKeys);
    return meta_bytes(slots, kv_heads) + (uint64_t)slots * kv_heads * tile_halves((int)head_dim) * 2;
}

hipError_t launch_attn_prefill(const PromptArgs &a, hipStream_t stream)
{
    return a.head_dim == 128 ? launch<128>(a, stream) : launch<64>(a, stream);
}

}  // namespace wq
