// Score modifications of block-sparse attention: tanh cap, distance bias,
// document and order masks.  For a query token i and a key token j of one head,
//   s = q_i . k_j / sqrt(d)
//   s <- cap tanh(s / cap)                                  (cap > 0)
//   s <- s - slope (wt |dt| + wh |dy| + ww |dx|)            (0 where i or j is a text token)
//   j is visible to i iff doc_j == doc_i >= 0 and order_j <= order_i.
//
// token_info_kernel lays the per-token values out in permuted order, so that
// one 64-key block's values are one contiguous piece, and summarises every
// block (range of documents and of orders): a pair of blocks none of whose
// token pairs is visible is left out of the attention's list before any of
// its work, and one whose pairs are all visible skips the per-score mask.
#pragma once
#include "geometry.cuh"
#include "ptx.cuh"

namespace rf2 {

struct TokenInfo {
    int2* mask;          // [B][T_b][kMaskSlots]: (document, order) of the 64 tokens (document < 0: padding, and past
                         // the sequence's end), then the block's summary again
    float4* pos;         // [T_b][kPosSlots]: (wt t, wh y, ww x, 1 for video tokens, 0 for text) of the 64 tokens,
                         // of the first token of every 4, and (1 if they give the others, else 0) at the end
    int4* summary;       // [B][T_b] (document min, max, order min, max); documents include padding as -1
};

// Modifications a kernel is compiled with.
constexpr int kModMask = 1, kModCap = 2, kModBias = 4;

constexpr int kMaskSlots = 64 + 2, kPosSlots = 64 + 16 + 1;

struct ModArgs {
    TokenInfo info;
    float cap_in;        // 1 / (sqrt(d) cap), 0 without the cap
    float cap;           // 0 without the cap
    float small;         // |product| up to which cap_small serves: half the cap in score units (0: never)
    float cap_small[4];  // log2(e) cap tanh(s cap_in) = s sum_k cap_small[k] s^2k there
    float cap_rcp2;      // -1 / (log2(e) cap)^2
    float step;          // ww: the position step between neighbours along x
    const float* slopes; // [heads] or null
    int32_t heads;
    int32_t masked;      // a document or order mask is given
};

constexpr float kLog2e = 1.4426950408889634f;

// (tanh x, 1 - tanh^2 x) from one exponential and one reciprocal: with
// e = e^(-2|x|) and r = 1 / (1 + e), |tanh x| = (1 - e) r and 1 - tanh^2 x =
// 4 e r^2.  The absolute error of tanh stays near 2^-22 (the hardware's
// tanh.approx has 2^-11, which times a cap of 50 would move scores by 0.02);
// the derivative is not formed by subtraction, so its error is relative: a few
// 1e-6 up to |x| = 10, where 1 - t t of a rounded t has no correct digit.
__device__ __forceinline__ float2 tanh_exp(float x)
{
    const float e = ex2_approx(fabsf(x) * (-2.f * kLog2e));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + 1.f));
    return make_float2(copysignf((1.f - e) * r, x), 4.f * e * (r * r));
}

// tanh(x) = x p(x^2) for |x| <= 1, p the minimax polynomial (relative error
// below 6.2e-7, fitted by Remez exchange); two lanes at a time.  The special
// function unit, which gives 4 results per cycle and SM sub-partition, is the
// scarce one next to a softmax: tanh_exp takes it twice per score, the
// polynomial leaves it to the exponential.
__device__ __forceinline__ float2 tanh_poly(float2 x)
{
    const float2 u = fmul2(x, x);
    float2 p = ffma2(u, make_float2(-0.003067060373723507f, -0.003067060373723507f),
                     make_float2(0.016743114218115807f, 0.016743114218115807f));
    p = ffma2(u, p, make_float2(-0.051605675369501114f, -0.051605675369501114f));
    p = ffma2(u, p, make_float2(0.13281433284282684f, 0.13281433284282684f));
    p = ffma2(u, p, make_float2(-0.3332904279232025f, -0.3332904279232025f));
    p = ffma2(u, p, make_float2(0.9999994039535522f, 0.9999994039535522f));
    return fmul2(x, p);
}

// One warp per block: lane l has tokens l and l + 32.
struct TokenInfoArgs {
    TokenInfo out;
    PermGeo g;
    int32_t B, Tb;
    const int32_t* document;
    const int32_t* order;
    float wt, wh, ww;
    int32_t masked, biased;
};

__device__ __forceinline__ void token_info(const TokenInfoArgs& a, int64_t w)
{
    const int lane = threadIdx.x & 31;
    const int32_t B = a.B, Tb = a.Tb;
    if (w >= (int64_t)B * Tb) return;
    const PermGeo& g = a.g;
    const TokenInfo& out = a.out;
    const int32_t* __restrict__ document = a.document;
    const int32_t* __restrict__ order = a.order;
    const float wt = a.wt, wh = a.wh, ww = a.ww;
    const int32_t masked = a.masked, biased = a.biased;
    const int32_t b = (int32_t)(w / Tb), j = (int32_t)(w - (int64_t)b * Tb);
    int dmin = INT32_MAX, dmax = -1, omin = INT32_MAX, omax = INT32_MIN;
    #pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int32_t p = j * kBlock + 32 * k + lane;
        int2 m = make_int2(-1, INT32_MAX);
        float4 pos = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p < g.N) {
            const int32_t src = perm_src(g, p);
            if (masked) {
                m.x = document ? max(__ldg(document + (int64_t)b * g.N + src), -1) : 0;
                m.y = order ? __ldg(order + (int64_t)b * g.N + src) : 0;
                dmin = min(dmin, m.x);
                dmax = max(dmax, m.x);
                if (m.x >= 0) { omin = min(omin, m.y); omax = max(omax, m.y); }
            }
            if (src < g.Nv) {
                const int32_t t = src / g.HW, hw = src - t * g.HW, y = hw / g.W;
                pos = make_float4(wt * t, wh * y, ww * (hw - y * g.W), 1.f);
            }
        }
        if (masked) out.mask[w * kMaskSlots + 32 * k + lane] = m;
        if (biased && b == 0) out.pos[(int64_t)j * kPosSlots + 32 * k + lane] = pos;
    }
    if (masked) {
        dmin = __reduce_min_sync(0xffffffffu, dmin);
        dmax = __reduce_max_sync(0xffffffffu, dmax);
        omin = __reduce_min_sync(0xffffffffu, omin);
        omax = __reduce_max_sync(0xffffffffu, omax);
        if (lane == 0) {
            const int4 s = make_int4(dmin, dmax, omin, omax);
            out.summary[w] = s;
            *reinterpret_cast<int4*>(out.mask + w * kMaskSlots + 64) = s;
        }
    }
    if (biased && b == 0) {
        // Every 4 tokens: consecutive along x of one grid row (or all text)?
        bool regular = true;
        if (lane < 16) {
            const int32_t p = j * kBlock + 4 * lane;
            float4 first = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p < g.N) {
                const int32_t src = perm_src(g, p);
                const int32_t x = src % g.W;
                if (src < g.Nv) {
                    const int32_t t = src / g.HW, y = (src - t * g.HW) / g.W;
                    first = make_float4(wt * t, wh * y, ww * x, 1.f);
                }
                for (int k = 1; k < 4 && p + k < g.N; ++k) {
                    const int32_t s = perm_src(g, p + k);
                    regular = regular && (src >= g.Nv || (s == src + k && s < g.Nv && x + k < g.W));
                }
            }
            out.pos[(int64_t)j * kPosSlots + 64 + lane] = first;
        }
        regular = __all_sync(0xffffffffu, regular);
        if (lane == 0) out.pos[(int64_t)j * kPosSlots + 80] = make_float4(regular ? 1.f : 0.f, 0.f, 0.f, 0.f);
    }
}

__global__ void __launch_bounds__(256) token_info_kernel(const TokenInfoArgs a)
{
    token_info(a, ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5);
}

// Block pair by the summaries of its query and key block: 0 no token pair
// visible, 1 all of them, 2 some (conservative: 2 may also be none or all).
__device__ __forceinline__ int block_visibility(const int4 q, const int4 k)
{
    if (q.y < 0 || k.y < 0) return 0;                          // padding only
    if (q.x > k.y || k.x > q.y || k.z > q.w) return 0;
    return (q.x == q.y && k.x == k.y && q.x == k.x && k.w <= q.z) ? 1 : 2;
}

// Pooled scores of one group of heads: block pairs without a visible token
// pair get a score below every real one, so that the selection takes them
// last.  (Finite: the selection interpolates between a row's scores.)
constexpr float kHiddenScore = -1e30f;

__global__ void __launch_bounds__(256) hide_scores_kernel(float* S, int32_t Tb, int32_t ld, int64_t h0, ModArgs m)
{
    const int32_t i = blockIdx.x;
    const int4* sum = m.info.summary + ((h0 + blockIdx.y) / m.heads) * Tb;
    const int4 q = sum[i];
    float* row = S + ((int64_t)blockIdx.y * Tb + i) * ld;
    for (int32_t j = threadIdx.x; j < Tb; j += blockDim.x)
        if (block_visibility(q, sum[j]) == 0) row[j] = kHiddenScore;
}

// The functions below take N (or 32) raw products of one query row (or, transposed,
// kKeyRow, of one key row) with tokens whose values are staged in shared
// memory, and turn them into scores in log2 units.
__device__ __forceinline__ int4 staged_summary(const int2* mask) { return *reinterpret_cast<const int4*>(mask + 64); }

struct RowInfo {
    int2 mask;               // the row token's document (-2: padding, sees nothing) and order
    float4 pos;              // w: slope * log2(e), 0 for text
};

__device__ __forceinline__ RowInfo load_row_info(const ModArgs& m, int64_t bh, int32_t Tb, int32_t p, bool valid)
{
    RowInfo r;
    r.mask = make_int2(-2, 0);
    r.pos = make_float4(0.f, 0.f, 0.f, 0.f);
    if (valid) {
        if (m.masked) {
            r.mask = m.info.mask[((bh / m.heads) * Tb + (p >> 6)) * kMaskSlots + (p & 63)];
            if (r.mask.x < 0) r.mask.x = -2;
        }
        if (m.slopes) {
            r.pos = m.info.pos[(int64_t)(p >> 6) * kPosSlots + (p & 63)];
            r.pos.w *= m.slopes[bh % m.heads] * kLog2e;
        }
    }
    return r;
}

// Scores in log2 units of raw products, s = log2(e) cap tanh(x), and with
// kGrad g = ds/dx = 1 - tanh^2.  Which polynomial serves a warp's chunk
// depends on its largest |x|: up to 1/2, i.e. scores up to half their cap, one
// of 4 terms in the raw product with every constant factor in its
// coefficients (5 operations a score); up to 1 the one of 6 terms (9); beyond,
// the exponential.  Relative error below 6.2e-7 of the polynomials; absolute
// 2^-22 of the exponential's tanh.
template <bool kGrad, int N>
__device__ __forceinline__ void cap_chunk(uint32_t (&s)[N], uint32_t (&g)[N], const ModArgs& m)
{
    float mx[2] = {0.f, 0.f};
    #pragma unroll
    for (int c = 0; c < N; c += 4) {
        mx[0] = fmaxf(mx[0], fmaxf(fabsf(__uint_as_float(s[c])), fabsf(__uint_as_float(s[c + 1]))));
        mx[1] = fmaxf(mx[1], fmaxf(fabsf(__uint_as_float(s[c + 2])), fabsf(__uint_as_float(s[c + 3]))));
    }
    const float largest = fmaxf(mx[0], mx[1]);
    if (!__any_sync(0xffffffffu, largest > m.small)) {
        const float2 c0 = make_float2(m.cap_small[0], m.cap_small[0]), c1 = make_float2(m.cap_small[1], m.cap_small[1]);
        const float2 c2 = make_float2(m.cap_small[2], m.cap_small[2]), c3 = make_float2(m.cap_small[3], m.cap_small[3]);
        #pragma unroll
        for (int c = 0; c < N; c += 2) {
            const float2 x = make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
            const float2 u = fmul2(x, x);
            const float2 y = fmul2(x, ffma2(u, ffma2(u, ffma2(u, c3, c2), c1), c0));
            s[c] = __float_as_uint(y.x);
            s[c + 1] = __float_as_uint(y.y);
            if (kGrad) {
                const float2 d = ffma2(fmul2(y, make_float2(m.cap_rcp2, m.cap_rcp2)), y, make_float2(1.f, 1.f));
                g[c] = __float_as_uint(d.x);
                g[c + 1] = __float_as_uint(d.y);
            }
        }
        return;
    }
    const float out = m.cap * kLog2e;
    if (!__any_sync(0xffffffffu, largest * m.cap_in > 1.f)) {
        const float2 in2 = make_float2(m.cap_in, m.cap_in), out2 = make_float2(out, out);
        #pragma unroll
        for (int c = 0; c < N; c += 2) {
            const float2 t = tanh_poly(fmul2(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), in2));
            const float2 y = fmul2(t, out2);
            s[c] = __float_as_uint(y.x);
            s[c + 1] = __float_as_uint(y.y);
            if (kGrad) {
                const float2 d = ffma2(make_float2(-t.x, -t.y), t, make_float2(1.f, 1.f));
                g[c] = __float_as_uint(d.x);
                g[c + 1] = __float_as_uint(d.y);
            }
        }
    } else {
        #pragma unroll
        for (int c = 0; c < N; ++c) {
            const float2 t = tanh_exp(__uint_as_float(s[c]) * m.cap_in);
            s[c] = __float_as_uint(out * t.x);
            if (kGrad) g[c] = __float_as_uint(t.y);
        }
    }
}

template <int N>
__device__ __forceinline__ void scale_chunk(uint32_t (&s)[N], float sl2, float add)
{
    const float2 sc = make_float2(sl2, sl2), ad = make_float2(add, add);
    #pragma unroll
    for (int c = 0; c < N; c += 2) {
        const float2 y = ffma2(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc, ad);
        s[c] = __float_as_uint(y.x);
        s[c + 1] = __float_as_uint(y.y);
    }
}

// Distance bias of N streamed tokens (from `first` on, of the block staged at
// `pos`).  A staged value reaches all lanes at 4 cycles of the shared
// memory pipe per 16 bytes, 64 tokens at 256 per warp: where every 4 tokens
// are neighbours along x, one value and the step between them serve the 4.
// kScale: s are raw products still, to be multiplied by sl2 along the way.
// `constant` is added to all.
template <bool kScale, int N>
__device__ __forceinline__ void bias_chunk(uint32_t (&s)[N], const RowInfo& r, const float4* pos, int first, float step,
                                           float sl2, float constant)
{
    auto add = [&](int c, float b) {
        const float x = __uint_as_float(s[c]);
        s[c] = __float_as_uint(kScale ? fmaf(x, sl2, b) : x + b);
    };
    if (pos[80].x != 0.f) {
        #pragma unroll
        for (int q = 0; q < N / 4; ++q) {
            const float4 k = pos[64 + (first >> 2) + q];
            const float f = -r.pos.w * k.w, dx = r.pos.z - k.z;
            const float base = fmaf(f, fabsf(r.pos.x - k.x) + fabsf(r.pos.y - k.y), constant);
            #pragma unroll
            for (int e = 0; e < 4; ++e) add(4 * q + e, fmaf(f, fabsf(dx - e * step), base));
        }
    } else {
        #pragma unroll
        for (int c = 0; c < N; ++c) {
            const float4 k = pos[first + c];
            add(c, fmaf(-r.pos.w * k.w, fabsf(r.pos.x - k.x) + fabsf(r.pos.y - k.y) + fabsf(r.pos.z - k.z), constant));
        }
    }
}

// Bit c: staged token c and the row's token see each other.
template <bool kKeyRow>
__device__ __forceinline__ uint32_t visible_bits(const RowInfo& r, const int2* mask)
{
    uint32_t bits = 0u;
    #pragma unroll
    for (int c = 0; c < 32; ++c) {
        const int2 k = mask[c];
        const bool vis = k.x == r.mask.x && (kKeyRow ? r.mask.y <= k.y : k.y <= r.mask.y);
        bits |= vis ? 1u << c : 0u;
    }
    return bits;
}

// The same by the summary of the staged block: 0 none of its tokens, 1 all, 2
// some (or not to be told).  A block of one document and one order (a frame,
// an image) never needs more.
template <bool kKeyRow>
__device__ __forceinline__ int row_visibility(const RowInfo& r, const int4 b)
{
    if (r.mask.x < b.x || r.mask.x > b.y) return 0;            // padding rows have document -2
    if (kKeyRow ? r.mask.y > b.w : r.mask.y < b.z) return 0;
    return (b.x == b.y && (kKeyRow ? r.mask.y <= b.z : r.mask.y >= b.w)) ? 1 : 2;
}

// Replaces the values whose bit is clear.  Hidden scores become 0 before the
// cap (whose choice of path must not depend on them) and -inf at the end.
template <int N>
__device__ __forceinline__ void hide(uint32_t (&s)[N], uint32_t bits, uint32_t value)
{
    #pragma unroll
    for (int c = 0; c < N; ++c) s[c] = (bits >> c & 1u) ? s[c] : value;
}
constexpr uint32_t kMinusInf = 0xff800000u;

// Zeroes the rows of a tile of 64 rows, 128 bytes each per chunk of 64
// columns (kChunk bytes apart), whose token is padding:
// their content may be anything, and 0 * NaN would reach every row of the
// product.  By one whole warp; the caller orders it before the tensor cores'
// reads (proxy fence, then the barrier they wait on).
template <int D, uint32_t kChunk>
__device__ __forceinline__ void zero_padding_rows(uint8_t* tile, const int2* mask, int lane)
{
    const uint32_t dead0 = __ballot_sync(0xffffffffu, mask[lane].x < 0);
    const uint32_t dead1 = __ballot_sync(0xffffffffu, mask[lane + 32].x < 0);
    // four rows of 128 bytes at a time
    #pragma unroll 4
    for (int r = lane >> 3; r < 64; r += 4) {
        const bool dead = ((r < 32 ? dead0 : dead1) >> (r & 31)) & 1u;
        #pragma unroll
        for (int c = 0; c < D / 64; ++c)
            if (dead) *reinterpret_cast<uint4*>(tile + c * kChunk + r * 128 + (lane & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
}

}  // namespace rf2
