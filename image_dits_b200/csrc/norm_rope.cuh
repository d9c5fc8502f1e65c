// RMS norm of each head's queries and keys, the 3D position rotation and the
// window permutation in one pass over Q, K and V, and its gradient.
//
// Row x (d channels of one head and token), weight w, angles a_p of its d/2
// channel pairs:
//   r = (mean x^2 + eps)^(-1/2),  z = x r w,
//   (y_a, y_b) = (z_a cos - z_b sin, z_a sin + z_b cos)    per pair (a, b),
// and, with g = dL/dy, its gradient
//   dz = the rotation turned back,  u = dz w,  h = x r,
//   dx = r (u - h mean(u h)),  dw = sum over rows of dz h.
// Statistics, rotation and sums are fp32; each output is rounded to bf16
// once.
//
// The angles of a pair depend on one grid coordinate only, so the rotation
// table holds one (cos, sin) row per coordinate value and axis (24 KB for a
// 21 x 45 x 80 grid at d = 128) instead of one per token.
//
// Both directions move every byte once.  HBM binds the longest calls (720p, 40
// heads, 4.6 GB in 780 us: 0.91 of a plain copy's rate).  Nothing is saturated
// in the 480p ones (0.72 forward, 0.69 backward; DRAM at 54% and 53%, issue
// slots at 58% and 46%): the forward call's last round of CTAs is half empty
// (1,548 on 444 slots), and the backward kernel has 16 warps an SM at 128
// registers and stages each item in the open.  A CTA takes one 64-token block
// of the permuted sequence and up to 24 (head, tensor) units of it: the source
// rows of the permutation and the (cos, sin) of every token and pair are laid
// down in shared memory once for all of them (33 KB at d = 128).  A warp takes
// a unit, 16 lanes (d = 128) or 8 (d = 64) to a row.  A lane holds four whole
// channel pairs, either way they are paired: channels 8c .. 8c+7 (interleaved,
// 16 bytes) or 4c .. 4c+3 and d/2 + 4c .. d/2 + 4c+3 (split, 2 x 8 bytes), so
// the rotation needs no other lane; the row's sum of squares is a butterfly.
// The loads of the next rows are issued before the current ones are worked on.
// Measured and not kept: a half-warp per unit, 8 lanes of 32 bytes to a row (half
// the shuffles, but 140 bytes of spills or half the warps): 10 to 30% slower.
#pragma once
#include "geometry.cuh"
#include "mask.cuh"
#include "ptx.cuh"

namespace rf2 {

// A bf16 tensor [B, H, N, d] by element strides (d contiguous).
struct RowView {
    uint16_t* data;
    int64_t sb, sh, sn;
};

struct NormRopeArgs {
    RowView x[3];            // q, k, v in token order (v.data may be null)
    void* yp[3];             // qp, kp, vp: permuted, dense (forward: written; backward: the gradients read)
    RowView dx[3];           // backward: gradients in token order
    const float* w[2];       // norm weights of q and k, or null
    const float2* rope;      // rotation table or null
    int32_t st2, sh2, sw2;   // pairs turned by t, y, x
    int32_t off_y, off_x, off_text;   // table offsets of the axes after t (in pairs)
    int32_t norm;
    float eps;
    PermGeo g;
    int32_t B, H, Tb, tensors;        // tensors: 2, or 3 with v
    int32_t chunks, per_item;         // items of a token block, and units of each
    float* means_hi;         // forward: block means of qp and kp (mask workspace), or null
    float* means_lo;
    float* dw_part;          // backward: [grid][2][D] partial weight gradients, or null
};

constexpr int kNormRopeThreads = 256;
// Units per CTA: 24, 16 or 8 (the 8 warps take one, two or three), the most
// that leaves `waves` rounds of resident CTAs (3 or 2 per SM of 148): few units
// repeat the staging, few CTAs leave SMs idle in the last round.  Measured:
// forward, 720p (5,910 CTAs of 24) 780 us, with 8 825; 480p + text (1,548 of
// 16) 135, with 24 143; backward, 480p 178 with 8, 241 with 24 (before the
// vote on rows without a gradient, which takes 3 us of it).
constexpr int kNormRopeForwardSlots = 444, kNormRopeForwardWaves = 3;
constexpr int kNormRopeBackwardSlots = 296, kNormRopeBackwardWaves = 8;
constexpr int kNormRopeMaxCtas = kNormRopeBackwardSlots;     // backward grid: rows of the partial weight gradients

template <int D>
struct NormRopeSmem {
    float2 cs[kBlock][D / 2];
    int32_t src[kBlock];
    int32_t off[3][kBlock];                   // table offset of a token's row of each axis, less the axis's first pair
    float dw[kNormRopeThreads / 32][2][D];    // backward
};

// The lane's four channel pairs (a, b) of a row, as two pairs of packed words:
// interleaved, words hold (a0, b0) .. (a3, b3); split, (a0, a1), (a2, a3) and
// (b0, b1), (b2, b3).
template <int D, bool kInter>
struct LaneRow {
    static constexpr int C = D / 8;
    // element offset of the lane's channels; the split layout's second half D/2 further on
    static __device__ __forceinline__ int first(int cidx) { return kInter ? 8 * cidx : 4 * cidx; }

    static __device__ __forceinline__ uint4 load(const uint16_t* p)
    {
        if (kInter) return __ldcs(reinterpret_cast<const uint4*>(p));
        const uint2 a = __ldcs(reinterpret_cast<const uint2*>(p)), b = __ldcs(reinterpret_cast<const uint2*>(p + D / 2));
        return make_uint4(a.x, a.y, b.x, b.y);
    }

    static __device__ __forceinline__ void store(uint16_t* p, const uint4 v)
    {
        if (kInter) {
            __stcs(reinterpret_cast<uint4*>(p), v);
        } else {
            __stcs(reinterpret_cast<uint2*>(p), make_uint2(v.x, v.y));
            __stcs(reinterpret_cast<uint2*>(p + D / 2), make_uint2(v.z, v.w));
        }
    }

    // the row's channels in memory order: words of (lo, hi)
    static __device__ __forceinline__ void unpack(const uint4 v, float2 (&f)[4])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        #pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
    }

    static __device__ __forceinline__ uint4 pack(const float2 (&f)[4])
    {
        return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                          pack_bf16x2(f[3].x, f[3].y));
    }

    // eight fp32 values (weights, sums) of the lane's channels
    static __device__ __forceinline__ void load_f32(const float* p, float2 (&f)[4])
    {
        #pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = make_float2(p[channel(2 * k)], p[channel(2 * k + 1)]);
    }
    static __device__ __forceinline__ int channel(int e) { return kInter || e < 4 ? e : D / 2 - 4 + e; }

    // Turns the pairs by (cos, sin), kBack: back.
    template <bool kBack>
    static __device__ __forceinline__ void turn(const float2* cs, float2 (&z)[4])
    {
        const float4 c01 = *reinterpret_cast<const float4*>(cs), c23 = *reinterpret_cast<const float4*>(cs + 2);
        const float c[4] = {c01.x, c01.z, c23.x, c23.z}, t[4] = {c01.y, c01.w, c23.y, c23.w};
        #pragma unroll
        for (int k = 0; k < 4; ++k) {
            float& a = kInter ? z[k].x : (k & 1 ? z[k >> 1].y : z[k >> 1].x);
            float& b = kInter ? z[k].y : (k & 1 ? z[2 + (k >> 1)].y : z[2 + (k >> 1)].x);
            const float sn = kBack ? -t[k] : t[k];
            const float u = a * c[k] - b * sn;
            b = a * sn + b * c[k];
            a = u;
        }
    }
};

// The item's permutation sources and rotation, into shared memory.
template <int D>
__device__ __forceinline__ void norm_rope_stage(const NormRopeArgs& a, NormRopeSmem<D>& sm, int32_t i)
{
    constexpr int P = D / 2;
    if (threadIdx.x < kBlock) {
        const int32_t pos = i * kBlock + threadIdx.x;
        int32_t src = pos < a.g.N ? perm_src(a.g, pos) : -1;
        if (RF2_CHECKED && pos < a.g.N && !in_range(src >= 0 && src < a.g.N)) src = -1;   // checked build: reported, skipped
        sm.src[threadIdx.x] = src;
        int32_t o0 = 0, o1 = 0, o2 = 0;
        if (src >= a.g.Nv) {
            o0 = o1 = o2 = a.off_text + (src - a.g.Nv) * P;
        } else if (src >= 0) {
            const int32_t t = src / a.g.HW, hw = src - t * a.g.HW;
            const int32_t y = hw / a.g.W, x = hw - y * a.g.W;
            o0 = t * a.st2;
            o1 = a.off_y + y * a.sh2 - a.st2;
            o2 = a.off_x + x * a.sw2 - a.st2 - a.sh2;
        }
        sm.off[0][threadIdx.x] = o0;
        sm.off[1][threadIdx.x] = o1;
        sm.off[2][threadIdx.x] = o2;
    }
    __syncthreads();
    if (a.rope) {
        // thread t: pair t % P of tokens t / P, t / P + 256 / P, ...
        const int p = threadIdx.x % P;
        const int axis = p < a.st2 ? 0 : p < a.st2 + a.sh2 ? 1 : 2;
        #pragma unroll 8
        for (int r = threadIdx.x / P; r < kBlock; r += kNormRopeThreads / P)
            sm.cs[r][p] = sm.src[r] >= 0 ? __ldg(a.rope + sm.off[axis][r] + p) : make_float2(1.f, 0.f);
    }
    __syncthreads();
}

// Item -> batch element, token block, first unit and their number.  A unit is
// a (tensor, head): heads of Q, then of K, then of V.
struct NormRopeItem { int32_t b, i, u0, n; };
__device__ __forceinline__ NormRopeItem norm_rope_item(const NormRopeArgs& a, int64_t item)
{
    NormRopeItem it;
    const int64_t blk = item / a.chunks;
    const int32_t c = (int32_t)(item - blk * a.chunks), units = a.H * a.tensors;
    it.b = (int32_t)(blk / a.Tb);
    it.i = (int32_t)(blk - (int64_t)it.b * a.Tb);
    it.u0 = c * a.per_item;
    it.n = min(a.per_item, units - it.u0);
    return it;
}

template <int D, bool kInter>
__global__ void __launch_bounds__(kNormRopeThreads, 3) norm_rope_kernel(const NormRopeArgs a)
{
    using Row = LaneRow<D, kInter>;
    constexpr int C = D / 8;          // lanes of a row
    constexpr int R = 32 / C;         // rows of a warp-wide access
    constexpr int kLoads = 4;         // accesses per batch
    constexpr int kSub = R * kLoads;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    NormRopeSmem<D>& sm = *reinterpret_cast<NormRopeSmem<D>*>(smem_raw);
    const NormRopeItem it = norm_rope_item(a, blockIdx.x);
    norm_rope_stage<D>(a, sm, it.i);
    const int lane = threadIdx.x & 31;
    const int cidx = lane % C, rsub = lane / C;
    const int32_t rows = min(kBlock, a.g.N - it.i * kBlock);
    for (int un = threadIdx.x >> 5; un < it.n; un += kNormRopeThreads / 32) {
        const int which = (it.u0 + un) / a.H, h = (it.u0 + un) - which * a.H;
        const bool copy = which == 2;
        const bool turn = a.rope != nullptr && !copy;
        const RowView& xv = a.x[which];
        const uint16_t* in = xv.data + it.b * xv.sb + h * xv.sh + Row::first(cidx);
        const int64_t bh = (int64_t)it.b * a.H + h;
        uint16_t* out = reinterpret_cast<uint16_t*>(a.yp[which]) + (bh * a.g.N + (int64_t)it.i * kBlock) * D + Row::first(cidx);
        float2 w[4], acc[4];
        #pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = make_float2(1.f, 1.f), acc[k] = make_float2(0.f, 0.f);
        if (!copy && a.w[which]) Row::load_f32(a.w[which] + Row::first(cidx), w);
        uint4 next[kLoads];
        auto fetch = [&](int r0) {
            #pragma unroll
            for (int q = 0; q < kLoads; ++q) {
                const int32_t src = sm.src[r0 + q * R + rsub];
                next[q] = make_uint4(0u, 0u, 0u, 0u);
                if (src >= 0) next[q] = Row::load(in + (int64_t)src * xv.sn);
            }
        };
        fetch(0);
        #pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += kSub) {
            uint4 v[kLoads];
            #pragma unroll
            for (int q = 0; q < kLoads; ++q) v[q] = next[q];
            if (r0 + kSub < rows) fetch(r0 + kSub);
            #pragma unroll
            for (int q = 0; q < kLoads; ++q) {
                const int r = r0 + q * R + rsub;
                const bool ok = r < rows && (!RF2_CHECKED || sm.src[r] >= 0);
                if (!copy) {
                    float2 z[4];
                    Row::unpack(v[q], z);
                    if (a.norm) {
                        float2 s2 = fmul2(z[0], z[0]);
                        #pragma unroll
                        for (int k = 1; k < 4; ++k) s2 = ffma2(z[k], z[k], s2);
                        float ss = s2.x + s2.y;
                        #pragma unroll
                        for (int off = 1; off < C; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
                        const float rs = rsqrtf(ss * (1.f / D) + a.eps);
                        #pragma unroll
                        for (int k = 0; k < 4; ++k) z[k] = fmul2(fmul2(z[k], make_float2(rs, rs)), w[k]);
                    }
                    if (turn) Row::template turn<false>(&sm.cs[r][4 * cidx], z);
                    v[q] = Row::pack(z);
                }
                if (ok) {
                    Row::store(out + r * D, v[q]);
                    float2 f[4];
                    Row::unpack(v[q], f);
                    #pragma unroll
                    for (int k = 0; k < 4; ++k) acc[k] = fadd2(acc[k], f[k]);
                }
            }
        }
        if (a.means_hi && !copy) {
            // the block mean, in the order permute_pool_kernel sums it
            #pragma unroll
            for (int off = C; off < 32; off <<= 1)
                #pragma unroll
                for (int k = 0; k < 4; ++k) {
                    acc[k].x += __shfl_xor_sync(0xffffffffu, acc[k].x, off);
                    acc[k].y += __shfl_xor_sync(0xffffffffu, acc[k].y, off);
                }
            if (lane < C) {
                const float fr = (float)rows;
                const int64_t at = (((int64_t)which * a.B * a.H + bh) * a.Tb + it.i) * D + Row::first(cidx);
                #pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float m0 = acc[k].x / fr, m1 = acc[k].y / fr;
                    const float h0 = to_tf32(m0), h1 = to_tf32(m1);
                    const int64_t e = at + Row::channel(2 * k);
                    *reinterpret_cast<float2*>(a.means_hi + e) = make_float2(h0, h1);
                    *reinterpret_cast<float2*>(a.means_lo + e) = make_float2(m0 - h0, m1 - h1);
                }
            }
        }
    }
}

// Gradients in token order from those of the permuted tensors.  The weight
// gradient is summed per lane over a unit's rows, then per warp in shared
// memory, and left as one partial row per CTA for norm_rope_dw_kernel: the
// grid is fixed by the sizes, so the order of the sums is too.
template <int D, bool kInter>
__global__ void __launch_bounds__(kNormRopeThreads, 2) norm_rope_backward_kernel(const NormRopeArgs a)
{
    using Row = LaneRow<D, kInter>;
    constexpr int C = D / 8;
    constexpr int R = 32 / C;
    constexpr int kLoads = 4;
    constexpr int kSub = R * kLoads;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    NormRopeSmem<D>& sm = *reinterpret_cast<NormRopeSmem<D>*>(smem_raw);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cidx = lane % C, rsub = lane / C;
    for (int e = threadIdx.x; e < kNormRopeThreads / 32 * 2 * D; e += kNormRopeThreads) (&sm.dw[0][0][0])[e] = 0.f;
    const int64_t items = (int64_t)a.B * a.Tb * a.chunks;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const NormRopeItem it = norm_rope_item(a, item);
        __syncthreads();                   // the previous item's rows are done with
        norm_rope_stage<D>(a, sm, it.i);
        const int32_t rows = min(kBlock, a.g.N - it.i * kBlock);
        for (int un = warp; un < it.n; un += kNormRopeThreads / 32) {
            const int which = (it.u0 + un) / a.H, h = (it.u0 + un) - which * a.H;
            const bool copy = which == 2;
            const bool turn = a.rope != nullptr && !copy, norm = a.norm && !copy;
            const RowView& xv = a.x[which];
            const RowView& gv = a.dx[which];
            const uint16_t* in = xv.data + it.b * xv.sb + h * xv.sh + Row::first(cidx);
            const uint16_t* gin = reinterpret_cast<const uint16_t*>(a.yp[which]) +
                                  (((int64_t)it.b * a.H + h) * a.g.N + (int64_t)it.i * kBlock) * D + Row::first(cidx);
            uint16_t* out = gv.data + it.b * gv.sb + h * gv.sh + Row::first(cidx);
            float2 w[4], acc[4];
            #pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = make_float2(1.f, 1.f), acc[k] = make_float2(0.f, 0.f);
            if (!copy && a.w[which]) Row::load_f32(a.w[which] + Row::first(cidx), w);
            uint4 ng[kLoads], nx[kLoads];
            auto fetch = [&](int r0) {
                #pragma unroll
                for (int q = 0; q < kLoads; ++q) {
                    const int r = r0 + q * R + rsub;
                    const int32_t src = sm.src[r];
                    ng[q] = nx[q] = make_uint4(0u, 0u, 0u, 0u);
                    if (src >= 0) {
                        ng[q] = Row::load(gin + r * D);
                        if (norm) nx[q] = Row::load(in + (int64_t)src * xv.sn);
                    }
                }
            };
            fetch(0);
            #pragma unroll 1
            for (int r0 = 0; r0 < rows; r0 += kSub) {
                uint4 v[kLoads], x[kLoads];
                #pragma unroll
                for (int q = 0; q < kLoads; ++q) v[q] = ng[q], x[q] = nx[q];
                if (r0 + kSub < rows) fetch(r0 + kSub);
                if (norm) {
                    // A row whose gradient is 0 throughout, as behind the sequence's end and in padding
                    // tokens, gives 0 and adds nothing to dw, whatever x holds: ones in its place.
                    auto nonzero = [](const uint4& g) { return ((g.x | g.y | g.z | g.w) & 0x7fff7fffu) != 0u; };
                    bool all = true;
                    #pragma unroll
                    for (int q = 0; q < kLoads; ++q) all = all && nonzero(v[q]);
                    if (!__all_sync(0xffffffffu, all)) {
                        const uint32_t lanes = (C == 16 ? 0xffffu : 0xffu) << (rsub * C);
                        #pragma unroll
                        for (int q = 0; q < kLoads; ++q)
                            if (!(__ballot_sync(0xffffffffu, nonzero(v[q])) & lanes))
                                x[q] = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
                    }
                }
                #pragma unroll
                for (int q = 0; q < kLoads; ++q) {
                    const int r = r0 + q * R + rsub;
                    const int32_t src = sm.src[r];
                    if (!copy) {
                        float2 dz[4];
                        Row::unpack(v[q], dz);
                        if (turn) Row::template turn<true>(&sm.cs[r][4 * cidx], dz);
                        if (norm) {
                            float2 hx[4], s2 = make_float2(0.f, 0.f), d2 = s2;
                            Row::unpack(x[q], hx);
                            #pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                s2 = ffma2(hx[k], hx[k], s2);
                                d2 = ffma2(fmul2(dz[k], w[k]), hx[k], d2);
                            }
                            float ss = s2.x + s2.y, dot = d2.x + d2.y;
                            #pragma unroll
                            for (int off = 1; off < C; off <<= 1) {
                                ss += __shfl_xor_sync(0xffffffffu, ss, off);
                                dot += __shfl_xor_sync(0xffffffffu, dot, off);
                            }
                            // dw += (r dz) x,  dx = (r dz) w - x r^3 mean(dz w x)
                            const float rs = rsqrtf(ss * (1.f / D) + a.eps);
                            const float m = -dot * (1.f / D) * rs * rs * rs;
                            #pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                dz[k] = fmul2(dz[k], make_float2(rs, rs));
                                acc[k] = ffma2(dz[k], hx[k], acc[k]);
                                dz[k] = ffma2(hx[k], make_float2(m, m), fmul2(dz[k], w[k]));
                            }
                        }
                        v[q] = Row::pack(dz);
                    }
                    if (src >= 0) Row::store(out + (int64_t)src * gv.sn, v[q]);
                }
            }
            if (a.dw_part && norm) {
                #pragma unroll
                for (int k = 0; k < 4; ++k) {
                    #pragma unroll
                    for (int off = C; off < 32; off <<= 1) {
                        acc[k].x += __shfl_xor_sync(0xffffffffu, acc[k].x, off);
                        acc[k].y += __shfl_xor_sync(0xffffffffu, acc[k].y, off);
                    }
                    if (lane < C) {
                        float* d = &sm.dw[warp][which][Row::first(cidx) + Row::channel(2 * k)];
                        d[0] += acc[k].x;
                        d[1] += acc[k].y;
                    }
                }
            }
        }
    }
    if (!a.dw_part) return;
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * D; e += kNormRopeThreads) {
        float s = 0.f;
        #pragma unroll
        for (int k = 0; k < kNormRopeThreads / 32; ++k) s += sm.dw[k][e / D][e % D];
        a.dw_part[(int64_t)blockIdx.x * 2 * D + e] = s;
    }
}

// Sum of the CTAs' partial weight gradients: 32 columns per CTA, 32 rows at a
// time, then over the 32 row sums.
template <int D>
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* part, int32_t n, float* dwq, float* dwk)
{
    __shared__ float s[32][33];
    const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + c;
    float acc = 0.f;
    for (int k = r; k < n; k += 32) acc += part[(int64_t)k * 2 * D + col];
    s[r][c] = acc;
    __syncthreads();
    if (r == 0) {
        float t = 0.f;
        #pragma unroll
        for (int k = 0; k < 32; ++k) t += s[k][c];
        float* out = col < D ? dwq : dwk;
        if (out) out[col % D] = t;
    }
}

}  // namespace rf2
