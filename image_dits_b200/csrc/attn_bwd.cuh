// Gradients of block-sparse attention on tcgen05.  With P_ij = exp(s_ij - lse_i)
// over the visible pairs (s: the modified scores of score_mod.cuh) and
// delta_i = dO_i . O_i,
//   dP = dO V^T,  dS = P (dP - delta) ds/dx     (ds/dx = 1 - tanh^2 under the cap),
//   dV = P^T dO,  dK = dS^T Q / sqrt(d),  dQ = dS K / sqrt(d).
//
// Two passes over the block pairs, so that every sum stays in one CTA's TMEM and
// nothing is added with atomics (results do not depend on timing):
//   row pass (kCol = false)  resident: a pair of query blocks (Q, dO); streamed:
//       the key blocks of their CSR rows (K, V); S = Q K^T, dP = dO V^T, dQ += dS K
//   column pass (kCol)       resident: a pair of key blocks (K, V); streamed: the
//       query blocks that keep them (Q, dO); S^T = K Q^T, dP^T = V dO^T,
//       dK += dS^T Q, dV += P^T dO
// i.e. 7 products per block pair where one pass with atomics needs 5.  The
// column pass finds its query blocks in the mask's transpose, a bit matrix
// that csr_transpose writes (7 MB for 40 heads of 1,182 blocks).
//
// One CTA (608 threads) per SM and resident pair, M = 128 as in the forward
// kernel.  Entries are the union of the pair's two lists, with one kept bit
// each, taken two at a time: a step is up to 128 streamed tokens, because an
// M128 x N128 x K16 product takes 64 cycles where two of N = 64 take 96 (the
// reads of both operands from shared memory bind the smaller one).
//   warps 0-15  softmax: four threads to a resident row (= TMEM lane), each
//               with 32 of the step's 128 columns; then the epilogue
//   warp 16     MMA issuer
//   warp 17     TMA: the first streamed tile (K / Q) and the streamed tokens'
//               info; the resident tiles are loaded by thread 0
//   warp 18     TMA: the second streamed tile (V / dO)
// (four stages of 32 KB at d = 128 in all).
// A step's softmax has two parts, A: probabilities from S, B: dS from dP, and
// the tensor pipe runs the products that do not wait for the part in progress.
//   column pass  TMEM: dK, dV, S, dP (all 512 columns).  P overwrites S, dS
//       overwrites dP.  Order: dV_p (after A_p), S_{p+1}, dK_p (after B_p),
//       dP_{p+1}: B_p runs beside dV_p and S_{p+1}, A_{p+1} beside dK_p and
//       dP_{p+1}.
//   row pass     TMEM: dQ, S, two dP buffers.  P stays in registers, so S is
//       free as soon as part A has loaded it.  Order: S_{p+1}, dP_{p+1}, dQ_p
//       (after B_p).
// Tensor cycles per step at d = 128: 2,048 (column; 128 more with the extra K
// step below), 1,536 (row).  Measured: 480p, 12 heads, keep 0.2: 7.3 ms.  P and dS
// are bf16, written over the first half of the 32 columns they come from.
//
// In the column pass a thread's columns are queries, and their log-sum-exp and
// delta would be read from shared memory by every thread (1,024 cycles of its
// 128 bytes a cycle per step, next to the products' own reads).  Instead one
// more K step of each product subtracts them: the streamed side has -lse
// sqrt(d) and -delta split into three bf16 each (24 bits), the resident side
// ones.  Under the cap the log-sum-exp comes after a function of the score,
// and only delta is subtracted that way.
//
// Waits are bounded and leave through the CTA's abort flag as in the forward
// kernel.
#pragma once
#include "attn.cuh"
#include "geometry.cuh"
#include "ptx.cuh"
#include "score_mod.cuh"

namespace rf2 {

template <int D>
struct BwdCfg {
    static constexpr int KCH = D / 64;
    static constexpr uint32_t CHUNK = 128 * 128;            // 64 columns of 128 rows
    static constexpr uint32_t TILE = CHUNK * KCH;           // a resident tile, or a step's streamed tile
    static constexpr uint32_t HALF = 64 * 128;              // the second entry's rows within a chunk
    // Stages of the two streamed tiles (the info goes with the first): the next load of a stage
    // starts when the last product that reads it is done, which for T1 is the step's last one.
    // (2 + 2 in the column pass: the same time.)
    static constexpr int S1 = 3, S2 = 1;
    static constexpr uint32_t TM_ACC1 = 0;                  // dQ, or dK
    static constexpr uint32_t TM_ACC2 = 128;                // column pass: dV
    static constexpr uint32_t TM_COLS = 512;
    static constexpr int SOFTMAX_WARPS = 16;                // (8, 64 columns a thread: 1.3x the time at 480p)
    static constexpr int HALVES = 16 / SOFTMAX_WARPS;       // 32-column pieces of a step per softmax thread
    static constexpr int MMA_WARP = SOFTMAX_WARPS;
    static constexpr int T1_WARP = SOFTMAX_WARPS + 1;
    static constexpr int T2_WARP = SOFTMAX_WARPS + 2;
    static constexpr int THREADS = 32 * (SOFTMAX_WARPS + 3);
    // Shared memory: [align slack][resident 1][resident 2][T1 stages][T2][extra K step][info stages][list][control]
    static constexpr uint32_t OFF_R1 = 0;
    static constexpr uint32_t OFF_R2 = TILE;
    static constexpr uint32_t OFF_T1 = 2 * TILE;
    static constexpr uint32_t OFF_T2 = OFF_T1 + S1 * TILE;
    // The extra K step of the column pass: tiles of 128 rows x 8 columns (16 bytes a row, 8-row
    // groups of 128 bytes, no swizzle), the other 8 columns of the step a shared tile of zeros.
    static constexpr uint32_t AUG = 128 * 16;
    static constexpr uint32_t AUG_HALF = 64 * 16;
    static constexpr uint32_t OFF_AUG_T = OFF_T2 + S2 * TILE;               // streamed, one per T1 stage
    static constexpr uint32_t OFF_AUG_S = OFF_AUG_T + S1 * AUG;             // resident ones of S
    static constexpr uint32_t OFF_AUG_P = OFF_AUG_S + AUG;                  // and of dP
    static constexpr uint32_t OFF_ZERO = OFF_AUG_P + AUG;
    static constexpr uint32_t INFO_MASK = kMaskSlots * 8;   // documents and orders
    static constexpr uint32_t INFO_POS = kPosSlots * 16;    // positions
    static constexpr uint32_t INFO_LSE = 64 * 4;            // log-sum-exp (column pass under the cap)
    static constexpr uint32_t INFO = INFO_MASK + INFO_POS + INFO_LSE;       // of one entry
    static constexpr uint32_t OFF_INFO = OFF_ZERO + AUG;
    static constexpr uint32_t OFF_LIST = OFF_INFO + S1 * 2 * INFO;
    static constexpr uint32_t CONTROL_BYTES = 256;
    __host__ __device__ static size_t list_bytes(int Tb) { return ((size_t)Tb * 2 + 15) & ~(size_t)15; }
    __host__ __device__ static size_t smem_bytes(int Tb) { return 1024 + OFF_LIST + list_bytes(Tb) + CONTROL_BYTES; }
    // TMEM columns of S, and of dP in step p
    __host__ __device__ static constexpr uint32_t tm_s(bool col) { return col ? 256 : 128; }
    __host__ __device__ static constexpr uint32_t tm_dp(bool col, int p) { return col ? 384 : 256 + 128 * (p & 1); }
};
// 227 KB per CTA, at the largest T_b (4096) and d
static_assert(1024 + BwdCfg<128>::OFF_LIST + 4096 * 2 + BwdCfg<128>::CONTROL_BYTES <= 232448, "shared memory");

// A list entry: block (12 bits: T_b <= 4096), then kept and partial bits of the two resident blocks.
__device__ __forceinline__ uint16_t bwd_entry(int block, uint32_t keptA, uint32_t keptB, uint32_t partA, uint32_t partB)
{
    return (uint16_t)(block | keptA << 12 | keptB << 13 | partA << 14 | partB << 15);
}

struct __align__(16) BwdCtl {
    uint64_t r_full;
    uint64_t t1_full[3], t1_free[3];
    uint64_t t2_full[1], t2_free[1];    // t2_free: column pass (the row pass frees T2 with dp_full)
    uint64_t s_full, dp_full[2];    // dp_full[1]: row pass
    uint64_t a_done;                // part A: S read (row pass) or P written (column pass)
    uint64_t b_done[2];             // part B: dS written; [1]: row pass, whose dP runs a step ahead
    uint64_t final, drain;
    uint32_t tmem_base;
    int32_t list_len;
    int32_t abort;
};
static_assert(sizeof(BwdCtl) <= 256, "control block must fit CONTROL_BYTES");

struct BwdArgs {
    const int32_t* row_start;    // row pass: the CSR mask
    const int32_t* row_count;
    const int32_t* col_idx;
    const uint32_t* tbits;       // column pass: [BH][ceil(T_b/32)][T_b], bit r of word (w, j): query block 32w + r keeps j
    const float* lse2;           // [BH][T_b * 64] lse * log2(e) of the queries
    const float* delta;          // [BH][T_b * 64]
    const uint4* aug;            // [BH][T_b * 64] the queries' columns of the extra K step
    uint16_t* dq;
    uint16_t* dk;
    uint16_t* dv;
    int* status;
    int32_t N, Tb, pairs, sink_pairs;
    float scale, scale_log2;     // 1/sqrt(d), log2(e)/sqrt(d)
    int64_t col_capacity;
    ModArgs mod;
};

constexpr int kBwdPrepThreads = 256;

// log2 units; of a query without visible keys and of the slots behind the last token: P = 2^(s - 1e30) = 0
// whatever the bias adds to the score (finite, as it goes through the extra K step)
constexpr float kDeadLse = 1e30f;

// x as the sum of three bf16, two packed words (hi, mid) and (lo, 0).
__device__ __forceinline__ uint2 split3(float x)
{
    const uint32_t hi = pack_bf16x2(x, 0.f) & 0xffffu;
    const float r = x - __uint_as_float(hi << 16);
    const uint32_t mid = pack_bf16x2(r, 0.f) & 0xffffu;
    const uint32_t lo = pack_bf16x2(r - __uint_as_float(mid << 16), 0.f) & 0xffffu;
    return make_uint2(hi | mid << 16, lo);
}

// Per query: lse * log2(e), dO . O and the columns of the extra K step.  A
// query without visible keys (lse = -inf) has delta 0, whatever dO holds.
// D/8 lanes to a row.
template <int D>
__device__ __forceinline__ void attn_stat(const uint4* __restrict__ op, const uint4* __restrict__ dop,
                                          const float* __restrict__ lse, float* __restrict__ lse2,
                                          float* __restrict__ delta, uint4* __restrict__ aug, int32_t N, int32_t Tb,
                                          int64_t BH, float unscale, int64_t block)
{
    constexpr int C = D / 8;
    const int64_t t = block * kBwdPrepThreads + threadIdx.x;
    const int64_t slot = t / C;
    const int c = (int)(t % C);
    const int64_t per = (int64_t)Tb * kBlock;
    if (slot >= BH * per) return;                  // whole warps leave together (per % 64 == 0)
    const int64_t bh = slot / per;
    const int32_t p = (int32_t)(slot - bh * per);
    float dot = 0.f, l = -INFINITY;
    if (p < N) {
        const int64_t at = (bh * N + p);
        l = lse[at];
        const uint4 x = __ldcs(op + at * C + c), y = __ldcs(dop + at * C + c);
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
        #pragma unroll
        for (int k = 0; k < 4; ++k)
            dot += __uint_as_float(xw[k] << 16) * __uint_as_float(yw[k] << 16) +
                   __uint_as_float(xw[k] & 0xffff0000u) * __uint_as_float(yw[k] & 0xffff0000u);
    }
    #pragma unroll
    for (int off = 1; off < C; off <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    if (c == 0) {
        const bool dead = l == -INFINITY;
        const float l2 = dead ? kDeadLse : l * kLog2e, dl = dead ? 0.f : dot;
        lse2[slot] = l2;
        delta[slot] = dl;
        // columns: -lse in units of the raw product (3 parts), -delta (3 parts), 0, 0
        const uint2 a = split3(-l2 * unscale), b = split3(-dl);
        aug[slot] = make_uint4(a.x, a.y | (b.x & 0xffffu) << 16, b.x >> 16 | b.y << 16, 0u);
    }
}

// The CSR mask's transpose as bits: one CTA per head and 32 query blocks.
__device__ __forceinline__ void csr_transpose(const int32_t* __restrict__ row_start,
                                              const int32_t* __restrict__ row_count, const int32_t* __restrict__ col_idx,
                                              uint32_t* __restrict__ tbits, int32_t Tb, int64_t col_capacity,
                                              int64_t block, uint32_t* words)
{
    const int W = (Tb + 31) >> 5;
    const int64_t bh = block / W;
    const int w = (int)(block - bh * W);
    for (int j = threadIdx.x; j < Tb; j += kBwdPrepThreads) words[j] = 0u;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    for (int r = threadIdx.x >> 5; r < 32; r += kBwdPrepThreads / 32) {
        if (32 * w + r >= Tb) break;
        const int64_t row = bh * Tb + 32 * w + r;
        const int32_t cnt = row_count[row], start = row_start[row];
        int len = min(max(cnt, 0), Tb);
        if (RF2_CHECKED && !in_range(cnt >= 0 && cnt <= Tb && start >= 0 && (int64_t)start + cnt <= col_capacity)) len = 0;
        for (int e = lane; e < len; e += 32) {
            const int32_t j = col_idx[(int64_t)start + e];
            if (in_range(j >= 0 && j < Tb) && j >= 0 && j < Tb) atomicOr(&words[j], 1u << r);
        }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < Tb; j += kBwdPrepThreads) tbits[(bh * W + w) * Tb + j] = words[j];
}

// What both passes need, in one launch: the first `t_blocks` CTAs transpose
// the mask, the next `i_blocks` write the token info, the rest the statistics.
template <int D>
__global__ void __launch_bounds__(kBwdPrepThreads) attn_bwd_prep_kernel(
    const uint4* __restrict__ op, const uint4* __restrict__ dop, const float* __restrict__ lse, BwdArgs a,
    float* lse2, float* delta, uint4* aug, uint32_t* tbits, int64_t BH, int64_t t_blocks, int64_t i_blocks,
    TokenInfoArgs info)
{
    extern __shared__ uint32_t words[];
    int64_t b = blockIdx.x;
    if (b < t_blocks) {
        csr_transpose(a.row_start, a.row_count, a.col_idx, tbits, a.Tb, a.col_capacity, b, words);
    } else if ((b -= t_blocks) < i_blocks) {
        token_info(info, b * (kBwdPrepThreads / 32) + (threadIdx.x >> 5));
    } else {
        attn_stat<D>(op, dop, lse, lse2, delta, aug, a.N, a.Tb, BH, 1.f / a.scale_log2, b - i_blocks);
    }
}

// One CTA's pass over resident pair `item` (of B*H*pairs).
template <int D, bool kCol, bool kCap>
__device__ __forceinline__ void bwd_pass(const CUtensorMap& tm_r1, const CUtensorMap& tm_r2, const CUtensorMap& tm_t1,
                                         const CUtensorMap& tm_t2, const BwdArgs& args, int64_t item)
{
    using Cfg = BwdCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    const uint32_t base_u32 = (raw_u32 + 1023u) & ~1023u;
    uint8_t* base = smem_raw + (base_u32 - raw_u32);
    uint16_t* list = reinterpret_cast<uint16_t*>(base + Cfg::OFF_LIST);
    BwdCtl* ctl = reinterpret_cast<BwdCtl*>(base + Cfg::OFF_LIST + Cfg::list_bytes(args.Tb));

    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const int lane = tid & 31;
    const int Tb = args.Tb;

    // A head's sink pairs (the longest lists) first, as in the forward kernel.
    const int64_t bh = item / args.pairs;
    int pair;
    {
        const int u = (int)(item - bh * args.pairs);
        pair = (u < args.sink_pairs) ? args.pairs - 1 - u : u - args.sink_pairs;
    }
    const int rb0 = 2 * pair;
    const bool has_b = rb0 + 1 < Tb;

    if (tid == 0) {
        mbar_init(smem_u32(&ctl->r_full), 1);
        #pragma unroll
        for (int i = 0; i < Cfg::S1; ++i) {
            mbar_init(smem_u32(&ctl->t1_full[i]), 1);
            mbar_init(smem_u32(&ctl->t1_free[i]), 1);
        }
        for (int i = 0; i < Cfg::S2; ++i) {
            mbar_init(smem_u32(&ctl->t2_full[i]), 1);
            mbar_init(smem_u32(&ctl->t2_free[i]), 1);
        }
        mbar_init(smem_u32(&ctl->s_full), 1);
        mbar_init(smem_u32(&ctl->dp_full[0]), 1);
        mbar_init(smem_u32(&ctl->dp_full[1]), 1);
        mbar_init(smem_u32(&ctl->a_done), Cfg::SOFTMAX_WARPS);
        mbar_init(smem_u32(&ctl->b_done[0]), Cfg::SOFTMAX_WARPS);
        mbar_init(smem_u32(&ctl->b_done[1]), Cfg::SOFTMAX_WARPS);
        mbar_init(smem_u32(&ctl->final), 1);
        mbar_init(smem_u32(&ctl->drain), 1);
        ctl->abort = 0;
        fence_mbar_init();
        mbar_arrive_expect_tx(smem_u32(&ctl->r_full), 2 * Cfg::TILE);
        tma_load_4d(base_u32 + Cfg::OFF_R1, &tm_r1, smem_u32(&ctl->r_full), 0, rb0 * 64, 0, (int)bh);
        tma_load_4d(base_u32 + Cfg::OFF_R2, &tm_r2, smem_u32(&ctl->r_full), 0, rb0 * 64, 0, (int)bh);
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(&ctl->tmem_base), Cfg::TM_COLS);
        tmem_relinquish();
    }
    if (kCol) {
        // the resident side of the extra K step: ones in columns 0-2 (S: the log-sum-exp's parts)
        // or 3-5 (dP: delta's); and the zeros
        constexpr uint32_t one = 0x3f80u, ones2 = one | one << 16;
        for (int r = tid; r < 128; r += Cfg::THREADS) {
            *reinterpret_cast<uint4*>(base + Cfg::OFF_AUG_S + r * 16) = make_uint4(ones2, one, 0u, 0u);
            *reinterpret_cast<uint4*>(base + Cfg::OFF_AUG_P + r * 16) = make_uint4(0u, one << 16, ones2, 0u);
            *reinterpret_cast<uint4*>(base + Cfg::OFF_ZERO + r * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
    }
    // ---- union of the pair's two lists: kept and partial bitmaps, built in the unused T1 stages
    const int W = (Tb + 31) >> 5;                          // <= 128 words
    uint32_t* bmA = reinterpret_cast<uint32_t*>(base + Cfg::OFF_T1);
    uint32_t* bmB = bmA + W;
    uint32_t* partA = bmB + W;
    uint32_t* partB = partA + W;
    int32_t* word_off = reinterpret_cast<int32_t*>(partB + W);
    for (int w = tid; w < 4 * W; w += Cfg::THREADS) bmA[w] = 0u;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    {
        const int4* sum = args.mod.info.summary + (bh / args.mod.heads) * Tb;
        int4 sumA = make_int4(0, 0, 0, 0), sumB = sumA;
        if (args.mod.masked) {
            sumA = sum[rb0];
            if (has_b) sumB = sum[rb0 + 1];
        }
        auto set_bit = [&](int half, int32_t j) {
            int vis = 1;
            if (args.mod.masked) {
                const int4 own = half ? sumB : sumA, other = sum[j];
                vis = kCol ? block_visibility(other, own) : block_visibility(own, other);
            }
            if (vis == 0) return;
            if (vis == 2) atomicOr(&(half ? partB : partA)[j >> 5], 1u << (j & 31));
            atomicOr(&(half ? bmB : bmA)[j >> 5], 1u << (j & 31));
        };
        for (int half = 0; half < (has_b ? 2 : 1); ++half) {
            if (kCol) {
                const uint32_t* col = args.tbits + bh * W * Tb + rb0 + half;
                for (int i = tid; i < Tb; i += Cfg::THREADS)
                    if (col[(int64_t)(i >> 5) * Tb] >> (i & 31) & 1u) set_bit(half, i);
            } else {
                const int64_t r = bh * Tb + rb0 + half;
                const int32_t cnt = args.row_count[r], start = args.row_start[r];
                int len = min(max(cnt, 0), Tb);
                if (RF2_CHECKED && !in_range(cnt >= 0 && cnt <= Tb && start >= 0 &&
                                             (int64_t)start + cnt <= args.col_capacity))
                    len = 0;
                for (int e = tid; e < len; e += Cfg::THREADS) {
                    const int32_t j = args.col_idx[(int64_t)start + e];
                    if (in_range(j >= 0 && j < Tb) && j >= 0 && j < Tb) set_bit(half, j);
                }
            }
        }
    }
    __syncthreads();
    if (warp == 0) {
        int cnt[4];
        int local = 0;
        #pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int w = lane * 4 + k;
            cnt[k] = (w < W) ? __popc(bmA[w] | bmB[w]) : 0;
            local += cnt[k];
        }
        int incl = local;
        #pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += v;
        }
        int run = incl - local;
        #pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int w = lane * 4 + k;
            if (w < W) word_off[w] = run;
            run += cnt[k];
        }
        if (lane == 31) ctl->list_len = incl;
    }
    __syncthreads();
    for (int w = tid; w < W; w += Cfg::THREADS) {
        const uint32_t a = bmA[w], b = bmB[w];
        uint32_t m = a | b;
        int pos = word_off[w];
        while (m) {
            const int bit = __ffs(m) - 1;
            m &= m - 1;
            list[pos++] = bwd_entry(w * 32 + bit, a >> bit & 1u, b >> bit & 1u, partA[w] >> bit & 1u, partB[w] >> bit & 1u);
        }
    }
    __syncthreads();
    const int L = ctl->list_len;
    volatile int* abort = &ctl->abort;
    const int P = (L + 1) >> 1;                  // steps
    auto block_of = [&](int e) -> int { return list[e] & 0xfff; };
    // dP buffer of a step, and the parity of its barriers
    auto dp_buf = [](int p) -> int { return kCol ? 0 : p & 1; };
    auto dp_par = [](int p) -> uint32_t { return (kCol ? p : p >> 1) & 1; };
    // stages of a step, and the parities of their barriers
    constexpr int S1 = Cfg::S1, S2 = Cfg::S2;
    auto st1 = [](int p) -> int { return p % S1; };
    auto par1 = [](int p) -> uint32_t { return (p / S1) & 1; };
    auto st2 = [](int p) -> int { return p % S2; };
    auto par2 = [](int p) -> uint32_t { return (p / S2) & 1; };
    // info of the step's entry i (0 or 1)
    auto info_at = [&](int p, int i) -> uint32_t { return Cfg::OFF_INFO + (st1(p) * 2 + i) * Cfg::INFO; };

    if (warp == Cfg::T1_WARP || warp == Cfg::T2_WARP) {
        // ------------------------------------------------ TMA producers
        if (lane == 0) {
            fence_proxy_async_smem();   // the stages held the bitmaps (generic accesses)
            const bool second = warp == Cfg::T2_WARP;
            const uint32_t info_bytes = second ? 0
                : (args.mod.masked ? Cfg::INFO_MASK : 0) + (args.mod.slopes ? Cfg::INFO_POS : 0) +
                  (kCol ? Cfg::AUG_HALF + (kCap ? Cfg::INFO_LSE : 0) : 0);
            int issued = -1;
            for (int p = 0; p < P; ++p) {
                const int n = min(2, L - 2 * p);
                bool ok = true;
                if (!second) {
                    if (p >= S1) ok = mbar_wait(smem_u32(&ctl->t1_free[st1(p)]), par1(p - S1), abort, args.status);
                } else if (p >= S2) {
                    ok = kCol ? mbar_wait(smem_u32(&ctl->t2_free[st2(p)]), par2(p - S2), abort, args.status)
                              : mbar_wait(smem_u32(&ctl->dp_full[dp_buf(p - 1)]), dp_par(p - 1), abort, args.status);
                }
                if (!ok) break;
                const uint32_t bar = smem_u32(second ? &ctl->t2_full[st2(p)] : &ctl->t1_full[st1(p)]);
                const uint32_t dst = base_u32 + (second ? Cfg::OFF_T2 + st2(p) * Cfg::TILE : Cfg::OFF_T1 + st1(p) * Cfg::TILE);
                mbar_arrive_expect_tx(bar, n * (Cfg::HALF * Cfg::KCH + info_bytes));
                for (int i = 0; i < n; ++i) {
                    const int j = block_of(2 * p + i);
                    #pragma unroll
                    for (int c = 0; c < Cfg::KCH; ++c)
                        tma_load_3d(dst + c * Cfg::CHUNK + i * Cfg::HALF, second ? &tm_t2 : &tm_t1, bar, c * 64, j * 64, (int)bh);
                    if (!second) {
                        const uint32_t at = base_u32 + info_at(p, i);
                        if (args.mod.masked)
                            bulk_load(at, args.mod.info.mask + ((bh / args.mod.heads) * Tb + j) * kMaskSlots, Cfg::INFO_MASK,
                                      bar);
                        if (args.mod.slopes)
                            bulk_load(at + Cfg::INFO_MASK, args.mod.info.pos + (int64_t)j * kPosSlots, Cfg::INFO_POS, bar);
                        if (kCol) {
                            const int64_t slot = (bh * Tb + j) * kBlock;
                            bulk_load(base_u32 + Cfg::OFF_AUG_T + st1(p) * Cfg::AUG + i * Cfg::AUG_HALF, args.aug + slot,
                                      Cfg::AUG_HALF, bar);
                            if (kCap)
                                bulk_load(at + Cfg::INFO_MASK + Cfg::INFO_POS, args.lse2 + slot, Cfg::INFO_LSE, bar);
                        }
                    }
                }
                issued = p;
            }
            // Drain: no copy may still be writing shared memory when the CTA exits.
            if (!second) {
                mbar_wait_drain(smem_u32(&ctl->r_full), 0);
                for (int p = max(issued - S1 + 1, 0); p <= issued; ++p) mbar_wait_drain(smem_u32(&ctl->t1_full[st1(p)]), par1(p));
            } else {
                for (int p = max(issued - S2 + 1, 0); p <= issued; ++p) mbar_wait_drain(smem_u32(&ctl->t2_full[st2(p)]), par2(p));
            }
        }
    } else if (warp == Cfg::MMA_WARP) {
        // ------------------------------------------------ MMA issuer: the whole warp runs the
        // loop, one lane issues
        {
            const bool lead = elect_one();
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            constexpr uint32_t IDESC_A = idesc_bf16_f32(128, D, 1);
            const uint64_t d1 = smem_desc_sw128(base_u32 + Cfg::OFF_R1, 16, 1024);
            const uint64_t d2 = smem_desc_sw128(base_u32 + Cfg::OFF_R2, 16, 1024);
            const uint64_t k1 = smem_desc_sw128(base_u32 + Cfg::OFF_T1, 16, 1024);             // streamed, K-major
            const uint64_t k2 = smem_desc_sw128(base_u32 + Cfg::OFF_T2, 16, 1024);
            const uint64_t m1 = smem_desc_sw128(base_u32 + Cfg::OFF_T1, Cfg::CHUNK, 1024);     // MN-major
            const uint64_t m2 = smem_desc_sw128(base_u32 + Cfg::OFF_T2, Cfg::CHUNK, 1024);
            // the extra K step: 16-byte rows, 8-row groups 128 bytes apart, columns 8-15 at the zeros
            auto aug_desc = [&](uint32_t off) -> uint64_t {
                return smem_desc_none(base_u32 + off, Cfg::OFF_ZERO - off, 128);
            };
            const uint64_t as = aug_desc(Cfg::OFF_AUG_S), ap = aug_desc(Cfg::OFF_AUG_P);
            // resident (128 x d) times the step's tile of N tokens (64 in a last step of one entry)
            auto scores_of = [&](uint32_t idesc, uint32_t dst, uint64_t res, uint64_t tile, uint64_t aug, bool has_aug, int p) {
                #pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * Cfg::CHUNK + (kk & 3) * 32) >> 4;
                    mma_ss_by(lead, dst, res + off, tile + off, idesc, kk > 0 ? 1u : 0u);
                }
                if (has_aug) mma_ss_by(lead, dst, aug, aug_desc(Cfg::OFF_AUG_T + st1(p) * Cfg::AUG), idesc, 1u);
            };
            auto mma_scores = [&](uint32_t dst, uint64_t res, uint64_t tile, uint64_t aug, bool has_aug, int p) {
                if (2 * p + 1 < L) scores_of(idesc_bf16_f32(128, 128, 0), dst, res, tile, aug, has_aug, p);
                else               scores_of(idesc_bf16_f32(128, 64, 0), dst, res, tile, aug, has_aug, p);
            };
            // acc += P or dS (TMEM, bf16) times the step's tile
            auto mma_acc = [&](uint32_t acc, uint32_t a, uint64_t tile, int p) {
                #pragma unroll
                for (int kk = 0; kk < 4; ++kk)          // 16 tokens a K step
                    mma_ts_by(lead, acc, a + (kk >> 1) * 32 + (kk & 1) * 8, tile + ((kk * 2048) >> 4), IDESC_A,
                              (p > 0 || kk > 0) ? 1u : 0u);
                if (2 * p + 1 < L) {
                    #pragma unroll
                    for (int kk = 4; kk < 8; ++kk)
                        mma_ts_by(lead, acc, a + (kk >> 1) * 32 + (kk & 1) * 8, tile + ((kk * 2048) >> 4), IDESC_A, 1u);
                }
            };
            auto commit = [&](uint64_t* bar) {
                if (lead) mma_commit(smem_u32(bar));
                __syncwarp();
            };
            auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
                const bool r = __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, abort, args.status));
                tc_fence_after();
                return r;
            };
            auto stage1 = [&](int p) -> uint32_t { return (st1(p) * Cfg::TILE) >> 4; };
            auto stage2 = [&](int p) -> uint32_t { return (st2(p) * Cfg::TILE) >> 4; };
            auto issue_s = [&](int p) -> bool {
                if (!wait(&ctl->t1_full[st1(p)], par1(p))) return false;
                mma_scores(tm + Cfg::tm_s(kCol), d1, k1 + stage1(p), as, kCol && !kCap, p);
                commit(&ctl->s_full);
                return true;
            };
            auto issue_dp = [&](int p) -> bool {
                if (!wait(&ctl->t2_full[st2(p)], par2(p))) return false;
                mma_scores(tm + Cfg::tm_dp(kCol, p), d2, k2 + stage2(p), ap, kCol, p);
                commit(&ctl->dp_full[dp_buf(p)]);
                return true;
            };
            bool ok = (L == 0) || (wait(&ctl->r_full, 0) && issue_s(0) && issue_dp(0));
            for (int p = 0; ok && p < P; ++p) {
                const bool more = p + 1 < P;
                if (!(ok = (kCol || more) ? wait(&ctl->a_done, p & 1) : true)) break;
                if (kCol) {
                    mma_acc(tm + Cfg::TM_ACC2, tm + Cfg::tm_s(kCol), m2 + stage2(p), p);
                    commit(&ctl->t2_free[st2(p)]);
                }
                if (more && !(ok = issue_s(p + 1))) break;
                if (!kCol && more && !(ok = issue_dp(p + 1))) break;
                if (!(ok = wait(&ctl->b_done[dp_buf(p)], dp_par(p)))) break;
                mma_acc(tm + Cfg::TM_ACC1, tm + Cfg::tm_dp(kCol, p), m1 + stage1(p), p);
                commit(&ctl->t1_free[st1(p)]);
                if (kCol && more) ok = issue_dp(p + 1);
            }
            commit(&ctl->final);
            commit(&ctl->drain);
            mbar_wait_drain(smem_u32(&ctl->drain), 0);
        }
    } else if (warp < Cfg::SOFTMAX_WARPS) {
        // ------------------------------------------------ softmax
        constexpr int NH = Cfg::HALVES;
        const int part = warp >> 2;                // the thread's columns: NH pieces of 32
        const int i = part * NH >> 1;              // the step's entry
        const int h0 = part * NH & 1;              // its first piece of the entry
        const int row = (warp & 3) * 32 + lane;    // resident row = TMEM lane
        const int half = row >> 6;
        const int32_t tok = rb0 * kBlock + row;    // the row's token (permuted)
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const RowInfo ri = load_row_info(args.mod, bh, Tb, tok, tok < args.N);
        float nlse = 0.f, ndelta = 0.f;            // row pass: minus the row's log-sum-exp and delta
        if (!kCol) {
            nlse = tok < args.N ? -args.lse2[bh * Tb * kBlock + tok] : -kDeadLse;
            ndelta = tok < args.N ? -args.delta[bh * Tb * kBlock + tok] : 0.f;
        }
        const uint32_t s_cols = tmem + lane_addr + Cfg::tm_s(kCol) + 64 * i + 32 * h0;
        const bool staged = args.mod.masked || args.mod.slopes || (kCol && kCap);
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, abort, args.status));
        };
        // the warp's TMEM accesses so far are done: one arrival per warp
        auto arrive = [&](uint64_t* bar) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(bar));
        };
        for (int p = 0; p < P; ++p) {
            const int e = 2 * p + i;
            const uint32_t ent = (e < L) ? list[e] : 0u;
            const bool kept = ent >> (12 + half) & 1u;
            const bool partial = ent >> (14 + half) & 1u;
            ok = wait(&ctl->s_full, p & 1);
            // the staged info (S_p done implies its copies have landed; this thread has to see them)
            if (ok && staged) ok = wait(&ctl->t1_full[st1(p)], par1(p));
            if (!ok) break;
            tc_fence_after();
            const uint8_t* info = base + info_at(p, i);
            const int2* mask = reinterpret_cast<const int2*>(info);
            const uint32_t dp_cols = tmem + lane_addr + Cfg::tm_dp(kCol, p) + 64 * i + 32 * h0;
            // ---- part A: s -> P ds/dx
            uint32_t s[NH][32], vis[NH];
            bool hidden[NH];                           // some row of the warp has a hidden token
            #pragma unroll
            for (int n = 0; n < NH; ++n) vis[n] = 0xffffffffu, hidden[n] = false;
            if (kept) {
                #pragma unroll
                for (int n = 0; n < NH; ++n) tmem_ld32(s_cols + 32 * n, s[n]);
                tmem_wait_ld();
                #pragma unroll
                for (int n = 0; n < NH; ++n) reg_fence(s[n]);
            }
            if (!kCol) arrive(&ctl->a_done);
            if (kept) {
                #pragma unroll
                for (int n = 0; n < NH; ++n) {
                    const int h = h0 + n;
                    if (partial) {
                        const int rv = row_visibility<kCol>(ri, staged_summary(mask));
                        if (__any_sync(0xffffffffu, rv == 2)) vis[n] = visible_bits<kCol>(ri, mask + 32 * h);
                        else vis[n] = rv ? 0xffffffffu : 0u;
                    }
                    const int nv = args.N - (int)(ent & 0xfff) * 64 - 32 * h;
                    if (!kCol && nv < 32) vis[n] &= nv > 0 ? (1u << nv) - 1u : 0u;
                    if (partial || (!kCol && nv < 32)) hidden[n] = __any_sync(0xffffffffu, vis[n] != 0xffffffffu);
                    uint32_t pk[16];
                    // under the cap in pieces of 16 columns, which keeps the derivatives in registers (4% at 480p)
                    constexpr int W = kCap ? 16 : 32;
                    #pragma unroll
                    for (int o = 0; o < 32; o += W) {
                        uint32_t x[W], f[W];
                        #pragma unroll
                        for (int c = 0; c < W; ++c) x[c] = s[n][o + c];
                        if (kCap) {
                            if (hidden[n]) hide(x, vis[n] >> o, 0u);
                            cap_chunk<true>(x, f, args.mod);
                        }
                        // row pass: less the row's log-sum-exp
                        if (args.mod.slopes)
                            bias_chunk<!kCap>(x, ri, reinterpret_cast<const float4*>(info + Cfg::INFO_MASK), 32 * h + o,
                                              args.mod.step, args.scale_log2, nlse);
                        else if (!kCol || !kCap)
                            scale_chunk(x, kCap ? 1.f : args.scale_log2, nlse);
                        if (hidden[n]) hide(x, vis[n] >> o, kMinusInf);
                        if (kCol && kCap) {            // the queries'
                            const float4* lse =
                                reinterpret_cast<const float4*>(info + Cfg::INFO_MASK + Cfg::INFO_POS) + 8 * h + o / 4;
                            #pragma unroll
                            for (int c = 0; c < W; c += 4) {
                                const float4 l = lse[c >> 2];
                                x[c] = __float_as_uint(__uint_as_float(x[c]) - l.x);
                                x[c + 1] = __float_as_uint(__uint_as_float(x[c + 1]) - l.y);
                                x[c + 2] = __float_as_uint(__uint_as_float(x[c + 2]) - l.z);
                                x[c + 3] = __float_as_uint(__uint_as_float(x[c + 3]) - l.w);
                            }
                        }
                        // 3 of 8 pairs without the special function unit (3-5% of the whole at 480p), except
                        // where hidden pairs have to come out as 0, and under the cap, whose polynomial fills
                        // the multipliers already
                        auto probs = [&](auto exp2s) {
                            #pragma unroll
                            for (int c = 0; c < W; c += 2) {
                                const float2 pr = exp2s(c, make_float2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])));
                                if (kCol) pk[(o + c) >> 1] = pack_bf16x2(pr.x, pr.y);
                                const float2 g = kCap ? fmul2(pr, make_float2(__uint_as_float(f[c]), __uint_as_float(f[c + 1]))) : pr;
                                s[n][o + c] = __float_as_uint(g.x);
                                s[n][o + c + 1] = __float_as_uint(g.y);
                            }
                        };
                        auto exact2 = [](int, float2 v) { return make_float2(ex2_approx(v.x), ex2_approx(v.y)); };
                        if (!kCap && !hidden[n])
                            probs([&](int c, float2 v) { return ((c >> 1) & 7) < 3 ? ex2_poly(v) : exact2(c, v); });
                        else
                            probs(exact2);
                    }
                    if (kCol) tmem_st16(s_cols + 32 * n, pk);
                }
            } else if (kCol && e < L) {
                uint32_t pk[16];
                #pragma unroll
                for (int k = 0; k < 16; ++k) pk[k] = 0u;
                #pragma unroll
                for (int n = 0; n < NH; ++n) tmem_st16(s_cols + 32 * n, pk);
            }
            if (kept && partial && h0 == 0 && staged_summary(mask).x < 0) {
                // padding tokens: their rows of T1 and T2 before the accumulating products read them
                zero_padding_rows<D, Cfg::CHUNK>(base + Cfg::OFF_T1 + st1(p) * Cfg::TILE + i * Cfg::HALF, mask, lane);
                if (kCol) {
                    ok = wait(&ctl->dp_full[0], p & 1);
                    if (!ok) break;
                    zero_padding_rows<D, Cfg::CHUNK>(base + Cfg::OFF_T2 + st2(p) * Cfg::TILE + i * Cfg::HALF, mask, lane);
                }
                fence_proxy_async_smem();
            }
            if (kCol) {
                tmem_wait_st();
                arrive(&ctl->a_done);
            }
            // ---- part B: dS = P ds/dx (dP - delta)
            ok = wait(&ctl->dp_full[dp_buf(p)], dp_par(p));
            if (!ok) break;
            tc_fence_after();
            if (e < L) {
                #pragma unroll
                for (int n = 0; n < NH; ++n) {
                    uint32_t dk[16];
                    if (kept) {
                        uint32_t g[32];
                        tmem_ld32(dp_cols + 32 * n, g);
                        tmem_wait_ld();
                        reg_fence(g);
                        #pragma unroll
                        for (int c = 0; c < 32; c += 2) {
                            float2 x = make_float2(__uint_as_float(g[c]), __uint_as_float(g[c + 1]));
                            if (!kCol) x = fadd2(x, make_float2(ndelta, ndelta));
                            x = fmul2(x, make_float2(__uint_as_float(s[n][c]), __uint_as_float(s[n][c + 1])));
                            g[c] = __float_as_uint(x.x);
                            g[c + 1] = __float_as_uint(x.y);
                        }
                        if (hidden[n]) hide(g, vis[n], 0u);        // dP of a padding token may be anything
                        #pragma unroll
                        for (int c = 0; c < 32; c += 2)
                            dk[c >> 1] = pack_bf16x2(__uint_as_float(g[c]), __uint_as_float(g[c + 1]));
                    } else {
                        #pragma unroll
                        for (int k = 0; k < 16; ++k) dk[k] = 0u;
                    }
                    tmem_st16(dp_cols + 32 * n, dk);
                }
                tmem_wait_st();
            }
            arrive(&ctl->b_done[dp_buf(p)]);
        }
        // ---- epilogue: the accumulators' columns, dQ or dK then dV, dealt out to the parts
        if (ok && L > 0) ok = wait(&ctl->final, 0);
        tc_fence_after();
        if (ok) {
            constexpr int COLS = (kCol ? 2 * D : D) * NH / 4;
            const bool second = kCol && i;
            const int c_first = part * COLS - (second ? D : 0);
            const uint32_t acc = tmem + lane_addr + (second ? Cfg::TM_ACC2 : Cfg::TM_ACC1);
            const float scale = second ? 1.f : args.scale;
            uint16_t* dst = (!kCol ? args.dq : second ? args.dv : args.dk) + (bh * args.N + tok) * D;
            #pragma unroll 1
            for (int c0 = c_first; c0 < c_first + COLS; c0 += 16) {
                uint32_t o[16];
                if (L > 0) {
                    tmem_ld16(acc + c0, o);
                    tmem_wait_ld();
                    reg_fence(o);
                } else {
                    #pragma unroll
                    for (int c = 0; c < 16; ++c) o[c] = 0u;
                }
                if (tok < args.N) {
                    uint4* d4 = reinterpret_cast<uint4*>(dst + c0);
                    #pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t w[4];
                        #pragma unroll
                        for (int k = 0; k < 4; ++k)
                            w[k] = pack_bf16x2(__uint_as_float(o[8 * c + 2 * k]) * scale,
                                               __uint_as_float(o[8 * c + 2 * k + 1]) * scale);
                        d4[c] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, Cfg::TM_COLS);
    }
}

// Tensor maps: 128-row boxes of Q, dO, K, V (resident), 64-row boxes (streamed).
struct BwdMaps { CUtensorMap q128, do128, k128, v128, q64, do64, k64, v64; };

// Both passes in one launch, the column CTAs first (they take longer): one
// ragged last round instead of two, and small calls run them side by side
// (1,024 tokens, 2 heads: 63 us as two launches, 33 in one).  Measured against
// alternating the passes head by head: 5 to 10% faster on the image shape and
// under the cap, 2% slower on the large unmodified ones.
template <int D, bool kCap>
__global__ void __launch_bounds__(BwdCfg<D>::THREADS, 1)
block_sparse_attn_bwd_kernel(const __grid_constant__ BwdMaps m, const __grid_constant__ BwdArgs args)
{
    const int64_t half = gridDim.x / 2;
    if (blockIdx.x < half) bwd_pass<D, true, kCap>(m.k128, m.v128, m.q64, m.do64, args, blockIdx.x);
    else                   bwd_pass<D, false, kCap>(m.q128, m.do128, m.k64, m.v64, args, blockIdx.x - half);
}

}  // namespace rf2
