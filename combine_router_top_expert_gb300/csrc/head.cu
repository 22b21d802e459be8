// head.cu - softmax cross entropy of a large vocabulary from the last hidden rows
// and the vocabulary's weights, with its gradient, without the logits.
//
// With x [T,H], W [V,H] and the label y_t of token t:
//   l[t,v] = <x_t, W_v>      lse_t = log sum_v exp l[t,v]      loss_t = lse_t - l[t,y_t]
//   dl[t,v] = c_t (exp(l[t,v] - lse_t) - [v == y_t])           c_t = scale * dloss_t
//   dX = dl W                dW = dl^T x
// Tokens whose label is outside 0..V-1 count for nothing: the live ones are
// gathered first (head_prep_kernel), so what their rows hold does not matter and
// none of the products is spent on them.
//
// Three products, each a persistent tcgen05 kernel over 256 x 256 tiles of 2-SM
// pairs (head_gemm_kernel):
//   logits  x W^T    both operands K-major; the epilogue reduces 128 columns of a row
//                    to (max, sum of exponentials, label's logit), so that a logit
//                    lives in tensor memory and registers only, and with a gradient
//                    writes dl (log-sum known) or the exponentials, which
//                    head_dl_kernel turns into dl in their place
//   dX      dl W     A K-major, B MN-major (the vocabulary is K)
//   dW      dl^T x   both MN-major (the tokens are K)
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "moves.cuh"
#include "tc.cuh"

namespace mok {

namespace {

constexpr int kBM = 256, kBN = 256;     // tile of a pair of CTAs
constexpr int kBK = 64;                 // K elements of a stage (128 bytes)
constexpr int kStages = 6;
constexpr int kEpiWarps = 8;            // two per TMEM lane quadrant, 128 columns each
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kOperandBytes = 128 * kBK * 2;          // a CTA's share of A or of B
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kBarOffset = kStages * kStageBytes;
constexpr int kSmemBytes = 1024 + kBarOffset + 256;
constexpr int kStatCols = 128;          // columns behind one (max, sum)
// K blocks of a logit that are summed in tensor memory; these sums are then added in
// registers. The tensor cores cut what they add to an accumulator instead of rounding
// it, which makes a long sum too small by up to 2^-24 of itself a step: H = 7168 in one
// sum moved a loss by 4.8e-6 of itself, in sums of 1024 by what the other roundings do.
constexpr int kLogitBlocks = 16;
constexpr float kLog2e = 1.4426950408889634f;
// An exponential e is kept as its root times 2^15, s = 2^15 exp((l - top) / 2): FP16 then has a relative error of
// 2^-11 in s, 2^-10 in e, down to e = 2^-58 (e itself would lose bits below 2^-29).
constexpr float kRootShift = 15.f;
constexpr float kRootScale = 1.f / (1 << 30);   // s * s * kRootScale = e

enum HeadEpi : int {
    kEpiStats = 0,   // (max, sum, label's logit)
    kEpiExp = 1,     // the same, and the exponentials
    kEpiDl = 2,      // dl from a known log-sum
    kEpiOut = 3,     // the product itself: BF16 rows, or fp32 rows, or a partial sum
};

struct HeadGemm {
    const int32_t* live;    // live tokens on the device, or NULL (all)
    int tokens;             // tokens of the piece (the live ones' upper bound)
    int M, N, K;            // K or M is the token count where m_live / k_live is set
    int m_live, k_live;
    int splits;             // parts of K, each a tile of its own
    int group;              // row tiles that are walked together
    // logits
    const void* labels;
    int labels_i64;
    const int32_t* rows;    // live token -> token, or NULL
    float2* stats;          // [tokens, stat tiles]
    int stat_tiles;
    float* label_logit;     // [tokens]
    const float* lse;       // [T]
    const float* dloss;     // [T] or NULL
    float scale;
    __nv_bfloat16* dl;      // [tokens rounded up to 256, ld]
    int64_t ld_dl;
    // products
    void* out;
    int out_f32;
    const float* add;       // fp32 rows that are added to the product, or NULL
    int64_t split_stride;   // elements between the parts' outputs
    const int32_t* out_rows;   // row -> output row, or NULL
    StatusBlock* status;
    unsigned long long timeout_ns;
};

__device__ __forceinline__ float exp2_approx(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ int64_t label_at(const void* labels, int i64, int64_t t) {
    return i64 ? __ldg(static_cast<const long long*>(labels) + t) : (int64_t)__ldg(static_cast<const int32_t*>(labels) + t);
}

struct Tile {
    int m, n, split;
};
// Row tiles in groups of p.group; inside a group column tiles in turn with the
// group's row tiles side by side, so that the pairs that run at once share tiles of
// both operands in L2.
__device__ __forceinline__ Tile head_tile(int g, int mt, int nt, int group) {
    Tile t;
    t.split = g / (mt * nt);
    g -= t.split * mt * nt;
    const int first = g / (group * nt) * group;
    const int rows = min(group, mt - first);
    g -= first * nt;
    t.m = first + g % rows;
    t.n = g / rows;
    return t;
}

// 32 lanes x 16 consecutive 32-bit columns of tensor memory.
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32"
        " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

template <bool A_MN, bool B_MN, int EPI>
__global__ void __launch_bounds__(kThreads, 1)
head_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmAll, const HeadGemm p) {
    // tmAll: the caller's own rows in place of the gathered ones, taken when every
    // token is live (logits: A, dW: B)
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ uint32_t s_tmem_base;
    const uint32_t smem_base = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t bar_base = smem_base + kBarOffset;
    auto full_bar = [&](int s) { return bar_base + 8u * s; };
    auto empty_bar = [&](int s) { return bar_base + 8u * (kStages + s); };
    auto accf_bar = [&](int a) { return bar_base + 8u * (2 * kStages + a); };
    auto acce_bar = [&](int a) { return bar_base + 8u * (2 * kStages + 2 + a); };
    const uint32_t drain_bar = bar_base + 8u * (2 * kStages + 4);
    auto a_tile = [&](int s) { return smem_base + s * kStageBytes; };
    auto b_tile = [&](int s) { return smem_base + s * kStageBytes + kOperandBytes; };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    StatusBlock* st = p.status;
    const uint64_t tmo = p.timeout_ns;
    if (threadIdx.x == 32) {
        for (int s = 0; s < kStages; ++s) {
            tc::mbar_init(full_bar(s), 1);
            tc::mbar_init(empty_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            tc::mbar_init(accf_bar(a), 1);
            tc::mbar_init(acce_bar(a), 32 * kEpiWarps * 2);   // both CTAs' epilogue threads
        }
        tc::mbar_init(drain_bar, 1);
        tc::fence_mbar_init();
    }
    if (threadIdx.x == 0) {
        tc::prefetch_tmap(&tmA);
        tc::prefetch_tmap(&tmB);
        tc::prefetch_tmap(&tmAll);
    }
    if (warp == 1) {
        tc::tmem_alloc_2sm(tc::smem_u32(&s_tmem_base), 512);
        tc::tmem_relinquish_2sm();
    }
    pdl_wait();
    pdl_allow_next();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    tc::cluster_sync();   // the peer's barriers and tensor memory exist
    const uint32_t tmem = s_tmem_base;
    const int rank = (int)tc::cluster_ctarank();

    const int live = p.live ? *p.live : p.tokens;
    const bool all = live == p.tokens;
    const int M = p.m_live ? live : p.M, K = p.k_live ? live : p.K;
    const int mt = (M + kBM - 1) / kBM, nt = (p.N + kBN - 1) / kBN;
    const int kbs = (K + kBK - 1) / kBK;
    const int total = mt * nt * p.splits;
    const int gstart = (int)blockIdx.x / 2, gstep = (int)gridDim.x / 2;
    constexpr int kSumBlocks = EPI == kEpiOut ? 1 << 30 : kLogitBlocks;   // K blocks of an accumulator's sum
    auto k_first = [&](int split) { return (int)((int64_t)kbs * split / p.splits); };

    if (warp == 0) {
        if (lane == 0) {
            const void* mapA = EPI != kEpiOut && all ? (const void*)&tmAll : (const void*)&tmA;
            const void* mapB = A_MN && B_MN && all ? (const void*)&tmAll : (const void*)&tmB;
            int stage = 0;
            uint32_t ph = 0;
            int last_par[kStages];
            for (int s = 0; s < kStages; ++s) last_par[s] = -1;
            bool ok = true;
            for (int g = gstart; g < total && ok; g += gstep) {
                const Tile t = head_tile(g, mt, nt, p.group);
                const int m0 = t.m * kBM + rank * 128, n0 = t.n * kBN + rank * 128;
                const int kend = k_first(t.split + 1);
                for (int kb = k_first(t.split); kb < kend; ++kb) {
                    if (!tc::mbar_wait(empty_bar(stage), ph ^ 1u, st, tmo, kSiteProducerEmpty)) { ok = false; break; }
                    // both halves signal the leader's barrier, which expects both
                    const uint32_t lead = tc::mapa_shared(full_bar(stage), 0);
                    if (rank == 0) tc::mbar_expect_tx(full_bar(stage), 2 * kStageBytes);
                    const int k0 = kb * kBK;
                    if constexpr (A_MN) {
                        tc::tma_load_2d_2sm(a_tile(stage), mapA, lead, m0, k0);
                        tc::tma_load_2d_2sm(a_tile(stage) + 8192, mapA, lead, m0 + 64, k0);
                    } else {
                        tc::tma_load_2d_2sm(a_tile(stage), mapA, lead, k0, m0);
                    }
                    if constexpr (B_MN) {
                        tc::tma_load_2d_2sm(b_tile(stage), mapB, lead, n0, k0);
                        tc::tma_load_2d_2sm(b_tile(stage) + 8192, mapB, lead, n0 + 64, k0);
                    } else {
                        tc::tma_load_2d_2sm(b_tile(stage), mapB, lead, k0, n0);
                    }
                    last_par[stage] = (int)ph;
                    if (++stage == kStages) { stage = 0; ph ^= 1u; }
                }
            }
            if (!ok) {
                // let every copy already issued land before the CTA exits
                for (int s = 0; s < kStages; ++s)
                    if (last_par[s] >= 0) tc::mbar_wait(full_bar(s), (uint32_t)last_par[s], st, tmo, kSiteDrain);
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            int stage = 0, acc = 0;
            uint32_t ph = 0, acc_ph = 0;
            bool ok = true, issued = false;
            for (int g = gstart; g < total && ok; g += gstep) {
                const int split = g / (mt * nt);
                const int kb0 = k_first(split), kb1 = k_first(split + 1);
                if (kb0 == kb1) continue;
                for (int kb = kb0; kb < kb1; ++kb) {
                    const bool first = (kb - kb0) % kSumBlocks == 0;
                    if (first) {
                        if (!tc::mbar_wait(acce_bar(acc), acc_ph ^ 1u, st, tmo, kSiteMmaAccEmpty)) { ok = false; break; }
                        tc::fence_after_sync();
                    }
                    const uint32_t d = tmem + (uint32_t)(acc * kBN);
                    if (!tc::mbar_wait(full_bar(stage), ph, st, tmo, kSiteMmaFull)) { ok = false; break; }
                    tc::fence_after_sync();
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk) {
                        const uint64_t ad = A_MN ? tc::make_sdesc(a_tile(stage) + kk * 2048, 8192, 1024, tc::kLayoutSW128)
                                                 : tc::make_sdesc(a_tile(stage) + kk * 32, 16, 1024, tc::kLayoutSW128);
                        const uint64_t bd = B_MN ? tc::make_sdesc(b_tile(stage) + kk * 2048, 8192, 1024, tc::kLayoutSW128)
                                                 : tc::make_sdesc(b_tile(stage) + kk * 32, 16, 1024, tc::kLayoutSW128);
                        tc::mma_bf16_2sm(d, ad, bd, tc::idesc_bf16(kBM, kBN, A_MN, B_MN), !first || kk > 0 ? 1u : 0u);
                    }
                    issued = true;
                    tc::mma_commit_2sm_multicast(empty_bar(stage), (uint16_t)0x3);
                    if (++stage == kStages) { stage = 0; ph ^= 1u; }
                    if (kb + 1 == kb1 || (kb + 1 - kb0) % kSumBlocks == 0) {
                        tc::mma_commit_2sm_multicast(accf_bar(acc), (uint16_t)0x3);
                        if (++acc == 2) { acc = 0; acc_ph ^= 1u; }
                    }
                }
            }
            if (!ok && issued) {
                // every MMA issued so far must finish before tensor memory is freed
                tc::mma_commit_2sm(drain_bar);
                tc::mbar_wait(drain_bar, 0, st, tmo, kSiteDrain);
            }
        }
    } else {
        const int q = warp & 3, half = (warp - 2) >> 2;   // TMEM lane quadrant, 128-column half of the tile
        int acc = 0;
        uint32_t acc_ph = 0;
        for (int g = gstart; g < total; g += gstep) {
            const Tile t = head_tile(g, mt, nt, p.group);
            const int blocks = k_first(t.split + 1) - k_first(t.split);
            float r[4][32];
            __syncwarp();
            bool ok = true;
            for (int b0 = 0; b0 < blocks; b0 += min(kSumBlocks, blocks - b0)) {
                if (!tc::mbar_wait(accf_bar(acc), acc_ph, st, tmo, kSiteEpiAccFull)) { ok = false; break; }
                __syncwarp();
                tc::fence_after_sync();
                const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kBN + half * 128);
                if (EPI == kEpiOut || b0 == 0) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        tc::tmem_ld_32x32b_x32(tbase + 32 * c, reinterpret_cast<uint32_t(&)[32]>(r[c]));
                    tc::tmem_ld_wait();
                } else {
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        uint32_t v[16];
                        tmem_ld_x16(tbase + 16 * c, v);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) r[c / 2][16 * (c % 2) + i] += __uint_as_float(v[i]);
                    }
                }
                tc::fence_before_sync();
                tc::mbar_arrive_cluster(tc::mapa_shared(acce_bar(acc), 0));
                if (++acc == 2) { acc = 0; acc_ph ^= 1u; }
            }
            if (!ok) break;
            if (blocks == 0) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 32; ++i) r[c][i] = 0.f;
            }
            const int row = t.m * kBM + rank * 128 + q * 32 + lane;
            const int col0 = t.n * kBN + half * 128;
            const int nv = min(128, p.N - col0);          // valid columns; none: <= 0
            if constexpr (EPI == kEpiStats || EPI == kEpiExp) {
                if (EPI == kEpiExp && row >= M && nv > 0) {
                    // rows behind the last live token are zeros: dW's last K block reads them
                    __nv_bfloat16* o = p.dl + (int64_t)row * p.ld_dl + col0;
                    const uint32_t z[8] = {};
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        if (16 * c < nv) tc::stg_v8(o + 16 * c, z);
                }
                if (row < M && nv > 0) {
                    const int64_t tok = p.rows && !all ? p.rows[row] : row;
                    int64_t lab = label_at(p.labels, p.labels_i64, tok);
                    if (lab < 0 || lab >= p.N) lab = -1;
                    const int lc = lab >= col0 && lab < col0 + nv ? (int)(lab - col0) : -1;
                    if (nv < 128) {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int i = 0; i < 32; ++i) r[c][i] = 32 * c + i < nv ? r[c][i] : -INFINITY;
                    }
                    float mx = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int i = 0; i < 32; ++i) mx = fmaxf(mx, r[c][i]);
                    const float base = kRootShift - (mx == -INFINITY ? 0.f : mx * (0.5f * kLog2e));
                    // the label's own term stays out of the sum, so that the others' share keeps its
                    // digits where the label takes nearly everything
                    float s[4] = {0.f, 0.f, 0.f, 0.f};
                    if constexpr (EPI == kEpiStats) {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const float e = exp2_approx(fmaf(r[c][i], 0.5f * kLog2e, base));
                                s[c] = 32 * c + i == lc ? s[c] : fmaf(e, e, s[c]);
                            }
                    } else {
                        // relative to the 128 columns' largest: head_dl_kernel makes dl of them
                        __nv_bfloat16* o = p.dl + (int64_t)row * p.ld_dl + col0;
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            if (16 * c >= nv) break;
                            uint32_t w[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                float e[2];
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const int j = 16 * c + 2 * i + h;
                                    e[h] = exp2_approx(fmaf(r[j / 32][j % 32], 0.5f * kLog2e, base));
                                    s[c / 2] = j == lc ? s[c / 2] : fmaf(e[h], e[h], s[c / 2]);
                                }
                                const __half2 v = __floats2half2_rn(e[0], e[1]);
                                w[i] = *reinterpret_cast<const uint32_t*>(&v);
                            }
                            tc::stg_v8(o + 16 * c, w);
                        }
                    }
                    if (lc >= 0) {
                        float own = 0.f;
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int i = 0; i < 32; ++i) own = 32 * c + i == lc ? r[c][i] : own;
                        p.label_logit[row] = own;
                    }
                    const float sum = ((s[0] + s[1]) + (s[2] + s[3])) * kRootScale;
                    p.stats[(int64_t)row * p.stat_tiles + col0 / kStatCols] = make_float2(mx, sum);
                }
            } else if constexpr (EPI == kEpiDl) {
                if (nv > 0) {
                    float coef = 0.f, base = 0.f;
                    int lc = -1;
                    // rows behind the last live token are zeros: dW's last K block reads them
                    const bool in = row < M;
                    if (in) {
                        const int64_t tok = p.rows && !all ? p.rows[row] : row;
                        const int64_t lab = label_at(p.labels, p.labels_i64, tok);
                        coef = p.scale * (p.dloss ? __ldg(p.dloss + tok) : 1.0f);
                        base = __ldg(p.lse + tok);
                        lc = lab >= col0 && lab < col0 + nv ? (int)(lab - col0) : -1;
                    }
                    __nv_bfloat16* o = p.dl + (int64_t)row * p.ld_dl + col0;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (32 * c >= nv) break;
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float v[2];
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                v[h] = in ? coef * exp2_approx((r[c][2 * i + h] - base) * kLog2e) : 0.f;
                            w[i] = pack_bf16x2(v[0], v[1]);
                        }
                        tc::stg_v8(o + 32 * c, w);
                        tc::stg_v8(o + 32 * c + 16, w + 8);
                    }
                    if (lc >= 0) {
                        float own = 0.f;
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int i = 0; i < 32; ++i) own = 32 * c + i == lc ? r[c][i] : own;
                        o[lc] = __float2bfloat16_rn(coef * expm1f(own - base));
                    }
                }
            } else {
                if (row < M && nv > 0) {
                    const int64_t orow = p.out_rows && !all ? p.out_rows[row] : row;
                    const int64_t at = t.split * p.split_stride + orow * p.N + col0;
#pragma unroll
                    for (int c = 0; c < 16; ++c) {     // N is a multiple of 8
                        if (8 * c >= nv) break;
                        float v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = r[c / 4][8 * (c % 4) + i];
                        if (p.add) {
                            const float4 a = *reinterpret_cast<const float4*>(p.add + at + 8 * c);
                            const float4 b = *reinterpret_cast<const float4*>(p.add + at + 8 * c + 4);
                            v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
                            v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
                        }
                        if (p.out_f32) {
                            float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at + 8 * c);
                            o[0] = make_float4(v[0], v[1], v[2], v[3]);
                            o[1] = make_float4(v[4], v[5], v[6], v[7]);
                        } else {
                            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + at + 8 * c) =
                                make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                           pack_bf16x2(v[6], v[7]));
                        }
                    }
                }
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    tc::cluster_sync();   // no CTA frees or leaves while its peer may still use the pair's resources
    if (warp == 1) tc::tmem_dealloc_2sm(tmem, 512);
}

// ------------------------------------------------------------------ live tokens

constexpr int kPrepThreads = 256;

__device__ __forceinline__ bool is_live(const void* labels, int i64, int64_t t, int V) {
    const int64_t y = label_at(labels, i64, t);
    return y >= 0 && y < V;
}

// CTA b takes `per` tokens: live ones get the next place (tokens in order), their
// rows are copied there unless every token is live, the others' outputs are zeroed.
// Each CTA counts the live tokens before its own from the labels themselves.
// Behind the last live row, rows up to the next multiple of kBK are zeroed: dW's
// last K block reads them. The first CTA clears the status block.
__global__ void __launch_bounds__(kPrepThreads)
head_prep_kernel(const uint4* __restrict__ x, int64_t ldx, const void* labels, int i64, int T, int V, int nv, int per,
                 int32_t* __restrict__ rows, int32_t* __restrict__ live, uint4* __restrict__ xc,
                 float* loss, float* lse, uint4* dx, int32_t* status) {
    __shared__ int32_t sh[3];
    __shared__ int32_t place[kPrepThreads];
    pdl_wait();
    pdl_allow_next();
    const int tid = threadIdx.x, lane = tid & 31;
    const int t0 = blockIdx.x * per, t1 = min(t0 + per, T);
    if (tid < 2) sh[tid] = 0;
    if (blockIdx.x == 0 && status && tid < kStatusBytes / 4) status[tid] = 0;
    __syncthreads();
    int before = 0, count = 0;
    for (int t = tid; t < T; t += kPrepThreads) {
        const int l = is_live(labels, i64, t, V) ? 1 : 0;
        count += l;
        before += t < t0 ? l : 0;
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, d);
        count += __shfl_xor_sync(0xffffffffu, count, d);
    }
    if (lane == 0) {
        atomicAdd(&sh[0], before);
        atomicAdd(&sh[1], count);
    }
    __syncthreads();
    const int total = sh[1];
    int next = sh[0];
    if (blockIdx.x == 0 && tid == 0) *live = total;
    const bool all = total == T;
    for (int c0 = t0; c0 < t1; c0 += 32) {
        // places of 32 tokens
        __syncthreads();
        if (tid < 32) {
            const int t = c0 + lane;
            const bool l = t < t1 && is_live(labels, i64, t, V);
            const unsigned b = __ballot_sync(0xffffffffu, l);
            place[lane] = l ? next + __popc(b & ((1u << lane) - 1)) : -1;
            if (lane == 0) sh[2] = __popc(b);
        }
        __syncthreads();
        next += sh[2];
        for (int j = 0; j < 32 && c0 + j < t1; ++j) {
            const int64_t t = c0 + j;
            const int to = place[j];
            if (to >= 0) {
                if (tid == 0) rows[to] = (int32_t)t;
                if (!all)
                    for (int v = tid; v < nv; v += kPrepThreads) xc[(int64_t)to * nv + v] = __ldg(x + t * ldx + v);
            } else {
                if (tid == 0 && loss) loss[t] = 0.f;
                if (tid == 0 && lse) lse[t] = 0.f;
                if (dx)
                    for (int v = tid; v < nv; v += kPrepThreads) dx[t * nv + v] = make_uint4(0, 0, 0, 0);
            }
        }
    }
    if (!all && t1 == T) {
        const int end = (total + kBK - 1) / kBK * kBK;
        for (int64_t v = (int64_t)total * nv + tid; v < (int64_t)end * nv; v += kPrepThreads)
            xc[v] = make_uint4(0, 0, 0, 0);
    }
}

// ------------------------------------------------------------------ log-sum and loss

constexpr int kRowThreads = 256;

// The sums of a row's stat tiles joined: the largest logit, the other tokens' sum
// relative to it and the label's term.
struct RowSum {
    float top, others, own;   // sum of all = others + own, over exp(top)
};
__device__ __forceinline__ RowSum join_row(const float2* stats, int n, float label_logit, float* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float m = -INFINITY;
    for (int i = threadIdx.x; i < n; i += kRowThreads) m = fmaxf(m, stats[i].x);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (lane == 0) red[warp] = m;
    __syncthreads();
    m = lane < kRowThreads / 32 ? red[lane] : -INFINITY;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float base = m == -INFINITY ? 0.f : m;
    float s = 0.f;
    for (int i = threadIdx.x; i < n; i += kRowThreads) {
        const float2 v = stats[i];
        s += v.y * exp2_approx((v.x == -INFINITY ? -INFINITY : v.x - base) * kLog2e);
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane == 0) red[32 + warp] = s;
    __syncthreads();
    s = lane < kRowThreads / 32 ? red[32 + lane] : 0.f;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    RowSum r;
    r.top = base;
    r.others = s;
    r.own = expf(label_logit - base);
    return r;
}

// A CTA per live token.
__global__ void __launch_bounds__(kRowThreads)
head_loss_kernel(const float2* __restrict__ stats, int stat_tiles, const float* __restrict__ label_logit,
                 const int32_t* __restrict__ rows, const int32_t* __restrict__ live, const void* labels, int i64, int V,
                 float* loss, float* lse) {
    __shared__ float red[64];
    pdl_wait();
    pdl_allow_next();
    const int i = blockIdx.x;
    if (live && i >= *live) return;
    const int64_t t = rows ? rows[i] : i;
    const bool on = rows || is_live(labels, i64, t, V);
    const RowSum r = join_row(stats + (int64_t)i * stat_tiles, stat_tiles, on ? label_logit[i] : 0.f, red);
    if (threadIdx.x != 0) return;
    // log(others + own) - log(own), by the form that loses no digits
    const float at = label_logit[i] - r.top;
    const float l = r.own > r.others ? log1pf(r.others / r.own) : logf(r.others + r.own) - at;
    if (loss) loss[t] = on ? l : 0.f;
    if (lse) lse[t] = on ? r.top + logf(r.others + r.own) : 0.f;
}

// The same with a gradient: then the row's exponentials, in their place, become
//   dl[v] = c e[v] exp(top of its 128 columns - lse),   dl[label] = -c others / (others + own)
__global__ void __launch_bounds__(kRowThreads)
head_dl_kernel(const float2* __restrict__ stats, int stat_tiles, const float* __restrict__ label_logit,
               const int32_t* __restrict__ rows, const int32_t* __restrict__ live, const void* labels, int i64,
               const float* __restrict__ dloss, float scale, __nv_bfloat16* dl, int64_t ld, int V, float* loss,
               float* lse) {
    __shared__ float red[64];
    pdl_wait();
    pdl_allow_next();
    const int i = blockIdx.x;
    if (i >= *live) return;
    const int64_t t = rows[i];
    const float2* st = stats + (int64_t)i * stat_tiles;
    const RowSum r = join_row(st, stat_tiles, label_logit[i], red);
    const float sum = r.others + r.own, log_sum = r.top + logf(sum);
    const float coef = scale * (dloss ? dloss[t] : 1.0f);
    const int label = (int)label_at(labels, i64, t);
    __nv_bfloat16* row = dl + i * ld;
    const float inv = coef / sum * kRootScale;
    for (int v = 8 * threadIdx.x; v < V; v += 8 * kRowThreads) {
        const uint4 e = *reinterpret_cast<const uint4*>(row + v);
        const float f = inv * exp2_approx((st[v / kStatCols].x - r.top) * kLog2e);
        const uint32_t w[4] = {e.x, e.y, e.z, e.w};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
            o[j] = pack_bf16x2(a.x * f * a.x, a.y * f * a.y);
        }
        *reinterpret_cast<uint4*>(row + v) = make_uint4(o[0], o[1], o[2], o[3]);
        if (label >= v && label < v + 8) row[label] = __float2bfloat16_rn(-coef * (r.others / sum));
    }
    if (threadIdx.x != 0) return;
    const float at = label_logit[i] - r.top;
    loss[t] = r.own > r.others ? log1pf(r.others / r.own) : logf(sum) - at;
    if (lse) lse[t] = log_sum;
}

// dx rows from the parts of K, added up in order.
__global__ void __launch_bounds__(256)
head_join_kernel(const float* __restrict__ part, int64_t stride, int splits, int nv, const int32_t* __restrict__ rows,
                 const int32_t* __restrict__ live, __nv_bfloat16* __restrict__ dx) {
    pdl_wait();
    pdl_allow_next();
    const int64_t i = blockIdx.x;
    if (i >= *live) return;
    const int64_t t = rows[i];
    for (int v = blockIdx.y * blockDim.x + threadIdx.x; v < nv; v += gridDim.y * blockDim.x) {
        float a[8] = {};
        for (int s = 0; s < splits; ++s) {
            const float4* q = reinterpret_cast<const float4*>(part + s * stride + (i * nv + v) * 8);
            const float4 b = q[0], c = q[1];
            a[0] += b.x; a[1] += b.y; a[2] += b.z; a[3] += b.w;
            a[4] += c.x; a[5] += c.y; a[6] += c.z; a[7] += c.w;
        }
        *reinterpret_cast<uint4*>(dx + (t * nv + v) * 8) = make_uint4(
            pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]), pack_bf16x2(a[6], a[7]));
    }
}

// ------------------------------------------------------------------ launches

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void* p = nullptr;
        return cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                           cudaSuccess && q == cudaDriverEntryPointSuccess
                   ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
    }();
    return fn;
}

// [rows, cols] BF16 with row pitch ld elements (a multiple of 8), read in boxes of
// 64 columns x box_rows with a 128-byte swizzle; what lies outside reads 0.
bool make_tmap_pitch(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)(ld * 2)};
    cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pairs of CTAs of a kernel that can be resident at once, asked once per kernel and
// device.
template <bool A_MN, bool B_MN, int EPI>
int resident_pairs(void (*kern)(CUtensorMap, CUtensorMap, CUtensorMap, HeadGemm), cudaLaunchConfig_t cfg, int num_sms) {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        cfg.gridDim = dim3(2 * (sm_count() / 2));
        if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
            cudaGetLastError();
            n = sm_count() / 2;
        }
        known[dev].store(n, std::memory_order_relaxed);
    }
    return std::min(n, num_sms / 2);
}


template <bool A_MN, bool B_MN, int EPI>
cudaError_t run_head_gemm(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& all, HeadGemm& p, int num_sms,
                          cudaStream_t s) {
    auto kern = head_gemm_kernel<A_MN, B_MN, EPI>;
    ensure_smem_attr(reinterpret_cast<const void*>(kern), kSmemBytes);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    const int64_t tiles = (int64_t)ceil_div(p.M, kBM) * ceil_div(p.N, kBN) * p.splits;
    const int pairs = (int)std::min<int64_t>(tiles, resident_pairs<A_MN, B_MN, EPI>(kern, cfg, num_sms));
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    cfg.gridDim = dim3(2 * pairs);
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a, b, all, p);
}

constexpr int kGroup = 16;              // row tiles of the walk's groups
constexpr int64_t kPieceBytes = (int64_t)4 << 30;
constexpr int kPieceMax = 65536;
// Logits without a gradient: up to one row tile, ignored tokens save nothing.
constexpr int kPlainRows = kBM;

int64_t pitch_dl(int V) { return align_up(V, 64); }

// Tokens of a piece: `want` where it is given, else as many as keep dl within
// kPieceBytes, in pieces of about the same size, whole row tiles.
int piece_tokens(int T, int V, int want) {
    int64_t most = want > 0 ? want : std::max<int64_t>(kPieceBytes / (pitch_dl(V) * 2) / kBM * kBM, kBM);
    most = std::min<int64_t>(most, kPieceMax);
    if (T <= most) return std::max(T, 1);
    if (want > 0) return (int)most;
    const int64_t pieces = (T + most - 1) / most;
    return (int)std::min<int64_t>(most, align_up((T + pieces - 1) / pieces, kBM));
}

// Parts of the vocabulary for dX: where the tiles alone leave most pairs without
// work, as many as fill them, each of 8 K blocks at least.
int dx_splits(int tokens, int H, int V, int pairs) {
    const int tiles = ceil_div(tokens, kBM) * ceil_div(H, kBN), kbs = ceil_div(V, kBK);
    if (2 * tiles > pairs) return 1;
    return std::max(1, std::min(pairs / tiles, kbs / 8));
}

struct HeadLayout {
    size_t rows, live, label, stats, xc, dl, part, acc, total;
    int piece, splits;
};

HeadLayout head_layout(int T, int H, int V, bool grad, bool acc, int want, int num_sms) {
    HeadLayout L{};
    size_t o = kStatusBytes;
    auto take = [&](int64_t bytes) {
        const size_t at = o;
        o += align_up(bytes, 1024);
        return at;
    };
    L.piece = piece_tokens(T, V, want);
    L.splits = grad ? dx_splits(L.piece, H, V, num_sms / 2) : 1;
    const int64_t cap = align_up(L.piece, kBM);
    o = align_up(o, 1024);
    L.live = take(4);
    L.rows = take(cap * 4);
    L.label = take(cap * 4);
    L.stats = take(cap * ceil_div(V, kStatCols) * 8);
    if (grad || T > kPlainRows) L.xc = take(cap * H * 2);
    if (grad) L.dl = take(cap * pitch_dl(V) * 2);
    if (L.splits > 1) L.part = take((int64_t)L.splits * cap * H * 4);
    if (acc && L.piece < T) L.acc = take((int64_t)V * H * 4);
    L.total = o;
    return L;
}

}  // namespace

size_t head_workspace_bytes(int T, int H, int V, bool grad, int piece, int num_sms) {
    return head_layout(T, H, V, grad, grad, piece, num_sms).total;
}

cudaError_t launch_head(const HeadLaunch& a, const GemmCommon& c, cudaStream_t s) {
    const int T = a.T, H = a.H, V = a.V;
    const bool grad = a.dx || a.dW;
    const HeadLayout L = head_layout(T, H, V, grad, grad, a.piece, c.num_sms);
    char* ws = static_cast<char*>(a.workspace);
    int32_t* live = reinterpret_cast<int32_t*>(ws + L.live);
    int32_t* rows = reinterpret_cast<int32_t*>(ws + L.rows);
    float* label = reinterpret_cast<float*>(ws + L.label);
    float2* stats = reinterpret_cast<float2*>(ws + L.stats);
    const int stat_tiles = ceil_div(V, kStatCols);
    const int nv = H / 8;
    cudaError_t e = cudaSuccess;
    if (T == 0) {
        e = cudaMemsetAsync(ws, 0, kStatusBytes, s);
        if (e == cudaSuccess && a.dW && !a.accumulate)
            e = cudaMemsetAsync(a.dW, 0, (size_t)V * H * (a.dW_f32 ? 4 : 2), s);
        return e;
    }
    const int label_bytes = a.labels_i64 ? 8 : 4;
    for (int t0 = 0; t0 < T && e == cudaSuccess; t0 += L.piece) {
        const int n = std::min(L.piece, T - t0);
        const int64_t cap = align_up(n, kBM);
        const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x) + t0 * a.ldx;
        const void* labels = static_cast<const char*>(a.labels) + (int64_t)t0 * label_bytes;
        float* loss = a.loss ? a.loss + t0 : nullptr;
        float* lse = a.lse ? a.lse + t0 : nullptr;
        __nv_bfloat16* dx = a.dx ? static_cast<__nv_bfloat16*>(a.dx) + (int64_t)t0 * H : nullptr;
        const bool gather = grad || T > kPlainRows;
        const bool forward = a.loss != nullptr;
        HeadGemm p{};
        p.status = c.status;
        p.timeout_ns = c.timeout_ns;
        p.tokens = n;
        p.group = kGroup;
        p.splits = 1;
        p.labels = labels;
        p.labels_i64 = a.labels_i64;
        p.scale = a.scale;
        CUtensorMap tx, txc, tw, tdl;
        if (!make_tmap_pitch(&tx, x, n, H, a.ldx, 128) || !make_tmap_pitch(&tw, a.W, V, H, H, 128)) return cudaErrorInvalidValue;
        txc = tx;
        if (gather) {
            const int per = std::max(8, ceil_div(n, 1024));
            e = launch_after(head_prep_kernel, dim3(ceil_div(n, per)), dim3(kPrepThreads), 0, s,
                             reinterpret_cast<const uint4*>(x), a.ldx / 8, labels, a.labels_i64, n, V, nv, per, rows, live,
                             reinterpret_cast<uint4*>(ws + L.xc), forward ? loss : nullptr,
                             forward ? lse : nullptr, reinterpret_cast<uint4*>(dx),
                             t0 == 0 ? reinterpret_cast<int32_t*>(ws) : nullptr);
            if (!make_tmap_pitch(&txc, ws + L.xc, cap, H, H, 128)) return cudaErrorInvalidValue;
            p.live = live;
            p.rows = rows;
            p.m_live = 1;
        } else {
            e = cudaMemsetAsync(ws, 0, kStatusBytes, s);
        }
        if (e != cudaSuccess) break;
        p.M = n;
        p.N = V;
        p.K = H;
        p.stats = stats;
        p.stat_tiles = stat_tiles;
        p.label_logit = label;
        if (!grad) {
            e = run_head_gemm<false, false, kEpiStats>(txc, tw, tx, p, c.num_sms, s);
            if (e == cudaSuccess)
                e = launch_after(head_loss_kernel, dim3(n), dim3(kRowThreads), 0, s, (const float2*)stats, stat_tiles,
                                 (const float*)label, (const int32_t*)(gather ? rows : nullptr),
                                 (const int32_t*)(gather ? live : nullptr), labels, a.labels_i64, V, loss, lse);
            continue;
        }
        p.dl = reinterpret_cast<__nv_bfloat16*>(ws + L.dl);
        p.ld_dl = pitch_dl(V);
        p.lse = lse;
        p.dloss = a.dloss ? a.dloss + t0 : nullptr;
        if (forward) {
            e = run_head_gemm<false, false, kEpiExp>(txc, tw, tx, p, c.num_sms, s);
            if (e == cudaSuccess)
                e = launch_after(head_dl_kernel, dim3(n), dim3(kRowThreads), 0, s, (const float2*)stats, stat_tiles,
                                 (const float*)label, (const int32_t*)rows, (const int32_t*)live, labels, a.labels_i64,
                                 p.dloss, a.scale, p.dl, p.ld_dl, V, loss, lse);
        } else {
            e = run_head_gemm<false, false, kEpiDl>(txc, tw, tx, p, c.num_sms, s);
        }
        if (e != cudaSuccess) break;
        if (dx) {
            HeadGemm q = p;
            CUtensorMap twm;
            if (!make_tmap_pitch(&tdl, p.dl, cap, V, p.ld_dl, 128) || !make_tmap_pitch(&twm, a.W, V, H, H, 64)) return cudaErrorInvalidValue;
            q.M = n;
            q.N = H;
            q.K = V;
            q.splits = L.splits;
            if (L.splits > 1) {
                q.out = ws + L.part;
                q.out_f32 = 1;
                q.split_stride = cap * H;
            } else {
                q.out = dx;
                q.out_rows = rows;
            }
            e = run_head_gemm<false, true, kEpiOut>(tdl, twm, tdl, q, c.num_sms, s);
            if (e == cudaSuccess && L.splits > 1)
                e = launch_after(head_join_kernel, dim3(n, std::min(ceil_div(nv, 64), 64)), dim3(64), 0, s,
                                 (const float*)(ws + L.part), cap * H, L.splits, nv, (const int32_t*)rows,
                                 (const int32_t*)live, dx);
            if (e != cudaSuccess) break;
        }
        if (a.dW) {
            HeadGemm q = p;
            CUtensorMap txm, txcm;
            if (!make_tmap_pitch(&tdl, p.dl, cap, V, p.ld_dl, 64) || !make_tmap_pitch(&txcm, ws + L.xc, cap, H, H, 64) ||
                !make_tmap_pitch(&txm, x, n, H, a.ldx, 64))
                return cudaErrorInvalidValue;
            q.M = V;
            q.N = H;
            q.K = n;
            q.m_live = 0;
            q.k_live = 1;
            // over several pieces the sum goes on in fp32 until the last one
            const bool first = t0 == 0, last = t0 + n >= T;
            float* acc = a.dW_f32 ? static_cast<float*>(a.dW) : reinterpret_cast<float*>(ws + L.acc);
            q.out_f32 = a.dW_f32 || !last;
            q.out = q.out_f32 ? (void*)acc : a.dW;
            q.add = first && !(a.dW_f32 && a.accumulate) ? nullptr : acc;
            e = run_head_gemm<true, true, kEpiOut>(tdl, txcm, txm, q, c.num_sms, s);
        }
    }
    return e;
}

}  // namespace mok
