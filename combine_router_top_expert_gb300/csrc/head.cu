// head.cu - softmax cross entropy of a large vocabulary from the last hidden rows
// and the vocabulary's weights, with its gradient, without the logits.
//
// With x [T,H], W [V,H] and the label y_t of token t:
//   l[t,v] = <x_t, W_v>      lse_t = log sum_v exp l[t,v]      loss_t = lse_t - l[t,y_t]
//   dl[t,v] = d_t (exp(l[t,v] - lse_t) - [v == y_t])           d_t = dloss_t / top
//   dX = c dl W              dW = c dl^T x                     c = scale * top
// with top the largest finite |dloss| (1 without dloss). dl is rounded to BF16, and an
// unlikely token's entry is nearly -d_t: with the whole coefficient in it all tokens'
// entries would be off by the same share, up to 2^-8 (scale = 1/4080: gradients 0.37%
// too short). So the common factor is taken out and multiplies the fp32 sums, and
// without dloss, or with equal ones, dl is the softmax less the label.
// Tokens whose label is outside 0..V-1 count for nothing, whatever their rows hold. In
// a call of more than one row tile the live ones are gathered first (head_prep_kernel),
// and none of the products is spent on the others.
//
// Three products, each a persistent tcgen05 kernel over 256 x 256 tiles of 2-SM
// pairs (head_gemm_kernel):
//   logits  x W^T    both operands K-major; the epilogue reduces 128 columns of a row
//                    to (max, sum of exponentials), so that a logit lives in tensor
//                    memory and registers only, and with a gradient writes dl (log-sum
//                    known) or the exponentials, which head_dl_kernel turns into dl in
//                    their place: 6TVH operations for a training call, none repeated
//   dX      dl W     A K-major, B MN-major (the vocabulary is K)
//   dW      dl^T x   both MN-major (the tokens are K)
// Few tokens are bound by the bytes of W (H = 7168, V = 131072, call after call: T = 64
// 294 to 312 us by the GPU at hand, 6.4 to 6.0 TB/s; T = 1 278 us), many by the tensor
// cores and what the power limit leaves of their clock (T = 2560, H = 7168, V = 50001,
// scoring: 975 us when the GPU is cool, 1110 to 1140 call after call, 1.9 and 1.6 PFLOP/s;
// T = 4096, V = 131072, training: 12.9 ms, and 14.3 to 15.6, 1.8 and 1.6 to 1.5 PFLOP/s).
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "moves.cuh"
#include "tc.cuh"

namespace mok {

namespace {

constexpr int kBM = 256, kBN = 256;     // tile of a pair of CTAs
constexpr int kBK = 64;                 // K elements of a stage (128 bytes)
constexpr int kMaxStages = 12;
constexpr int kEpiWarps = 8;            // two per TMEM lane quadrant, 128 columns each
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kOperandBytes = 128 * kBK * 2;          // a CTA's share of A or of B
constexpr int kBarOffset = 6 * 2 * kOperandBytes;     // the ring: 6 stages, or more that hold few rows of A
constexpr int kPassBytes = 4096;                      // an epilogue warp's staging: 32 rows x 128 bytes
constexpr int kStageOutOffset = kBarOffset + 1024;
constexpr int kSmemBytes = 1024 + kStageOutOffset + kEpiWarps * kPassBytes;
// K blocks of a logit that are summed in tensor memory; these sums are then added in
// registers. The tensor cores cut what they add to an accumulator instead of rounding
// it, which makes a long sum too small by up to 2^-24 of itself a step: H = 7168 in one
// sum moved a loss by 4.8e-6 of itself, in sums of 1024 by what the other roundings do.
// (dl from a known log-sum is rounded to BF16: there one sum does.)
constexpr int kLogitBlocks = 16;
constexpr float kLog2e = 1.4426950408889634f;
// An exponential e is kept as its root times 2^15, s = 2^15 exp((l - top) / 2): FP16 then has a relative error of
// 2^-11 in s, 2^-10 in e, down to e = 2^-58 (e itself would lose bits below 2^-29).
constexpr float kRootShift = 15.f;
constexpr float kRootScale = 1.f / (1 << 30);   // s * s * kRootScale = e

enum Early : int { kEarlyNone = 0, kEarlyA = 1, kEarlyB = 2 };

enum HeadEpi : int {
    kEpiStats = 0,   // (max, sum)
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
    int a_mn;               // A is MN-major (two products in one launch; else the kernel's own type says it)
    int a_bytes;            // what a CTA loads of A: its share, or the rows there are where one CTA holds them all
    int a_room;             // its room in a stage
    int stages;
    int a_groups, b_groups; // MN-major: the operand's map has groups of 64 columns as its last axis
    int early;              // operands whose first blocks may be loaded before the kernel ahead has ended
    int wait_late;          // the operands were complete before the kernel ahead began: it is waited for at the end
    // logits
    const void* labels;
    int labels_i64;
    const int32_t* rows;    // live token -> token, or NULL
    float2* stats;          // [tokens, stat tiles]
    int stat_tiles;
    const float* label_logit;   // [tokens]
    const float* lse;       // [T]
    const float* dloss;     // [T] or NULL
    const float* factors;   // {top, c}, written by the call's first kernel
    __nv_bfloat16* dl;      // [dl_rows, ld_dl]
    int64_t ld_dl;
    int64_t dl_rows;
    // products
    int tma_out;            // rows leave as tmOut's boxes; else (scattered, or added to) by the warps' stores
    void* out;
    int out_f32;
    int scaled;             // times c (else what c is to multiply is joined first)
    const float* add;       // fp32 rows that are added to the product, or NULL
    const int32_t* out_rows;   // row -> output row, or NULL
    int zero_dead;          // rows whose label is not below live_below are zeros
    int live_below;
    int withhold;           // test hook: the first pair's producers stop before the last K block of a tile
    StatusBlock* status;
    unsigned long long timeout_ns;
};

// A product with its operands. all: the caller's own rows in place of the gathered ones,
// taken when every token is live (logits: for A, dW: for B). out: what the epilogue
// writes, as [parts][rows][columns] in boxes of 32 rows x 128 bytes (p.tma_out).
struct HeadJob {
    CUtensorMap a, b, all, out;
    HeadGemm p;
};
// One product, or two that do not depend on each other (dX and dW): the first `lead`
// pairs take a tile of the first product each and then share the first `lead_tiles` of
// the second one's, the other pairs share the rest of those.
template <int N>
struct HeadJobs {
    HeadJob job[N];
    int lead, lead_tiles;
};

__device__ __forceinline__ float exp2_approx(float v) {
    float r;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));   // volatile: kept in place, or the epilogues spill
    return r;
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared16(uint32_t a, __nv_bfloat16 v) {
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(a), "h"(__bfloat16_as_ushort(v)) : "memory");
}

// After a wait that gave up: a phase that is to complete by what is already under way
// (copies, MMAs), waited for whatever the abort flag says, for 10 ms at most.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = globaltimer_ns();
    while (!tc::mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < 10000000ull) {
    }
}

// Arrive on an mbarrier of the pair. What is released is tensor memory that was read;
// a release at cluster scope would also wait for the thread's stores on their way (1 to
// 2 us a tile).
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
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

// A box of a three-dimensional map, as tma_load_2d_2sm.
__device__ __forceinline__ void tma_load_3d_2sm(uint32_t dst, const void* tmap, uint32_t bar, int32_t x, int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// Sizes of a product with the live tokens in place.
struct HeadSize {
    int M, mt, nt, kbs, total;
    bool all;
};

// Warp 0 loads (one thread: TMA boxes into the ring), warp 1 of the pair's leader issues the
// MMAs, warps 2 to 9 turn a tile's sums into what the product is for, while the next tile is
// summed in the other half of tensor memory. 256 x 256 is the largest tile that leaves two
// halves; a K block of it costs the pair 0.27 us of MMA and brings 64 KB, 18 TB/s over the
// GPU, about what L2 gives: narrower tiles bring more for the same work and were no faster,
// and for few rows, where most of the MMA is spent on rows that there are not, HBM is the
// bound all the same. T = 2560, H = 7168, V = 32768, the kernels by themselves: logits 622 us
// (86% of the tensor cores' cycles; V = 50001: 92%), with exponentials 637, dX 686, dW 650
// (76%; MN-major operands: the power limit sets their clock). Kept out because they gained
// nothing: clusters of four with multicast, five stages with a second staging buffer, each
// pair's walk of K begun elsewhere, waits that sleep (the clock rose by 5%, the time too).
template <bool A_MN, bool B_MN, int EPI, int N>
__global__ void __launch_bounds__(kThreads, 1)
head_gemm_kernel(const __grid_constant__ HeadJobs<N> jobs) {
    const HeadGemm& p0 = jobs.job[0].p;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ uint32_t s_tmem_base;
    const uint32_t smem_base = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t bar_base = smem_base + kBarOffset;
    auto full_bar = [&](int s) { return bar_base + 8u * s; };
    auto empty_bar = [&](int s) { return bar_base + 8u * (kMaxStages + s); };
    auto accf_bar = [&](int a) { return bar_base + 8u * (2 * kMaxStages + a); };
    auto acce_bar = [&](int a) { return bar_base + 8u * (2 * kMaxStages + 2 + a); };
    const uint32_t drain_bar = bar_base + 8u * (2 * kMaxStages + 4);
    // the stages' rows of A, then room for the rest of a tile behind the last one, then their rows of B
    const uint32_t a_room = p0.a_room;
    const int stages = p0.stages;
    const uint32_t b_base = smem_base + (stages - 1) * a_room + kOperandBytes;
    auto a_tile = [&](int s) { return smem_base + s * a_room; };
    auto b_tile = [&](int s) { return b_base + s * kOperandBytes; };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    StatusBlock* st = p0.status;
    const uint64_t tmo = p0.timeout_ns;
    if (threadIdx.x == 32) {
        for (int s = 0; s < stages; ++s) {
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
        for (int j = 0; j < N; ++j) {
            tc::prefetch_tmap(&jobs.job[j].a);
            tc::prefetch_tmap(&jobs.job[j].b);
            tc::prefetch_tmap(&jobs.job[j].all);
        }
    }
    if (a_room < kOperandBytes && warp >= 2) {
        // Zeros where no row is loaded: a CTA without tokens, and behind the last stage. Products with whatever
        // lay there were discarded too, but took power: call after call the SM clock fell to 1560 MHz (T = 1, H =
        // 7168, V = 131072: 312 us; this 2010 MHz, 278).
        const uint32_t from = tc::cluster_ctarank() == 0 ? stages * a_room : 0;
        for (uint32_t a = smem_base + from + (threadIdx.x - 64) * 16; a < b_base; a += 32 * kEpiWarps * 16)
            tc::st_shared_v4(a, 0, 0, 0, 0);
        tc::fence_proxy_async_shared();
    }
    if (warp == 1) {
        tc::tmem_alloc_2sm(tc::smem_u32(&s_tmem_base), 512);
        tc::tmem_relinquish_2sm();
    }
    // The kernel behind this one may begin once all that this one reads is complete
    // (a wait_late kernel reads on that ground); early kernels wait in their roles.
    if (!p0.early) {
        if (!p0.wait_late) pdl_wait();
        pdl_allow_next();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    tc::cluster_sync();   // the peer's barriers and tensor memory exist
    const uint32_t tmem = s_tmem_base;
    const int rank = (int)tc::cluster_ctarank();

    const int pair = (int)blockIdx.x / 2, pairs = (int)gridDim.x / 2;
    auto size_of = [&](const HeadGemm& p) {
        HeadSize z;
        const int live = p.live ? *p.live : p.tokens;
        z.all = live == p.tokens;
        z.M = p.m_live ? live : p.M;
        z.mt = (z.M + kBM - 1) / kBM;
        z.nt = (p.N + kBN - 1) / kBN;
        z.kbs = ((p.k_live ? live : p.K) + kBK - 1) / kBK;
        z.total = z.mt * z.nt * p.splits;
        return z;
    };
    // this pair's tiles of product j: from g0 to before g1
    struct Range {
        int g0, g1, step;
    };
    auto range_of = [&](int j, const HeadSize& z) {
        Range r{pair, z.total, pairs};
        if (N == 2 && j == 1) {
            const bool in_lead = pair < jobs.lead;
            const int64_t tiles = in_lead ? jobs.lead_tiles : z.total - jobs.lead_tiles;
            const int k = in_lead ? pair : pair - jobs.lead, of = in_lead ? jobs.lead : pairs - jobs.lead;
            const int base = in_lead ? 0 : jobs.lead_tiles;
            r = Range{base + (int)(tiles * k / of), base + (int)(tiles * (k + 1) / of), 1};
        }
        return r;
    };
    constexpr int kSumBlocks = EPI == kEpiStats || EPI == kEpiExp ? kLogitBlocks : 1 << 30;   // K blocks of an accumulator's sum
    // first K block of a part (products below 2^25)
    auto k_first = [](const HeadGemm& p, const HeadSize& z, int split) {
        return p.splits == 1 ? z.kbs * split : z.kbs * split / p.splits;
    };

    if (warp == 0) {
        if (lane == 0) {
            // both halves of a pair signal the leader's barrier, which expects both
            auto load_a = [&](const HeadJob& J, const HeadSize& z, int stage, const Tile& t, int kb) {
                const HeadGemm& p = J.p;
                const void* map = EPI != kEpiOut && z.all ? (const void*)&J.all : (const void*)&J.a;
                const uint32_t lead = tc::mapa_shared(full_bar(stage), 0);
                const int m0 = t.m * kBM + rank * 128, k0 = kb * kBK;
                if (N == 2 ? p.a_mn != 0 : A_MN) {
                    if (p.a_groups) {
                        tma_load_3d_2sm(a_tile(stage), map, lead, 0, k0, m0 / 64);
                    } else {
                        tc::tma_load_2d_2sm(a_tile(stage), map, lead, m0, k0);
                        tc::tma_load_2d_2sm(a_tile(stage) + 8192, map, lead, m0 + 64, k0);
                    }
                } else if (p.a_bytes == kOperandBytes || rank == 0) {
                    // (few rows: the leader alone has some, and the MMAs' other rows are the next stages' or zeros)
                    tc::tma_load_2d_2sm(a_tile(stage), map, lead, k0, m0);
                }
            };
            auto load_b = [&](const HeadJob& J, const HeadSize& z, int stage, const Tile& t, int kb) {
                const HeadGemm& p = J.p;
                const void* map = (N == 2 ? p.a_mn != 0 : A_MN) && z.all ? (const void*)&J.all : (const void*)&J.b;
                const uint32_t lead = tc::mapa_shared(full_bar(stage), 0);
                const int n0 = t.n * kBN + rank * 128, k0 = kb * kBK;
                if constexpr (B_MN) {
                    if (p.b_groups) {
                        tma_load_3d_2sm(b_tile(stage), map, lead, 0, k0, n0 / 64);
                    } else {
                        tc::tma_load_2d_2sm(b_tile(stage), map, lead, n0, k0);
                        tc::tma_load_2d_2sm(b_tile(stage) + 8192, map, lead, n0 + 64, k0);
                    }
                } else {
                    tc::tma_load_2d_2sm(b_tile(stage), map, lead, k0, n0);
                }
            };
            auto bytes_of = [](const HeadGemm& p) {
                return (uint32_t)((p.a_bytes == kOperandBytes ? 2 : 1) * p.a_bytes + 2 * kOperandBytes);
            };
            int stage = 0, ahead = 0;   // ahead: blocks whose early operands are on their way
            uint32_t ph = 0;
            int last_par[kMaxStages];
            for (int s = 0; s < kMaxStages; ++s) last_par[s] = -1;
            bool ok = true;
            if (p0.early) {
                const HeadJob& J = jobs.job[0];
                const HeadSize z = size_of(p0);
                for (int g = pair; g < z.total && ahead < stages && !(p0.withhold && pair == 0); g += pairs) {
                    const Tile t = head_tile(g, z.mt, z.nt, p0.group);
                    const int kend = k_first(p0, z, t.split + 1);
                    for (int kb = k_first(p0, z, t.split); kb < kend && ahead < stages; ++kb, ++ahead) {
                        if (rank == 0) tc::mbar_expect_tx(full_bar(ahead), bytes_of(p0));
                        if (p0.early & kEarlyA) load_a(J, z, ahead, t, kb);
                        if (p0.early & kEarlyB) load_b(J, z, ahead, t, kb);
                    }
                }
                pdl_wait();
                pdl_allow_next();
            }
#pragma unroll 1
            for (int j = 0; j < N && ok; ++j) {
                const HeadJob& J = jobs.job[j];
                const HeadGemm& p = J.p;
                const HeadSize z = size_of(p);
                const Range r = range_of(j, z);
                const uint32_t bytes = bytes_of(p);
                for (int g = r.g0; g < r.g1 && ok; g += r.step) {
                    const Tile t = head_tile(g, z.mt, z.nt, p.group);
                    const int kend = k_first(p, z, t.split + 1);
                    for (int kb = k_first(p, z, t.split); kb < kend; ++kb) {
                        if (p0.withhold && pair == 0 && kb + 1 == kend) { ok = false; break; }
                        const bool begun = ahead > 0;   // only in the first round of stages, which are free
                        if (begun) {
                            --ahead;
                        } else {
                            if (!tc::mbar_wait(empty_bar(stage), ph ^ 1u, st, tmo, kSiteProducerEmpty)) { ok = false; break; }
                            if (rank == 0) tc::mbar_expect_tx(full_bar(stage), bytes);
                        }
                        if (!begun || !(p0.early & kEarlyA)) load_a(J, z, stage, t, kb);
                        if (!begun || !(p0.early & kEarlyB)) load_b(J, z, stage, t, kb);
                        last_par[stage] = (int)ph;
                        if (++stage == stages) { stage = 0; ph ^= 1u; }
                    }
                }
            }
            if (!ok) {
                // every copy already issued lands before the pair exits: the leader sees it on its barriers, where
                // both CTAs' bytes arrive; the time covers those of a stage that the other CTA never reached
                if (rank == 0)
                    for (int s = 0; s < stages; ++s)
                        if (last_par[s] >= 0) drain_wait(full_bar(s), (uint32_t)last_par[s]);
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 200000ull) {
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            if (p0.early) pdl_wait();
            // Of a descriptor only the start address changes (16-byte units, in the low word), so an MMA
            // costs two additions: what this thread does between MMAs is not hidden behind them. Building
            // each descriptor from its fields and waiting for every stage by itself left the tensor cores
            // idle a quarter of the time (T = 2560, H = 7168, V = 50001, score: 1090 us, this 954).
            constexpr uint32_t kHi = 64u | 1u << 14 | tc::kLayoutSW128 << 29;
            constexpr uint32_t kLoB = (B_MN ? 512u : 1u) << 16, kStepB = B_MN ? 128u : 2u;
            uint32_t idesc = 0, step_a = 0, al0 = 0;
            const uint32_t bl0 = b_tile(0) >> 4 | kLoB;
            auto mma4 = [&](uint32_t d, int sg, uint32_t more) {
                const uint32_t al = al0 + (uint32_t)sg * (a_room >> 4);
                const uint32_t bl = bl0 + (uint32_t)sg * (kOperandBytes >> 4);
                const uint32_t sa = N == 2 ? step_a : A_MN ? 128u : 2u;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    tc::mma_bf16_2sm(d, (uint64_t)kHi << 32 | (al + kk * sa), (uint64_t)kHi << 32 | (bl + kk * kStepB),
                                     idesc, kk > 0 ? 1u : more);
            };
            int stage = 0, acc = 0;
            uint32_t ph = 0, acc_ph = 0;
            bool ok = true, issued = false;
#pragma unroll 1
            for (int j = 0; j < N && ok; ++j) {
                const HeadGemm& p = jobs.job[j].p;
                const HeadSize z = size_of(p);
                const Range r = range_of(j, z);
                const bool a_mn = N == 2 ? p.a_mn != 0 : A_MN;
                idesc = tc::idesc_bf16(kBM, kBN, a_mn, B_MN);
                step_a = a_mn ? 128u : 2u;
                al0 = a_tile(0) >> 4 | (a_mn ? 512u : 1u) << 16;
                for (int g = r.g0; g < r.g1 && ok; g += r.step) {
                    const int split = g / (z.mt * z.nt);
                    int left = k_first(p, z, split + 1) - k_first(p, z, split);
                    while (left > 0 && ok) {
                        const int n = min(left, kSumBlocks);
                        left -= n;
                        if (!tc::mbar_wait(acce_bar(acc), acc_ph ^ 1u, st, tmo, kSiteMmaAccEmpty)) { ok = false; break; }
                        const uint32_t d = tmem + (uint32_t)(acc * kBN);
                        uint32_t more = 0;
                        for (int i = 0; i < n; i += 2) {
                            const int s1 = stage + 1 == stages ? 0 : stage + 1;
                            const uint32_t p1 = stage + 1 == stages ? ph ^ 1u : ph;
                            const bool two = i + 1 < n;
                            if (!tc::mbar_wait(full_bar(stage), ph, st, tmo, kSiteMmaFull)) { ok = false; break; }
                            if (two && !tc::mbar_wait(full_bar(s1), p1, st, tmo, kSiteMmaFull)) { ok = false; break; }
                            tc::fence_after_sync();
                            mma4(d, stage, more);
                            more = 1;
                            tc::mma_commit_2sm_multicast(empty_bar(stage), (uint16_t)0x3);
                            stage = s1; ph = p1;
                            if (two) {
                                mma4(d, stage, 1);
                                tc::mma_commit_2sm_multicast(empty_bar(stage), (uint16_t)0x3);
                                if (++stage == stages) { stage = 0; ph ^= 1u; }
                            }
                        }
                        issued = true;
                        if (!ok) break;
                        tc::mma_commit_2sm_multicast(accf_bar(acc), (uint16_t)0x3);
                        if (++acc == 2) { acc = 0; acc_ph ^= 1u; }
                    }
                }
            }
            if (!ok && issued) {
                // every MMA issued so far must finish before tensor memory is freed
                tc::mma_commit_2sm(drain_bar);
                drain_wait(drain_bar, 0);
            }
        }
    } else {
        if (p0.early) pdl_wait();
        const int q = warp & 3, half = (warp - 2) >> 2;   // TMEM lane quadrant, half of the tile's columns
        // 32 rows x 128 bytes are put down by row (a thread each), in the 128-byte swizzle, and leave as one box;
        // or they are taken up by eighths of a row, so that a store instruction writes four whole 128-byte lines (a
        // thread writing its own row touches 32 lines with each).
        const uint32_t pass = smem_base + kStageOutOffset + (uint32_t)(warp - 2) * kPassBytes;
        auto begin_pass = [&]() {
            if (lane == 0) tc::bulk_wait_read<0>();   // the box that left from here before
            __syncwarp();
        };
        auto send_pass = [&](const HeadJob& J, int x, int y, int z) {
            tc::fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
                tc::tma_store_3d(&J.out, pass, x, y, z);
                tc::bulk_commit();
            }
        };
        auto put = [&](int eighth, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
            tc::st_shared_v4(pass + lane * 128 + ((eighth ^ (lane & 7)) << 4), a, b, c, d);
        };
        auto take = [&](int i0, auto& v) {     // rows 4i + lane / 8 from i = i0 on, eighth lane % 8
#pragma unroll
            for (int i = 0; i < (int)(sizeof(v) / sizeof(uint4)); ++i) {
                const int row = 4 * (i0 + i) + (lane >> 3);
                v[i] = ld_shared16(pass + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
            }
        };
        int acc = 0;
        uint32_t acc_ph = 0;
        bool ok = true;
#pragma unroll 1
        for (int j = 0; j < N && ok; ++j) {
            const HeadJob& J = jobs.job[j];
            const HeadGemm& p = J.p;
            const HeadSize z = size_of(p);
            const Range range = range_of(j, z);
            const int M = z.M;
            const bool all = z.all;
            const float by = EPI == kEpiOut && p.scaled ? __ldcg(p.factors + 1) : 1.0f;
            for (int g = range.g0; g < range.g1; g += range.step) {
                const Tile t = head_tile(g, z.mt, z.nt, p.group);
                const int blocks = k_first(p, z, t.split + 1) - k_first(p, z, t.split);
                const int row0 = t.m * kBM + rank * 128 + q * 32, row = row0 + lane;
                const int col0 = t.n * kBN + half * 128;
                const int nv = min(128, p.N - col0);          // valid columns; none: <= 0
                const bool in = row < M;
                // what belongs to the row, fetched while the tile is being summed
                int lab = -1;                                 // its label
                float mul = 0.f, base = 0.f;
                float label_at_lse = 0.f;                     // its label's logit less its log-sum
                int orow = in ? row : -1;                     // its output row
                bool dead = false;
                // (dl: rows behind the last live token, up to the tile's end, are written as zeros: dW's last K block
                // reads some of them)
                if constexpr (EPI != kEpiOut) {
                    if (in) {
                        const int64_t tok = p.rows && !all ? p.rows[row] : row;
                        const int64_t y = label_at(p.labels, p.labels_i64, tok);
                        if (y >= 0 && y < p.N) lab = (int)y;
                        if (EPI == kEpiDl && lab >= 0) {
                            mul = p.dloss ? __ldg(p.dloss + tok) / __ldcg(p.factors) : 1.0f;
                            const float lse = __ldg(p.lse + tok);
                            base = -kLog2e * lse;
                            label_at_lse = __ldcg(p.label_logit + row) - lse;
                        }
                    }
                } else {
                    if (in && p.out_rows && !all) orow = p.out_rows[row];
                    dead = p.zero_dead && in && !is_live(p.labels, p.labels_i64, row, p.live_below);
                }
                __syncwarp();
                // rows of no token (but for those that dW's last K block reads): the sums are let go unread
                if (row0 >= (p.m_live ? (M + kBK - 1) / kBK * kBK : M)) {
                    for (int b0 = 0; b0 < blocks && ok; b0 += min(kSumBlocks, blocks - b0)) {
                        if (!tc::mbar_wait(accf_bar(acc), acc_ph, st, tmo, kSiteEpiAccFull)) { ok = false; break; }
                        mbar_arrive_pair(tc::mapa_shared(acce_bar(acc), 0));
                        if (++acc == 2) { acc = 0; acc_ph ^= 1u; }
                    }
                    if (!ok) break;
                    continue;
                }
                const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(half * 128);
                if constexpr (EPI == kEpiOut || EPI == kEpiDl) {
                    // 64 columns at a time: tensor memory, registers, staging, memory
                    if (blocks > 0) {
                        if (!tc::mbar_wait(accf_bar(acc), acc_ph, st, tmo, kSiteEpiAccFull)) { ok = false; break; }
                        __syncwarp();
                        tc::fence_after_sync();
                    }
                    const uint32_t tbase = lanes + (uint32_t)(acc * kBN);
                    const int64_t at = col0;
                    int o[8];                           // output rows of this lane's eighths
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xffffffffu, orow, 4 * i + (lane >> 3));
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        float r[2][32];
                        if (blocks > 0) {
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                tc::tmem_ld_32x32b_x32(tbase + 64 * h + 32 * c, reinterpret_cast<uint32_t(&)[32]>(r[c]));
                            tc::tmem_ld_wait();
                            if (h == 1) {
                                tc::fence_before_sync();
                                mbar_arrive_pair(tc::mapa_shared(acce_bar(acc), 0));
                                if (++acc == 2) { acc = 0; acc_ph ^= 1u; }
                            }
                        } else {
#pragma unroll
                            for (int c = 0; c < 2; ++c)
#pragma unroll
                                for (int i = 0; i < 32; ++i) r[c][i] = 0.f;
                        }
                        if (64 * h >= nv) continue;
                        uint4 v[8];
                        if constexpr (EPI == kEpiDl) {
                            begin_pass();
#pragma unroll
                            for (int e8 = 0; e8 < 8; ++e8) {
                                uint32_t w[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const int j = 8 * e8 + 2 * i;
                                    float2 e = make_float2(r[j / 32][j % 32], r[j / 32][j % 32 + 1]);
                                    e = __ffma2_rn(e, make_float2(kLog2e, kLog2e), make_float2(base, base));
                                    e = __fmul2_rn(make_float2(exp2_approx(e.x), exp2_approx(e.y)), make_float2(mul, mul));
                                    w[i] = lab >= 0 ? pack_bf16x2(e.x, e.y) : 0u;
                                }
                                put(e8, w[0], w[1], w[2], w[3]);
                            }
                            const int j = lab - col0 - 64 * h;      // the label's column of these 64
                            if (lab >= 0 && j >= 0 && j < 64)
                                st_shared16(pass + lane * 128 + (((j >> 3) ^ (lane & 7)) << 4) + 2 * (j & 7),
                                            __float2bfloat16_rn(mul * expm1f(label_at_lse)));
                            if (row0 < p.dl_rows) send_pass(J, col0 + 64 * h, row0, 0);
                            continue;
                        }
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                const float2 e = __fmul2_rn(make_float2(r[c][i], r[c][i + 1]), make_float2(by, by));
                                r[c][i] = e.x;
                                r[c][i + 1] = e.y;
                            }
                        if (!p.out_f32 && !p.add) {
                            begin_pass();
#pragma unroll
                            for (int e8 = 0; e8 < 8; ++e8) {
                                uint32_t w[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const int j = 8 * e8 + 2 * i;
                                    w[i] = dead ? 0u : pack_bf16x2(r[j / 32][j % 32], r[j / 32][j % 32 + 1]);
                                }
                                put(e8, w[0], w[1], w[2], w[3]);
                            }
                            if (p.tma_out) {
                                if (row0 < M) send_pass(J, col0 + 64 * h, row0, 0);
                                continue;
                            }
                            __syncwarp();
                            take(0, v);
                            const int cc = 64 * h + 8 * (lane & 7);
                            __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.out) + at + cc;
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                if (o[i] >= 0 && cc < nv) *reinterpret_cast<uint4*>(to + (int64_t)o[i] * p.N) = v[i];
                            __syncwarp();
                            continue;
                        }
#pragma unroll
                        for (int c = 0; c < 2; ++c) {      // 32 fp32 columns, 128 bytes of a row
                            const int cc = 64 * h + 32 * c + 4 * (lane & 7);
                            begin_pass();
#pragma unroll
                            for (int e8 = 0; e8 < 8; ++e8)
                                put(e8, __float_as_uint(r[c][4 * e8]), __float_as_uint(r[c][4 * e8 + 1]),
                                    __float_as_uint(r[c][4 * e8 + 2]), __float_as_uint(r[c][4 * e8 + 3]));
                            if (p.tma_out) {
                                if (row0 < M && 64 * h + 32 * c < nv) send_pass(J, col0 + 64 * h + 32 * c, row0, t.split);
                                continue;
                            }
                            __syncwarp();
                            take(0, v);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                if (o[i] < 0 || cc >= nv) continue;
                                const int64_t to = at + (int64_t)o[i] * p.N + cc;
                                float4 f = make_float4(__uint_as_float(v[i].x), __uint_as_float(v[i].y),
                                                       __uint_as_float(v[i].z), __uint_as_float(v[i].w));
                                if (p.add) {
                                    const float4 g4 = *reinterpret_cast<const float4*>(p.add + to);
                                    f.x += g4.x; f.y += g4.y; f.z += g4.z; f.w += g4.w;
                                }
                                if (p.out_f32)
                                    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + to) = f;
                                else
                                    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + to) =
                                        make_uint2(pack_bf16x2(f.x, f.y), pack_bf16x2(f.z, f.w));
                            }
                            __syncwarp();
                        }
                    }
                    continue;
                } else {
                    float r[4][32];
                    for (int b0 = 0; b0 < blocks; b0 += min(kSumBlocks, blocks - b0)) {
                        if (!tc::mbar_wait(accf_bar(acc), acc_ph, st, tmo, kSiteEpiAccFull)) { ok = false; break; }
                        __syncwarp();
                        tc::fence_after_sync();
                        const uint32_t tbase = lanes + (uint32_t)(acc * kBN);
                        if (b0 == 0) {
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
                        mbar_arrive_pair(tc::mapa_shared(acce_bar(acc), 0));
                        if (++acc == 2) { acc = 0; acc_ph ^= 1u; }
                    }
                    if (!ok) break;
                    if (nv <= 0) {
                        // nothing of the last tile
                        if (in) p.stats[(int64_t)row * p.stat_tiles + 2 * t.n + half] = make_float2(-INFINITY, 0.f);
                        continue;
                    }
                    const int lc = lab >= col0 && lab < col0 + nv ? lab - col0 : -1;
                    if (nv < 128) {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int i = 0; i < 32; ++i) r[c][i] = 32 * c + i < nv ? r[c][i] : -INFINITY;
                    }
                    mul = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int i = 0; i < 32; ++i) mul = fmaxf(mul, r[c][i]);
                    base = kRootShift - (mul == -INFINITY ? 0.f : mul * (0.5f * kLog2e));
                    // the label's own term stays out of the sum, so that the others' share keeps its
                    // digits where the label takes nearly everything
                    if (__any_sync(0xffffffffu, lc >= 0)) {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int i = 0; i < 32; ++i) r[c][i] = 32 * c + i == lc ? -INFINITY : r[c][i];
                    }
                    float2 s[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[c] = make_float2(0.f, 0.f);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {      // 64 columns, 128 bytes of a row
                        if (64 * h >= nv) break;
                        if constexpr (EPI != kEpiStats) begin_pass();
#pragma unroll
                        for (int e8 = 0; e8 < 8; ++e8) {
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int j = 64 * h + 8 * e8 + 2 * i;
                                float2 v = make_float2(r[j / 32][j % 32], r[j / 32][j % 32 + 1]);
                                v = __ffma2_rn(v, make_float2(0.5f * kLog2e, 0.5f * kLog2e), make_float2(base, base));
                                v = make_float2(exp2_approx(v.x), exp2_approx(v.y));
                                s[j / 32] = __ffma2_rn(v, v, s[j / 32]);
                                const __half2 v2 = __float22half2_rn(v);
                                w[i] = in ? *reinterpret_cast<const uint32_t*>(&v2) : 0u;
                            }
                            if (EPI != kEpiStats) put(e8, w[0], w[1], w[2], w[3]);
                        }
                        if (EPI != kEpiStats && row0 < p.dl_rows) send_pass(J, col0 + 64 * h, row0, 0);
                    }
                    if (in) {
                        const float sum = ((s[0].x + s[0].y) + (s[1].x + s[1].y)) + ((s[2].x + s[2].y) + (s[3].x + s[3].y));
                        p.stats[(int64_t)row * p.stat_tiles + 2 * t.n + half] = make_float2(mul, sum * kRootScale);
                    }
                }
            }
        }
    }
    if (EPI != kEpiStats && warp >= 2 && lane == 0) tc::bulk_wait<0>();   // every box has left and arrived
    if (p0.wait_late && threadIdx.x == 0) pdl_wait();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    tc::cluster_sync();   // no CTA frees or leaves while its peer may still use the pair's resources
    if (warp == 1) tc::tmem_dealloc_2sm(tmem, 512);
}

// ------------------------------------------------------------------ live tokens

constexpr int kRowThreads = 256;

// Sum over the CTA's threads (whole warps), the same in each; red holds 33 floats.
__device__ __forceinline__ float cta_sum(float v, float* red) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < (int)blockDim.x / 32 ? red[lane] : 0.f;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

__device__ __forceinline__ float dot8(const uint4& a, const uint4& b, float s) {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) s = fmaf(bf16_hi(u[i]), bf16_hi(v[i]), fmaf(bf16_lo(u[i]), bf16_lo(v[i]), s));
    return s;
}

// A label's logit in fp32 by this thread's vectors (id of n): the tensor cores' sums
// are cut, and the loss of a well-predicted token is a small difference to this one.
__device__ __forceinline__ float label_dot(const uint4* x, const uint4* w, int nv, int id, int n) {
    float s = 0.f;
    for (int v = id; v < nv; v += n) s = dot8(__ldg(x + v), __ldg(w + v), s);
    return s;
}

// |d| as bits whose order is its own; 0 for NaN and infinity, which stay their token's.
__device__ __forceinline__ unsigned finite_bits(float d) {
    const unsigned u = __float_as_uint(d) & 0x7fffffffu;
    return u < 0x7f800000u ? u : 0u;
}
// {top, c}; without live tokens c is 0, whatever the scale (1 / 0, say): gradients are zeros.
__device__ __forceinline__ void put_factors(float* factors, unsigned top_bits, bool any, float scale) {
    const float top = top_bits ? __uint_as_float(top_bits) : 1.0f;
    factors[0] = top;
    factors[1] = any ? scale * top : 0.f;
}

// For up to one row tile of tokens: a CTA per token copies its row, zeros for a token
// without a label, for dW (whose K the tokens are), and forms the label's logit if
// asked. The first CTA clears the status block, and one behind the tokens' forms the
// gradient's factors. Without xc: the status block alone. Bound by its launch: 5 us by
// itself at T = 8, less than 1 in a chain of launches.
__global__ void __launch_bounds__(kRowThreads)
head_start_kernel(const uint4* __restrict__ x, int64_t ldx, const uint4* __restrict__ W, const void* labels, int i64,
                  int V, int nv, const float* __restrict__ dloss, float scale, float* factors, uint4* __restrict__ xc,
                  float* label_logit, int32_t* status) {
    __shared__ float red[33];
    __shared__ unsigned top;
    pdl_wait();
    pdl_allow_next();
    const int64_t t = blockIdx.x;
    if (t == 0 && status && threadIdx.x < kStatusBytes / 4) status[threadIdx.x] = 0;
    if (!xc) return;
    if (t == gridDim.x - 1) {   // at most kPlainRows tokens, one a thread
        if (threadIdx.x == 0) top = 0;
        const bool in = threadIdx.x < gridDim.x - 1;
        const float d = in && dloss ? __ldg(dloss + threadIdx.x) : 0.f;
        const bool l = in && is_live(labels, i64, threadIdx.x, V);
        const int any = __syncthreads_or(l);
        if (l) atomicMax(&top, finite_bits(d));
        __syncthreads();
        if (threadIdx.x == 0) put_factors(factors, top, any, scale);
        return;
    }
    const bool on = is_live(labels, i64, t, V);
    for (int v = threadIdx.x; v < nv; v += kRowThreads)
        xc[t * nv + v] = on ? __ldg(x + t * ldx + v) : make_uint4(0, 0, 0, 0);
    if (label_logit && on) {
        const float s = cta_sum(label_dot(x + t * ldx, W + label_at(labels, i64, t) * nv, nv, threadIdx.x, kRowThreads), red);
        if (threadIdx.x == 0) label_logit[t] = s;
    }
}

// For more tokens. CTA b takes `span` tokens from b * span on, kPrepTokens at a time:
// live ones get the next place (tokens in order), their rows are copied there unless
// every token is live, and their labels' logits are formed; the others' outputs are
// zeroed. Each CTA counts the live tokens before its own from the labels themselves.
// Behind the last live row, rows up to the next multiple of kBK are zeroed: dW's last K
// block reads them. The first CTA clears the status block and, with a gradient, forms its
// factors. Bound by the loads in flight, so
// four tokens' rows are read side by side: 25 us at T = 2560, H = 7168 (73 MB, 2.9 TB/s from
// a cold start). Beside the logits' kernel in a kernel of its own, the labels' logits cost
// as much time as here (scoring T = 1000, H = 4096, V = 20000: 115.8 and 117.1 us; with a
// gradient, H = 1024: 124.9 and 122.5).
constexpr int kPrepTokens = 4;
__global__ void __launch_bounds__(kRowThreads)
head_prep_kernel(const uint4* __restrict__ x, int64_t ldx, const uint4* __restrict__ W, const void* labels, int i64,
                 int T, int V, int nv, int span, int32_t* __restrict__ rows, int32_t* __restrict__ live,
                 uint4* __restrict__ xc, float* __restrict__ label_logit, float* loss, float* lse, uint4* dx,
                 const float* __restrict__ dloss, float scale, float* factors, int32_t* status) {
    __shared__ int32_t sh[2];
    __shared__ unsigned top;
    __shared__ int32_t place[kPrepTokens];
    __shared__ float red[kPrepTokens][kRowThreads / 32];
    pdl_wait();
    pdl_allow_next();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t0 = blockIdx.x * span, t1 = min(t0 + span, T);
    if (tid < 2) sh[tid] = 0;
    if (tid == 2) top = 0;
    if (blockIdx.x == 0 && status && tid < kStatusBytes / 4) status[tid] = 0;
    __syncthreads();
    int before = 0, count = 0;
    unsigned bits = 0;
    const float* weights = blockIdx.x == 0 ? dloss : nullptr;
#pragma unroll 8
    for (int t = tid; t < T; t += kRowThreads) {
        const int l = is_live(labels, i64, t, V) ? 1 : 0;
        count += l;
        before += t < t0 ? l : 0;
        const unsigned b = weights ? finite_bits(__ldg(weights + t)) : 0u;
        bits = l ? max(bits, b) : bits;
    }
    bits = __reduce_max_sync(0xffffffffu, bits);
    before = __reduce_add_sync(0xffffffffu, before);
    count = __reduce_add_sync(0xffffffffu, count);
    if (lane == 0) {
        atomicAdd(&sh[0], before);
        atomicAdd(&sh[1], count);
        atomicMax(&top, bits);
    }
    __syncthreads();
    const int total = sh[1];
    int next = sh[0];
    if (blockIdx.x == 0 && tid == 0) {
        *live = total;
        if (factors) put_factors(factors, top, total > 0, scale);
    }
    const bool all = total == T;
    for (int c0 = t0; c0 < t1; c0 += kPrepTokens) {
        const int n = min(kPrepTokens, t1 - c0);
        const bool l = lane < n && is_live(labels, i64, c0 + lane, V);
        const unsigned b = __ballot_sync(0xffffffffu, l);
        __syncthreads();
        if (warp == 0 && lane < n) {
            const int to = l ? next + __popc(b & ((1u << lane) - 1)) : -1;
            place[lane] = to;
            if (l) {
                rows[to] = c0 + lane;
            } else {
                if (loss) loss[c0 + lane] = 0.f;
                if (lse) lse[c0 + lane] = 0.f;
            }
        }
        next += __popc(b);
        __syncthreads();
        int to[kPrepTokens];
        const uint4 *xr[kPrepTokens], *wr[kPrepTokens];
        float dot[kPrepTokens];
#pragma unroll
        for (int j = 0; j < kPrepTokens; ++j) {
            to[j] = j < n ? place[j] : -2;
            xr[j] = x + (int64_t)(c0 + j) * ldx;
            wr[j] = to[j] >= 0 ? W + label_at(labels, i64, c0 + j) * nv : W;
            dot[j] = 0.f;
        }
        for (int v = tid; v < nv; v += kRowThreads) {
            uint4 a[kPrepTokens], w[kPrepTokens];
#pragma unroll
            for (int j = 0; j < kPrepTokens; ++j)
                if (to[j] >= 0) {
                    a[j] = __ldg(xr[j] + v);
                    w[j] = __ldg(wr[j] + v);
                }
#pragma unroll
            for (int j = 0; j < kPrepTokens; ++j) {
                if (to[j] >= 0) {
                    dot[j] = dot8(a[j], w[j], dot[j]);
                    if (!all) xc[(int64_t)to[j] * nv + v] = a[j];
                } else if (to[j] == -1 && dx) {
                    dx[(int64_t)(c0 + j) * nv + v] = make_uint4(0, 0, 0, 0);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kPrepTokens; ++j) {
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], d);
            if (lane == 0) red[j][warp] = dot[j];
        }
        __syncthreads();
        if (tid < n && place[tid] >= 0) {
            float s = 0.f;
            for (int i = 0; i < kRowThreads / 32; ++i) s += red[tid][i];
            label_logit[place[tid]] = s;
        }
    }
    if (!all && t1 == T) {
        const int end = (total + kBK - 1) / kBK * kBK;
        for (int64_t v = (int64_t)total * nv + tid; v < (int64_t)end * nv; v += kRowThreads)
            xc[v] = make_uint4(0, 0, 0, 0);
    }
}

// ------------------------------------------------------------------ log-sum and loss

// The sums of a row's stat tiles joined: the largest logit, the other tokens' sum
// relative to it and the label's term.
struct RowSum {
    float top, others, own;   // sum of all = others + own, over exp(top)
};
__device__ __forceinline__ RowSum join_row(const float2* stats, int n, float label_logit, float* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // a thread's first pair stays in registers between the two passes
    const float2 v0 = (int)threadIdx.x < n ? __ldcg(stats + threadIdx.x) : make_float2(-INFINITY, 0.f);
    float m = fmaxf(label_logit, v0.x);   // the label's, at its place in the order, if the tiles' own is a little lower
    for (int i = threadIdx.x + kRowThreads; i < n; i += kRowThreads) m = fmaxf(m, __ldcg(stats + i).x);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (lane == 0) red[warp] = m;
    __syncthreads();
    m = lane < kRowThreads / 32 ? red[lane] : -INFINITY;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float base = m == -INFINITY ? 0.f : m;
    auto term = [&](const float2& v) { return v.y * exp2_approx((v.x == -INFINITY ? -INFINITY : v.x - base) * kLog2e); };
    float s = term(v0);
    for (int i = threadIdx.x + kRowThreads; i < n; i += kRowThreads) s += term(__ldcg(stats + i));
    s = cta_sum(s, red + 32);
    RowSum r;
    r.top = base;
    r.others = s;
    r.own = expf(label_logit - base);
    return r;
}

// log(others + own) - log(own), by the form that loses no digits.
__device__ __forceinline__ float row_loss(const RowSum& r, float label_logit) {
    return r.own > r.others ? log1pf(r.others / r.own) : logf(r.others + r.own) - (label_logit - r.top);
}

// A CTA per live token. For one row tile the label's logit is formed here, while the
// logits' kernel still runs: x, W and labels are the caller's and the list of live tokens
// is the kernel's before that one, all complete before that one began. Bound by the
// latency of its two passes over the row's V / 128 pairs: 12 us at T = 2560, V = 32768.
__global__ void __launch_bounds__(kRowThreads)
head_loss_kernel(const float2* __restrict__ stats, int stat_tiles, const uint4* __restrict__ x, int64_t ldx,
                 const uint4* __restrict__ W, int nv, const int32_t* __restrict__ rows, const int32_t* __restrict__ live,
                 const float* label_logit, const void* labels, int i64, int V, float* loss, float* lse) {
    __shared__ float red[128];
    pdl_allow_next();
    const int i = blockIdx.x;
    if (live && i >= *live) {
        pdl_wait();   // this kernel ends after the one ahead
        return;
    }
    const int64_t t = rows ? rows[i] : i;
    const bool on = is_live(labels, i64, t, V);
    float own = 0.f;
    if (live) own = __ldcg(label_logit + i);
    else if (on) own = cta_sum(label_dot(x + t * ldx, W + label_at(labels, i64, t) * nv, nv, threadIdx.x, kRowThreads), red + 96);
    pdl_wait();
    const RowSum r = join_row(stats + (int64_t)i * stat_tiles, stat_tiles, on ? own : -INFINITY, red);
    if (threadIdx.x != 0) return;
    loss[t] = on ? row_loss(r, own) : 0.f;
    if (lse) lse[t] = on ? r.top + logf(r.others + r.own) : 0.f;
}

// The same with a gradient: then the row's exponentials, in their place, become
//   dl[v] = d e[v] exp(top of its columns - lse),   dl[label] = -d others / (others + own)
// and zeros for a token without a label (rows == NULL; else only live tokens are here).
// Few rows are cut along the vocabulary (gridDim.y), each part joining the sums itself.
// One pass over the bytes, read and written: 322 us at T = 4096, V = 131072 (6.7 TB/s),
// 57 us at T = 2560, V = 32768. Roundings: the exponential is s * s of an FP16 root
// (2^-10 relative), dl goes to BF16 (2^-8) because it is an operand of both products; the
// label's dl comes from the exact fp32 sums.
__global__ void __launch_bounds__(kRowThreads)
head_dl_kernel(const float2* __restrict__ stats, int stat_tiles, const uint4* __restrict__ x, int64_t ldx,
               const uint4* __restrict__ W, int nv, const int32_t* __restrict__ rows, const int32_t* __restrict__ live,
               const float* label_logit, const void* labels, int i64, const float* __restrict__ dloss, const float* factors,
               __nv_bfloat16* dl, int64_t ld, int V, float* loss, float* lse) {
    __shared__ float red[128];
    pdl_allow_next();
    const int i = blockIdx.x;
    if (live && i >= *live) {
        pdl_wait();
        return;
    }
    const int64_t t = rows ? rows[i] : i;
    const bool on = is_live(labels, i64, t, V);
    const int label = on ? (int)label_at(labels, i64, t) : 0;
    float own = 0.f;
    if (live) own = __ldcg(label_logit + i);
    else if (on) own = cta_sum(label_dot(x + t * ldx, W + (int64_t)label * nv, nv, threadIdx.x, kRowThreads), red + 96);
    const float coef = dloss ? dloss[t] / __ldcg(factors) : 1.0f;
    pdl_wait();
    __nv_bfloat16* row = dl + i * ld;
    const int vecs = (V + 7) / 8, per = (vecs + (int)gridDim.y - 1) / (int)gridDim.y;
    const int v0 = (int)blockIdx.y * per, v1 = min(v0 + per, vecs);
    if (!on) {
        for (int v = v0 + threadIdx.x; v < v1; v += kRowThreads) *reinterpret_cast<uint4*>(row + 8 * v) = make_uint4(0, 0, 0, 0);
        if (threadIdx.x == 0 && blockIdx.y == 0) {
            loss[t] = 0.f;
            if (lse) lse[t] = 0.f;
        }
        return;
    }
    const float2* st = stats + (int64_t)i * stat_tiles;
    // a thread's first eight exponentials are on their way while the sums are joined
    const int first = v0 + threadIdx.x;
    uint4 e0 = make_uint4(0, 0, 0, 0);
    float top0 = 0.f;
    if (first < v1) {
        e0 = __ldcg(reinterpret_cast<const uint4*>(row + 8 * first));
        top0 = __ldcg(st + first / 16).x;
    }
    const RowSum r = join_row(st, stat_tiles, own, red);
    const float sum = r.others + r.own;
    const float inv = coef / sum * kRootScale;
    auto form = [&](int v, const uint4& e, float top) {
        const float f = inv * exp2_approx((top - r.top) * kLog2e);
        const uint32_t w[4] = {e.x, e.y, e.z, e.w};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
            o[j] = pack_bf16x2(a.x * f * a.x, a.y * f * a.y);
        }
        *reinterpret_cast<uint4*>(row + 8 * v) = make_uint4(o[0], o[1], o[2], o[3]);
        if (label >> 3 == v) row[label] = __float2bfloat16_rn(-coef * (r.others / sum));
    };
    if (first < v1) form(first, e0, top0);
#pragma unroll 4
    for (int v = first + kRowThreads; v < v1; v += kRowThreads)
        form(v, __ldcg(reinterpret_cast<const uint4*>(row + 8 * v)), __ldcg(st + v / 16).x);
    if (threadIdx.x != 0 || blockIdx.y != 0) return;
    loss[t] = row_loss(r, own);
    if (lse) lse[t] = r.top + logf(sum);
}

// dx rows from the parts of K, four columns a thread. WAYS = 1: a thread adds up all parts in
// order. WAYS = 4, where that leaves most threads without work: the warp's four groups of
// eight lanes add up every fourth part each, then these sums in a fixed order, so that a
// thread's loads are one or two trips to L2 (T = 100, H = 512, V = 8191, whole calls: 27.7
// us, 30.3 with one way; T = 14, H = 496, V = 65750: 61.7 and 67.6; but T = 300, H = 2048,
// V = 32768: 168.6 and 163.5, bound by the bytes). Without a list of rows, a token without
// a label gets zeros. The sums are multiplied by c. A kernel of dW's own is launched behind this one and needs nothing
// of it, so it may begin at once; two to four CTAs an SM took the same time, one 2% more.
constexpr int kJoinThreads = 256;
template <int WAYS>
__global__ void __launch_bounds__(kJoinThreads)
head_join_kernel(const float4* part, int64_t stride, int splits, int n, int nq, const int32_t* __restrict__ rows,
                 const int32_t* __restrict__ live, const void* labels, int i64, int V, const float* factors,
                 uint2* __restrict__ dx) {
    pdl_allow_next();
    const float c = __ldcg(factors + 1);   // complete since before the kernel ahead began, as the labels
    pdl_wait();
    const int64_t total = (int64_t)(live ? *live : n) * nq;
    constexpr int kLanes = 32 / WAYS;
    const int lane = threadIdx.x & 31, way = lane / kLanes;
    for (int64_t at0 = ((int64_t)blockIdx.x * kJoinThreads + threadIdx.x - lane) / WAYS; at0 < total;
         at0 += (int64_t)gridDim.x * (kJoinThreads / WAYS)) {
        const int64_t at = at0 + lane % kLanes;
        const bool in = at < total;
        const int64_t t = !in ? 0 : rows ? rows[at / nq] : at / nq;
        const bool on = in && (rows || is_live(labels, i64, t, V));
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        if (on) {
#pragma unroll 8
            for (int s = way; s < splits; s += WAYS) {
                const float4 b = __ldcg(part + s * stride + at);
                a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
            }
        }
#pragma unroll
        for (int d = kLanes; d < 32; d <<= 1) {
            a.x += __shfl_xor_sync(0xffffffffu, a.x, d);
            a.y += __shfl_xor_sync(0xffffffffu, a.y, d);
            a.z += __shfl_xor_sync(0xffffffffu, a.z, d);
            a.w += __shfl_xor_sync(0xffffffffu, a.w, d);
        }
        if (in && way == 0)
            dx[t * nq + at % nq] = on ? make_uint2(pack_bf16x2(a.x * c, a.y * c), pack_bf16x2(a.z * c, a.w * c)) : make_uint2(0, 0);
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

// The same for an MN-major operand whose rows are whole groups of 64 columns: [groups][rows][64], in boxes of two
// groups x 64 rows, so that one copy brings a CTA's 128 columns of a K block (two copies for each operand were as much
// as the producer could issue: dW at T = 2560, H = 7168, V = 32768 took 641 us, this 626).
bool make_tmap_groups(CUtensorMap* m, const void* base, int64_t rows, int64_t groups, int64_t ld) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)groups};
    cuuint64_t strides[2] = {(cuuint64_t)(ld * 2), 128};
    cuuint32_t box[3] = {64, 64, 2};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What an epilogue writes: [parts][rows][cols] of 2- or 4-byte elements, row pitch ld, in boxes of 32 rows x 128 bytes.
bool make_tmap_out(CUtensorMap* m, void* base, int bytes, int64_t parts, int64_t rows, int64_t cols, int64_t ld) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)parts};
    cuuint64_t strides[2] = {(cuuint64_t)(ld * bytes), (cuuint64_t)(rows * ld * bytes)};
    cuuint32_t box[3] = {(cuuint32_t)(128 / bytes), 32, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pairs of CTAs of a kernel that can be resident at once, asked once per kernel and
// device.
template <bool A_MN, bool B_MN, int EPI, int N>
int resident_pairs(void (*kern)(HeadJobs<N>), cudaLaunchConfig_t cfg, int num_sms) {
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

// What a product reads.
struct Operand {
    const void* base;
    int64_t rows, cols, ld;
};

// A product's maps and ring. `all`: the operand that replaces A (logits) or B (dW) when
// every token is live. Boxes: two groups of 64 columns x 64 rows of K where the operand is
// MN-major, else a CTA's rows.
bool make_job(HeadJob& J, bool a_mn, bool b_mn, int epi, const Operand& a, const Operand& b, const Operand& all,
              const HeadGemm& params) {
    J.p = params;
    HeadGemm& p = J.p;
    // up to 128 rows (of a count that the host knows): boxes of as many, and a longer ring. 128-row boxes that are
    // mostly outside the tensor took as long as full ones (T = 1, H = 1024, V = 32768: 25.9 us, this 19.7)
    const int rows = !a_mn && !p.m_live && p.M <= 128 ? (int)align_up(p.M, 8) : 128;
    p.a_mn = a_mn;
    p.a_bytes = p.a_room = rows * kBK * 2;
    p.stages = std::min(kMaxStages, (kBarOffset - kOperandBytes + p.a_room) / (p.a_room + kOperandBytes));
    p.a_groups = a_mn && a.cols % 64 == 0;
    p.b_groups = b_mn && b.cols % 64 == 0;
    auto map = [](CUtensorMap* m, const Operand& o, bool groups, int box_rows) {
        return groups ? make_tmap_groups(m, o.base, o.rows, o.cols / 64, o.ld)
                      : make_tmap_pitch(m, o.base, o.rows, o.cols, o.ld, box_rows);
    };
    const int box_a = a_mn ? kBK : rows, box_b = b_mn ? kBK : 128;
    if (!map(&J.a, a, p.a_groups, box_a) || !map(&J.b, b, p.b_groups, box_b)) return false;
    const Operand& other = epi == kEpiOut ? b : a;       // what `all` stands in for
    J.all = epi == kEpiOut ? J.b : J.a;
    if (all.base != other.base && !map(&J.all, all, epi == kEpiOut && p.b_groups, epi == kEpiOut ? box_b : box_a)) return false;
    p.tma_out = epi != kEpiOut || (!p.out_rows && !p.add && !p.zero_dead);
    J.out = J.a;
    if (epi == kEpiExp || epi == kEpiDl) return make_tmap_out(&J.out, p.dl, 2, 1, p.dl_rows, p.ld_dl, p.ld_dl);
    if (epi == kEpiOut && p.tma_out) return make_tmap_out(&J.out, p.out, p.out_f32 ? 4 : 2, p.splits, p.M, p.N, p.N);
    return true;
}

int64_t tiles_of(const HeadGemm& p) { return (int64_t)ceil_div(p.M, kBM) * ceil_div(p.N, kBN) * p.splits; }

// Cycles of a tile of dX and of dW, about 700 a K block and 4000 at least for the latter's
// way out, and of each pair where all share both products.
double dx_tile_cycles(const HeadGemm& x) { return 700.0 * ceil_div(x.K, kBK) / x.splits; }
double dw_tile_cycles(const HeadGemm& w) { return std::max(700 * ceil_div(w.K, kBK), 4000); }
double pair_cycles(const HeadGemm& x, const HeadGemm& w, int pairs) {
    return (tiles_of(x) * dx_tile_cycles(x) + tiles_of(w) * dw_tile_cycles(w)) / std::max(pairs, 1);
}
// Up to here dX and dW go in one launch: a launch less counts for more than what the
// fixed shares lose (T = 100, H = 512, V = 8191: 30.6 us in one launch, 33.1 in two;
// T = 700, H = 1000, V = 20000: 119 and 114).
constexpr double kOneLaunchCycles = 2e4;

template <bool A_MN, bool B_MN, int EPI, int N>
cudaError_t launch_jobs(HeadJobs<N>& jobs, int num_sms, cudaStream_t s) {
    auto kern = head_gemm_kernel<A_MN, B_MN, EPI, N>;
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
    int pairs = resident_pairs<A_MN, B_MN, EPI, N>(kern, cfg, num_sms);
    if constexpr (N == 1) {
        pairs = (int)std::min<int64_t>(tiles_of(jobs.job[0].p), pairs);
    } else {
        // the pairs with a tile of dX take as many fewer of dW's as that one costs
        HeadGemm &x = jobs.job[0].p, &w = jobs.job[1].p;
        x.a_room = w.a_room;
        x.stages = w.stages;
        const int64_t tiles = tiles_of(w);
        jobs.lead = (int)std::min<int64_t>(tiles_of(x), pairs);
        const double cx = dx_tile_cycles(x), cw = dw_tile_cycles(w), each = pair_cycles(x, w, pairs);
        jobs.lead_tiles = jobs.lead == pairs ? (int)tiles
                                             : (int)std::min<double>(tiles, std::max(0.0, (each - cx) / cw * jobs.lead));
    }
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    cfg.gridDim = dim3(2 * pairs);
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, jobs);
}

template <bool A_MN, bool B_MN, int EPI>
cudaError_t run_head_gemm(const Operand& a, const Operand& b, const Operand& all, const HeadGemm& p, int num_sms,
                          cudaStream_t s) {
    HeadJobs<1> jobs{};
    if (!make_job(jobs.job[0], A_MN, B_MN, EPI, a, b, all, p)) return cudaErrorInvalidValue;
    return launch_jobs<A_MN, B_MN, EPI, 1>(jobs, num_sms, s);
}

constexpr int kGroup = 16;              // row tiles of the walk's groups
constexpr int64_t kPieceBytes = (int64_t)4 << 30;
constexpr int kPieceMax = 65536;
// Up to one row tile, ignored tokens cost no products: nothing is gathered then.
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

// Parts of the vocabulary for dX where its tiles alone leave most pairs without work: as
// many as give each pair one, of 8 K blocks at least.
int dx_splits(int tokens, int H, int V, int pairs) {
    const int tiles = ceil_div(tokens, kBM) * ceil_div(H, kBN);
    return 2 * tiles > pairs ? 1 : std::max(1, std::min(pairs / tiles, ceil_div(V, kBK) / 8));
}

// Parts of a row for head_dl_kernel: three CTAs an SM, each with a vector a thread at least.
int dl_parts(int rows, int V) {
    return std::max(1, std::min(3 * sm_count() / rows, ceil_div(V, 8 * kRowThreads)));
}

struct HeadLayout {
    size_t rows, live, label, stats, xc, dl, part, acc, total;
    int piece, splits;
};

// grad: the gradients that a call forms (HeadGrad bits). dX's parts are held with dx alone, and dW's running sum where a
// BF16 one is formed in several pieces (an fp32 one is its own sum).
HeadLayout head_layout(int T, int H, int V, int grad, int want, int num_sms) {
    HeadLayout L{};
    size_t o = 1024;   // the status block
    auto take = [&](int64_t bytes) {
        const size_t at = o;
        o += align_up(bytes, 1024);
        return at;
    };
    L.piece = piece_tokens(T, V, want);
    L.splits = grad & kHeadDx ? dx_splits(L.piece, H, V, num_sms / 2) : 1;
    const int64_t cap = T > kPlainRows ? align_up(L.piece, kBM) : L.piece;   // gathered rows fill tiles
    L.live = take(12);   // and the gradient's two factors
    L.rows = take(cap * 4);
    L.label = take(cap * 4);
    L.stats = take(L.piece * (int64_t)(2 * ceil_div(V, kBN)) * 8);
    if (grad || T > kPlainRows) L.xc = take(cap * H * 2);
    if (grad) L.dl = take(cap * pitch_dl(V) * 2);
    if (L.splits > 1) L.part = take((int64_t)L.splits * L.piece * H * 4);
    if (grad & kHeadDw && L.piece < T) L.acc = take((int64_t)V * H * 4);
    L.total = o;
    return L;
}

}  // namespace

size_t head_workspace_bytes(int T, int H, int V, int grad, int piece, int num_sms) {
    return head_layout(T, H, V, grad, piece, num_sms).total;
}

cudaError_t launch_head(const HeadLaunch& a, const GemmCommon& c, cudaStream_t s) {
    const int T = a.T, H = a.H, V = a.V;
    const bool grad = a.dx || a.dW, forward = a.loss != nullptr;
    const HeadLayout L = head_layout(T, H, V, head_grads(a.dx, a.dW, a.dW_f32), a.piece, c.num_sms);
    char* ws = static_cast<char*>(a.workspace);
    float2* stats = reinterpret_cast<float2*>(ws + L.stats);
    float* label = reinterpret_cast<float*>(ws + L.label);
    uint4* xc = reinterpret_cast<uint4*>(ws + L.xc);
    __nv_bfloat16* dl = reinterpret_cast<__nv_bfloat16*>(ws + L.dl);
    const uint4* W = static_cast<const uint4*>(a.W);
    float* factors = grad ? reinterpret_cast<float*>(ws + L.live) + 1 : nullptr;
    const int nv = H / 8;
    cudaError_t e = cudaSuccess;
    if (T == 0) {
        e = cudaMemsetAsync(ws, 0, kStatusBytes, s);
        if (e == cudaSuccess && a.dW && !a.accumulate)
            e = cudaMemsetAsync(a.dW, 0, (size_t)V * H * (a.dW_f32 ? 4 : 2), s);
        return e;
    }
    for (int t0 = 0; t0 < T; t0 += L.piece) {
        const int n = std::min(L.piece, T - t0);
        const int64_t cap = align_up(n, kBM);
        const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x) + t0 * a.ldx;
        const void* labels = static_cast<const char*>(a.labels) + (int64_t)t0 * (a.labels_i64 ? 8 : 4);
        float* loss = forward ? a.loss + t0 : nullptr;
        float* lse = a.lse ? a.lse + t0 : nullptr;
        const float* dloss = a.dloss ? a.dloss + t0 : nullptr;
        __nv_bfloat16* dx = a.dx ? static_cast<__nv_bfloat16*>(a.dx) + (int64_t)t0 * H : nullptr;
        // one row tile (of a call of that size, not of a piece): tokens as they are; more: the live ones gathered
        const bool gather = T > kPlainRows;
        int32_t* live = gather ? reinterpret_cast<int32_t*>(ws + L.live) : nullptr;
        int32_t* rows = gather ? reinterpret_cast<int32_t*>(ws + L.rows) : nullptr;
        const uint4* xv = reinterpret_cast<const uint4*>(x);
        float* logit = forward ? nullptr : label;
        int32_t* status = t0 == 0 ? reinterpret_cast<int32_t*>(ws) : nullptr;
        if (gather) {
            const int span = kPrepTokens * ceil_div(n, kPrepTokens * 1024);
            e = launch_after(head_prep_kernel, dim3(ceil_div(n, span)), dim3(kRowThreads), 0, s, xv, a.ldx / 8, W, labels,
                             a.labels_i64, n, V, nv, span, rows, live, xc, label, loss, forward ? lse : nullptr,
                             reinterpret_cast<uint4*>(dx), dloss, a.scale, factors, status);
        } else {
            e = launch_after(head_start_kernel, dim3(grad ? n + 1 : 1), dim3(kRowThreads), 0, s, xv, a.ldx / 8, W, labels,
                             a.labels_i64, V, nv, dloss, a.scale, factors, grad ? xc : nullptr, logit, status);
        }
        if (e != cudaSuccess) return e;
        HeadGemm p{};
        p.status = c.status;
        p.timeout_ns = c.timeout_ns;
        p.withhold = a.withhold;
        p.live = live;
        p.rows = rows;
        p.tokens = n;
        p.group = kGroup;
        p.splits = 1;
        p.labels = labels;
        p.labels_i64 = a.labels_i64;
        p.label_logit = label;
        p.factors = factors;
        p.lse = lse;
        p.dloss = dloss;
        p.stats = stats;
        p.dl = dl;
        p.ld_dl = pitch_dl(V);
        p.dl_rows = gather ? cap : n;
        p.M = n;
        p.m_live = gather;
        p.N = V;
        p.K = H;
        p.stat_tiles = 2 * ceil_div(V, kBN);
        p.early = gather ? kEarlyNone : kEarlyA | kEarlyB;
        const Operand ox{x, n, H, a.ldx}, ow{a.W, V, H, H};
        const Operand oxc = gather ? Operand{xc, cap, H, H} : ox;
        if (!grad) {
            e = run_head_gemm<false, false, kEpiStats>(oxc, ow, ox, p, c.num_sms, s);
            if (e == cudaSuccess)
                e = launch_after(head_loss_kernel, dim3(n), dim3(kRowThreads), 0, s, (const float2*)stats, p.stat_tiles,
                                 xv, a.ldx / 8, W, nv, (const int32_t*)rows, (const int32_t*)live, (const float*)label, labels,
                                 a.labels_i64, V, loss, lse);
            if (e != cudaSuccess) return e;
            continue;
        }
        if (forward) {
            e = run_head_gemm<false, false, kEpiExp>(oxc, ow, ox, p, c.num_sms, s);
            if (e == cudaSuccess)
                e = launch_after(head_dl_kernel, dim3(n, dl_parts(n, V)), dim3(kRowThreads), 0, s, (const float2*)stats, p.stat_tiles,
                                 xv, a.ldx / 8, W, nv, (const int32_t*)rows, (const int32_t*)live,
                                 (const float*)label, labels, a.labels_i64, dloss, (const float*)factors, dl, p.ld_dl, V, loss, lse);
        } else {
            e = run_head_gemm<false, false, kEpiDl>(oxc, ow, ox, p, c.num_sms, s);
        }
        if (e != cudaSuccess) return e;
        p.early = kEarlyNone;
        const Operand odl{dl, p.dl_rows, V, p.ld_dl};
        const int splits = L.splits;
        HeadGemm px = p, pw = p;
        if (dx) {
            px.N = H;
            px.K = V;
            px.splits = splits;
            px.early = gather ? kEarlyNone : kEarlyB;
            if (splits > 1) {
                px.out = ws + L.part;
                px.out_f32 = 1;
            } else {
                px.scaled = 1;
                px.out = dx;
                px.out_rows = rows;
                px.zero_dead = !gather;
                px.live_below = V;
            }
        }
        // dl's rows are padded to whole groups; what lies behind V belongs to rows of dW that there are not
        const Operand odl64{dl, odl.rows, p.ld_dl, p.ld_dl}, clean{xc, n, H, H};
        const Operand &owx = gather ? oxc : clean, &owall = gather ? ox : clean;
        if (a.dW) {
            pw.M = V;
            pw.N = H;
            pw.K = n;
            pw.m_live = 0;
            pw.k_live = gather;
            pw.scaled = 1;
            // over several pieces the sum goes on in fp32 until the last one
            const bool first = t0 == 0, last = t0 + n >= T;
            float* acc = a.dW_f32 ? static_cast<float*>(a.dW) : reinterpret_cast<float*>(ws + L.acc);
            pw.out_f32 = a.dW_f32 || !last;
            pw.out = pw.out_f32 ? (void*)acc : a.dW;
            pw.add = first && !(a.dW_f32 && a.accumulate) ? nullptr : acc;
        }
        auto join = [&]() {
            const int nq = H / 4, most = 3 * sm_count();
            const int64_t at_once = (int64_t)most * kJoinThreads, quads = (int64_t)n * nq;
            const bool four = 4 * quads <= at_once;
            const int ctas = (int)std::min<int64_t>(((four ? 4 : 1) * quads + kJoinThreads - 1) / kJoinThreads, most);
            return launch_after(four ? head_join_kernel<4> : head_join_kernel<1>, dim3(ctas), dim3(kJoinThreads), 0, s, (const float4*)(ws + L.part),
                                (int64_t)n * nq, splits, n, nq, (const int32_t*)rows, (const int32_t*)live, labels,
                                a.labels_i64, V, (const float*)factors, reinterpret_cast<uint2*>(dx));
        };
        if (dx && a.dW && splits > 1 && pair_cycles(px, pw, c.num_sms / 2) < kOneLaunchCycles) {
            HeadJobs<2> jobs{};
            if (!make_job(jobs.job[0], false, true, kEpiOut, odl, ow, ow, px) ||
                !make_job(jobs.job[1], true, true, kEpiOut, odl64, owx, owall, pw))
                return cudaErrorInvalidValue;
            e = launch_jobs<false, true, kEpiOut, 2>(jobs, c.num_sms, s);
            if (e == cudaSuccess) e = join();
        } else {
            if (dx) e = run_head_gemm<false, true, kEpiOut>(odl, ow, ow, px, c.num_sms, s);
            if (e == cudaSuccess && dx && splits > 1) e = join();
            if (a.dW && e == cudaSuccess) {
                // dl and x were complete before dX's kernel let the next ones begin
                pw.wait_late = dx != nullptr;
                e = run_head_gemm<true, true, kEpiOut>(odl64, owx, owall, pw, c.num_sms, s);
            }
        }
        if (e != cudaSuccess) return e;
    }
    return e;
}

}  // namespace mok
