// few.cu - the whole routed layer for a few tokens (T <= 128) in two kernels:
// the router (logits, top-k), then everything else (both expert GEMMs, weighted
// sum, shared expert).
//
// With few tokens the layer is bound by reading each selected expert's weights
// once: a 128-row tile of packed weights takes longer to arrive than its
// product with up to 128 token columns takes on the tensor cores. So the
// weights are the M side of the MMAs and all T tokens are the N side, for every
// active expert: no gather, no per-expert token lists, no padding of rows. A
// token's result from an expert that it did not select is dropped (gate/up: the
// row is never read with a weight; down: the accumulation skips the column).
//
//   phase 1   h_e = SwiGLU(W_gu[e] x^T)       units: (expert, row tile, K block)
//   phase 2   out = sum_e w_e * (W_dn[e] h_e^T)   units: (row tile, expert, K block)
//
// Each phase's K blocks form one sequence that is cut into contiguous ranges of
// about equal length, one per CTA (at tile boundaries where that leaves few CTAs
// idle). A row tile cut between CTAs goes through fp32 partial sums in the
// workspace: each CTA that shares the tile waits for the others' partials and adds
// up its own part of the token columns, always in CTA order, so no bit depends on
// timing and the additions are spread over the SMs. In phase 1 every CTA takes its
// cut tiles first, so that this runs while the weights of its whole tiles stream (64
// MXFP8 tokens 246 us against 257 with the exchange at the phase's end, 125 BF16
// tokens 462 against 476; sizes as below).
// h is rounded once, to BF16 (MXFP8 layers: to MXFP8), because it is the operand of
// the second product on the tensor cores, as in the layer's stages. Phase 2
// multiplies each expert's accumulator by the routing weight in fp32 and adds it up
// in registers; nothing between h and the output is rounded.
//
// Both kernels, H = 7168, I = 2048, E = 32, k = 8 (share of the time that the active
// experts' weights need at the copy rate; the layer's stages take 191, 518, 526, 531
// and, MXFP8, 135, 312, 315 us):
//   BF16    1 token 120 us (87%), 16 tokens 419 (98%), 64 434, 125 462 (90%)
//   MXFP8   1 token 75 us, 64 tokens 246 (87%), 65 292, 128 306 (70%)
// What is missing: the launches, the router and the first weights' way in (7 us with
// one token, 12 with 125), the way from the last gate/up tile to the first down one
// (4 to 10) and the partial sums at the end (6 to 15). From 65 MXFP8 tokens on, the
// 128-column form: its ring has four stages, its one accumulator lets no MMA run
// while it is read, and its sums spill (the products alone would take about a
// third of the time). Middle layers pay the fixed part in full (H = 2048, I = 1024,
// E = 16, k = 4: 32 BF16 tokens 52 us, the bytes need 30).
//
// CTA layout (one per SM, cooperative launch: phase 2 waits for other CTAs'
// phase 1 through per-expert counters):
//   warp 0      TMA of the weight boxes (and their block scales)
//   warp 1      allocates tensor memory, issues tcgen05.mma
//   warp 2      TMA of the token boxes; in phase 2 it first waits for the
//               expert's h, while warp 0 is already a ring of weights ahead
//   warps 3-10  epilogue: two warps per TMEM lane quadrant, half the token
//               columns each
// Every wait is bounded (StatusBlock); nothing traps.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "gemm.cuh"
#include "moves.cuh"
#include "quant.cuh"

namespace mok {

namespace {

// ---------------------------------------------------------------------------
// Kernel 1: router logits in the fixed order of the routing kernels (32 fma
// chains, chain c over h = 256 i + 8 c + m, then adds at distance 16, 8, 4, 2,
// 1, then the bias), the top-k with its weights, the MXFP8 rows of x, and the
// zeroed counters of kernel 2.
//
// A cluster of CL (8 or 16) CTAs takes 8 tokens x 32 experts. CTA r holds the
// chains r, r + CL, ..., so the tree's first levels stay inside it and one value
// per (token, expert) goes to the first CTA. A warp runs one chain for some of the
// tokens, one expert a lane. The work is about 100 KB of W_r per CTA (CL = 8): what
// counts is to have the loads in flight early, so W_r and x stream through a ring
// of cp.async stages that holds H <= 8192 whole. The products are packed fp32 pairs
// of two tokens (a pair's halves are separate chains). With more than 32 experts the
// clusters of a token group count themselves in, and the last one takes the top-k
// from the logits of all.
//
// H = 7168, E = 32, k = 8, from the kernel's start: one token 4.0 us, 64 tokens 7.2,
// 125 tokens 8.4, of which the loads' way in takes 1 to 2, the products 1.3 to 4.8
// (latency of shared memory and of the chains, two warps to a scheduler), the cluster
// and the top-k 1.5.
// ---------------------------------------------------------------------------
constexpr int kLgThreads = 256;
// Clusters up to which 16 CTAs are taken (H = 7168, 32 experts, the whole layer with
// I = 128: 24.4 us against 25.4 with one token, 51.1 against 52.0 with 16; 69.4 against
// 68.2 with 64 tokens, whose 8 wide clusters do not all fit at once).
constexpr int kLgWideClusters = 4;
constexpr int kLgTokens = 8;       // tokens per cluster
constexpr int kLgRows = 128;       // rows of W_r per stage and CTA
constexpr int kLgWBytes = kLgRows * 32 * 4;
constexpr int kLgXBytes = kLgTokens * kLgRows * 2;
constexpr int kLgStageBytes = kLgWBytes + kLgXBytes;
// after the ring: this CTA's chain sums, the CTAs' sums (written by all of them in
// the first one), the logits
__host__ __device__ constexpr int lg_part_bytes(int cl) { return 32 / cl * kLgTokens * 32 * 4; }
__host__ __device__ constexpr int lg_red_bytes(int cl) { return cl * kLgTokens * 32 * 4; }
__host__ __device__ constexpr int lg_smem_bytes(int cl, int stages) {
    return stages * kLgStageBytes + lg_part_bytes(cl) + lg_red_bytes(cl) + kLgTokens * kMaxE * 4;
}

struct FewLogitsParams {
    const __nv_bfloat16* x;
    const float* W_r;
    const float* bias;
    int T, H, E, k;
    int32_t* idx;         // [T, k]
    float* w;             // [T, k]
    int32_t* topk_idx;    // the caller's copies, or NULL
    float* topk_w;
    float* logits;        // [T, E] and
    int* arrived;         // [token groups] zeroed counts: E > 32 only
    uint8_t* xq;          // MXFP8: [T, H] E4M3, else NULL
    uint8_t* xsf;         // chunk order, one 512-byte chunk per 128 columns
    int* zero;            // status block and counters of kernel 2
    int zero_words;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    const int n = valid ? 16 : 0;   // 0: the destination is filled with zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool valid) {
    const int n = valid ? 4 : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Top-k of one token by one warp (larger logit first, lower expert on ties,
// -0 = +0): experts lane, lane + 32, ... (NQ of them, E <= 32 NQ); keys order like the
// logits, 0 is "taken". The weights are the softmax over the selected logits. `sel`
// holds the selected experts meanwhile (256 bytes of this warp's).
template <int NQ>
__device__ __forceinline__ void few_topk(const float* lg, uint8_t* sel, const FewLogitsParams& p, int64_t t) {
    const int lane = threadIdx.x & 31;
    uint32_t key[NQ];
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
        key[q] = 0;
        if (lane + 32 * q < p.E) {
            const uint32_t b = __float_as_uint(lg[lane + 32 * q] + 0.0f);
            key[q] = max(b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u), 1u);
        }
    }
    float l0 = 0.f, den = 0.f;
    for (int j = 0; j < p.k; ++j) {
        uint32_t best = key[0];
        int be = lane;
#pragma unroll
        for (int q = 1; q < NQ; ++q)
            if (key[q] > best) {
                best = key[q];
                be = lane + 32 * q;
            }
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        int e;
        if constexpr (NQ == 1) e = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
        else e = (int)__reduce_min_sync(0xffffffffu, best == top ? (unsigned)be : 0xffffu);
#pragma unroll
        for (int q = 0; q < NQ; ++q)
            if (e == lane + 32 * q) key[q] = 0;
        const float l = __uint_as_float(top ^ ((top >> 31) ? 0x80000000u : 0xffffffffu));
        if (j == 0) l0 = l;
        den += expf(l - l0);   // j ascending; identical in every lane
        if (lane == 0) sel[j] = (uint8_t)e;
    }
    __syncwarp();
    for (int j = lane; j < p.k; j += 32) {
        const int e = sel[j];
        const float w = expf(lg[e] - l0) / den;
        p.idx[t * p.k + j] = e;
        p.w[t * p.k + j] = w;
        if (p.topk_idx) p.topk_idx[t * p.k + j] = e;
        if (p.topk_w) p.topk_w[t * p.k + j] = w;
    }
}

// Grid: (CL * ceil(E / 32), token groups), clusters of CL along x.
template <int CL, int STAGES>
__global__ void __launch_bounds__(kLgThreads)
few_logits_kernel(const FewLogitsParams p) {
    constexpr int NCH = 32 / CL;               // chains of a CTA; also tokens of a warp
    constexpr int kChunkRows = 8 * NCH;        // rows of W_r per 256-wide chunk of h
    constexpr int kChunks = kLgRows / kChunkRows;
    extern __shared__ __align__(128) unsigned char lg_smem[];
    __shared__ int s_last;
    float* part = reinterpret_cast<float*>(lg_smem + STAGES * kLgStageBytes);   // [chain][token][expert]
    float* red = part + lg_part_bytes(CL) / 4;                                  // [CTA][token][expert]
    float* lg = red + lg_red_bytes(CL) / 4;                                     // [token][kMaxE]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)tc::cluster_ctarank();
    const int e0 = ((int)blockIdx.x / CL) * 32, t0 = (int)blockIdx.y * kLgTokens;
    const int ntok = min(kLgTokens, p.T - t0);
    const int nchunks = ceil_div(p.H, 256);
    const int total = ceil_div(nchunks, kChunks);        // stages
    const int cl = warp % NCH, tw = NCH * (warp / NCH);  // this warp's chain and first token
    const bool vec = (p.E & 3) == 0 && (reinterpret_cast<uintptr_t>(p.W_r) & 15) == 0;

    // every CTA of the cluster runs before any writes to the first one's shared
    // memory: arrive here, wait below
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    pdl_wait();
    pdl_allow_next();

    // row r of a chunk's share: chain rank + CL (r / 8), h = 256 i + 8 chain + r % 8
    auto h_of = [&](int i, int r) { return 256 * i + 8 * (rank + CL * (r >> 3)) + (r & 7); };
    // this thread's copies of a stage: of W_r the vector v0 of rows r0, r0 + 32, ...
    // (whole chunks apart), of x 8 h of one token
    constexpr int kRowStep = kLgThreads / 8, kChunkStep = kRowStep / kChunkRows;
    static_assert(kRowStep % kChunkRows == 0, "whole chunks apart");
    const int r0 = tid >> 3, v0 = tid & 7;
    const int hw = h_of(r0 / kChunkRows, r0 % kChunkRows);
    const bool e_in = e0 + 4 * v0 < p.E;
    const float* wp = p.W_r + (int64_t)hw * p.E + e0 + 4 * v0;
    const int xi = tid / (kLgTokens * NCH), xt = (tid / NCH) % kLgTokens;   // [chunk][token][chain][8 h]
    const int hx = h_of(xi, 8 * (tid % NCH));
    const __nv_bfloat16* xp = p.x + (int64_t)(t0 + xt) * p.H + hx;
    auto issue = [&](int n) {
        if (n < total) {
            const int c0 = n * kChunks;
            const uint32_t ws = tc::smem_u32(lg_smem + (n % STAGES) * kLgStageBytes), xs = ws + kLgWBytes;
            if (vec) {
#pragma unroll
                for (int q = 0; q < kLgRows / kRowStep; ++q) {
                    const int h = 256 * (c0 + q * kChunkStep);   // from this thread's first
                    const bool in = hw + h < p.H && e_in;
                    cp_async16(ws + (r0 + q * kRowStep) * 128 + v0 * 16, in ? wp + (int64_t)h * p.E : p.W_r, in);
                }
            } else {
                for (int j = tid; j < kLgRows * 32; j += kLgThreads) {
                    const int r = j >> 5, v = j & 31;
                    const int h = h_of(c0 + r / kChunkRows, r % kChunkRows), e = e0 + v;
                    const bool in = h < p.H && e < p.E;
                    cp_async4(ws + (r * 32 + v) * 4, in ? p.W_r + (int64_t)h * p.E + e : p.W_r, in);
                }
            }
            if (tid < kLgRows) {
                const bool in = hx + 256 * c0 < p.H && xt < ntok;
                cp_async16(xs + tid * 16, in ? xp + 256 * c0 : p.x, in);
            }
        }
        cp_async_commit();   // one group per stage, empty past the end
    };
    for (int n = 0; n < STAGES - 1; ++n) issue(n);

    // while the first copies are in flight: the counters of kernel 2, and x in
    // 8 bits (one block of 32 a thread; the bytes of mok_quantize_rows)
    if (e0 == 0) {
        const int part_of = (int)blockIdx.y * CL + rank;
        for (int i = part_of * kLgThreads + tid; i < p.zero_words; i += (int)gridDim.y * CL * kLgThreads)
            p.zero[i] = 0;
    }
    if (p.xq && e0 == 0) {
        const int nb = p.H / 32;
        for (int j = rank * kLgThreads + tid; j < ntok * nb; j += CL * kLgThreads) {
            const int t = t0 + j / nb, b = j % nb;
            uint4 o0, o1;
            const uint32_t code = quantize_block32(p.x + (int64_t)t * p.H + b * 32, o0, o1);
            uint4* dst = reinterpret_cast<uint4*>(p.xq + (int64_t)t * p.H + b * 32);
            dst[0] = o0;
            dst[1] = o1;
            p.xsf[(b >> 2) * 512 + sf_chunk_offset(t, b & 3)] = (uint8_t)code;
        }
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");

    float2 acc2[NCH / 2] = {};
    for (int n = 0; n < total; ++n) {
        cp_async_wait<STAGES - 2>();
        __syncthreads();              // stage n has landed for every thread; stage n - 1 is consumed
        issue(n + STAGES - 1);
        const float* ws = reinterpret_cast<const float*>(lg_smem + (n % STAGES) * kLgStageBytes);
        const unsigned char* xs = lg_smem + (n % STAGES) * kLgStageBytes + kLgWBytes;
        if (tw < ntok) {
            // without branches, so that the loads of all chunks run ahead: what lies
            // past H or past the last token was filled with zeros and adds nothing
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                float w[8];
#pragma unroll
                for (int m = 0; m < 8; ++m) w[m] = ws[(i * kChunkRows + 8 * cl + m) * 32 + lane];
#pragma unroll
                for (int u = 0; u < NCH; u += 2) {
                    float f0[8], f1[8];
                    unpack8(*reinterpret_cast<const uint4*>(xs + ((i * kLgTokens + tw + u) * NCH + cl) * 16), f0);
                    unpack8(*reinterpret_cast<const uint4*>(xs + ((i * kLgTokens + tw + u + 1) * NCH + cl) * 16), f1);
#pragma unroll
                    for (int m = 0; m < 8; ++m)
                        acc2[u / 2] = __ffma2_rn(make_float2(f0[m], f1[m]), make_float2(w[m], w[m]), acc2[u / 2]);
                }
            }
        }
    }
    // the tree over the 32 chains: distances 16 (and 8 with four chains a CTA)
    // here, the others over the CTAs, then the bias
    constexpr int P = kLgTokens * 32;
    const int o = warp * 32 + lane;                      // token = warp
#pragma unroll
    for (int u = 0; u < NCH; ++u) part[(cl * kLgTokens + tw + u) * 32 + lane] = (u & 1) ? acc2[u / 2].y : acc2[u / 2].x;
    __syncthreads();
    float v;
    if constexpr (NCH == 4) v = (part[o] + part[2 * P + o]) + (part[P + o] + part[3 * P + o]);
    else v = part[o] + part[P + o];
    static_assert(NCH == 4 || NCH == 2, "chains per CTA");
    const uint32_t dst = tc::mapa_shared(tc::smem_u32(red + rank * P + o), 0);
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst), "f"(v) : "memory");
    tc::cluster_sync();
    if (rank != 0) return;
    float s[CL];
#pragma unroll
    for (int c = 0; c < CL; ++c) s[c] = red[c * P + o];
#pragma unroll
    for (int d = CL / 2; d >= 1; d >>= 1)
#pragma unroll
        for (int c = 0; c < d; ++c) s[c] = s[c] + s[c + d];
    const int e = e0 + lane;
    const float l = e < p.E && p.bias ? s[0] + p.bias[e] : s[0];
    if (gridDim.x == CL) {                               // 32 experts at most: these are all logits
        lg[warp * kMaxE + lane] = l;
        __syncwarp();
    } else {
        if (e < p.E && warp < ntok) p.logits[(int64_t)(t0 + warp) * p.E + e] = l;
        __syncthreads();
        if (tid == 0) {
            __threadfence();
            s_last = atomicAdd(p.arrived + blockIdx.y, 1) == (int)(gridDim.x / CL) - 1;
            __threadfence();
        }
        __syncthreads();
        if (!s_last) return;
        if (warp < ntok)
            for (int i = lane; i < p.E; i += 32) lg[warp * kMaxE + i] = __ldcg(p.logits + (int64_t)(t0 + warp) * p.E + i);
        __syncwarp();
    }
    if (warp >= ntok) return;
    uint8_t* sel = reinterpret_cast<uint8_t*>(part) + warp * kMaxE;   // (the sums in it were read above)
    if (p.E <= 32) few_topk<1>(lg + warp * kMaxE, sel, p, t0 + warp);
    else few_topk<kMaxE / 32>(lg + warp * kMaxE, sel, p, t0 + warp);
}

// ---------------------------------------------------------------------------
// Kernel 2
// ---------------------------------------------------------------------------
constexpr int kFewThreads = 352;
// Units that a part of a tile has at least: a shorter one costs more in shared
// tiles than it saves in streaming (H = 2048, I = 512, 8 MXFP8 experts, 128 tokens: 61
// us at 1, 57 at 2, 45 at 4, 52 at 8; H = 640, I = 1024, 2 tokens: 33.7, 33.6,
// 31.4, 34.9; layers that fill every SM do not change).
constexpr int kFewMinUnits = 4;
constexpr int kFewMaxParts = 1 << 20;   // parts of a phase, where tiles are cut at all
constexpr int kFewEpi = 256;      // epilogue threads
constexpr int kFewEpiBar = 1;     // their named barrier

struct FewParams {
    int T, H, I, E, k, Is;
    int R1, R2, Rs1;              // packed weight rows per tile: gate/up, down, shared gate/up
    const int32_t* idx;           // [T, k] routing of kernel 1
    const float* w;
    const uint8_t* gu_sf;
    const uint8_t* dn_sf;
    const uint8_t* xsf;
    void* h;                      // [active experts * T, I]
    uint8_t* hsf;                 // [active experts][I / 128] chunks of 512 bytes
    __nv_bfloat16* hs;            // [T, Is]
    float* part;                  // [2 phases][CTAs][2][256][T rounded up to 8]
    int* hready;                  // [E + 1] finished items of h per active expert (the shared one last)
    int* cnt1;                    // arrivals per gate/up tile
    int* cnt2;                    // arrivals per down tile
    __nv_bfloat16* out;
    StatusBlock* status;
    unsigned long long timeout_ns;
    int withhold;                 // test hook: CTA 0 counts nothing of its gate/up phase in
};

template <bool MX, int NT>
struct FewCfg {
    static constexpr int kBK = MX ? 128 : 64;              // K elements per block of 128 bytes
    static constexpr int kBytesA = 256 * 128;
    static constexpr int kBytesB = NT * 128;
    static constexpr int kSf = MX ? 3 * 512 : 0;           // two weight chunks, one token chunk
    static constexpr int kStage = kBytesA + kBytesB;
    static constexpr int kFixed = 1024 /* alignment */ + 512 /* barriers */ + kFewMaxPairs * 5 + 256 * 2 + 2 * 128 * 4;
    static constexpr int kLimit = 227 * 1024 - 1024 /* the kernel's static shared memory */;
    static constexpr int kStagesFit = (kLimit - kFixed) / (kStage + kSf);
    static constexpr int kStages = kStagesFit > 6 ? 6 : kStagesFit;
    static constexpr int kSfOffset = kStages * kStage;
    static constexpr int kBarOffset = kSfOffset + kStages * kSf;
    static constexpr int kTabOffset = kBarOffset + 512;
    static constexpr int kSmem = kBarOffset + kFixed;
    // a CTA's time for one unit (few_parts): more tokens leave a shorter ring
    static constexpr float kUnitUs = NT >= 64 ? 0.68f : MX ? 0.58f : NT == 32 ? 0.55f : 0.5f;
    static constexpr float kDrainUs = NT == 128 ? 2.5f : NT == 64 ? 1.3f : NT == 32 ? 0.8f : 0.5f;
    // two accumulators where tensor memory holds them (all but MXFP8 with 128
    // tokens), so that the MMAs of a job run while the one before is read
    static constexpr int kAccs = 4 * NT + (MX ? 12 * kStages : 0) <= 512 ? 2 : 1;
    static constexpr int kAccCols = kAccs * 2 * NT;
    static constexpr int kTmemNeed = kAccCols + (MX ? 12 * kStages : 0);
    static constexpr int kTmemCols = kTmemNeed <= 32 ? 32 : kTmemNeed <= 64 ? 64 : kTmemNeed <= 128 ? 128
                                   : kTmemNeed <= 256 ? 256 : 512;
    static_assert(kStages >= 3 && kSmem <= kLimit && kTmemNeed <= 512, "few-token kernel budget");
};

// The layer's work as two sequences of K blocks (units), and how they are cut:
// each row tile into p parts of about equal length, the parts in order over G
// CTAs (CTA c takes the parts P c / G .. P (c + 1) / G).
struct FewWork {
    int A;                       // active routed experts
    int t1, kb1, ts1, kbs1;      // gate/up: tiles per expert and K blocks per tile, routed and shared
    int t2, kb2, kbs2;           // down: tiles, K blocks per tile and expert, routed and shared
    int p1, ps1, P1, G1;         // gate/up: parts per routed and shared tile, all parts, CTAs
    int p2, P2, G2;              // down
    int b1, e1, b2, e2;          // this CTA's units of the phases
    int wb, we;                  // those of its whole gate/up tiles: the others are cut (at most one at each end)

    __device__ __forceinline__ int upt2() const { return A * kb2 + kbs2; }
    // first unit of part x of a phase (x = all parts: the end)
    __device__ __forceinline__ int unit1(int x) const {
        const int routed = A * t1 * p1;
        if (x < routed) return x / p1 * kb1 + kb1 * (x % p1) / p1;
        const int y = x - routed;
        return A * t1 * kb1 + (ps1 ? y / ps1 * kbs1 + kbs1 * (y % ps1) / ps1 : 0);
    }
    __device__ __forceinline__ int unit2(int x) const { return x / p2 * upt2() + upt2() * (x % p2) / p2; }
    // (at most kFewMaxParts parts and a few hundred CTAs: products fit 32 bits)
    __device__ __forceinline__ int start1(int c) const { return unit1(P1 * c / G1); }
    __device__ __forceinline__ int start2(int c) const { return unit2(P2 * c / G2); }
    // the CTA that takes part x
    __device__ __forceinline__ int owner1(int x) const { return ((x + 1) * G1 - 1) / P1; }
    __device__ __forceinline__ int owner2(int x) const { return ((x + 1) * G2 - 1) / P2; }
};

// Parts per tile for `tiles` tiles (counted in routed tiles of kb units) on M
// CTAs. A phase takes as long as the memory needs for all of its bytes, or as the
// busiest CTA needs for its units if that is longer, and a cut tile costs the
// exchange of its partial sums on top; so tiles stay whole, and SMs idle, wherever
// the remaining ones keep the memory busy. The three times are measured on this
// GPU (H = 7168, I = 2048, BF16, 16 tokens: 512 gate/up tiles, whole on 128 CTAs
// 433 us, in halves on 147 437; MXFP8 with 64 tokens 289 and 281):
//   kUnitsPerUs   32 KB units that the memory delivers
//   unit_us       a CTA's time for a unit with all of its ring in flight
//   drain_us      a CTA's time for reading an accumulator, once for each of the
//                 tile's `segs` experts
//   kShareUs      write, count, wait and add up of a shared tile, and kPartUs for
//                 each of its parts
// Parts have at least kFewMinUnits units. All 32 lanes call it; lane i tries i + 1.
__device__ __forceinline__ int few_parts(int tiles, int kb, int segs, int M, float unit_us, float drain_us) {
    constexpr float kUnitsPerUs = 207.f, kShareUs = 3.5f, kPartUs = 0.25f;
    const int n = (int)(threadIdx.x & 31) + 1;
    float us = 1e9f;
    if (n == 1 || (n * kFewMinUnits <= kb && tiles <= kFewMaxParts / n)) {
        const int q = ceil_div(tiles * n, M);   // parts of the busiest CTA
        us = fmaxf((float)tiles * (float)kb / kUnitsPerUs,
                   fmaxf((float)(q * ceil_div(kb, n)) * unit_us, (float)(q * ceil_div(segs, n)) * drain_us));
        if (n > 1) us += kShareUs + kPartUs * (float)n;
    }
    // the least time, the fewest parts among (nearly) equal ones
    const uint32_t key = (__float_as_uint(us) & ~31u) | (uint32_t)(n - 1);
    return (int)(__reduce_min_sync(0xffffffffu, key) & 31u) + 1;
}

struct FewJob {
    int phase;       // 0 gate/up, 1 down
    int a;           // active expert (A: the shared one)
    int tile;        // gate/up: row tile of the expert; down: row tile
    int gtile;       // index of the tile's arrival counter
    int kb, n;       // K blocks kb .. kb + n - 1
    int u0;          // first unit of the tile
    int c0, c1;      // the CTAs that share the tile
    bool last;       // this CTA's last job of the tile
};

// A row tile that this CTA shares with others, to be finished at the end of
// the phase.
struct FewShared {
    int a, tile, gtile;
    int c0, c1;      // the CTAs that share it
    int u0;
};

// This CTA's part of the gate/up tile that holds unit u.
__device__ __forceinline__ FewJob few_job_up(const FewWork& w, int u) {
    const int routed = w.A * w.t1 * w.kb1;
    const bool sh = u >= routed;
    const int kbt = sh ? w.kbs1 : w.kb1, p = sh ? w.ps1 : w.p1;
    const int v = sh ? u - routed : u;
    const int g = v / kbt;
    FewJob j;
    j.phase = 0;
    j.last = true;
    j.u0 = u - v % kbt;
    j.kb = max(w.b1 - j.u0, 0);
    j.n = min(w.e1 - j.u0, kbt) - j.kb;
    j.a = sh ? w.A : g / w.t1;
    j.tile = sh ? g : g % w.t1;
    j.gtile = sh ? w.A * w.t1 + g : g;
    const int x = (sh ? w.A * w.t1 * w.p1 : 0) + g * p;
    j.c0 = w.owner1(x);
    j.c1 = w.owner1(x + p - 1);
    return j;
}

// Calls f(job) for this CTA's jobs of a phase in order; false as soon as f
// returns false.
//
// Gate/up: first the tiles that it shares with other CTAs (CUT: at the end and at
// the start of its range), then its whole ones (WHOLE), whose weights stream while
// the partial sums are exchanged.
template <bool CUT, bool WHOLE, typename F>
__device__ __forceinline__ bool few_jobs_up(const FewWork& w, F&& f) {
    int next = w.wb;   // of the whole ones
    for (int step = CUT ? 0 : 2;;) {
        int u;
        if (step == 0) {
            step = 1;
            if (w.we == w.e1) continue;
            u = w.we;
        } else if (step == 1) {
            step = 2;
            if (w.wb == w.b1) continue;
            u = w.b1;
        } else {
            if (!WHOLE || next >= w.we) return true;
            u = next;
        }
        const FewJob j = few_job_up(w, u);
        if (u == next) next += j.n;
        if (!f(j)) return false;
    }
}
template <typename F>
__device__ __forceinline__ bool few_jobs_down(const FewWork& w, F&& f) {
    int u = w.b2;
    const int end = w.e2;
    const int upt = w.upt2();
    FewJob j;
    j.phase = 1;
    while (u < end) {
        j.tile = j.gtile = u / upt;
        j.u0 = j.tile * upt;
        const int r = u - j.u0;
        const bool sh = r >= w.A * w.kb2;
        j.a = sh ? w.A : r / w.kb2;
        j.kb = sh ? r - w.A * w.kb2 : r % w.kb2;
        j.n = min((sh ? w.kbs2 : w.kb2) - j.kb, end - u);
        u += j.n;
        j.last = u == end || u == j.u0 + upt;
        j.c0 = w.owner2(j.tile * w.p2);
        j.c1 = w.owner2((j.tile + 1) * w.p2 - 1);
        if (!f(j)) return false;
    }
    return true;
}
template <typename F>
__device__ __forceinline__ void few_jobs(const FewWork& w, F&& f) {
    if (few_jobs_up<true, true>(w, f)) few_jobs_down(w, f);
}

__device__ __forceinline__ int few_ld_acquire(const int* p) {
    int v;
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void few_red_release(int* p, int v) {
    asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Bounded wait until *p >= target (acquire). False: gave up (recorded).
__device__ bool few_wait_counter(const int* p, int target, StatusBlock* st, uint64_t tmo) {
    if (few_ld_acquire(p) >= target) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (few_ld_acquire(p) >= target) return true;
        if ((it & 31) == 0) {
            if (abort_requested(st)) return false;
            if (globaltimer_ns() - t0 > tmo) {
                record_failure(st, MOK_ERR_TIMEOUT, kSiteCounter);
                return false;
            }
        }
    }
}

// Wait, whatever the abort flag says, until copies or MMAs in flight have
// landed, at most tmo.
__device__ void few_drain(uint32_t bar, uint32_t parity, uint64_t tmo) {
    const uint64_t t0 = globaltimer_ns();
    while (!tc::mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < tmo) {
    }
}

// AND over the epilogue's threads (all of them call it), so that they leave a
// loop together.
__device__ __forceinline__ bool epi_and(bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.red.and.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)pred), "n"(kFewEpiBar), "n"(kFewEpi)
        : "memory");
    __syncwarp();
    return r != 0;
}
__device__ __forceinline__ void epi_sync() {
    __syncwarp();
    asm volatile("bar.sync %0, %1;" ::"n"(kFewEpiBar), "n"(kFewEpi) : "memory");
}

// CH (8 or 16) consecutive 32-bit columns of this warp's 32 lanes.
template <int CH>
__device__ __forceinline__ void few_tmem_ld(uint32_t a, float (&v)[CH]) {
    uint32_t r[CH];
    if constexpr (CH == 8) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(a)
                     : "memory");
    } else {
        static_assert(CH == 16, "columns per load");
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14,"
            " %15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
              "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(a)
            : "memory");
    }
    tc::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < CH; ++i) v[i] = __uint_as_float(r[i]);
}

template <bool MX, int NT>
__global__ void __launch_bounds__(kFewThreads, 1)
few_ffn_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmXq,
               const __grid_constant__ CUtensorMap tmGU, const __grid_constant__ CUtensorMap tmDN,
               const __grid_constant__ CUtensorMap tmH, const __grid_constant__ CUtensorMap tmSGU,
               const __grid_constant__ CUtensorMap tmSDN, const __grid_constant__ CUtensorMap tmHs,
               const FewParams p) {
    using C = FewCfg<MX, NT>;
    constexpr int S = C::kStages;
    extern __shared__ __align__(1024) unsigned char few_smem[];
    __shared__ uint32_t s_tmem;
    __shared__ uint32_t s_hit[kMaxE / 32];
    __shared__ int s_cut[13];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(few_smem) + 1023) & ~uintptr_t(1023));
    const uint32_t base = tc::smem_u32(smem);
    const uint32_t bar = base + C::kBarOffset;
    auto fullA = [&](int s) { return bar + 8u * s; };
    auto fullB = [&](int s) { return bar + 8u * (S + s); };
    auto empty = [&](int s) { return bar + 8u * (2 * S + s); };
    auto accf = [&](int a) { return bar + 8u * (3 * S + a); };
    auto acce = [&](int a) { return bar + 8u * (3 * S + C::kAccs + a); };
    const uint32_t drain = bar + 8u * (3 * S + 2 * C::kAccs);
    auto a_tile = [&](int s) { return base + s * C::kStage; };
    auto b_tile = [&](int s) { return base + s * C::kStage + C::kBytesA; };
    auto sf_tile = [&](int s) { return base + C::kSfOffset + s * C::kSf; };
    float* s_w = reinterpret_cast<float*>(smem + C::kTabOffset);              // [T*k] routing weights
    uint8_t* s_idx = smem + C::kTabOffset + kFewMaxPairs * 4;                 // [T*k] experts
    uint16_t* s_act = reinterpret_cast<uint16_t*>(smem + C::kTabOffset + kFewMaxPairs * 5);   // [A] active experts
    float* s_row = reinterpret_cast<float*>(smem + C::kTabOffset + kFewMaxPairs * 5 + 512);   // [2][128]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    StatusBlock* st = p.status;
    const uint64_t tmo = p.timeout_ns;
    const int T = p.T, E = p.E, k = p.k;

    if (threadIdx.x < kMaxE / 32) s_hit[threadIdx.x] = 0;
    if (threadIdx.x == 0) {
        const CUtensorMap* maps[8] = {&tmGU, MX ? &tmXq : &tmX, &tmDN, &tmH, &tmSGU, &tmX, &tmSDN, &tmHs};
        for (int i = 0; i < (p.Is ? 8 : 4); ++i) tc::prefetch_tmap(maps[i]);
    }
    if (threadIdx.x == 64) {
        for (int s = 0; s < S; ++s) {
            tc::mbar_init(fullA(s), 1);
            tc::mbar_init(fullB(s), 1);
            tc::mbar_init(empty(s), 1);
        }
        for (int a = 0; a < C::kAccs; ++a) {
            tc::mbar_init(accf(a), 1);
            tc::mbar_init(acce(a), kFewEpi);
        }
        tc::mbar_init(drain, 1);
        tc::fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(tc::smem_u32(&s_tmem), C::kTmemCols);
        tc::tmem_relinquish();
    }
    __syncthreads();

    pdl_wait();   // the routing, the MXFP8 rows and the zeroed counters are kernel 1's
    pdl_allow_next();
    {
        // all loads first: kFewMaxPairs are 6 rounds of the CTA at most
        constexpr int R = (kFewMaxPairs + kFewThreads - 1) / kFewThreads;
        int e[R];
        float v[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = threadIdx.x + r * kFewThreads;
            if (i < T * k) {
                e[r] = p.idx[i];
                v[r] = p.w[i];
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = threadIdx.x + r * kFewThreads;
            if (i < T * k) {
                s_idx[i] = (uint8_t)e[r];
                s_w[i] = v[r];
                atomicOr(&s_hit[e[r] >> 5], 1u << (e[r] & 31));
            }
        }
    }
    __syncthreads();
    // the active experts in ascending order (warp 0), and the cut of the two
    // phases (warps 1 and 2; a K block of the MXFP8 experts holds twice the
    // elements of the BF16 shared expert's, so a shared tile counts as kbs1 / kb1
    // routed ones)
    FewWork w;
    w.A = 0;
#pragma unroll
    for (int q = 0; q < kMaxE / 32; ++q) w.A += __popc(s_hit[q]);
    w.t1 = 2 * p.I / p.R1;
    w.kb1 = p.H / C::kBK;
    w.ts1 = p.Is ? 2 * p.Is / p.Rs1 : 0;
    w.kbs1 = p.Is ? p.H / 64 : 0;
    w.t2 = p.H / p.R2;
    w.kb2 = p.I / C::kBK;
    w.kbs2 = p.Is / 64;
    const int M = (int)gridDim.x, me = (int)blockIdx.x;
    if (warp == 0) {
        int n = 0;
        for (int q = 0; 32 * q < E; ++q) {
            const uint32_t m = s_hit[q];
            if ((m >> lane) & 1u) s_act[n + __popc(m & ((1u << lane) - 1))] = (uint16_t)(32 * q + lane);
            n += __popc(m);
        }
    } else if (warp == 1) {
        const int heavy = w.ts1 ? (MX ? 2 : 1) : 0;
        w.p1 = few_parts(w.A * w.t1 + w.ts1 * heavy, w.kb1, 1, M, C::kUnitUs, C::kDrainUs);
        w.ps1 = w.p1 * heavy;
        w.P1 = w.A * w.t1 * w.p1 + w.ts1 * w.ps1;
        w.G1 = ceil_div(w.P1, ceil_div(w.P1, M));
        // lanes 0 and 1: first unit of this CTA and of the next
        const int u = me < w.G1 ? w.start1(min(me + (lane & 1), w.G1)) : 0;
        if (lane < 2) s_cut[4 + lane] = u;
        w.b1 = w.wb = __shfl_sync(0xffffffffu, u, 0);
        w.e1 = w.we = __shfl_sync(0xffffffffu, u, 1);
        if (w.b1 < w.e1) {
            const FewJob t = few_job_up(w, w.e1 - 1);
            if (t.c0 != t.c1) w.we = t.u0 + t.kb;
            if (t.u0 > w.b1) {
                const FewJob h = few_job_up(w, w.b1);
                if (h.c0 != h.c1) w.wb = h.u0 + h.kb + h.n;
            }
        }
        if (lane == 0) {
            s_cut[11] = w.wb;
            s_cut[12] = w.we;
            s_cut[0] = w.p1;
            s_cut[1] = w.ps1;
            s_cut[2] = w.P1;
            s_cut[3] = w.G1;
        }
    } else if (warp == 2) {
        w.p2 = few_parts(w.t2, w.upt2(), w.A + (w.kbs2 > 0), M, C::kUnitUs, C::kDrainUs);
        w.P2 = w.t2 * w.p2;
        w.G2 = ceil_div(w.P2, ceil_div(w.P2, M));
        const int u = me < w.G2 ? w.start2(min(me + (lane & 1), w.G2)) : 0;
        if (lane < 2) s_cut[9 + lane] = u;
        if (lane == 0) {
            s_cut[6] = w.p2;
            s_cut[7] = w.P2;
            s_cut[8] = w.G2;
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem;
    w.p1 = s_cut[0];
    w.ps1 = s_cut[1];
    w.P1 = s_cut[2];
    w.G1 = s_cut[3];
    w.b1 = s_cut[4];
    w.e1 = s_cut[5];
    w.p2 = s_cut[6];
    w.P2 = s_cut[7];
    w.G2 = s_cut[8];
    w.b2 = s_cut[9];
    w.e2 = s_cut[10];
    w.wb = s_cut[11];
    w.we = s_cut[12];

    if (warp == 0) {
        // ------------------------------------------------------------ weights
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            int last_par[S];
            for (int i = 0; i < S; ++i) last_par[i] = -1;
            few_jobs(w, [&](const FewJob& j) {
                const bool sh = j.a == w.A;
                const int e = sh ? 0 : s_act[j.a];
                const int rows = j.phase ? p.R2 : sh ? p.Rs1 : p.R1;
                const int row0 = (j.phase ? e * p.H : e * 2 * p.I) + j.tile * rows;
                const CUtensorMap* tm = j.phase ? (sh ? &tmSDN : &tmDN) : (sh ? &tmSGU : &tmGU);
                const int bk = sh ? 64 : C::kBK;
                for (int i = 0; i < j.n; ++i) {
                    if (!tc::mbar_wait(empty(s), ph ^ 1u, st, tmo, kSiteProducerEmpty)) return false;
                    const int kb = j.kb + i;
                    uint32_t bytes = (uint32_t)rows * 128u;
                    if constexpr (MX) {
                        if (!sh) bytes += 512u * (uint32_t)ceil_div(rows, 128);
                    }
                    tc::mbar_expect_tx(fullA(s), bytes);
                    tc::tma_load_2d(a_tile(s), tm, fullA(s), kb * bk, row0);
                    if constexpr (MX) {
                        if (!sh) {
                            if (rows == 224) {   // scales packed per 224-row tile: two chunks side by side
                                tc::bulk_load(sf_tile(s), p.dn_sf + ((int64_t)(row0 / 224) * (p.I / 128) + kb) * 1024, 1024,
                                              fullA(s));
                            } else {
                                const uint8_t* sf = j.phase ? p.dn_sf : p.gu_sf;
                                const int nkc = (j.phase ? p.I : p.H) / 128;
                                for (int b = 0; b < rows / 128; ++b)
                                    tc::bulk_load(sf_tile(s) + 512 * b, sf + ((int64_t)(row0 / 128 + b) * nkc + kb) * 512, 512,
                                                  fullA(s));
                            }
                        }
                    }
                    last_par[s] = (int)ph;
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
                return true;
            });
            // the CTA may end early because of another warp or CTA, but not before
            // its copies have landed
            for (int q = 0; q < S; ++q)
                if (last_par[q] >= 0) few_drain(fullA(q), (uint32_t)last_par[q], tmo);
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ tokens
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            int last_par[S];
            for (int i = 0; i < S; ++i) last_par[i] = -1;
            int ready = -1;   // the expert whose h is known to be complete
            few_jobs(w, [&](const FewJob& j) {
                const bool sh = j.a == w.A;
                if (j.phase && ready != j.a) {
                    // (items of 32 rows, or MXFP8 features, and 8 tokens)
                    const int items = (sh ? 2 * p.Is : MX ? p.I : 2 * p.I) / 32 * ceil_div(T, 8);
                    if (!few_wait_counter(p.hready + j.a, items, st, tmo)) return false;
                    tc::fence_proxy_async_global();
                    ready = j.a;
                }
                const CUtensorMap* tm = j.phase ? (sh ? &tmHs : &tmH) : (MX && !sh ? &tmXq : &tmX);
                const int row0 = j.phase && !sh ? j.a * T : 0;
                const int bk = sh ? 64 : C::kBK;
                for (int i = 0; i < j.n; ++i) {
                    if (!tc::mbar_wait(empty(s), ph ^ 1u, st, tmo, kSiteProducerEmpty)) return false;
                    const int kb = j.kb + i;
                    tc::mbar_expect_tx(fullB(s), (uint32_t)C::kBytesB + (MX && !sh ? 512u : 0u));
                    tc::tma_load_2d(b_tile(s), tm, fullB(s), kb * bk, row0);
                    if constexpr (MX) {
                        if (!sh)
                            tc::bulk_load(sf_tile(s) + 1024,
                                          j.phase ? p.hsf + ((int64_t)j.a * (p.I / 128) + kb) * 512 : p.xsf + (int64_t)kb * 512,
                                          512, fullB(s));
                    }
                    last_par[s] = (int)ph;
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
                return true;
            });
            for (int q = 0; q < S; ++q)
                if (last_par[q] >= 0) few_drain(fullB(q), (uint32_t)last_par[q], tmo);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0, acc_ph = 0;
            int ac = 0;   // accumulator of this job
            bool issued = false;
            few_jobs(w, [&](const FewJob& j) {
                const bool sh = j.a == w.A;
                const int rows = j.phase ? p.R2 : sh ? p.Rs1 : p.R1;
                const bool two = rows > 128;   // two 128-row blocks
                if (!tc::mbar_wait(acce(ac), acc_ph ^ 1u, st, tmo, kSiteMmaAccEmpty)) return false;
                tc::fence_after_sync();
                const uint32_t d0 = tmem + (uint32_t)(ac * 2 * NT), d1 = d0 + NT;
                for (int i = 0; i < j.n; ++i) {
                    if (!tc::mbar_wait(fullA(s), ph, st, tmo, kSiteMmaFull)) return false;
                    if (!tc::mbar_wait(fullB(s), ph, st, tmo, kSiteMmaFull)) return false;
                    tc::fence_after_sync();
                    // descriptors of the stage; K step kk starts 32 bytes (2
                    // descriptor units) further, row block b 16 KB
                    const uint64_t ad = tc::make_sdesc(a_tile(s), 16, 1024, tc::kLayoutSW128);
                    const uint64_t bd = tc::make_sdesc(b_tile(s), 16, 1024, tc::kLayoutSW128);
                    const uint32_t on = i > 0 ? 1u : 0u;
                    if (MX && !sh) {
                        const uint32_t sf = tmem + (uint32_t)(C::kAccCols + 12 * s);
                        const uint64_t sd = tc::make_sdesc(sf_tile(s), 0, 128, tc::kLayoutNone);
                        tc::tmem_cp_32x128b_warpx4(sf, sd);
                        if (two) tc::tmem_cp_32x128b_warpx4(sf + 4, sd + 32);
                        tc::tmem_cp_32x128b_warpx4(sf + 8, sd + 64);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            tc::mma_mxf8(d0, ad + 2 * kk, bd + 2 * kk, tc::idesc_mxf8(128, NT, kk, kk), sf, sf + 8,
                                         kk ? 1u : on);
                            if (two)
                                tc::mma_mxf8(d1, ad + 1024 + 2 * kk, bd + 2 * kk, tc::idesc_mxf8(128, NT, kk, kk),
                                             sf + 4, sf + 8, kk ? 1u : on);
                        }
                    } else {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            tc::mma_bf16(d0, ad + 2 * kk, bd + 2 * kk, tc::idesc_bf16(128, NT, false, false), kk ? 1u : on);
                            if (two)
                                tc::mma_bf16(d1, ad + 1024 + 2 * kk, bd + 2 * kk, tc::idesc_bf16(128, NT, false, false),
                                             kk ? 1u : on);
                        }
                    }
                    issued = true;
                    tc::mma_commit(empty(s));
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
                tc::mma_commit(accf(ac));
                if (++ac == C::kAccs) { ac = 0; acc_ph ^= 1u; }
                return true;
            });
            if (issued) {   // the MMAs issued so far end before tensor memory is freed
                tc::mma_commit(drain);
                few_drain(drain, 0, tmo);
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        constexpr int NC = NT / 2;                  // token columns of a thread
        constexpr int CH = 8;                       // columns at a time
        const int q = warp & 3;                     // TMEM lane quadrant of this warp
        const int half = (warp - 3) >> 2;
        const int et = threadIdx.x - 96;            // 0 .. 255
        const int row = 32 * q + lane;              // row in each 128-row block
        const int col0 = half * NC;                 // first token column of this thread
        const uint32_t tq0 = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)col0;
        int ac = 0;   // accumulator of this job
        const int c_me = (int)blockIdx.x;
        uint32_t ph = 0;
        int wbuf = 0;

        // this CTA's shared tiles of a phase, at most two: the ones that its range
        // starts and ends in
        FewShared pend[2];
        int n_pend = 0;
        const int tpad = ceil_div(T, 8) * 8;
        // a partial tile: blocks of 32 rows x 8 tokens (1 KB each, a row's 8 tokens
        // adjacent), by row group and token chunk
        const int64_t part_stride = 256 * (int64_t)tpad;
        auto block = [&](int g, int t0) { return ((g * (tpad / 8) + t0 / 8) * 32 + lane) * 8; };
        auto slots = [&](int phase) { return p.part + (int64_t)phase * gridDim.x * 2 * part_stride; };
        // CTA c's partial of a tile whose first unit is u0: only the first
        // sharer may have started before the tile
        auto slot_of = [&](int phase, int c, bool began_before) {
            return slots(phase) + (2 * (int64_t)c + (began_before ? 1 : 0)) * part_stride;
        };

        // MXFP8 h of one token and 32 features (group g of the tile's 128, one a
        // lane) from their gate and up values
        auto store_h_mx = [&](int a, int tile, int g, int t, float gate, float up) {
            const float hv = silu_f(gate) * up;
            const uint32_t am = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(hv)));
            const uint32_t code = e8m0_code(__uint_as_float(am));
            const int64_t r = (int64_t)a * T + t;
            static_cast<uint8_t*>(p.h)[r * p.I + tile * 128 + 32 * g + lane] =
                (uint8_t)f32x2_to_e4m3x2(hv * e8m0_inv_scale(code), 0.f);
            if (lane == 0) p.hsf[((int64_t)a * (p.I / 128) + tile) * 512 + sf_chunk_offset(t, g)] = (uint8_t)code;
        };
        // SwiGLU of one token column: v0, v1 are this thread's values in the
        // tile's two row blocks (all lanes of the warp call it)
        auto store_h = [&](int a, int tile, int t, float v0, float v1) {
            const bool sh = a == w.A;
            if (MX && !sh) {
                // gate rows 0..127, up rows 128..255 of the same features
                store_h_mx(a, tile, q, t, v0, v1);
            } else {
                // lanes 0-15 hold gate rows, 16-31 the up rows of the same 16
                // features: the lower half forms h of the first row block, the
                // upper half that of the second
                const int rows = sh ? p.Rs1 : p.R1, ld = sh ? p.Is : p.I;
                const bool lower = lane < 16;
                const float other = __shfl_xor_sync(0xffffffffu, lower ? v1 : v0, 16);
                const float hv = silu_f(lower ? v0 : other) * (lower ? other : v1);
                if (lower || rows > 128) {
                    __nv_bfloat16* hb = sh ? p.hs : static_cast<__nv_bfloat16*>(p.h) + (int64_t)a * T * p.I;
                    const int f = tile * (rows / 2) + (lower ? 0 : 64) + 16 * q + (lane & 15);
                    hb[(int64_t)t * ld + f] = __float2bfloat16_rn(hv);
                }
            }
        };
        auto store_out = [&](int tile, int t, float v0, float v1) {
            __nv_bfloat16* o = p.out + (int64_t)t * p.H + tile * p.R2;
            o[row] = __float2bfloat16_rn(v0);
            if (128 + row < p.R2) o[128 + row] = __float2bfloat16_rn(v1);
        };
        // 8 tokens (from column cc of this thread) of a partial tile: one 32-byte
        // store for each of this thread's rows
        auto put_part = [&](float* mine, int cc, bool two, const float (&v0)[CH], const float (&v1)[CH]) {
            uint32_t u[8];
            float* dst = mine + block(q, col0 + cc);
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(v0[i]);
            tc::stg_v8(dst, u);
            if (two) {
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(v1[i]);
                tc::stg_v8(dst + 128 * tpad, u);
            }
        };
        // A tile is finished in items of one warp: 8 tokens x 32 weight rows (MXFP8
        // gate/up: 32 features, i.e. 32 gate and 32 up rows).
        auto groups_of = [&](int phase, bool sh) {
            return phase ? p.R2 / 32 : sh ? p.Rs1 / 32 : MX ? 4 : p.R1 / 32;
        };
        // n items of an expert's h are written (their readers are TMA loads):
        // publish them. The barrier and the release order every thread's writes
        // before the count.
        auto publish_h = [&](int a, int n) {
            tc::fence_proxy_async_global();
            epi_sync();
            if (et == 0 && !(p.withhold && c_me == 0)) few_red_release(p.hready + a, n);
        };
        // this CTA's partial of a shared tile is written: count it in and
        // remember the tile
        auto share = [&](const FewJob& j) {
            epi_sync();
            if (et == 0 && !(p.withhold && c_me == 0 && !j.phase))
                few_red_release((j.phase ? p.cnt2 : p.cnt1) + j.gtile, 1);
            const FewShared f{j.a, j.tile, j.gtile, j.c0, j.c1, j.u0};
            if (n_pend == 0) pend[0] = f;
            else pend[1] = f;
            ++n_pend;
        };
        // after the cut tiles of a phase: of each, sharer i of n adds up the partials of
        // its share of the items, in CTA order
        auto finish = [&](int phase) {
#pragma unroll 1
            for (int i = 0; i < n_pend; ++i) {
                const FewShared f = i == 0 ? pend[0] : pend[1];
                const bool sh = f.a == w.A;
                const int n = f.c1 - f.c0 + 1, me_ = c_me - f.c0;
                const int groups = groups_of(phase, sh), items = groups * (tpad / 8);
                const int from = items * me_ / n, to = items * (me_ + 1) / n;
                if (from == to) continue;
                bool ok = true;
                if (et == 0) ok = few_wait_counter((phase ? p.cnt2 : p.cnt1) + f.gtile, n, st, tmo);
                if (!epi_and(ok)) return false;
                const bool pairs = MX && !phase && !sh;   // gate and up rows 128 apart
                const int lead = (phase ? w.start2(f.c0) : w.start1(f.c0)) < f.u0 ? 1 : 0;
                const float* src = slots(phase) + 2 * (int64_t)f.c0 * part_stride;
                constexpr int kWarps = kFewEpi / 32;
                // NI items of a warp at a time (the second one clamped to the last
                // item, so that the loads need no branch)
                auto run = [&](auto tag) {
                    constexpr int NI = decltype(tag)::value;
#pragma unroll 1
                    for (int it0 = from + (et >> 5); it0 < to; it0 += NI * kWarps) {
                        float v[NI][8] = {}, up[NI][8] = {};
                        const float* at[NI];
#pragma unroll
                        for (int u = 0; u < NI; ++u) {
                            const int it = min(it0 + u * kWarps, to - 1);
                            at[u] = src + block(it % groups, it / groups * 8);
                        }
                        auto add = [&](float (&x)[8], const float* q) {
                            const float4 lo = __ldcg(reinterpret_cast<const float4*>(q));
                            const float4 hi = __ldcg(reinterpret_cast<const float4*>(q) + 1);
                            x[0] += lo.x; x[1] += lo.y; x[2] += lo.z; x[3] += lo.w;
                            x[4] += hi.x; x[5] += hi.y; x[6] += hi.z; x[7] += hi.w;
                        };
#pragma unroll 4
                        for (int c = 0; c < n; ++c) {
                            const int64_t o = (2 * (int64_t)c + (c == 0 ? lead : 0)) * part_stride;
#pragma unroll
                            for (int u = 0; u < NI; ++u) {
                                add(v[u], at[u] + o);
                                if (pairs) add(up[u], at[u] + o + 128 * tpad);
                            }
                        }
#pragma unroll
                        for (int u = 0; u < NI; ++u) {
                            const int it = it0 + u * kWarps;
                            if (it >= to) break;
                            const int g = it % groups, t0 = it / groups * 8;
                            if (phase) {
                                __nv_bfloat16* o = p.out + (int64_t)t0 * p.H + f.tile * p.R2 + 32 * g + lane;
#pragma unroll
                                for (int t = 0; t < 8; ++t)
                                    if (t0 + t < T) o[(int64_t)t * p.H] = __float2bfloat16_rn(v[u][t]);
                            } else if (pairs) {
#pragma unroll
                                for (int t = 0; t < 8; ++t)
                                    if (t0 + t < T) store_h_mx(f.a, f.tile, g, t0 + t, v[u][t], up[u][t]);
                            } else {
                                // lanes 0-15 gate, 16-31 up of the same 16 features: the
                                // lower half forms the first four tokens, the upper half
                                // the others
                                const bool lower = lane < 16;
                                const int ld = sh ? p.Is : p.I, fe = f.tile * (groups * 16) + 16 * g + (lane & 15);
                                __nv_bfloat16* hb = sh ? p.hs : static_cast<__nv_bfloat16*>(p.h) + (int64_t)f.a * T * p.I;
#pragma unroll
                                for (int t = 0; t < 4; ++t) {
                                    const float other = __shfl_xor_sync(0xffffffffu, lower ? v[u][4 + t] : v[u][t], 16);
                                    const float hv = silu_f(lower ? v[u][t] : other) * (lower ? other : v[u][4 + t]);
                                    const int tt = t0 + t + (lower ? 0 : 4);
                                    if (tt < T) hb[(int64_t)tt * ld + fe] = __float2bfloat16_rn(hv);
                                }
                            }
                        }
                    }
                };
                if (NT >= 64 && to - from > kWarps) run(std::integral_constant<int, 2>{});
                else run(std::integral_constant<int, 1>{});
                if (!phase) publish_h(f.a, to - from);
            }
            n_pend = 0;
            return true;
        };

        // gate/up: the accumulator of each job, cut tiles first
        auto up = [&](const FewJob& j, auto tag) {
            constexpr bool whole = decltype(tag)::value;
            const bool two = (j.a == w.A ? p.Rs1 : p.R1) > 128;
            float* mine = slot_of(0, c_me, w.b1 < j.u0);
            if (!epi_and(tc::mbar_wait(accf(ac), ph, st, tmo, kSiteEpiAccFull))) return false;
            tc::fence_after_sync();
            const uint32_t tq = tq0 + (uint32_t)(ac * 2 * NT);
#pragma unroll 1
            for (int cc = 0; cc < NC && col0 + cc < T; cc += CH) {
                float v0[CH], v1[CH];
                few_tmem_ld<CH>(tq + cc, v0);
                few_tmem_ld<CH>(tq + NT + cc, v1);
                if constexpr (whole) {
#pragma unroll
                    for (int i = 0; i < CH; ++i)
                        if (col0 + cc + i < T) store_h(j.a, j.tile, col0 + cc + i, v0[i], v1[i]);
                } else {
                    put_part(mine, cc, two, v0, v1);
                }
            }
            tc::fence_before_sync();
            tc::mbar_arrive(acce(ac));
            if (++ac == C::kAccs) { ac = 0; ph ^= 1u; }
            if constexpr (whole) publish_h(j.a, groups_of(0, j.a == w.A) * (tpad / 8));
            else share(j);
            return true;
        };
        bool ok = few_jobs_up<true, false>(w, [&](const FewJob& j) { return up(j, std::false_type{}); });
        ok = ok && finish(0);
        ok = ok && few_jobs_up<false, true>(w, [&](const FewJob& j) { return up(j, std::true_type{}); });
        float acc[2][NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) acc[0][i] = acc[1][i] = 0.f;
        ok = ok && few_jobs_down(w, [&](const FewJob& j) {
            if (et < T) {
                // this expert's routing weights per token; -1: not selected
                float wt = -1.f;
                if (j.a == w.A) wt = 1.f;
                else
                    for (int i = 0; i < k; ++i)
                        if (s_idx[et * k + i] == s_act[j.a]) wt = s_w[et * k + i];
                s_row[wbuf * 128 + et] = wt;
            }
            if (!epi_and(tc::mbar_wait(accf(ac), ph, st, tmo, kSiteEpiAccFull))) return false;
            tc::fence_after_sync();
            const uint32_t tq = tq0 + (uint32_t)(ac * 2 * NT);
            const float* wr = s_row + wbuf * 128 + col0;
            wbuf ^= 1;
#pragma unroll
            for (int cc = 0; cc < NC; cc += CH) {
                if (col0 + cc < T) {
                    float v0[CH], v1[CH];
                    few_tmem_ld<CH>(tq + cc, v0);
                    few_tmem_ld<CH>(tq + NT + cc, v1);
#pragma unroll
                    for (int i = 0; i < CH; ++i) {
                        const float wt = col0 + cc + i < T ? wr[cc + i] : -1.f;
                        if (!(wt < 0.f)) {   // (a NaN weight, from a row without numbers, goes through)
                            acc[0][cc + i] = fmaf(wt, v0[i], acc[0][cc + i]);
                            acc[1][cc + i] = fmaf(wt, v1[i], acc[1][cc + i]);
                        }
                    }
                }
            }
            tc::fence_before_sync();
            tc::mbar_arrive(acce(ac));
            if (++ac == C::kAccs) { ac = 0; ph ^= 1u; }
            if (j.last) {
                const bool whole = j.c0 == j.c1;
                const bool two = p.R2 > 128;
                float* mine = slot_of(1, c_me, w.b2 < j.u0);
#pragma unroll
                for (int cc = 0; cc < NC; cc += CH) {
                    float v0[CH], v1[CH];
#pragma unroll
                    for (int i = 0; i < CH; ++i) {
                        v0[i] = acc[0][cc + i];
                        v1[i] = acc[1][cc + i];
                        acc[0][cc + i] = acc[1][cc + i] = 0.f;
                    }
                    if (col0 + cc < T) {
                        if (whole) {
#pragma unroll
                            for (int i = 0; i < CH; ++i)
                                if (col0 + cc + i < T) store_out(j.tile, col0 + cc + i, v0[i], v1[i]);
                        } else {
                            put_part(mine, cc, two, v0, v1);
                        }
                    }
                }
                if (!whole) share(j);
            }
            return true;
        });
        if (ok) finish(1);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 1) tc::tmem_dealloc(tmem, C::kTmemCols);
}

int few_columns(int T) { return T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128; }

struct FewLayout {
    size_t counters, arrived, logits, idx, w, xq, xsf, h, hsf, hs, part, total;
    int n_counters, n1;   // ints: E + 1 ready counts, n1 gate/up tiles, down tiles
};

int gu_rows(int I) { return std::min(256, 2 * I); }

FewLayout few_layout(const mok_problem* p, int ctas) {
    FewLayout L{};
    const bool mx = p->dtype == MOK_MXFP8;
    const int64_t T = p->T, H = p->H, I = p->I;
    const int64_t act = std::min<int64_t>(p->E, T * p->k);
    const int r2 = down_tile_n(p->H, mx);
    L.n1 = (int)(act * (2 * I / gu_rows(p->I))) + (p->I_shared ? 2 * p->I_shared / gu_rows(p->I_shared) : 0);
    L.n_counters = p->E + 1 + L.n1 + (int)(H / r2);
    size_t o = kStatusBytes;
    L.counters = o; o += align_up((int64_t)L.n_counters * 4, 256);
    L.arrived = o; if (p->E > 32) o += align_up(ceil_div(p->T, kLgTokens) * 4, 256);
    L.logits = o; if (p->E > 32) o += align_up(T * p->E * 4, 256);
    L.idx = o; o += align_up(T * p->k * 4, 256);
    L.w = o; o += align_up(T * p->k * 4, 256);
    L.xq = o; if (mx) o += align_up(T * H, 256);
    L.xsf = o; if (mx) o += H / 128 * 512;
    L.h = o; o += align_up(act * T * I * (mx ? 1 : 2), 256);
    L.hsf = o; if (mx) o += act * (I / 128) * 512;
    L.hs = o; o += align_up(T * p->I_shared * 2, 256);
    L.part = o; o += (size_t)2 * ctas * 2 * 256 * align_up(T, 8) * 4;
    L.total = o;
    return L;
}

template <int CL, int STAGES>
cudaError_t run_logits(const FewLogitsParams& p, cudaStream_t s) {
    auto kern = few_logits_kernel<CL, STAGES>;
    const int smem = lg_smem_bytes(CL, STAGES);
    ensure_smem_attr(reinterpret_cast<const void*>(kern), smem);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CL;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(CL * ceil_div(p.E, 32), ceil_div(p.T, kLgTokens));
    cfg.blockDim = dim3(kLgThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

// Clusters of 16 CTAs are beyond the portable 8: whether this device can hold one
// (asked once per device).
bool wide_clusters_ok() {
    static std::atomic<int8_t> known[64];   // 0: not asked, 1: yes, 2: no
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    if (const int8_t k = known[dev].load(std::memory_order_relaxed)) return k == 1;
    auto kern = few_logits_kernel<16, 5>;
    const int smem = lg_smem_bytes(16, 5);
    ensure_smem_attr(reinterpret_cast<const void*>(kern), smem);
    int n = 0;
    bool ok = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
    if (ok) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 16;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(16);
        cfg.blockDim = dim3(kLgThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        ok = cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n > 0;
    }
    if (!ok) cudaGetLastError();
    known[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
    return ok;
}

template <bool MX, int NT>
cudaError_t run_ffn(const CUtensorMap* tm, const FewParams& p, int grid, cudaStream_t s) {
    using C = FewCfg<MX, NT>;
    auto kern = few_ffn_kernel<MX, NT>;
    ensure_smem_attr(reinterpret_cast<const void*>(kern), C::kSmem);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tm[0], tm[1], tm[2], tm[3], tm[4], tm[5], tm[6], tm[7], p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool MX>
cudaError_t run_ffn(const CUtensorMap* tm, const FewParams& p, int grid, cudaStream_t s) {
    switch (few_columns(p.T)) {
        case 16: return run_ffn<MX, 16>(tm, p, grid, s);
        case 32: return run_ffn<MX, 32>(tm, p, grid, s);
        case 64: return run_ffn<MX, 64>(tm, p, grid, s);
        default: return run_ffn<MX, 128>(tm, p, grid, s);
    }
}

}  // namespace

size_t few_workspace_bytes(const mok_problem* p, int ctas) { return few_layout(p, ctas).total; }

cudaError_t launch_few(const FewLaunch& a, const GemmCommon& c, cudaStream_t s) {
    const mok_problem* q = a.p;
    const bool mx = q->dtype == MOK_MXFP8;
    const int T = q->T, H = q->H, I = q->I, E = q->E, Is = q->I_shared;
    const FewLayout L = few_layout(q, c.num_sms);
    char* ws = static_cast<char*>(a.workspace);
    const int64_t act = std::min<int64_t>(E, (int64_t)T * q->k);

    FewLogitsParams lp{};
    lp.x = static_cast<const __nv_bfloat16*>(a.x);
    lp.W_r = a.W_r;
    lp.bias = a.bias;
    lp.T = T;
    lp.H = H;
    lp.E = E;
    lp.k = q->k;
    lp.idx = reinterpret_cast<int32_t*>(ws + L.idx);
    lp.w = reinterpret_cast<float*>(ws + L.w);
    lp.logits = reinterpret_cast<float*>(ws + L.logits);
    lp.arrived = reinterpret_cast<int*>(ws + L.arrived);
    lp.topk_idx = a.topk_idx;
    lp.topk_w = a.topk_w;
    lp.xq = mx ? reinterpret_cast<uint8_t*>(ws + L.xq) : nullptr;
    lp.xsf = mx ? reinterpret_cast<uint8_t*>(ws + L.xsf) : nullptr;
    lp.zero = reinterpret_cast<int*>(ws);
    lp.zero_words = (int)(kStatusBytes / 4) + L.n_counters;

    FewParams p{};
    p.T = T; p.H = H; p.I = I; p.E = E; p.k = q->k; p.Is = Is;
    p.R1 = gu_rows(I);
    p.R2 = down_tile_n(H, mx);
    p.Rs1 = Is ? gu_rows(Is) : 0;
    p.idx = lp.idx;
    p.w = lp.w;
    p.gu_sf = a.gu_sf;
    p.dn_sf = a.dn_sf;
    p.xsf = lp.xsf;
    p.h = ws + L.h;
    p.hsf = mx ? reinterpret_cast<uint8_t*>(ws + L.hsf) : nullptr;
    p.hs = reinterpret_cast<__nv_bfloat16*>(ws + L.hs);
    p.part = reinterpret_cast<float*>(ws + L.part);
    p.hready = reinterpret_cast<int*>(ws + L.counters);
    p.cnt1 = p.hready + E + 1;
    p.cnt2 = p.cnt1 + L.n1;
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.status = c.status;
    p.timeout_ns = c.timeout_ns;
    p.withhold = a.withhold;

    CUtensorMap tm[8];
    const int NT = few_columns(T), eb = mx ? 1 : 2;
    bool ok = make_tmap_swizzled(&tm[0], a.x, T, H, 2, NT) &&
              make_tmap_swizzled(&tm[2], a.gu, (int64_t)E * 2 * I, H, eb, p.R1) &&
              make_tmap_swizzled(&tm[3], a.dn, (int64_t)E * H, I, eb, p.R2) &&
              make_tmap_swizzled(&tm[4], p.h, act * T, I, eb, NT);
    tm[1] = tm[0];
    if (ok && mx) ok = make_tmap_swizzled(&tm[1], lp.xq, T, H, 1, NT);
    tm[5] = tm[2];
    tm[6] = tm[3];
    tm[7] = tm[4];
    if (ok && Is)
        ok = make_tmap_swizzled(&tm[5], a.sgu, 2 * (int64_t)Is, H, 2, p.Rs1) &&
             make_tmap_swizzled(&tm[6], a.sdn, H, Is, 2, p.R2) && make_tmap_swizzled(&tm[7], p.hs, T, Is, 2, NT);
    if (!ok) return cudaErrorInvalidValue;

    cudaError_t e = cudaSuccess;
    const int groups = ceil_div(T, kLgTokens), clusters = groups * ceil_div(E, 32);
    if (E > 32) e = cudaMemsetAsync(ws + L.arrived, 0, groups * 4, s);
    // few clusters are spread over 16 CTAs each; up to 64 CTAs of 8-wide clusters
    // hold all of H <= 8192 in their rings, an SM to each (55.1 us against 56.9 with
    // the short ring at 32 tokens, sizes as above); more keep the ring short so that two
    // CTAs share an SM
    if (e == cudaSuccess)
        e = clusters <= kLgWideClusters && wide_clusters_ok() ? run_logits<16, 5>(lp, s)
            : clusters <= 8                                   ? run_logits<8, 9>(lp, s)
                                                              : run_logits<8, 5>(lp, s);
    if (e != cudaSuccess) return e;
    return mx ? run_ffn<true>(tm, p, c.num_sms, s) : run_ffn<false>(tm, p, c.num_sms, s);
}

}  // namespace mok
