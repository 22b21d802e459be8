// grads.cu - the global norm of many gradients, and clipping by it.
//
//   norm = sqrt(sum over all tensors of g^2)
//   g' = g * min(1, max_norm / (norm + 1e-6))       (in place, or into out)
//
// Two passes over the bytes: every CTA sums the squares of its chunks, then every
// CTA adds up all CTAs' sums (in the same order, so all get the same norm) and
// scales chunks. The second pass goes through the chunks backwards, so that it
// begins with what the first pass left in L2. Bound by memory, with nothing of three
// passes (read; read, write) to save where the tensors are larger than L2: a layer's
// 3.3 GB in 1481 us against 1475 at the copy rate; 2^29 BF16 values summed at 6.6 TB/s,
// read and scaled at 6.5. Small calls are bound by the two launches and the norm's FP64
// between them (30 tensors, 4.7 MB: 8.0 us).
#include <algorithm>

#include <cuda_fp16.h>

#include "common.cuh"
#include "moves.cuh"

namespace mok {

namespace {

constexpr int kGradThreads = 512;
constexpr int kGradVecs = 4;                                  // 16-byte vectors of a thread and chunk
constexpr int kChunkBytes = kGradThreads * kGradVecs * 16;
constexpr int kGradTable = 120;                               // tensors of a launch (kernel parameters hold 4 KB)
constexpr int kMaxParts = 1024;

struct GradTable {
    const void* g[kGradTable];
    void* out[kGradTable];
    int64_t n[kGradTable];             // elements << 2 | type
    int32_t first[kGradTable + 1];     // first chunk
    int32_t count;
};

// Last tensor whose first chunk is at or before c.
__device__ __forceinline__ int tensor_of(const GradTable& t, int c) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= c) lo = mid; else hi = mid - 1;
    }
    return lo;
}

template <int ELEM>
__device__ __forceinline__ float elem_at(const void* p, int64_t i) {
    if (ELEM == MOK_ELEM_F32) return static_cast<const float*>(p)[i];
    if (ELEM == MOK_ELEM_F16) return __half2float(static_cast<const __half*>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
template <int ELEM>
__device__ __forceinline__ void put_elem(void* p, int64_t i, float v) {
    if (ELEM == MOK_ELEM_F32) static_cast<float*>(p)[i] = v;
    else if (ELEM == MOK_ELEM_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}
// The two values of a 32-bit word of a 16-bit type.
template <int ELEM>
__device__ __forceinline__ float2 word_values(uint32_t w) {
    if (ELEM == MOK_ELEM_F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return make_float2(bf16_lo(w), bf16_hi(w));
}
template <int ELEM>
__device__ __forceinline__ uint32_t scale_word(uint32_t w, float c) {
    if (ELEM == MOK_ELEM_F32) return __float_as_uint(__uint_as_float(w) * c);
    const float2 v = word_values<ELEM>(w);
    if (ELEM == MOK_ELEM_F16) {
        const __half2 h = __floats2half2_rn(v.x * c, v.y * c);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    return pack_bf16x2(v.x * c, v.y * c);
}

// Sum of squares of a thread's part of a chunk. In fp32; where that overflows or
// is so small that squares were lost, again in fp64 (gradients near 1e-20 or 1e20
// keep their norm).
template <int ELEM>
__device__ double chunk_squares(const void* base, int64_t n, int64_t c0) {
    constexpr int kPer = ELEM == MOK_ELEM_F32 ? 4 : 8;     // elements of a vector
    const int64_t e0 = c0 * (kChunkBytes / (16 / kPer));
    const int64_t left = min(n - e0, (int64_t)kChunkBytes / (16 / kPer));
    double total = 0.0;
    if ((reinterpret_cast<uintptr_t>(base) & 15) == 0) {
        const uint4* v = reinterpret_cast<const uint4*>(base) + e0 / kPer;
        const int nv = (int)(left / kPer);
        uint4 a[kGradVecs];
#pragma unroll
        for (int i = 0; i < kGradVecs; ++i) {
            const int j = threadIdx.x + i * kGradThreads;
            a[i] = j < nv ? __ldg(v + j) : make_uint4(0, 0, 0, 0);
        }
        float2 s = make_float2(0.f, 0.f);
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < kGradVecs; ++i) {
            const uint32_t w[4] = {a[i].x, a[i].y, a[i].z, a[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                any |= w[j];
                if (ELEM == MOK_ELEM_F32) {
                    const float x = __uint_as_float(w[j]);
                    if (j & 1) s.y = fmaf(x, x, s.y);
                    else s.x = fmaf(x, x, s.x);
                } else {
                    const float2 x = word_values<ELEM>(w[j]);
                    s = __ffma2_rn(x, x, s);
                }
            }
        }
        const float f = s.x + s.y;
        if (any != 0 && !(f > 1e-30f && f < 1e38f)) {
#pragma unroll 1
            for (int i = 0; i < kGradVecs * 4; ++i) {
                const uint32_t w = i < 4 ? (i == 0 ? a[0].x : i == 1 ? a[0].y : i == 2 ? a[0].z : a[0].w)
                                 : i < 8 ? (i == 4 ? a[1].x : i == 5 ? a[1].y : i == 6 ? a[1].z : a[1].w)
                                 : i < 12 ? (i == 8 ? a[2].x : i == 9 ? a[2].y : i == 10 ? a[2].z : a[2].w)
                                          : (i == 12 ? a[3].x : i == 13 ? a[3].y : i == 14 ? a[3].z : a[3].w);
                if (ELEM == MOK_ELEM_F32) {
                    const double x = __uint_as_float(w);
                    total += x * x;
                } else {
                    const float2 x = word_values<ELEM>(w);
                    total += (double)x.x * x.x + (double)x.y * x.y;
                }
            }
        } else {
            total = f;
        }
        // the last elements of the tensor
        const int64_t t = (int64_t)nv * kPer + threadIdx.x;
        if (t < left) {
            const double x = elem_at<ELEM>(base, e0 + t);
            total += x * x;
        }
    } else {
        for (int64_t i = threadIdx.x; i < left; i += kGradThreads) {
            const double x = elem_at<ELEM>(base, e0 + i);
            total += x * x;
        }
    }
    return total;
}

// Sum of a value per thread, in the CTA's first thread (fixed order). FP64 arithmetic is
// slow here, two lanes a cycle for the whole SM, so one warp does it. With the first
// chunk's load below this took a call of 30 small tensors from 19.8 to 8.0 us.
__device__ __forceinline__ double cta_sum_f64(double v, double* all) {
    all[threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.x >= 32) return 0.0;
    v = 0.0;
#pragma unroll
    for (int i = 0; i < kGradThreads / 32; ++i) v += all[threadIdx.x + 32 * i];
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// part[b] = (add ? part[b] : 0) + the squares of CTA b's chunks
__global__ void __launch_bounds__(kGradThreads, 2)
grad_squares_kernel(const __grid_constant__ GradTable t, double* part, int add) {
    __shared__ double all[kGradThreads];
    pdl_wait();
    pdl_allow_next();
    const int chunks = t.first[t.count];
    double s = 0.0;
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int i = tensor_of(t, c);
        const int64_t n = t.n[i] >> 2;
        const int elem = (int)(t.n[i] & 3);
        const int64_t c0 = c - t.first[i];
        if (elem == MOK_ELEM_F32) s += chunk_squares<MOK_ELEM_F32>(t.g[i], n, c0);
        else if (elem == MOK_ELEM_F16) s += chunk_squares<MOK_ELEM_F16>(t.g[i], n, c0);
        else s += chunk_squares<MOK_ELEM_BF16>(t.g[i], n, c0);
    }
    s = cta_sum_f64(s, all);
    if (threadIdx.x == 0) part[blockIdx.x] = (add ? part[blockIdx.x] : 0.0) + s;
}

// sqrt of the sum of all partial sums, in the CTA's first warp, the same in every CTA.
__device__ __forceinline__ double norm_of(const double* part, int parts) {
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += 32) s += __ldcg(part + i);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    return threadIdx.x == 0 ? sqrt(s) : 0.0;
}

__global__ void __launch_bounds__(32)
grad_norm_kernel(const double* part, int parts, float* norm) {
    pdl_wait();
    pdl_allow_next();
    const double v = norm_of(part, parts);
    if (threadIdx.x == 0) *norm = (float)v;
}

// A CTA's chunk: where it is, and its vectors on their way (aligned tensors).
struct Chunk {
    const void* src;
    void* dst;
    int64_t e0;        // first element
    int left;          // elements
    int elem;
    bool vec;
    uint4 a[kGradVecs];
};

__device__ __forceinline__ void load_chunk(const GradTable& t, int k, Chunk& c) {
    const int i = tensor_of(t, k);
    c.src = t.g[i];
    c.dst = t.out[i];
    c.elem = (int)(t.n[i] & 3);
    const int per = c.elem == MOK_ELEM_F32 ? 4 : 8;
    c.e0 = (int64_t)(k - t.first[i]) * (kChunkBytes / 16 * per);
    c.left = (int)min((t.n[i] >> 2) - c.e0, (int64_t)kChunkBytes / 16 * per);
    c.vec = ((reinterpret_cast<uintptr_t>(c.src) | reinterpret_cast<uintptr_t>(c.dst)) & 15) == 0;
    if (!c.vec) return;
    const uint4* v = reinterpret_cast<const uint4*>(c.src) + c.e0 / per;
    const int nv = c.left / per;
#pragma unroll
    for (int j = 0; j < kGradVecs; ++j) {
        const int at = threadIdx.x + j * kGradThreads;
        if (at < nv) c.a[j] = v[at];
    }
}

template <int ELEM>
__device__ __forceinline__ void scale_chunk(const Chunk& c, float f) {
    constexpr int kPer = ELEM == MOK_ELEM_F32 ? 4 : 8;
    int from = 0;
    if (c.vec) {
        uint4* o = reinterpret_cast<uint4*>(c.dst) + c.e0 / kPer;
        const int nv = c.left / kPer;
#pragma unroll
        for (int j = 0; j < kGradVecs; ++j) {
            const int at = threadIdx.x + j * kGradThreads;
            if (at < nv)
                o[at] = make_uint4(scale_word<ELEM>(c.a[j].x, f), scale_word<ELEM>(c.a[j].y, f),
                                   scale_word<ELEM>(c.a[j].z, f), scale_word<ELEM>(c.a[j].w, f));
        }
        from = nv * kPer;
    }
    for (int i = from + threadIdx.x; i < c.left; i += kGradThreads)
        put_elem<ELEM>(c.dst, c.e0 + i, elem_at<ELEM>(c.src, c.e0 + i) * f);
}

// The first chunk is loaded while the norm is still being formed: the gradients were
// complete before the kernel that sums them began.
__global__ void __launch_bounds__(kGradThreads, 2)
grad_scale_kernel(const __grid_constant__ GradTable t, const double* part, int parts, double max_norm, float* norm) {
    __shared__ float factor;
    pdl_allow_next();
    int k = t.first[t.count] - 1 - (int)blockIdx.x;
    Chunk c;
    if (k >= 0) load_chunk(t, k, c);
    pdl_wait();
    if (threadIdx.x < 32) {
        const double v = norm_of(part, parts);
        if (threadIdx.x == 0) {
            if (blockIdx.x == 0) *norm = (float)v;
            const double ratio = max_norm / (v + MOK_CLIP_EPS);
            float f = ratio >= 1.0 ? 1.0f : (float)ratio;
            if (isnan(f) && !isnan(v)) f = 1.0f;   // an infinite norm is not above an infinite bound; NaN stays NaN
            factor = f;
        }
    }
    __syncthreads();
    const float f = factor;
    while (k >= 0) {
        if (f != 1.0f || c.dst != c.src) {
            if (c.elem == MOK_ELEM_F32) scale_chunk<MOK_ELEM_F32>(c, f);
            else if (c.elem == MOK_ELEM_F16) scale_chunk<MOK_ELEM_F16>(c, f);
            else scale_chunk<MOK_ELEM_BF16>(c, f);
        }
        k -= gridDim.x;
        if (k >= 0) load_chunk(t, k, c);
    }
}

// The next tensors for one launch, from `i` on: as many as the table holds and their chunks'
// numbers allow; empty ones are left out. Returns the one after them. A tensor of more than a
// chunk that does not begin on 16 bytes (a view into a larger buffer) is listed as its first
// elements and the aligned rest, if its output (read for `outs`) lies the same way. 2^29 BF16
// values at an odd element: norm 164 us and clipping into such an output 526, as aligned
// ones; by elements throughout, 1965 and 3633.
int fill_table(GradTable& t, int32_t count, const mok_grad_tensor* list, int i, bool outs) {
    t.count = 0;
    t.first[0] = 0;
    auto put = [&](const char* g, const char* out, int64_t n, int elem) {
        const int64_t chunks = (n * elem_bytes(elem) + kChunkBytes - 1) / kChunkBytes;
        t.g[t.count] = g;
        t.out[t.count] = const_cast<char*>(out);
        t.n[t.count] = n << 2 | elem;
        t.first[t.count + 1] = t.first[t.count] + (int32_t)chunks;
        ++t.count;
    };
    for (; i < count; ++i) {
        const int64_t n = list[i].n, bytes = n * elem_bytes(list[i].elem);
        if (n == 0) continue;
        const char* g = static_cast<const char*>(list[i].g);
        const char* out = outs && list[i].out ? static_cast<const char*>(list[i].out) : g;
        const uintptr_t at = reinterpret_cast<uintptr_t>(g);
        const int head = bytes > kChunkBytes && ((at ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0 ? (int)(-at & 15) : 0;
        const int64_t chunks = bytes / kChunkBytes + 2;
        if (t.count + (head ? 2 : 1) > kGradTable || (t.count > 0 && t.first[t.count] + chunks > ((int64_t)1 << 30))) break;
        const int first = head / elem_bytes(list[i].elem);
        if (head) put(g, out, first, list[i].elem);
        put(g + head, out + head, n - first, list[i].elem);
    }
    return i;
}

}  // namespace

size_t grad_workspace_bytes() { return kMaxParts * sizeof(double); }

cudaError_t launch_grad_clip(int32_t count, const mok_grad_tensor* list, bool scale, double max_norm, float* norm,
                             void* ws, cudaStream_t s) {
    double* part = static_cast<double*>(ws);
    const int grid = std::min(2 * sm_count(), kMaxParts);
    GradTable t;
    cudaError_t e = cudaSuccess;
    int i = 0, add = 0;
    do {   // once without tensors, too: the partial sums are then zeros
        i = fill_table(t, count, list, i, false);
        e = launch_after(grad_squares_kernel, dim3(grid), dim3(kGradThreads), 0, s, t, part, add);
        add = 1;
    } while (e == cudaSuccess && i < count);
    if (!scale) {
        if (e == cudaSuccess)
            e = launch_after(grad_norm_kernel, dim3(1), dim3(32), 0, s, (const double*)part, grid, norm);
        return e;
    }
    i = 0;
    do {
        i = fill_table(t, count, list, i, true);
        if (e == cudaSuccess)
            e = launch_after(grad_scale_kernel, dim3(grid), dim3(kGradThreads), 0, s, t, (const double*)part, grid,
                             max_norm, norm);
    } while (e == cudaSuccess && i < count);
    return e;
}

}  // namespace mok
