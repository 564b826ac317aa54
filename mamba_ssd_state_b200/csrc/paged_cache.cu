// paged_cache.cu -- chunk memories into the pages of their sequences and back.
//
//   write  memory first[b] + i of sequence b = dH[b, :, i]    for i < count[b]
//   read   dH[b, :, i] = memory first[b] + i of sequence b
// as elements of dtype (a copy) or as 4-bit codes with a scale for every 32
// values along N (dart_paged.cuh): the scale is the least power of two that
// holds the block's largest magnitude, the codes round to nearest even.
//
// Bound by HBM: a memory of N P values is read once and written once.  Dense rows
// go along P and codes along N, so the 4-bit form passes through shared memory:
// global memory sees whole rows only.  Going in, a thread owns the 32 values of a
// block for two columns and has them in flight before the range is checked; a
// block is one memory.  Coming out, a block takes a memory of several heads, whose
// codes are all in flight at once behind one look at the range and the table
// (one head a block: 155 us for 16 x 63 memories of 32 heads, four: 79).
// Codes are made and widened by the hardware's E2M1 conversions (nearest, ties
// to even; every code is exact in float16).
//
// A sequence is moved whole or not at all: every block checks the sequence's
// range and the pages it touches before it moves its own memory.
#include <cuda_fp16.h>

#include "dart_paged.cuh"

namespace dart {
namespace {

constexpr int kThreads = 256;

// The page of slot first + i, or -1 when this sequence is not to be moved (or
// has no memory i).  All threads of the block take part.
__device__ __forceinline__ int checked_page(const CacheCopyArgs& a, int b, int i, int& slot) {
    const int count = a.count[b], first = a.first[b];
    const long long last = (long long)first + count;
    const bool range = count >= 0 && count <= a.C && first >= 0 && last <= (long long)a.cache.width * a.cache.R;
    const int* row = a.cache.table + (size_t)b * a.cache.width;
    int bad = !range;
    if (range && count > 0)
        for (int k = first / a.cache.R + threadIdx.x; k <= (int)((last - 1) / a.cache.R); k += blockDim.x)
            bad |= row[k] < 0 || row[k] >= a.cache.npages;
    if (__syncthreads_or(bad)) {
        if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) flag_status(a.status, kStatusDevice);
        return -1;
    }
    if (i >= count) return -1;
    slot = (first + i) % a.cache.R;
    return row[(first + i) / a.cache.R];
}

// grid (C, H, B); kWrite: dH -> page, else page -> dH.
template <bool kWrite>
__global__ void __launch_bounds__(kThreads) cache_copy_kernel(CacheCopyArgs a, int vecs) {
    const int i = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    int slot = 0;
    const int page = checked_page(a, b, i, slot);
    if (page < 0) return;
    uint4* dense = static_cast<uint4*>(a.dH) + (((size_t)b * a.H + h) * a.C + i) * vecs;
    uint4* paged = static_cast<uint4*>(a.cache.pages) + memory_index(a.cache, a.H, page, h, slot) * vecs;
    const uint4* src = kWrite ? dense : paged;
    uint4* dst = kWrite ? paged : dense;
#pragma unroll 4
    for (int v = threadIdx.x; v < vecs; v += blockDim.x) dst[v] = ld_stream_u4(src + v);
}

// Two neighbouring columns of a row.
__device__ __forceinline__ float2 load2(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 load2(const __nv_bfloat16* p) {
    const unsigned w = *reinterpret_cast<const unsigned*>(p);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ void store2(float* p, float u, float v) { *reinterpret_cast<float2*>(p) = make_float2(u, v); }
__device__ __forceinline__ void store2(__nv_bfloat16* p, float u, float v) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(u, v);
}

// A code word holds the 8 codes of column p with n = 32k + {0, 16} + 4q + j;
// row p has N/8 of them, word q (N/32) + k.
// The 8 values of a code word.
__device__ __forceinline__ void code_values(uint32_t w, float (&v)[8]) {
    uint32_t r[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

constexpr int kP = 64;   // columns of the 4-bit shapes

template <typename T, int N>
__global__ void __launch_bounds__(N) cache_write_mxfp4_kernel(CacheCopyArgs a) {
    constexpr int K = N / 32, W = N / 8;          // blocks and code words of a column
    constexpr int WS = W + 1;                     // padded: lanes write words of different columns
    const int i = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    __shared__ uint32_t codes[kP * WS];
    __shared__ __align__(16) uint8_t scales[kP * K];
    const T* src = static_cast<const T*>(a.dH) + (((size_t)b * a.H + h) * a.C + i) * (size_t)(N * kP);
    const int p = 2 * (threadIdx.x % 32), k = threadIdx.x / 32;
    float2 v[32];                                 // dH has this memory, whatever the counts say
#pragma unroll
    for (int r = 0; r < 32; ++r) v[r] = load2(src + (32 * k + r) * kP + p);
    int slot = 0;
    const int page = checked_page(a, b, i, slot);
    if (page < 0) return;
    scales[p * K + k] = (uint8_t)mxfp4_block<N>([&](int r) { return v[r].x; }, codes + p * WS + k);
    scales[(p + 1) * K + k] = (uint8_t)mxfp4_block<N>([&](int r) { return v[r].y; }, codes + (p + 1) * WS + k);
    __syncthreads();
    const size_t m = memory_index(a.cache, a.H, page, h, slot);
    uint4* cdst = static_cast<uint4*>(a.cache.pages) + m * (kP * W / 4);
    uint4* sdst = reinterpret_cast<uint4*>(a.cache.scales) + m * (kP * K / 16);
    for (int w = threadIdx.x; w < kP * W / 4; w += N) {
        const uint32_t* c = codes + w * 4 / W * WS + w * 4 % W;
        cdst[w] = make_uint4(c[0], c[1], c[2], c[3]);
    }
    if (threadIdx.x < kP * K / 16) sdst[threadIdx.x] = reinterpret_cast<const uint4*>(scales)[threadIdx.x];
}

constexpr int kHeads = 4;   // memories (of neighbouring heads) of a reading block

template <typename T, int N>
__global__ void __launch_bounds__(kThreads) cache_read_mxfp4_kernel(CacheCopyArgs a) {
    constexpr int K = N / 32, W = N / 8;
    constexpr int WS = W + 1;                     // padded rows: lanes read words of different columns
    constexpr int V = kP * W / 4;                 // 16-byte vectors of a memory's codes
    const int i = blockIdx.x, h0 = blockIdx.y * kHeads, b = blockIdx.z, heads = min(kHeads, a.H - h0);
    int slot = 0;
    const int page = checked_page(a, b, i, slot);
    if (page < 0) return;
    __shared__ uint32_t codes[kHeads][kP * WS];
    __shared__ __align__(16) uint8_t scales[kHeads][kP * K];
    uint4 c[kHeads];
    uint32_t sc[kHeads];
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
        if (h >= heads) break;
        const size_t m = memory_index(a.cache, a.H, page, h0 + h, slot);
        if (threadIdx.x < V) c[h] = ld_stream_u4(static_cast<const uint4*>(a.cache.pages) + m * V + threadIdx.x);
        if (threadIdx.x < kP * K / 4) sc[h] = __ldg(reinterpret_cast<const uint32_t*>(a.cache.scales) + m * (kP * K / 4) + threadIdx.x);
    }
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
        if (h >= heads) break;
        if (threadIdx.x < V) {
            uint32_t* d = codes[h] + threadIdx.x * 4 / W * WS + threadIdx.x * 4 % W;
            d[0] = c[h].x; d[1] = c[h].y; d[2] = c[h].z; d[3] = c[h].w;
        }
        if (threadIdx.x < kP * K / 4) reinterpret_cast<uint32_t*>(scales[h])[threadIdx.x] = sc[h];
    }
    __syncthreads();
    const int p = 2 * (threadIdx.x % (kP / 2));
    for (int h = 0; h < heads; ++h) {
        T* dst = static_cast<T*>(a.dH) + (((size_t)b * a.H + h0 + h) * a.C + i) * (size_t)(N * kP);
#pragma unroll
        for (int w = threadIdx.x / (kP / 2); w < W; w += kThreads / (kP / 2)) {
            const int q = w / K, k = w % K;
            float u[8], v[8];
            code_values(codes[h][p * WS + w], u);
            code_values(codes[h][(p + 1) * WS + w], v);
            const float s0 = mxfp4_scale(scales[h][p * K + k]), s1 = mxfp4_scale(scales[h][(p + 1) * K + k]);
#pragma unroll
            for (int j = 0; j < 8; ++j) store2(dst + (32 * k + 16 * (j / 4) + 4 * q + j % 4) * kP + p, u[j] * s0, v[j] * s1);
        }
    }
}

template <bool kWrite>
cudaError_t launch(const CacheCopyArgs& a, dart_dtype dt, cudaStream_t st) {
    const dim3 grid(a.C, a.H, a.B);
    if (!a.cache.mxfp4) {
        const int vecs = a.N * a.P * (dt == DART_F32 ? 4 : 2) / 16;
        cache_copy_kernel<kWrite><<<grid, vecs < kThreads ? (vecs + 31) / 32 * 32 : kThreads, 0, st>>>(a, vecs);
    } else if (kWrite) {
        if (a.N == 128 && dt == DART_F32) cache_write_mxfp4_kernel<float, 128><<<grid, 128, 0, st>>>(a);
        else if (a.N == 128) cache_write_mxfp4_kernel<__nv_bfloat16, 128><<<grid, 128, 0, st>>>(a);
        else if (dt == DART_F32) cache_write_mxfp4_kernel<float, 64><<<grid, 64, 0, st>>>(a);
        else cache_write_mxfp4_kernel<__nv_bfloat16, 64><<<grid, 64, 0, st>>>(a);
    } else {
        const dim3 few(a.C, (a.H + kHeads - 1) / kHeads, a.B);
        if (a.N == 128 && dt == DART_F32) cache_read_mxfp4_kernel<float, 128><<<few, kThreads, 0, st>>>(a);
        else if (a.N == 128) cache_read_mxfp4_kernel<__nv_bfloat16, 128><<<few, kThreads, 0, st>>>(a);
        else if (dt == DART_F32) cache_read_mxfp4_kernel<float, 64><<<few, kThreads, 0, st>>>(a);
        else cache_read_mxfp4_kernel<__nv_bfloat16, 64><<<few, kThreads, 0, st>>>(a);
    }
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace

bool paged_supported(int N, int P, int mxfp4) {
    return (N == 128 && P == 64) || (N == 64 && P == 64) || (!mxfp4 && N == 16 && P == 16);
}

cudaError_t launch_cache_write(const CacheCopyArgs& a, dart_dtype dt, cudaStream_t st) { return launch<true>(a, dt, st); }
cudaError_t launch_cache_read(const CacheCopyArgs& a, dart_dtype dt, cudaStream_t st) { return launch<false>(a, dt, st); }

}  // namespace dart
