// paged_cache.cu -- chunk memories into the pages of their sequences and back.
//
//   write  memory first[b] + i of sequence b = dH[b, :, i]    for i < count[b]
//   read   dH[b, :, i] = memory first[b] + i of sequence b
// as elements of dtype (a copy) or as 4-bit codes with a scale for every 32
// values along N (dart_paged.cuh): the scale is the least power of two that
// holds the block's largest magnitude, the codes round to nearest even.
//
// Bound by HBM: a memory of N P values is read once and written once.  One
// block moves one memory.  Dense rows go along P and codes along N, so the
// 4-bit form passes through shared memory: there a thread owns 32 values of
// one column going in, and 8 values of two columns coming out, while global
// memory sees whole rows only.
//
// A sequence is moved whole or not at all: every block checks the sequence's
// range and the pages it touches before it moves its own memory.
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

// A code word holds the 8 codes of column p with n = 32k + {0, 16} + 4q + j;
// row p has N/8 of them, word q (N/32) + k.
template <typename T, int N, int P>
__global__ void __launch_bounds__(kThreads) cache_write_mxfp4_kernel(CacheCopyArgs a) {
    constexpr int K = N / 32, W = N / 8;          // blocks and code words of a column
    static_assert(P * K <= kThreads && P == 64, "one thread per block of 32 values");
    const int i = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    int slot = 0;
    const int page = checked_page(a, b, i, slot);
    if (page < 0) return;
    __shared__ __align__(16) uint32_t codes[P * W];
    __shared__ __align__(16) uint8_t scales[P * K];
    const T* src = static_cast<const T*>(a.dH) + (((size_t)b * a.H + h) * a.C + i) * (size_t)(N * P);
    if (threadIdx.x < P * K) {
        const int p = threadIdx.x % P, k = threadIdx.x / P;
        float v[32];
        float amax = 0.f;
        bool finite = true;
#pragma unroll
        for (int r = 0; r < 32; ++r) v[r] = ldf(src + (32 * k + r) * P + p);
#pragma unroll
        for (int r = 0; r < 32; ++r) {
            amax = fmaxf(amax, fabsf(v[r]));
            finite &= fabsf(v[r]) < INFINITY;
        }
        const int e = mxfp4_exponent(finite ? amax : 0.f);
        const float inv = mxfp4_pow2(-e);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t w = 0;
#pragma unroll
            for (int c = 0; c < 8; ++c) w |= mxfp4_code(v[16 * (c / 4) + 4 * q + c % 4] * inv) << (4 * c);
            codes[p * W + q * K + k] = finite ? w : 0u;
        }
        scales[p * K + k] = finite ? (uint8_t)(e + 127) : (uint8_t)255;
    }
    __syncthreads();
    const size_t m = memory_index(a.cache, a.H, page, h, slot);
    uint4* cdst = static_cast<uint4*>(a.cache.pages) + m * (P * W / 4);
    uint4* sdst = reinterpret_cast<uint4*>(a.cache.scales) + m * (P * K / 16);
    if (threadIdx.x < P * W / 4) cdst[threadIdx.x] = reinterpret_cast<const uint4*>(codes)[threadIdx.x];
    if (threadIdx.x < P * K / 16) sdst[threadIdx.x] = reinterpret_cast<const uint4*>(scales)[threadIdx.x];
}

__device__ __forceinline__ void store2(float* p, float u, float v) { *reinterpret_cast<float2*>(p) = make_float2(u, v); }
__device__ __forceinline__ void store2(__nv_bfloat16* p, float u, float v) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(u, v);
}

template <typename T, int N, int P>
__global__ void __launch_bounds__(kThreads) cache_read_mxfp4_kernel(CacheCopyArgs a) {
    constexpr int K = N / 32, W = N / 8;
    constexpr int WS = W + 1;                     // padded rows: lanes read words of different columns
    const int i = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    int slot = 0;
    const int page = checked_page(a, b, i, slot);
    if (page < 0) return;
    __shared__ uint32_t codes[P * WS];
    __shared__ uint8_t scales[P * K];
    const size_t m = memory_index(a.cache, a.H, page, h, slot);
    const uint4* csrc = static_cast<const uint4*>(a.cache.pages) + m * (P * W / 4);
    const uint32_t* ssrc = reinterpret_cast<const uint32_t*>(a.cache.scales) + m * (P * K / 4);
    if (threadIdx.x < P * W / 4) {
        const uint4 c = ld_stream_u4(csrc + threadIdx.x);
        uint32_t* d = codes + threadIdx.x * 4 / W * WS + threadIdx.x * 4 % W;
        d[0] = c.x; d[1] = c.y; d[2] = c.z; d[3] = c.w;
    }
    if (threadIdx.x < P * K / 4) reinterpret_cast<uint32_t*>(scales)[threadIdx.x] = ssrc[threadIdx.x];
    __syncthreads();
    T* dst = static_cast<T*>(a.dH) + (((size_t)b * a.H + h) * a.C + i) * (size_t)(N * P);
    const int p = 2 * (threadIdx.x % (P / 2));
    for (int w = threadIdx.x / (P / 2); w < W; w += kThreads / (P / 2)) {
        const int q = w / K, k = w % K;
        const uint32_t c0 = codes[p * WS + w], c1 = codes[(p + 1) * WS + w];
        const float s0 = mxfp4_scale(scales[p * K + k]), s1 = mxfp4_scale(scales[(p + 1) * K + k]);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int n = 32 * k + 16 * (c / 4) + 4 * q + c % 4;
            store2(dst + n * P + p, mxfp4_level(c0 >> (4 * c) & 15u) * s0, mxfp4_level(c1 >> (4 * c) & 15u) * s1);
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
        if (a.N == 128 && dt == DART_F32) cache_write_mxfp4_kernel<float, 128, 64><<<grid, kThreads, 0, st>>>(a);
        else if (a.N == 128) cache_write_mxfp4_kernel<__nv_bfloat16, 128, 64><<<grid, kThreads, 0, st>>>(a);
        else if (dt == DART_F32) cache_write_mxfp4_kernel<float, 64, 64><<<grid, kThreads, 0, st>>>(a);
        else cache_write_mxfp4_kernel<__nv_bfloat16, 64, 64><<<grid, kThreads, 0, st>>>(a);
    } else {
        if (a.N == 128 && dt == DART_F32) cache_read_mxfp4_kernel<float, 128, 64><<<grid, kThreads, 0, st>>>(a);
        else if (a.N == 128) cache_read_mxfp4_kernel<__nv_bfloat16, 128, 64><<<grid, kThreads, 0, st>>>(a);
        else if (dt == DART_F32) cache_read_mxfp4_kernel<float, 64, 64><<<grid, kThreads, 0, st>>>(a);
        else cache_read_mxfp4_kernel<__nv_bfloat16, 64, 64><<<grid, kThreads, 0, st>>>(a);
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
