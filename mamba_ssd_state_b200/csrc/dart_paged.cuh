// dart_paged.cuh -- argument blocks, launchers and device helpers of the paged
// memory cache (paged_cache.cu, ssd_extend.cu, sma_paged*.cu), used by the C
// ABI in dart_abi.cu.
//
// Memory m of sequence b is slot m % R of page table[b, m / R].  A page holds
// R memories of every head: [npages, H, R, N, P] elements of dtype, or, in the
// 4-bit format, codes [npages, H, R, P, N/2] and scales [npages, H, R, P, N/32].
#pragma once

#include "dart_common.cuh"

namespace dart {

struct PagedCache {
    int mxfp4;           // 0: elements of dtype, 1: E2M1 codes and E8M0 scales
    int npages, R, width;
    void* pages;
    uint8_t* scales;     // mxfp4 only
    const int* table;    // [B, width]
};

struct CacheCopyArgs {   // write: dH -> pages; read: pages -> dH
    int B, C, H, P, N;
    void* dH;            // [B,H,C,N,P] dtype
    const int* first;    // [B] first memory slot of the sequence
    const int* count;    // [B] memories to move, <= C
    PagedCache cache;
    int* status;
};

struct ExtendArgs {
    int B, T, H, P, N, S, G;   // T packed token rows
    const void* x; const float* dt; const float* A; const void* Bm; const void* Cm;
    const int* cu;             // [B+1]
    const float* state; float* state_out;   // [B,H,N,P]; may be the same
    const float* cur; float* cur_out;       // [B,H,N,P]; may be the same
    PagedCache cache;
    const int* nchunks; const int* pos; int* nchunks_out; int* pos_out;   // [B]
    float* y;                  // [T,H,P]
    int* mem_count;            // [T]
    int* status;
};

struct SmaPagedArgs {
    int B, T, H, P, N, G;
    const void* Q; const void* E; const void* Cm;   // [T,H,N], [T,H,P], [T,G,N]
    const int* cu;             // [B+1]
    PagedCache cache;
    const int* mem_count;      // [T]
    float g; const float* y_ssd; float* out;        // [T,H,P]
    float* part;               // workspace
    int* status;
};

// Largest number of memories a sequence's table may name: 2^26 tokens of context at S = 256.
constexpr long long kPagedMaxMemories = 1 << 18;

bool paged_supported(int N, int P, int mxfp4);
cudaError_t launch_cache_write(const CacheCopyArgs& a, dart_dtype dt, cudaStream_t st);
cudaError_t launch_cache_read(const CacheCopyArgs& a, dart_dtype dt, cudaStream_t st);
cudaError_t launch_ssd_extend(const ExtendArgs& a, dart_dtype dt, cudaStream_t st);
size_t sma_paged_workspace_bytes(int P);
// Tiles a call may come to, and the most a call may have.
long long sma_paged_tiles(int B, int T);
long long sma_paged_max_tiles();
cudaError_t launch_sma_paged(const SmaPagedArgs& a, dart_dtype dt, cudaStream_t st);

#ifdef __CUDACC__
// Index of memory `slot` of head h in page `page` (in memories).
__device__ __forceinline__ size_t memory_index(const PagedCache& c, int H, int page, int h, int slot) {
    return ((size_t)page * H + h) * c.R + slot;
}

// Sequence b's rows of the packed tokens; false when they are not rows at all.
__device__ __forceinline__ bool token_range(const int* cu, int b, int T, int& t0, int& t1) {
    t0 = cu[b];
    t1 = cu[b + 1];
    return t0 >= 0 && t0 <= t1 && t1 <= T;
}

// ------------------------------------------------------------ 4-bit memories
// The 32 values V[32k .. 32k+31, p] share the scale 2^(s-127); codes are E2M1
// (sign, then 0 0.5 1 1.5 2 3 4 6).  The code of V[16i + 4q + j, p] stands at
// place q (N/4) + 4i + j of row p, so that the codes a lane of a 16x8x16 matrix
// product needs of one row are contiguous.  A block that holds a value that is
// not finite has the scale byte 255 and reads as NaN.

// Scale exponent of a block whose largest magnitude is amax (finite): the least
// k with amax <= 6 * 2^k, within [-126, 126].
__device__ __forceinline__ int mxfp4_exponent(float amax) {
    if (amax == 0.f) return -126;
    int e;
    const float f = frexpf(amax, &e);          // amax = f 2^e, f in [0.5, 1)
    return min(max(f <= 0.75f ? e - 3 : e - 2, -126), 126);
}
__device__ __forceinline__ float mxfp4_pow2(int k) { return __int_as_float((k + 127) << 23); }   // |k| <= 126
__device__ __forceinline__ float mxfp4_scale(unsigned s) {   // 2^(s-127), 2^-127 as a subnormal; 255 is NaN
    return __uint_as_float(s == 255u ? 0x7fffffffu : s == 0u ? 0x00400000u : s << 23);
}
// E2M1 code of v (already divided by the scale, |v| <= 6): nearest, ties to even.
__device__ __forceinline__ unsigned mxfp4_code(float v) {
    const float a = fabsf(v);
    const float step = a < 2.f ? 0.5f : a < 4.f ? 1.f : 2.f;
    const float near = rintf(a / step) * step;   // step is a power of two: the division is exact
    const float c = near < 2.f ? 2.f * near : near < 4.f ? near + 2.f : 0.5f * near + 4.f;
    return (unsigned)c | (__float_as_uint(v) >> 31 << 3);
}
__device__ __forceinline__ float mxfp4_level(unsigned code) {
    const unsigned m = code & 7u;
    // 0.5 m below 1, else (1 + low/2) 2^(m/2 - 1)
    const float v = m < 2u ? 0.5f * (float)m : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
    return code & 8u ? -v : v;
}
#endif

}  // namespace dart
