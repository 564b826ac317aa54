// dart_paged.cuh -- argument blocks, launchers and device helpers of the paged
// memory cache (paged_cache.cu, ssd_extend.cu, sma_paged*.cu), used by the C
// ABI in dart_abi.cu.
//
// Memory m of sequence b is slot m % R of page table[b, m / R].  A page holds
// R memories of every head: [npages, H, R, N, P] elements of dtype, or, in the
// 4-bit format, codes [npages, H, R, P, N/2] and scales [npages, H, R, P, N/32].
#pragma once

#include <atomic>

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

// Largest number of memories a sequence's table may name: 2^24 tokens of context at S = 256
// (and the units of 4096 tiles, at 5 a memory, stay within 31 bits).
constexpr long long kPagedMaxMemories = 1 << 16;

bool paged_supported(int N, int P, int mxfp4);
cudaError_t launch_cache_write(const CacheCopyArgs& a, dart_dtype dt, cudaStream_t st);
cudaError_t launch_cache_read(const CacheCopyArgs& a, dart_dtype dt, cudaStream_t st);
cudaError_t launch_ssd_extend(const ExtendArgs& a, dart_dtype dt, cudaStream_t st);
// ssd_extend_mma.cu: bfloat16 tokens with P = 64, long runs.
bool ssd_extend_mma_applicable(const ExtendArgs& a, dart_dtype dt);
cudaError_t launch_ssd_extend_mma(const ExtendArgs& a, cudaStream_t st);
// Multiprocessors of the current device, looked up once; 0 on failure.
int paged_sm_count();
// Allows a kernel its dynamic shared memory on the current device, once for each
// (ready: one per kernel; threads that race set the same attribute twice).
cudaError_t paged_allow_smem(const void* kernel, int bytes, std::atomic<unsigned long long>& ready);
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
// Whether an earlier sequence may own rows from t0 on: one of entries first, first +
// step, ... before b says so, itself within the T rows.  Where no entry before b does,
// the rows of sequences whose own two entries are in order do not meet.
__device__ __forceinline__ bool rows_taken(const int* cu, int b, int T, int t0, int first, int step) {
    bool taken = false;
    for (int k = first; k < b; k += step) taken |= cu[k] > t0 && cu[k] <= T;
    return taken;
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
// Encodes the 8 values v[0 .. 7] (divided by their scale) as a word, the first in the lowest nibble.
__device__ __forceinline__ uint32_t mxfp4_word(const float (&v)[8]) {
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w) : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return w;
}
// The 32 values get(0 .. 31) of block k of a column: its four code words go to
// word[q N/32], its scale is returned as a byte.
template <int N, class Get>
__device__ __forceinline__ unsigned mxfp4_block(Get get, uint32_t* word) {
    float v[32], amax = 0.f;
    bool finite = true;
#pragma unroll
    for (int r = 0; r < 32; ++r) {
        v[r] = get(r);
        amax = fmaxf(amax, fabsf(v[r]));
        finite &= fabsf(v[r]) < INFINITY;
    }
    const int e = mxfp4_exponent(finite ? amax : 0.f);
    const float inv = mxfp4_pow2(-e);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = v[16 * (j / 4) + 4 * q + j % 4] * inv;
        word[q * (N / 32)] = finite ? mxfp4_word(u) : 0u;
    }
    return finite ? (unsigned)(e + 127) : 255u;
}

// ----------------------------------------------- what a run of tokens has to do
struct ExtendPlan {
    int t0, len;     // rows of the sequence's tokens; len 0 where there is nothing to do, or it cannot be done
    int n, pos;      // memories and place in the chunk before the run
};

// A thread's share of the entries of cu_tokens up to sequence b's, asked for before the
// state is.  kMany: for batches of more than kEach entries a thread, whose loop waits for
// every load that is under way; with it in every call 64 single tokens took 47 us instead
// of 45, and 64 runs of 48 163 instead of 152.  All threads of a block.
template <bool kMany>
struct EarlierEntries {
    static constexpr int kEach = 4;
    int entry[kEach];
    bool taken = false;
    __device__ __forceinline__ EarlierEntries(const ExtendArgs& a, int b) {
        const int tid = threadIdx.x, threads = blockDim.x;
#pragma unroll
        for (int i = 0; i < kEach; ++i) entry[i] = a.cu[min(tid + i * threads, b)];
        if constexpr (kMany) taken = rows_taken(a.cu, b, a.T, a.cu[b], tid + kEach * threads, threads);
    }
};

// Checks the run of sequence b: its rows, its counters, and that the pages of the
// memories that close have room and are pages.  One block per sequence (`first`)
// writes its counters and counts and flags what is wrong.  All threads of a block.
template <bool kMany>
__device__ __forceinline__ ExtendPlan plan_extend(const ExtendArgs& a, int b, bool first, const EarlierEntries<kMany>& earlier) {
    const int tid = threadIdx.x, threads = blockDim.x;
    ExtendPlan p;
    int t1;
    const bool range = token_range(a.cu, b, a.T, p.t0, t1);
    p.n = a.nchunks[b];
    p.pos = a.pos[b];
    bool taken = earlier.taken;
#pragma unroll
    for (int i = 0; i < earlier.kEach; ++i) taken |= earlier.entry[i] > p.t0 && earlier.entry[i] <= a.T;
    p.len = range ? t1 - p.t0 : 0;
    const bool counters = p.n >= 0 && p.pos >= 0 && p.pos < a.S;
    const long long closes = counters ? ((long long)p.pos + p.len) / a.S : 0;
    const int R = a.cache.R;
    const int* row = a.cache.table + (size_t)b * a.cache.width;
    int bad = !range || !counters || p.n + closes > (long long)a.cache.width * R;
    if (!bad && closes > 0)
        for (int k = p.n / R + tid; k <= (int)((p.n + closes - 1) / R); k += threads) bad |= row[k] < 0 || row[k] >= a.cache.npages;
    bad = __syncthreads_or(bad || taken);
    if (first) {
        const bool own = range && !(bad && __syncthreads_or(taken));      // the rows are this sequence's, if anyone's
        if (bad && tid == 0) flag_status(a.status, kStatusDevice);
        if (tid == 0) {
            a.nchunks_out[b] = bad ? p.n : (int)(p.n + closes);
            a.pos_out[b] = bad ? p.pos : (int)((p.pos + (long long)p.len) - closes * a.S);
        }
        if (own)
            for (int t = p.t0 + tid; t < t1; t += threads) a.mem_count[t] = bad ? -1 : (int)(p.n + ((long long)p.pos + (t - p.t0)) / a.S);
    }
    if (bad) p.len = 0;
    return p;
}

// Columns p0 .. p0 + PS - 1 of a finished memory, from shared memory d [N][PS] to
// slot `slot` of sequence b, head h.  All threads of a block.
template <typename T, int N, int P, int PS>
__device__ __forceinline__ void append_memory(const ExtendArgs& a, int b, int h, int slot, int p0, const float* d, int tid, int threads) {
    const int R = a.cache.R;
    const size_t mem = memory_index(a.cache, a.H, a.cache.table[(size_t)b * a.cache.width + slot / R], h, slot % R);
    if (!a.cache.mxfp4) {
        T* to = static_cast<T*>(a.cache.pages) + mem * (size_t)(N * P) + p0;
        for (int i = tid; i < N * PS; i += threads) to[(size_t)(i / PS) * P + i % PS] = Elem<T>::from_f(d[i]);
    } else if constexpr (N % 32 == 0) {
        uint32_t* codes = static_cast<uint32_t*>(a.cache.pages) + mem * (size_t)(N * P / 8);
        uint8_t* scales = a.cache.scales + mem * (size_t)(N * P / 32);
        for (int i = tid; i < PS * (N / 32); i += threads) {
            const int p = i % PS, k = i / PS;
            scales[(p0 + p) * (N / 32) + k] =
                (uint8_t)mxfp4_block<N>([&](int r) { return d[(32 * k + r) * PS + p]; }, codes + (size_t)(p0 + p) * (N / 8) + k);
        }
    }
}
#endif

}  // namespace dart
