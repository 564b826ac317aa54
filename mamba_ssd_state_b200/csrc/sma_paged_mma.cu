// sma_paged_mma.cu -- state-memory attention of runs of few tokens over paged
// memories, bfloat16 or 4-bit, P = 64.
//
// For up to 8 tokens t of one (sequence, head) and every visible memory M (N x P):
//   U = M^T [Q_t ...] (P x tokens),  V = M^T [C_t ...],  s_t = U_t . E_t / sqrt(N),
//   online softmax over the memories, o_t = sum w_t V_t.
// A memory is read once for all tokens of the tile, so the kernel is bound by
// HBM as long as the products keep up: 4 N P a token do on tensor cores and do
// not on CUDA cores (8 tokens: 262 thousand multiply-adds a memory of 16 KB).
// The products are small (M = P, N = 8 columns), which is the shape of the
// warp-level m16n8k16; a 128-row tile of tcgen05 would be 1/16 full.
//
// Every warp is a worker of its own, with its run of units, its ring of stages in
// shared memory and its softmax: it starts the copy that refills a stage as soon
// as it has read it, running ahead of itself over the ends of items, and never
// waits for another warp.  (With one copying warp and eight that shared the
// pieces of a block, the joins and loads at the ends of items were what bound
// short ones: 616 us where this takes 465 for 64 sequences of one token and 128 memories.)
//
// M^T is the A operand: bfloat16 through ldmatrix.trans; codes become float16
// in registers (E2M1 values are exact there), laid out in memory so that a lane
// finds the codes of its fragments in its own 16 bytes of a column.  The columns
// of B are tokens: with up to 4 tokens one tile of 8 columns holds Q and C, else
// one tile each.  float16 operands hold Q and C scaled by a power of two per
// token, so that a value is off by at most 2^-39 of its row's largest; float32 inputs
// are split into a high and a low float16 half (2^-23 of the value, or 2^-39 as above).
// A block of 32 codes is two k steps: their product is multiplied by the block's
// scale in float32 before it is added, so a scale costs 4 multiply-adds for
// every 2 products and no bit.  That holds for scale bytes 1 .. 192 (values of up
// to 2^67); a piece that meets another one is done again on CUDA cores, about 10
// (one token) to 35 times (six) as slow, for the whole range of the format.
#include <cuda_fp16.h>
#include <float.h>
#include <limits.h>
#include <string.h>

#include "sm100.cuh"
#include "sma_paged.cuh"
#include "tensor_map.h"

namespace dart {
namespace {

using namespace sm100;

constexpr int kP = 64;
constexpr int kCap = 4096;                      // tiles of a call
constexpr int kLeast = 4;                       // units below which a run is not cut

// A memory takes 2.0 us of a warp with two tiles of columns and 1.6 with one
// (4-bit; counted the same, the runs with more rows ended a fifth later).
struct RowCost { static __device__ __forceinline__ int of(int rows) { return rows > 4 ? 5 : 4; } };
using Tiles = TileList<kCap, RowCost>;

struct Params {
    CUtensorMap map;      // bfloat16 memories: (P, rows of N), boxes of one memory
    SmaPagedArgs a;
};

// What a memory is kept as, and the stages it passes through: kPieces of them.
template <int N> struct Bf16Mem {
    static constexpr bool kFp4 = false;
    static constexpr int kWarps = 8, kStages = 2;             // 128 KB of copies in flight
    static constexpr int kRows = 64, kPieces = N / kRows;     // rows of a stage
    static constexpr uint32_t kStageBytes = kRows * kP * 2;
    static __device__ __forceinline__ void copy(const Params& prm, size_t mem, int piece, uint32_t dst, uint32_t full) {
        tma_load_2d(dst, &prm.map, full, 0, (int)(mem * N) + piece * kRows);
    }
};
template <int N> struct Fp4Mem {
    static constexpr bool kFp4 = true;
    static constexpr int kWarps = 12, kStages = 3, kPieces = 1;
    static constexpr uint32_t kCodeBytes = N * kP / 2, kScaleBytes = N * kP / 32;
    static constexpr uint32_t kStageBytes = kCodeBytes + kScaleBytes;
    static __device__ __forceinline__ void copy(const Params& prm, size_t mem, int, uint32_t dst, uint32_t full) {
        bulk_load(dst, static_cast<const uint8_t*>(prm.a.cache.pages) + mem * kCodeBytes, kCodeBytes, full);
        bulk_load(dst + kCodeBytes, prm.a.cache.scales + mem * kScaleBytes, kScaleBytes, full);
    }
};

template <typename M>
struct Smem {
    uint8_t ring[M::kWarps][M::kStages][M::kStageBytes];    // first: tiles are 1024-byte aligned
    uint64_t full[M::kWarps][M::kStages];
    int abort_flag;
    Tiles tiles;
};

template <int I> struct Piece { static constexpr int value = I; };


__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(0.f));
}
// 2^x, good to 2^-22; 0 below 2^-126.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The four bytes of w, two codes each, as pairs of float16.
__device__ __forceinline__ void widen_codes(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(w));
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// The power of two that a column of float16 operands is multiplied by: its largest
// value goes to [2^14, 2^15); one that is not finite stays as it is.
__device__ __forceinline__ int column_exponent(float amax) {
    const int e = (int)(__float_as_uint(amax) >> 23);      // biased exponent, 0 for 0 and subnormals
    return amax > 0.f && e < 255 ? min(max(14 - (e - 127), -126), 126) : 0;
}

// A lane's columns of B: PARTS float16 halves (or bfloat16 as it is) of N / 16
// k steps.  Slots 2q, 2q+1, 2q+8, 2q+9 of k step i stand for rows
// 16i + 4q + {0,1,2,3} with codes, and for 16i + {2q, 2q+1, 2q+8, 2q+9} else
// (there the rows of a ldmatrix are eight neighbours, in eight different banks).
template <typename M, int N, int PARTS>
struct Column {
    uint32_t b[PARTS][N / 16][2];

    // The values of a row of Q or C as they are (zeros for an unused column,
    // src == nullptr): loads that wait for nothing.
    template <typename T>
    struct Raw {
        float f[N / 16][4];
        __device__ __forceinline__ void load(const T* src) {
            const int q = threadIdx.x & 3;
#pragma unroll
            for (int i = 0; i < N / 16; ++i) {
                if constexpr (M::kFp4) {          // rows 16i + 4q ..
                    load4(src ? src + 16 * i + 4 * q : nullptr, f[i]);
                } else {                          // rows 16i + 2q, + 1, and 8 further on
                    load2(src ? src + 16 * i + 2 * q : nullptr, f[i]);
                    load2(src ? src + 16 * i + 2 * q + 8 : nullptr, f[i] + 2);
                }
            }
        }
        static __device__ __forceinline__ void load2(const T* p, float* to) {
            static_assert(sizeof(T) == 2, "bfloat16 memories have bfloat16 tokens");
            const uint32_t u = p ? __ldg(reinterpret_cast<const uint32_t*>(p)) : 0u;
            to[0] = __uint_as_float(u << 16);
            to[1] = __uint_as_float(u & 0xffff0000u);
        }
        static __device__ __forceinline__ void load4(const T* p, float* to) {
            if constexpr (sizeof(T) == 4) {
                const float4 u = p ? __ldg(reinterpret_cast<const float4*>(p)) : make_float4(0.f, 0.f, 0.f, 0.f);
                to[0] = u.x; to[1] = u.y; to[2] = u.z; to[3] = u.w;
            } else {
                const uint2 u = p ? __ldg(reinterpret_cast<const uint2*>(p)) : make_uint2(0u, 0u);
                to[0] = __uint_as_float(u.x << 16); to[1] = __uint_as_float(u.x & 0xffff0000u);
                to[2] = __uint_as_float(u.y << 16); to[3] = __uint_as_float(u.y & 0xffff0000u);
            }
        }
    };

    // Takes the values in.  Returns the power of two that the column was multiplied
    // by (its lanes are those of equal lane / 4).
    template <typename T>
    __device__ __forceinline__ float take(const Raw<T>& raw) {
        const auto& f = raw.f;
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < N / 16; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) amax = fmaxf(amax, fabsf(f[i][j]));
        float scale = 1.f;
        if constexpr (M::kFp4) {
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            scale = mxfp4_pow2(column_exponent(amax));
        }
#pragma unroll
        for (int i = 0; i < N / 16; ++i) {
            if constexpr (M::kFp4) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float u = f[i][2 * j] * scale, v = f[i][2 * j + 1] * scale;
                    b[0][i][j] = pack_half(u, v);
                    if constexpr (PARTS == 2) {
                        const __half2 h = *reinterpret_cast<const __half2*>(&b[0][i][j]);
                        b[1][i][j] = pack_half(u - __low2float(h), v - __high2float(h));
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(f[i][2 * j], f[i][2 * j + 1]);   // exact: it was bfloat16
                    b[0][i][j] = *reinterpret_cast<const uint32_t*>(&h);
                }
            }
        }
        return scale;
    }
};

// acc[t][m] += (piece of a memory in `stage`)^T times the columns; scale bytes are
// ordinary ones (or what comes out is not used).
template <typename M, int N, int NT, int PARTS, int PIECE>
__device__ __forceinline__ void multiply(const uint8_t* stage, const Column<M, N, PARTS> (&col)[NT], float (&acc)[NT][4][4]) {
    const int lane = threadIdx.x & 31;
    if constexpr (!M::kFp4) {
        const int mi = lane >> 3, r = lane & 7;
        const uint32_t base = smem_u32(stage) + (uint32_t)((mi >> 1) * 8 + r) * 128u;
#pragma unroll
        for (int i = 0; i < M::kRows / 16; ++i) {
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                uint32_t a[4];
                ldmatrix_x4_trans(base + (uint32_t)i * 2048u + (uint32_t)(((2 * m + (mi & 1)) ^ r) << 4), a);
#pragma unroll
                for (int t = 0; t < NT; ++t) mma_bf16(acc[t][m], a, col[t].b[0][PIECE * (M::kRows / 16) + i]);
            }
        }
    } else {
        // Products that do not wait for each other stand together: MG groups of 16
        // columns of the memory, as many as the registers take.
        constexpr int K = N / 32, MG = NT == 1 ? 4 : 2;
        const int g = lane >> 2, q = lane & 3;
        const uint8_t* scales = stage + M::kCodeBytes;
#pragma unroll
        for (int m0 = 0; m0 < 4; m0 += MG) {
            uint32_t w[MG][2][K], sc[MG][2];       // code words and scale bytes of two rows of a group
#pragma unroll
            for (int m = 0; m < MG; ++m)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int p = 16 * (m0 + m) + g + 8 * r;
                    if constexpr (K == 4) {
                        const uint4 u = *reinterpret_cast<const uint4*>(stage + p * (N / 2) + q * 16);
                        w[m][r][0] = u.x; w[m][r][1] = u.y; w[m][r][2] = u.z; w[m][r][3] = u.w;
                        sc[m][r] = *reinterpret_cast<const uint32_t*>(scales + p * 4);
                    } else {
                        const uint2 u = *reinterpret_cast<const uint2*>(stage + p * (N / 2) + q * 8);
                        w[m][r][0] = u.x; w[m][r][1] = u.y;
                        sc[m][r] = *reinterpret_cast<const uint16_t*>(scales + p * 2);
                    }
                }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                uint32_t a0[MG][4], a1[MG][4];     // the two k steps of a block
#pragma unroll
                for (int m = 0; m < MG; ++m) {
                    uint32_t u[4], v[4];
                    widen_codes(w[m][0][k], u);
                    widen_codes(w[m][1][k], v);
                    a0[m][0] = u[0]; a0[m][1] = v[0]; a0[m][2] = u[1]; a0[m][3] = v[1];
                    a1[m][0] = u[2]; a1[m][1] = v[2]; a1[m][2] = u[3]; a1[m][3] = v[3];
                }
                float d[NT][MG][4];
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int m = 0; m < MG; ++m) mma_f16_first(d[t][m], a0[m], col[t].b[0][2 * k]);
#pragma unroll
                for (int h = 0; h < PARTS; ++h) {
                    if (h > 0) {
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int m = 0; m < MG; ++m) mma_f16(d[t][m], a0[m], col[t].b[h][2 * k]);
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int m = 0; m < MG; ++m) mma_f16(d[t][m], a1[m], col[t].b[h][2 * k + 1]);
                }
#pragma unroll
                for (int m = 0; m < MG; ++m) {
                    // 2^(s - 127) of the two rows
                    const float s0 = __uint_as_float((k < 3 ? sc[m][0] << (23 - 8 * k) : sc[m][0] >> 1) & 0x7f800000u);
                    const float s1 = __uint_as_float((k < 3 ? sc[m][1] << (23 - 8 * k) : sc[m][1] >> 1) & 0x7f800000u);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        acc[t][m0 + m][0] = fmaf(d[t][m][0], s0, acc[t][m0 + m][0]);
                        acc[t][m0 + m][1] = fmaf(d[t][m][1], s0, acc[t][m0 + m][1]);
                        acc[t][m0 + m][2] = fmaf(d[t][m][2], s1, acc[t][m0 + m][2]);
                        acc[t][m0 + m][3] = fmaf(d[t][m][3], s1, acc[t][m0 + m][3]);
                    }
                }
            }
        }
    }
}

// Not 0 where one of the scale bytes that this lane looks at is no ordinary one, 1 .. 192:
// scaled columns times larger ones may overflow where the true sums do not, and 0 and 255
// do not stand for the exponents that multiply() takes them for.  (A look at every word
// where it is multiplied by, and the products anew on the spot, cost up to 4%; this costs
// less than the look for 255 alone did: drafts 131 -> 125 us.)
template <typename M>
__device__ __forceinline__ uint32_t odd_scales(const uint8_t* stage) {
    constexpr int kWords = M::kScaleBytes / 128;             // of a lane
    const uint32_t* words = reinterpret_cast<const uint32_t*>(stage + M::kCodeBytes) + (threadIdx.x & 31) * kWords;
    uint32_t odd = 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        const uint32_t less = words[i] - 0x01010101u;        // its bytes' upper two bits are set from 193 on, and where 0 borrows
        odd |= less & less << 1;
    }
    return odd & 0x80808080u;
}

// A piece whose memories hold scale bytes that are not ordinary, anew: token by token on
// CUDA cores, from the pages, a lane with the columns `lane` and `lane + 32`.  A block's
// product meets the powers of two of its scale and of its row of Q or C in one step, so
// that nothing overflows or vanishes on the way that does not in the sum.  Not inlined: its
// registers would be the products'.
template <typename T, typename M, int N, int TT>
__device__ __noinline__ void run_piece_any_scale(const SmaPagedArgs& a, const int* table, int t0, int rows, int h, int first, int last,
                                                 int bad, bool whole, int run, int which) {
    constexpr int K = N / 32;
    const int lane = threadIdx.x & 31, grp = group_of(h, a.H, a.G);
    for (int t = 0; t < rows; ++t) {
        const size_t tok = (size_t)(t0 + t);
        const T* src[2] = {static_cast<const T*>(a.Q) + (tok * a.H + h) * N, static_cast<const T*>(a.Cm) + (tok * a.G + grp) * N};
        float pre[2], e[2];
        int exponent[2];
        for (int i = 0; i < 2; ++i) {
            float amax = 0.f;
            for (int n = 0; n < N; ++n) amax = fmaxf(amax, fabsf(ldf(src[i] + n)));
            exponent[i] = column_exponent(amax);
            pre[i] = mxfp4_pow2(exponent[i]);
            e[i] = ldf(static_cast<const T*>(a.E) + (tok * a.H + h) * kP + lane + 32 * i);
        }
        const int count = a.mem_count[tok];
        float m = -FLT_MAX, l = 0.f, o[2] = {0.f, 0.f};
        for (int c = first; c < min(last, count); ++c) {
            const size_t mem = memory_index(a.cache, a.H, table[c / a.cache.R], h, c % a.cache.R);
            const uint32_t* codes = static_cast<const uint32_t*>(a.cache.pages) + mem * (M::kCodeBytes / 4);
            const uint8_t* scales = a.cache.scales + mem * M::kScaleBytes;
            float uv[2][2] = {};                              // of Q and C, of the two columns
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int p = lane + 32 * j;
#pragma unroll 1
                for (int k = 0; k < K; ++k) {
                    float d[2] = {0.f, 0.f};
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t w[4];
                        widen_codes(codes[p * (N / 8) + q * K + k], w);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 two = __half22float2(*reinterpret_cast<const __half2*>(&w[i / 2]));
                            const int n = 32 * k + 16 * (i / 4) + 4 * q + i % 4;
#pragma unroll
                            for (int r = 0; r < 2; ++r) d[r] = fmaf(i & 1 ? two.y : two.x, ldf(src[r] + n) * pre[r], d[r]);
                        }
                    }
                    const int s = scales[p * K + k];
#pragma unroll
                    for (int r = 0; r < 2; ++r) uv[r][j] += s == 255 ? __int_as_float(0x7fffffff) : ldexpf(d[r], s - 127 - exponent[r]);
                }
            }
            const float sc = warp_sum(fmaf(uv[0][0], e[0], uv[0][1] * e[1])) * (kLog2e * rsqrtf((float)N));
            const float mn = fmaxf(m, sc), f = exp2f(m - mn), wt = exp2f(sc - mn);
            l = fmaf(l, f, wt);
            m = mn;
#pragma unroll
            for (int j = 0; j < 2; ++j) o[j] = wt != 0.f ? fmaf(o[j], f, wt * uv[1][j]) : o[j];
        }
        const bool left = count < 0 || count > bad;           // a row that is not to be computed
        if (!whole) {
            float* row = piece_rows<TT, kP>(a.part, run, which) + t * (kP + 4);
            if (lane == 0) { row[kP] = m; row[kP + 1] = left ? -1.f : l; }
            row[lane] = o[0];
            row[lane + 32] = o[1];
        } else if (!left) {
            const size_t at = (tok * a.H + h) * kP + lane;
            const float f = l == 0.f ? 0.f : (a.y_ssd ? a.g : 1.f) / l;
#pragma unroll
            for (int j = 0; j < 2; ++j) a.out[at + 32 * j] = fmaf(f, o[j], a.y_ssd ? a.y_ssd[at + 32 * j] : 0.f);
        }
    }
}

// One piece of the run.  NT = 1: columns 0-3 of the tile are Q and 4-7 C of up to
// 4 tokens; NT = 2: a tile each of up to 8.
template <typename T, typename M, int N, int TT, int NT, int PARTS>
__device__ __forceinline__ void run_piece(const Params& prm, Smem<M>& s, const Walk& w, int run, int t0, int rows,
                                          Feed<M, Tiles>& feed, int& taken, const WaitCtx& wc, bool& ok) {
    const SmaPagedArgs& a = prm.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
    const int grp = group_of(w.h, a.H, a.G);
    const T *Q = static_cast<const T*>(a.Q), *C = static_cast<const T*>(a.Cm), *E = static_cast<const T*>(a.E);
    auto q_row = [&](int t) { return t < rows ? Q + ((size_t)(t0 + t) * a.H + w.h) * N : nullptr; };
    auto c_row = [&](int t) { return t < rows ? C + ((size_t)(t0 + t) * a.G + grp) * N : nullptr; };
    Column<M, N, PARTS> col[NT];
    // this lane's two tokens, as columns of the results, and what their scores and values are to be multiplied by
    const int tk = NT == 2 ? 2 * q : 2 * (q & 1);
    float e[4][4];        // E of (token, column) as the results are laid out
    int count[2];         // of the two tokens
    float qs[2], vs[2];
    {   // all loads first
        typename Column<M, N, PARTS>::template Raw<T> raw[NT];
        if constexpr (NT == 2) {
            raw[0].load(q_row(g));
            raw[1].load(c_row(g));
        } else {
            raw[0].load(g < 4 ? q_row(g) : c_row(g - 4));
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            count[j] = tk + j < rows ? a.mem_count[t0 + tk + j] : -1;
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    e[m][2 * r + j] = tk + j < rows && (NT == 2 || q < 2)
                                          ? ldf(E + ((size_t)(t0 + tk + j) * a.H + w.h) * kP + 16 * m + g + 8 * r) : 0.f;
        }
        float scale[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) scale[t] = col[t].take(raw[t]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            qs[j] = kLog2e * rsqrtf((float)N) / __shfl_sync(0xffffffffu, scale[0], 4 * (tk + j));
            vs[j] = 1.f / __shfl_sync(0xffffffffu, scale[NT - 1], 4 * ((NT == 2 ? 0 : 4) + tk + j));
        }
    }
    const int* table = a.cache.table + (size_t)s.tiles.seq(w.k) * a.cache.width;
    const int bad = readable_memories(table, a.cache, w.first_memory(), w.last_memory());
    int fewest = INT_MAX; // memories that every row of the tile sees (rows that are not to be computed apart)
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (count[j] >= 0 && count[j] <= bad) fewest = min(fewest, count[j]);
    fewest = __reduce_min_sync(0xffffffffu, fewest);
    // Scores: the lanes of a column (equal lane % 4) hold parts of those of its two
    // tokens; the even of lane / 4 take the first one's, the odd the second's.
    const int mine = g & 1;
    const float qm = mine ? qs[1] : qs[0];
    // lanes that have the weights of this lane's tokens (the C columns take those of the Q columns)
    const int from = NT == 2 ? q : q & 1;
    float mx = -FLT_MAX, l = 0.f, o[4][4];      // of token tk + mine; o of both
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[m][r] = 0.f;

    uint32_t odd = 0;     // 4-bit: scale bytes that the products below are not made for
    const int last = min(w.last_memory(), bad);
    for (int c = w.first_memory(); c < last; ++c) {
        float acc[NT][4][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[t][m][r] = 0.f;
        auto take = [&](auto piece) {
            const int st = taken % M::kStages;
            const uint32_t bar = smem_u32(&s.full[warp][st]), phase = (uint32_t)(taken / M::kStages) & 1u;
            // bfloat16 memories are waited for longer than a look takes (64 single tokens 462 us, 465 with it)
            if (ok) ok = M::kFp4 ? wait_warp(bar, phase, wc, 1) : mbar_wait_warp(bar, phase, wc, 1);
            ++taken;
            if (!ok) return;
            if constexpr (M::kFp4) odd |= odd_scales<M>(s.ring[warp][st]);
            multiply<M, N, NT, PARTS, decltype(piece)::value>(s.ring[warp][st], col, acc);
            __syncwarp();        // every lane has read the stage
            feed.fill(prm, s.tiles, s.ring[warp], s.full[warp]);
        };
        take(Piece<0>{});
        if constexpr (M::kPieces == 2) take(Piece<1>{});
        float v[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            v[j] = 0.f;
#pragma unroll
            for (int m = 0; m < 4; ++m) v[j] = fmaf(acc[0][m][j], e[m][j], fmaf(acc[0][m][2 + j], e[m][2 + j], v[j]));
        }
        float sc = (mine ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, mine ? v[0] : v[1], 4);
        sc += __shfl_xor_sync(0xffffffffu, sc, 8);
        sc += __shfl_xor_sync(0xffffffffu, sc, 16);
        sc *= qm;
        const bool all = c < fewest;                // every row sees this memory
        if (!all && c >= (mine ? count[1] : count[0])) sc = -INFINITY;
        if (__any_sync(0xffffffffu, sc > mx)) {     // few memories move a maximum
            const float mn = fmaxf(mx, sc), f = exp2_fast(mx - mn);
            l *= f;
            mx = mn;
            const float f0 = __shfl_sync(0xffffffffu, f, from), f1 = __shfl_sync(0xffffffffu, f, from + 4);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                o[m][0] *= f0; o[m][1] *= f1; o[m][2] *= f0; o[m][3] *= f1;
            }
        }
        const float wm = exp2_fast(sc - mx);
        l += wm;
        const float w0 = __shfl_sync(0xffffffffu, wm, from), w1 = __shfl_sync(0xffffffffu, wm, from + 4);
        if (all) {
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                o[m][0] = fmaf(w0, acc[NT - 1][m][0], o[m][0]);
                o[m][1] = fmaf(w1, acc[NT - 1][m][1], o[m][1]);
                o[m][2] = fmaf(w0, acc[NT - 1][m][2], o[m][2]);
                o[m][3] = fmaf(w1, acc[NT - 1][m][3], o[m][3]);
            }
        } else {
            // what a row does not see it does not read, whatever the value is
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                if (w0 != 0.f) { o[m][0] = fmaf(w0, acc[NT - 1][m][0], o[m][0]); o[m][2] = fmaf(w0, acc[NT - 1][m][2], o[m][2]); }
                if (w1 != 0.f) { o[m][1] = fmaf(w1, acc[NT - 1][m][1], o[m][1]); o[m][3] = fmaf(w1, acc[NT - 1][m][3], o[m][3]); }
            }
        }
    }
    const float ml[2] = {__shfl_sync(0xffffffffu, mx, from), __shfl_sync(0xffffffffu, mx, from + 4)};
    const float ll[2] = {__shfl_sync(0xffffffffu, l, from), __shfl_sync(0xffffffffu, l, from + 4)};
    // a whole item is written out, a part of one kept for the combine kernel
    const bool whole = w.whole();
    const int which = w.c > 0 ? 0 : 1;
    if (!whole && lane == 0) *piece_header(a.part, run, which) = PieceHeader{w.last == w.units ? 2 : 1, t0, rows, w.h};
    if constexpr (M::kFp4) {
        if (__any_sync(0xffffffffu, odd != 0)) {
            run_piece_any_scale<T, M, N, TT>(a, table, t0, rows, w.h, w.first_memory(), last, bad, whole, run, which);
            return;
        }
    }
    if (NT == 1 && q < 2) return;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int t = tk + j;
        if (t >= rows) continue;
        const bool left = count[j] < 0 || count[j] > bad;     // a row that is not to be computed
        if (whole) {
            if (left) continue;
            const size_t at = ((size_t)(t0 + t) * a.H + w.h) * kP + g;
            const float f = ll[j] == 0.f ? 0.f : (a.y_ssd ? a.g : 1.f) * vs[j] / ll[j];
            float y[4][2];      // all loads before the first store: out may be y_ssd itself
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int r = 0; r < 2; ++r) y[m][r] = a.y_ssd ? a.y_ssd[at + 16 * m + 8 * r] : 0.f;
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int r = 0; r < 2; ++r) a.out[at + 16 * m + 8 * r] = fmaf(f, o[m][2 * r + j], y[m][r]);
        } else {
            float* row = piece_rows<TT, kP>(a.part, run, which) + t * (kP + 4);
            if (g == 0) { row[kP] = ml[j]; row[kP + 1] = left ? -1.f : ll[j]; }
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int r = 0; r < 2; ++r) row[g + 16 * m + 8 * r] = o[m][2 * r + j] * vs[j];
        }
    }
}

template <typename T, typename M, int N, int TT, int PARTS>
__global__ void __launch_bounds__(32 * M::kWarps, 1) sma_paged_mma_kernel(const __grid_constant__ Params prm) {
    extern __shared__ uint8_t raw[];
    Smem<M>& s = *reinterpret_cast<Smem<M>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const SmaPagedArgs& a = prm.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < M::kWarps * M::kStages; ++i) mbar_init(smem_u32(&s.full[0][0] + i), 1);
        s.abort_flag = 0;
        fence_mbar_init();
    }
    // neighbours in the order of units go to different blocks: a few units spread over all of them
    const int runs = gridDim.x * M::kWarps, run = warp * gridDim.x + blockIdx.x;
    griddep_wait();
    if (lane < 2) piece_header(a.part, run, lane)->state = 0;
    __syncwarp();
    build_tiles<TT>(a, s.tiles);
    if (s.tiles.n == 0) return;
    const WaitCtx wc{&s.abort_flag, a.status, 10};
    bool ok = true;
    int taken = 0;
    Walk w = start_walk(s.tiles, a.H, run, runs, kLeast);
    Feed<M, Tiles> feed;
    feed.begin(a, s.tiles, w);
    for (int i = 0; i < M::kStages; ++i) feed.fill(prm, s.tiles, s.ring[warp], s.full[warp]);
    for (; next_piece(w); advance(s.tiles, w, a.H)) {
        const int t0 = s.tiles.t0[w.k], rows = s.tiles.rows(w.k);
        if (w.memories() == 0) {      // nothing to see: the readout is 0
            for (int i = lane; i < rows * kP; i += 32) {
                const int c = a.mem_count[t0 + i / kP];
                const size_t at = ((size_t)(t0 + i / kP) * a.H + w.h) * kP + i % kP;
                if (c == 0) a.out[at] = a.y_ssd ? a.y_ssd[at] : 0.f;
            }
            continue;
        }
        if (TT == 8 && rows > 4) {
            if constexpr (TT == 8) run_piece<T, M, N, TT, 2, PARTS>(prm, s, w, run, t0, rows, feed, taken, wc, ok);
        } else {
            run_piece<T, M, N, TT, 1, PARTS>(prm, s, w, run, t0, rows, feed, taken, wc, ok);
        }
    }
    if (!ok) feed.drain(s.full[warp]);      // else every copy has been waited for
}

template <typename T, typename M, int N, int TT, int PARTS>
cudaError_t run(const SmaPagedArgs& a, cudaStream_t st) {
    auto kern = sma_paged_mma_kernel<T, M, N, TT, PARTS>;
    const int smem = (int)sizeof(Smem<M>) + 1024, sms = paged_sm_count();
    static_assert(sizeof(Smem<M>) + 1024 <= 232448, "shared memory");
    if (sms <= 0) return cudaErrorInvalidDevice;
    Params prm;
    memset(&prm.map, 0, sizeof(prm.map));
    prm.a = a;
    if constexpr (!M::kFp4) {
        const uint64_t rows = (uint64_t)a.cache.npages * a.H * a.cache.R * N;
        if (rows > 0x7fffffffull) return cudaErrorInvalidValue;      // 256 GB and more of memories
        const uint64_t dims[2] = {kP, rows}, strides[1] = {kP * 2};
        const uint32_t box[2] = {kP, (uint32_t)M::kRows};
        if (!encode_tile_map_bf16(&prm.map, 2, a.cache.pages, dims, strides, box)) return cudaErrorInvalidValue;
    }
    static std::atomic<unsigned long long> ready{0};   // devices whose kernel has its shared memory allowed
    cudaError_t e = paged_allow_smem(reinterpret_cast<const void*>(kern), smem, ready);
    if (e != cudaSuccess) return e;
    const int blocks = min(sms, kMaxRuns / M::kWarps);
    if ((e = launch_dependent(kern, dim3(blocks), dim3(32 * M::kWarps), smem, st, 1, prm)) != cudaSuccess) return e;
    count_launches(1);
    return launch_sma_paged_combine(a, blocks * M::kWarps, TT, st);
}

}  // namespace

cudaError_t launch_sma_paged_mma(const SmaPagedArgs& a, dart_dtype dt, cudaStream_t st) {
    if (a.cache.mxfp4) {
        if (dt == DART_F32) return a.N == 128 ? run<float, Fp4Mem<128>, 128, 4, 2>(a, st) : run<float, Fp4Mem<64>, 64, 4, 2>(a, st);
        return a.N == 128 ? run<__nv_bfloat16, Fp4Mem<128>, 128, 8, 1>(a, st) : run<__nv_bfloat16, Fp4Mem<64>, 64, 8, 1>(a, st);
    }
    return a.N == 128 ? run<__nv_bfloat16, Bf16Mem<128>, 128, 8, 1>(a, st) : run<__nv_bfloat16, Bf16Mem<64>, 64, 8, 1>(a, st);
}

}  // namespace dart
