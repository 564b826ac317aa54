// ssd_extend_mma.cu -- runs of many new tokens (pieces of a prompt) through the
// recurrence on tensor cores, bfloat16 inputs, P = 64.
//
// The rule is ssd_extend.cu's, evaluated in blocks of up to 64 tokens that end at
// the end of a chunk.  With cum_t the sum of dt A up to token t of the block and
// H, D the matrices before it,
//   y_t = exp(cum_t) C_t^T H + sum_{s <= t} exp(cum_t - cum_s) dt_s (C_t . B_s) x_s,
//   H' = exp(cum_end) H + S,  D' = exp(cum_end) D + S,
//   S = sum_s B_s (exp(cum_end - cum_s) dt_s x_s)^T.
// Token by token a thread needs 4 N P operations a token from the CUDA cores and
// waits for shared memory at every one (four pieces of up to 256 tokens, 32
// heads, chunks of 64: 117 us); the products of a block keep the state in
// registers too and take 39 us (37 with chunks of 128).  They are warp-level m16n8k16: the state is both the accumulator of one
// block's S and, as it lies, the A operand of the next block's C^T H.
//
// float32 results from bfloat16 products: C, B and x are exact; H, the decayed
// Gram matrix and the weighted x are float32 and go in as three bfloat16 parts
// (24 bits), so every product is exact and every sum is in float32.  Decays are
// exponentials of differences of prefix sums that are kept as two floats (their
// difference is good to 2^-24 as long as the block's |dt A| sum to less than 2^29).
//
// No token's value reaches an earlier token, whatever it is: a column of the Gram
// matrix that a row does not see is 0 by selection, and where an x of the block is
// not finite (0 times it is NaN) the rows are summed over what they see by CUDA
// cores.  A state that is not finite gives y that are not finite, NaN where the
// token-by-token kernel may have an infinity.
//
// A block of 256 threads owns PS columns of one (sequence, head): warp w holds 16
// of them and N PS / 128 rows of H^T and D^T.  The partial sums of y meet in
// shared memory, in a fixed order.  The next tokens' B, C and x are on their way
// (cp.async) while a block is computed.
#include "dart_paged.cuh"
#include "sm100.cuh"

namespace dart {
namespace {

constexpr int kThreads = 256, kWarps = 8;
constexpr int kTB = 64;       // tokens of a block
constexpr int kP = 64;

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void ldsm(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {   // zeros where it is not
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
// u and v as three pairs of bfloat16 that add up to them (24 bits).
__device__ __forceinline__ void split3(float u, float v, uint32_t (&r)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(u, v);
        r[i] = *reinterpret_cast<const uint32_t*>(&h);
        u -= __low2float(h);
        v -= __high2float(h);
    }
}

template <int N, int PS>
struct Smem {
    static constexpr int kRowN = N + 8, kRowP = PS + 8;     // padded rows: ldmatrix rows fall into different banks
    static constexpr int kPW = PS / 16, kNW = kWarps / kPW; // warps along the columns, along the rows of the state
    __nv_bfloat16 B[2][kTB][kRowN], C[2][kTB][kRowN], x[2][kTB][kRowP];
    __nv_bfloat16 wx[3][kTB][kRowP];
    float y[2 + kNW][kTB][PS + 4];                           // partial sums
    float d[N * PS];                                         // D on its way to a page
    float dt[2][kTB];
    // of the block in each buffer: cum (base 2) in two parts, exp(cum), exp(cum_end - cum) dt, exp(cum_end)
    float hi[2][kTB], lo[2][kTB], grow[2][kTB], w[2][kTB], total[2];
};

template <int N, int PS, bool kMany>
__global__ void __launch_bounds__(kThreads, 1) ssd_extend_mma_kernel(ExtendArgs a) {
    using T = __nv_bfloat16;
    using S = Smem<N, PS>;
    constexpr int NW = N / S::kNW, NT = NW / 8;              // rows of H held by a warp, as tiles of 8
    extern __shared__ __align__(16) uint8_t raw[];
    S& s = *reinterpret_cast<S*>(raw);
    const int p0 = blockIdx.x * PS, h = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    sm100::griddep_wait();
    const EarlierEntries<kMany> earlier(a, b);
    const int wp = warp % S::kPW, wn = warp / S::kPW;        // this warp's 16 columns and NW rows of the state
    const size_t bh = (size_t)b * a.H + h;
    // element (p, n) of H^T: columns p0 + 16 wp + g (+ 8), rows NW wn + 8 j + 2 q (+ 1)
    const size_t at = (bh * N + NW * wn + 2 * q) * kP + p0 + 16 * wp + g;
    float H[NT][4], D[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const size_t e = at + (8 * j + (r & 1)) * kP + 8 * (r >> 1);
            H[j][r] = a.state[e];
            D[j][r] = a.cur[e];
        }
    const ExtendPlan plan = plan_extend(a, b, p0 == 0 && h == 0, earlier);
    auto store = [&]() {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const size_t e = at + (8 * j + (r & 1)) * kP + 8 * (r >> 1);
                a.state_out[e] = H[j][r];
                a.cur_out[e] = D[j][r];
            }
    };
    if (plan.len == 0) {   // the sequence stays as it is
        if (a.state_out != a.state || a.cur_out != a.cur) store();
        return;
    }
    const int grp = group_of(h, a.H, a.G), t1 = plan.t0 + plan.len;
    const float Ah = a.A[h];
    auto fetch = [&](int base, int m, int buf) {
        for (int i = tid; i < kTB * (N / 8); i += kThreads) {
            const int r = i / (N / 8), c = 8 * (i % (N / 8));
            const size_t e = ((size_t)(base + (r < m ? r : 0)) * a.G + grp) * N + c;
            copy16(smem_addr(&s.B[buf][r][c]), static_cast<const T*>(a.Bm) + e, r < m);
            copy16(smem_addr(&s.C[buf][r][c]), static_cast<const T*>(a.Cm) + e, r < m);
        }
        for (int i = tid; i < kTB * (PS / 8); i += kThreads) {
            const int r = i / (PS / 8), c = 8 * (i % (PS / 8));
            copy16(smem_addr(&s.x[buf][r][c]), static_cast<const T*>(a.x) + ((size_t)(base + (r < m ? r : 0)) * a.H + h) * kP + p0 + c, r < m);
        }
        if (warp == 4)       // which sums them up
#pragma unroll
            for (int t = lane; t < kTB; t += 32)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(&s.dt[buf][t])),
                             "l"(a.dt + (size_t)(base + (t < m ? t : 0)) * a.H + h), "r"(t < m ? 4 : 0) : "memory");
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // Decays of the block in a buffer, by one warp: sums of dt A log2(e) in float64, two tokens a lane.
    auto decays = [&](int k) {
        const double la = (double)Ah * 1.4426950408889634;
        const double u = la * s.dt[k][2 * lane];
        double c = u + la * s.dt[k][2 * lane + 1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double before = __shfl_up_sync(0xffffffffu, c, o);
            if (lane >= o) c += before;
        }
        const double end = __shfl_sync(0xffffffffu, c, 31);   // tokens past the block's add nothing
        double first = __shfl_up_sync(0xffffffffu, c, 1);      // up to the lane's first token: nothing of its second one
        first = lane > 0 ? first + u : u;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const double cum = i ? c : first;
            const int t = 2 * lane + i;
            s.hi[k][t] = (float)cum;
            s.lo[k][t] = (float)(cum - (double)(float)cum);
            s.grow[k][t] = exp2f((float)cum);
            s.w[k][t] = exp2f((float)(end - cum)) * s.dt[k][t];
        }
        if (lane == 0) s.total[k] = exp2f((float)end);
    };
    int slot = plan.n, left = a.S - plan.pos, buf = 0;       // tokens up to the end of the chunk
    int m = min(min(kTB, plan.len), left);
    fetch(plan.t0, m, 0);
    auto wait_copies = [&]() { asm volatile("cp.async.wait_group 0;" ::: "memory"); };
    if (warp == 4) {
        wait_copies();
        __syncwarp();
        decays(0);
    }
    // y of m tokens from row `base` on, and the memory that closed with the last one
    auto finish = [&](int base, int m, bool closed) {
        constexpr int COLS = PS / 4, ROWS = kThreads / COLS;      // threads of a row, rows at a time
        const int c = 4 * (tid % COLS), r0 = tid / COLS;
        float* to = a.y + ((size_t)(base + r0) * a.H + h) * kP + p0 + c;
#pragma unroll
        for (int u = 0; u < kTB / ROWS; ++u) {
            const int t = r0 + u * ROWS;
            if (t < m) {
                float4 v[2 + S::kNW];
#pragma unroll
                for (int k = 0; k < 2 + S::kNW; ++k) v[k] = *reinterpret_cast<const float4*>(&s.y[k][t][c]);
                if (t < 32) v[1] = make_float4(0.f, 0.f, 0.f, 0.f);      // no column of the second half is seen
#pragma unroll
                for (int k = 1; k < 2 + S::kNW; ++k) v[0] = make_float4(v[0].x + v[k].x, v[0].y + v[k].y, v[0].z + v[k].z, v[0].w + v[k].w);
                *reinterpret_cast<float4*>(to + (size_t)u * ROWS * a.H * kP) = v[0];
            }
        }
        if (closed) {
            append_memory<T, N, kP, PS>(a, b, h, slot, p0, s.d, tid, kThreads);
            ++slot;
        }
    };
    int done = 0;                     // tokens of the block before, whose y is still in parts
    bool closed = false;
    for (int base = plan.t0; base < t1; buf ^= 1) {
        const bool closes = m == left;
        const int next = base + m, left2 = closes ? a.S : left - m, m2 = min(min(kTB, t1 - next), left2);
        wait_copies();
        __syncthreads();
        if (done > 0) finish(base - done, done, closed);
        // ---- the weighted x in three parts
        bool odd = false;                                     // a value of it is not finite
        for (int i = tid; i < kTB * (PS / 2); i += kThreads) {
            const int r = i / (PS / 2), c = 2 * (i % (PS / 2));
            const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&s.x[buf][r][c]);
            odd |= !(fabsf(__low2float(v)) < INFINITY && fabsf(__high2float(v)) < INFINITY);
            uint32_t part[3];
            split3(s.w[buf][r] * __low2float(v), s.w[buf][r] * __high2float(v), part);
#pragma unroll
            for (int k = 0; k < 3; ++k) *reinterpret_cast<uint32_t*>(&s.wx[k][r][c]) = part[k];
        }
        odd = __syncthreads_or(odd);
        if (m2 > 0) fetch(next, m2, buf ^ 1);
        const int li = lane & 7, lm = lane >> 3;              // row and matrix of a ldmatrix address
        // ---- inside the block: 16 rows t by 32 columns s of the decayed Gram matrix, times x
        {
            const int tt = 16 * (warp & 3), ss = 32 * (warp >> 2);
            if (ss <= tt + 15) {
                float G[4][4] = {};
#pragma unroll
                for (int k = 0; k < N / 16; ++k) {
                    uint32_t ca[4];
                    ldsm(smem_addr(&s.C[buf][tt + (lm & 1) * 8 + li][16 * k + (lm >> 1) * 8]), ca);
#pragma unroll
                    for (int j = 0; j < 4; j += 2) {
                        if (ss + 8 * j > tt + 15) continue;
                        uint32_t bb[4];      // tiles j and j + 1 of 8 columns
                        ldsm(smem_addr(&s.B[buf][ss + 8 * j + (lm >> 1) * 8 + li][16 * k + (lm & 1) * 8]), bb);
                        mma(G[j], ca, bb[0], bb[1]);
                        mma(G[j + 1], ca, bb[2], bb[3]);
                    }
                }
                // the decayed G[j][r] of row tt + g + 8 (r / 2), column ss + 8 j + 2 q + r % 2; 0 where the row does not see it
                auto decayed = [&](int j, int r) {
                    const int t = tt + g + 8 * (r >> 1), c = ss + 8 * j + 2 * q + (r & 1);
                    return c <= t && c < m ? exp2f((s.hi[buf][t] - s.hi[buf][c]) + (s.lo[buf][t] - s.lo[buf][c])) * s.dt[buf][c] * G[j][r] : 0.f;
                };
                float(*y)[PS + 4] = s.y[warp >> 2];
                if (odd) {
                    // 0 times a later token's infinity or NaN would reach earlier ones: only what a row sees is multiplied
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r) G[j][r] = decayed(j, r);
#pragma unroll 1
                    for (int p = 0; p < PS; ++p) {
                        float u[2] = {0.f, 0.f};              // rows tt + g and tt + g + 8
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const int t = tt + g + 8 * (r >> 1), c = ss + 8 * j + 2 * q + (r & 1);
                                if (c <= t) u[r >> 1] = fmaf(G[j][r], __bfloat162float(s.x[buf][c][p]), u[r >> 1]);
                            }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            u[i] += __shfl_xor_sync(0xffffffffu, u[i], 1);
                            u[i] += __shfl_xor_sync(0xffffffffu, u[i], 2);
                            if (q == 0) y[tt + g + 8 * i][p] = u[i];
                        }
                    }
                } else {
                    uint32_t A3[3][2][4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int r = 0; r < 4; r += 2) {
                            uint32_t part[3];
                            split3(decayed(j, r), decayed(j, r + 1), part);
#pragma unroll
                            for (int k = 0; k < 3; ++k) A3[k][j >> 1][(j & 1) * 2 + (r >> 1)] = part[k];
                        }
                    float Y[PS / 8][4] = {};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (ss + 16 * k > tt + 15) continue;
                        uint32_t xb[PS / 16][4];
#pragma unroll
                        for (int j = 0; j < PS / 16; ++j) ldsm_t(smem_addr(&s.x[buf][ss + 16 * k + (lm & 1) * 8 + li][16 * j + (lm >> 1) * 8]), xb[j]);
#pragma unroll
                        for (int i = 0; i < 3; ++i)      // products of one part after the other: neighbours do not wait for each other
#pragma unroll
                            for (int j = 0; j < PS / 8; ++j) mma(Y[j], A3[i][k], xb[j >> 1][2 * (j & 1)], xb[j >> 1][2 * (j & 1) + 1]);
                    }
#pragma unroll
                    for (int j = 0; j < PS / 8; ++j) {
                        *reinterpret_cast<float2*>(&y[tt + g][8 * j + 2 * q]) = make_float2(Y[j][0], Y[j][1]);
                        *reinterpret_cast<float2*>(&y[tt + g + 8][8 * j + 2 * q]) = make_float2(Y[j][2], Y[j][3]);
                    }
                }
            }
        }
        // ---- from before the block: (H^T C^T) in columns t; the accumulator of H^T as it lies is the A operand
        {
            float Y[kTB / 8][4] = {};
#pragma unroll
            for (int k = 0; k < NT / 2; ++k) {
                uint32_t part[4][3];
                split3(H[2 * k][0], H[2 * k][1], part[0]);
                split3(H[2 * k][2], H[2 * k][3], part[1]);
                split3(H[2 * k + 1][0], H[2 * k + 1][1], part[2]);
                split3(H[2 * k + 1][2], H[2 * k + 1][3], part[3]);
                uint32_t cb[kTB / 16][4];
#pragma unroll
                for (int j = 0; j < kTB / 16; ++j) ldsm(smem_addr(&s.C[buf][16 * j + (lm >> 1) * 8 + li][NW * wn + 16 * k + (lm & 1) * 8]), cb[j]);
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const uint32_t ha[4] = {part[0][i], part[1][i], part[2][i], part[3][i]};
#pragma unroll
                    for (int j = 0; j < kTB / 8; ++j) mma(Y[j], ha, cb[j >> 1][2 * (j & 1)], cb[j >> 1][2 * (j & 1) + 1]);
                }
            }
            float(*y)[PS + 4] = s.y[2 + wn];
#pragma unroll
            for (int j = 0; j < kTB / 8; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t = 8 * j + 2 * q + (r & 1);
                    y[t][16 * wp + g + 8 * (r >> 1)] = s.grow[buf][t] * Y[j][r];
                }
        }
        // ---- the state after the block
        {
            float U[NT][4] = {};
#pragma unroll
            for (int k = 0; k < kTB / 16; ++k) {
                if (16 * k >= m) continue;
                uint32_t xa[3][4];
#pragma unroll
                for (int i = 0; i < 3; ++i) ldsm_t(smem_addr(&s.wx[i][16 * k + (lm >> 1) * 8 + li][16 * wp + (lm & 1) * 8]), xa[i]);
                uint32_t bb[NT / 2][4];
#pragma unroll
                for (int j = 0; j < NT / 2; ++j) ldsm_t(smem_addr(&s.B[buf][16 * k + (lm & 1) * 8 + li][NW * wn + 16 * j + (lm >> 1) * 8]), bb[j]);
#pragma unroll
                for (int i = 0; i < 3; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j) mma(U[j], xa[i], bb[j >> 1][2 * (j & 1)], bb[j >> 1][2 * (j & 1) + 1]);
            }
            const float total = s.total[buf];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    H[j][r] = fmaf(total, H[j][r], U[j][r]);
                    D[j][r] = fmaf(total, D[j][r], U[j][r]);
                }
        }
        if (closes) {                  // D is the chunk's memory
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    s.d[(NW * wn + 8 * j + 2 * q + (r & 1)) * PS + 16 * wp + g + 8 * (r >> 1)] = D[j][r];
                    D[j][r] = 0.f;
                }
        }
        if (warp == 4 && m2 > 0) {     // ahead of the others: it has no part in the Gram matrix
            wait_copies();
            __syncwarp();
            decays(buf ^ 1);
        }
        done = m;
        closed = closes;
        base = next;
        left = left2;
        m = m2;
    }
    __syncthreads();
    finish(t1 - done, done, closed);
    store();
}

template <int N, int PS, bool kMany>
cudaError_t run(const ExtendArgs& a, cudaStream_t st) {
    auto kern = ssd_extend_mma_kernel<N, PS, kMany>;
    const int smem = (int)sizeof(Smem<N, PS>);
    static_assert(sizeof(Smem<N, PS>) <= 232448, "shared memory");
    static std::atomic<unsigned long long> ready{0};   // devices whose kernel has its shared memory allowed
    cudaError_t e = paged_allow_smem(reinterpret_cast<const void*>(kern), smem, ready);
    if (e != cudaSuccess) return e;
    if ((e = launch_dependent(kern, dim3(kP / PS, a.H, a.B), dim3(kThreads), smem, st, 1, a)) == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace

bool ssd_extend_mma_applicable(const ExtendArgs& a, dart_dtype dt) {
    // A block costs the same with few tokens as with 64, and ends with its chunk.  64 sequences of 32 heads,
    // token by token / here: 12 tokens on average 90 / 136 us, 24 tokens 145 / 156, 35 tokens 198 / 178, 48
    // tokens 258 / 190; 4 sequences: 14 tokens 11 / 15 us, 27 tokens 18 / 16, 58 tokens 32 / 17.  Four pieces
    // of up to 256 tokens, token by token / here, before the former's last step (3% of it): 151 / 187 us with
    // chunks of 8, 138 / 103 of 16, 117 / 39 of 64.
    return dt == DART_BF16 && a.P == kP && (a.N == 128 || a.N == 64) && a.S >= 16 && a.T >= 24 * (long long)a.B;
}

cudaError_t launch_ssd_extend_mma(const ExtendArgs& a, cudaStream_t st) {
    // half the columns a block where whole ones would leave half of the machine idle
    const bool half = 2ll * a.B * a.H <= paged_sm_count();
    if (a.B > EarlierEntries<true>::kEach * kThreads) return a.N == 128 ? run<128, 64, true>(a, st) : run<64, 64, true>(a, st);
    if (a.N == 128) return half ? run<128, 32, false>(a, st) : run<128, 64, false>(a, st);
    return half ? run<64, 32, false>(a, st) : run<64, 64, false>(a, st);
}

}  // namespace dart
