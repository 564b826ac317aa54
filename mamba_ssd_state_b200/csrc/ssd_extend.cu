// ssd_extend.cu -- a run of new tokens per sequence through the recurrence,
// from the middle of a chunk on, appending the memories that close on the way
// to the sequence's pages.
//
// Per sequence, head and token (the same rule as the decode step, for several
// tokens): a = exp(dt A), H = a H + dt B x^T, D = a D + dt B x^T, y = H^T C; at
// the last token of a chunk D goes to the next memory slot and restarts at 0.
//
// Both matrices are N x P and their columns are independent, so a block owns a
// slice of the columns of one (sequence, head) and keeps them in registers from
// the first token to the last: one read and one write of H and D, the floor of
// short runs.  A thread owns one column and N / RG rows of it; the RG partial
// sums of a y meet in shared memory once for every kTile tokens.
#include "dart_paged.cuh"

namespace dart {
namespace {

constexpr int kTile = 16;   // tokens staged in shared memory at a time

template <typename T, int N, int P, int PS, int kThreads>
__global__ void __launch_bounds__(kThreads) ssd_extend_kernel(ExtendArgs a) {
    constexpr int RG = kThreads / PS;      // row groups
    constexpr int RPT = N / RG;            // rows of a thread
    static_assert(RPT >= 1 && RPT % 4 == 0, "rows per thread");
    const int p0 = blockIdx.x * PS, h = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, col = tid % PS, rg = tid / PS, n0 = rg * RPT;
    __shared__ __align__(16) float Bs[kTile][N], Cs[kTile][N];
    __shared__ float xs[kTile][PS], dts[kTile], as[kTile];
    __shared__ float ys[kTile][RG][PS];
    __shared__ float amax_s[RG][PS];

    // ---- what this sequence has to do, and whether it can be done
    int t0, t1;
    const bool range = token_range(a.cu, b, a.T, t0, t1);
    const int n = a.nchunks[b], pos = a.pos[b];
    const int len = range ? t1 - t0 : 0;
    const bool counters = n >= 0 && pos >= 0 && pos < a.S;
    const long long closes = counters ? ((long long)pos + len) / a.S : 0;
    const int R = a.cache.R;
    const int* row = a.cache.table + (size_t)b * a.cache.width;
    int bad = !range || !counters || n + closes > (long long)a.cache.width * R;
    if (!bad && closes > 0)
        for (int k = n / R + tid; k <= (int)((n + closes - 1) / R); k += kThreads) bad |= row[k] < 0 || row[k] >= a.cache.npages;
    bad = __syncthreads_or(bad);
    const bool first = p0 == 0 && h == 0;
    if (first) {
        if (bad && tid == 0) flag_status(a.status, kStatusDevice);
        if (tid == 0) {
            a.nchunks_out[b] = bad ? n : (int)(n + closes);
            a.pos_out[b] = bad ? pos : (int)((pos + (long long)len) - closes * a.S);
        }
        if (range)
            for (int t = t0 + tid; t < t1; t += kThreads) a.mem_count[t] = bad ? -1 : (int)(n + ((long long)pos + (t - t0)) / a.S);
    }
    const size_t bh = (size_t)b * a.H + h;
    if (bad || len == 0) {   // the sequence stays as it is
        if (a.state_out != a.state || a.cur_out != a.cur)
            for (int r = 0; r < RPT; ++r) {
                const size_t at = (bh * N + n0 + r) * P + p0 + col;
                a.state_out[at] = a.state[at];
                a.cur_out[at] = a.cur[at];
            }
        return;
    }

    float H[RPT], D[RPT];
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        const size_t at = (bh * N + n0 + r) * P + p0 + col;
        H[r] = a.state[at];
        D[r] = a.cur[at];
    }
    const float Ah = a.A[h];
    const int grp = group_of(h, a.H, a.G);
    int slot = n, left = a.S - pos;        // tokens up to the end of the chunk
    for (int base = t0; base < t1; base += kTile) {
        const int m = min(kTile, t1 - base);
        __syncthreads();
        for (int i = tid; i < m * N; i += kThreads) {
            const size_t at = ((size_t)(base + i / N) * a.G + grp) * N + i % N;
            Bs[i / N][i % N] = ldf(static_cast<const T*>(a.Bm) + at);
            Cs[i / N][i % N] = ldf(static_cast<const T*>(a.Cm) + at);
        }
        for (int i = tid; i < m * PS; i += kThreads)
            xs[i / PS][i % PS] = ldf(static_cast<const T*>(a.x) + ((size_t)(base + i / PS) * a.H + h) * P + p0 + i % PS);
        if (tid < m) {
            const float dt = a.dt[(size_t)(base + tid) * a.H + h];
            dts[tid] = dt;
            as[tid] = expf(dt * Ah);
        }
        __syncthreads();
        for (int i = 0; i < m; ++i) {
            const float dx = dts[i] * xs[i][col], al = as[i];
            float y = 0.f;
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
                const float in = Bs[i][n0 + r] * dx;
                H[r] = fmaf(al, H[r], in);
                D[r] = fmaf(al, D[r], in);
                y = fmaf(Cs[i][n0 + r], H[r], y);
            }
            ys[i][rg][col] = y;
            if (--left == 0) {             // the chunk closes: D is its memory
                const size_t mem = memory_index(a.cache, a.H, row[slot / R], h, slot % R);
                if (!a.cache.mxfp4) {
                    T* dst = static_cast<T*>(a.cache.pages) + mem * (size_t)(N * P);
#pragma unroll
                    for (int r = 0; r < RPT; ++r) dst[(size_t)(n0 + r) * P + p0 + col] = Elem<T>::from_f(D[r]);
                } else if constexpr (N % 32 == 0 && PS * (N / 32) <= kThreads) {
                    // the largest magnitude of each block of 32 rows, over the threads that share it
                    constexpr int BPT = RPT < 32 ? 1 : RPT / 32;       // blocks of a thread
                    constexpr int TPB = RPT < 32 ? 32 / RPT : 1;       // threads of a block
                    constexpr int RB = RPT < 32 ? RPT : 32;
                    uint8_t* codes = static_cast<uint8_t*>(a.cache.pages) + mem * (size_t)(N * P / 2);
                    uint8_t* scales = a.cache.scales + mem * (size_t)(N * P / 32);
#pragma unroll
                    for (int k = 0; k < BPT; ++k) {
                        float amax = 0.f;
#pragma unroll
                        for (int r = 0; r < RB; ++r) amax = fabsf(D[k * 32 + r]) <= amax ? amax : fabsf(D[k * 32 + r]);   // keeps a NaN
                        if (TPB > 1) {
                            amax_s[rg][col] = amax;
                            __syncthreads();
#pragma unroll
                            for (int o = 0; o < TPB; ++o) {
                                const float v = amax_s[rg / TPB * TPB + o][col];
                                amax = v <= amax ? amax : v;
                            }
                            __syncthreads();
                        }
                        const bool finite = amax < INFINITY;
                        const int e = mxfp4_exponent(finite ? amax : 0.f);
                        const float inv = mxfp4_pow2(-e);
#pragma unroll
                        for (int r = 0; r < RB; r += 4) {
                            unsigned w = 0;
#pragma unroll
                            for (int j = 0; j < 4; ++j) w |= mxfp4_code(D[k * 32 + r + j] * inv) << (4 * j);
                            const int nn = n0 + k * 32 + r;            // codes of rows nn .. nn + 3
                            *reinterpret_cast<uint16_t*>(codes + (size_t)(p0 + col) * (N / 2) + (nn % 16 / 4) * (N / 8) + 2 * (nn / 16)) =
                                (uint16_t)(finite ? w : 0u);
                        }
                        if ((n0 + k * 32) % 32 == 0) scales[(p0 + col) * (N / 32) + (n0 + k * 32) / 32] = (uint8_t)(finite ? e + 127 : 255);
                    }
                }
#pragma unroll
                for (int r = 0; r < RPT; ++r) D[r] = 0.f;
                left = a.S;
                ++slot;
            }
        }
        __syncthreads();
        for (int i = tid; i < m * PS; i += kThreads) {
            float y = 0.f;
#pragma unroll
            for (int g = 0; g < RG; ++g) y += ys[i / PS][g][i % PS];
            a.y[((size_t)(base + i / PS) * a.H + h) * P + p0 + i % PS] = y;
        }
    }
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        const size_t at = (bh * N + n0 + r) * P + p0 + col;
        a.state_out[at] = H[r];
        a.cur_out[at] = D[r];
    }
}

template <int N, int P, int PS, int kThreads>
cudaError_t run(const ExtendArgs& a, dart_dtype dt, cudaStream_t st) {
    const dim3 grid(P / PS, a.H, a.B);
    if (dt == DART_F32)
        ssd_extend_kernel<float, N, P, PS, kThreads><<<grid, kThreads, 0, st>>>(a);
    else
        ssd_extend_kernel<__nv_bfloat16, N, P, PS, kThreads><<<grid, kThreads, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace

cudaError_t launch_ssd_extend(const ExtendArgs& a, dart_dtype dt, cudaStream_t st) {
    if (a.N == 128 && a.P == 64) return run<128, 64, 32, 256>(a, dt, st);
    if (a.N == 64 && a.P == 64) return run<64, 64, 32, 256>(a, dt, st);
    if (a.N == 16 && a.P == 16) return run<16, 16, 16, 64>(a, dt, st);
    return cudaErrorInvalidValue;
}

}  // namespace dart
