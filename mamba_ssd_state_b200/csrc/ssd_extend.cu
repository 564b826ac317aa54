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
// short runs (64 sequences of one token, 32 heads: 269 MB in 44 us, 93% of measured
// HBM).  The loads of the state go out before the run is looked at, with
// streaming hints (3 us less).  A thread owns four columns and RPT rows: 8 rows
// give it sixteen wide loads in flight, and 128 registers for them (512 threads
// an SM) measured 44 us where 4 rows of twice the threads took 47, five blocks an
// SM 46 and six 52, and slices of 16 columns 50.  Partial sums of y meet over a
// warp's rows by shuffles and over the warps in shared memory, once for every
// kTile tokens.  Long runs of bfloat16 tokens are bound by the 4 N P operations a
// token instead and go to ssd_extend_mma.cu.
#include "dart_paged.cuh"
#include "sm100.cuh"

namespace dart {
namespace {

constexpr int kTile = 8;   // tokens staged in shared memory at a time

template <typename T, int N, int P, int PS, int RPT, bool kMany>
__global__ void __launch_bounds__(PS / 4 * N / RPT, 512 / (PS / 4 * N / RPT)) ssd_extend_kernel(ExtendArgs a) {
    constexpr int CT = PS / 4, kThreads = CT * (N / RPT);   // threads across the columns, of the block
    constexpr int WARPS = kThreads / 32;
    static_assert(kThreads % 32 == 0 && 32 % CT == 0, "whole warps of whole rows");
    const int p0 = blockIdx.x * PS, h = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, col = 4 * (tid % CT), n0 = tid / CT * RPT;
    __shared__ __align__(16) float Bs[kTile][N], Cs[kTile][N], xs[kTile][PS];
    __shared__ float dts[kTile], as[kTile];
    __shared__ __align__(16) float ys[kTile][WARPS][PS], ds[N * PS];
    sm100::griddep_wait();
    const EarlierEntries<kMany> earlier(a, b);
    const size_t bh = (size_t)b * a.H + h, at = (bh * N + n0) * P + p0 + col;
    float H[RPT][4], D[RPT][4];
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        const float4 u = __ldcs(reinterpret_cast<const float4*>(a.state + at + r * P)), v = __ldcs(reinterpret_cast<const float4*>(a.cur + at + r * P));
        H[r][0] = u.x; H[r][1] = u.y; H[r][2] = u.z; H[r][3] = u.w;
        D[r][0] = v.x; D[r][1] = v.y; D[r][2] = v.z; D[r][3] = v.w;
    }
    const ExtendPlan plan = plan_extend(a, b, p0 == 0 && h == 0, earlier);
    if (plan.len == 0 && a.state_out == a.state && a.cur_out == a.cur) return;   // the sequence stays as it is
    const float Ah = a.A[h];
    const int grp = group_of(h, a.H, a.G), t1 = plan.t0 + plan.len;
    int slot = plan.n, left = a.S - plan.pos;        // tokens up to the end of the chunk
    for (int base = plan.t0; base < t1; base += kTile) {
        const int m = min(kTile, t1 - base);
        __syncthreads();
        for (int i = tid; i < m * N; i += kThreads) {
            const size_t e = ((size_t)(base + i / N) * a.G + grp) * N + i % N;
            Bs[i / N][i % N] = ldf(static_cast<const T*>(a.Bm) + e);
            Cs[i / N][i % N] = ldf(static_cast<const T*>(a.Cm) + e);
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
            const float4 x4 = *reinterpret_cast<const float4*>(&xs[i][col]);
            const float dt = dts[i], al = as[i];
            const float dx[4] = {dt * x4.x, dt * x4.y, dt * x4.z, dt * x4.w};
            float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
                const float bn = Bs[i][n0 + r], cn = Cs[i][n0 + r];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float in = bn * dx[c];
                    H[r][c] = fmaf(al, H[r][c], in);
                    D[r][c] = fmaf(al, D[r][c], in);
                    y[c] = fmaf(cn, H[r][c], y[c]);
                }
            }
#pragma unroll
            for (int o = CT; o < 32; o <<= 1)
#pragma unroll
                for (int c = 0; c < 4; ++c) y[c] += __shfl_xor_sync(0xffffffffu, y[c], o);
            if (lane < CT) *reinterpret_cast<float4*>(&ys[i][warp][col]) = make_float4(y[0], y[1], y[2], y[3]);
            if (--left == 0) {             // the chunk closes: D is its memory
                __syncthreads();           // the last one has left ds
#pragma unroll
                for (int r = 0; r < RPT; ++r) {
                    *reinterpret_cast<float4*>(&ds[(n0 + r) * PS + col]) = make_float4(D[r][0], D[r][1], D[r][2], D[r][3]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) D[r][c] = 0.f;
                }
                __syncthreads();
                append_memory<T, N, P, PS>(a, b, h, slot, p0, ds, tid, kThreads);
                left = a.S;
                ++slot;
            }
        }
        __syncthreads();
        for (int i = tid; i < m * PS; i += kThreads) {
            float y = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) y += ys[i / PS][w][i % PS];
            a.y[((size_t)(base + i / PS) * a.H + h) * P + p0 + i % PS] = y;
        }
    }
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        __stcs(reinterpret_cast<float4*>(a.state_out + at + r * P), make_float4(H[r][0], H[r][1], H[r][2], H[r][3]));
        __stcs(reinterpret_cast<float4*>(a.cur_out + at + r * P), make_float4(D[r][0], D[r][1], D[r][2], D[r][3]));
    }
}

template <typename T, int N, int P, int PS, int RPT>
cudaError_t run(const ExtendArgs& a, cudaStream_t st) {
    constexpr int threads = PS / 4 * N / RPT;
    const bool many = a.B > EarlierEntries<true>::kEach * threads;
    auto kern = many ? ssd_extend_kernel<T, N, P, PS, RPT, true> : ssd_extend_kernel<T, N, P, PS, RPT, false>;
    const cudaError_t e = launch_dependent(kern, dim3(P / PS, a.H, a.B), dim3(threads), 0, st, 1, a);
    if (e == cudaSuccess) count_launches(1);
    return e;
}
template <int N, int P, int PS, int RPT>
cudaError_t run(const ExtendArgs& a, dart_dtype dt, cudaStream_t st) {
    return dt == DART_F32 ? run<float, N, P, PS, RPT>(a, st) : run<__nv_bfloat16, N, P, PS, RPT>(a, st);
}

}  // namespace

cudaError_t launch_ssd_extend(const ExtendArgs& a, dart_dtype dt, cudaStream_t st) {
    if (ssd_extend_mma_applicable(a, dt)) return launch_ssd_extend_mma(a, st);
    if (a.N == 128 && a.P == 64) return run<128, 64, 32, 8>(a, dt, st);
    if (a.N == 64 && a.P == 64) return run<64, 64, 32, 8>(a, dt, st);
    if (a.N == 16 && a.P == 16) return run<16, 16, 16, 2>(a, dt, st);
    return cudaErrorInvalidValue;
}

}  // namespace dart
