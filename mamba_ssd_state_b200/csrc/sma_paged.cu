// sma_paged.cu -- state-memory attention of packed new tokens over paged chunk
// memories, on CUDA cores: float32, and the shape (16, 16).
//
// Per token t, head h and visible memory M_c (N x P):
//   u = Q_t^T M_c,  v = C_t^T M_c,  s = u . E_t / sqrt(N),
//   o = sum_c softmax_c(s) v_c,  out = y_ssd + g o        (o = 0 with none visible).
//
// A warp takes a memory at a time, a lane two of its columns: it streams the
// rows past up to 8 tokens held as pairs, so a value is loaded once for
// 2 x 8 products.  Scores are summed over the warp, the softmax runs online in
// base 2, and v is folded into the lane's own columns, so that the eight warps
// of a block meet only at the end of a piece.
#include "sm100.cuh"
#include "sma_paged.cuh"

namespace dart {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTT = 8;        // tokens of a tile
constexpr int kCap = 4096;    // tiles of a call
constexpr int kLeast = 8;     // units below which a run is not cut

template <int N, int P>
struct Smem {
    TileList<kCap> tiles;
    float qc[N][2 * kTT];              // Q (times log2(e) / sqrt(N)) and C of the tile's tokens
    float m[kWarps][kTT], l[kWarps][kTT];
    float o[kWarps][kTT][P];
    int count[kTT], bad;
};

// Rows of a memory as (n, two columns) for this lane, eight at a time.
template <typename T, int N, int P>
struct Rows {
    static constexpr int LPR = P / 2, RPW = 32 / LPR;      // lanes of a row, rows of a warp load
    static constexpr int STEPS = N / RPW, BATCH = STEPS < 8 ? STEPS : 8;
    const T* at;
    __device__ Rows(const PagedCache& c, size_t mem, int lane)
        : at(static_cast<const T*>(c.pages) + mem * (size_t)(N * P) + (lane / LPR) * P + 2 * (lane % LPR)) {}
    __device__ __forceinline__ static int row(int step, int lane) { return step * RPW + lane / LPR; }
    __device__ __forceinline__ void load(int step, float2 (&v)[BATCH]) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const T* p = at + (size_t)(step + i) * RPW * P;
            if constexpr (sizeof(T) == 4) {
                v[i] = __ldcs(reinterpret_cast<const float2*>(p));
            } else {
                const unsigned w = __ldcs(reinterpret_cast<const unsigned*>(p));
                v[i] = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
            }
        }
    }
};

// This warp's memories of a piece for the first NT tokens of the tile.
template <typename T, int N, int P, int NT>
__device__ __forceinline__ void run_piece(const SmaPagedArgs& a, Smem<N, P>& s, const Walk& w, const int* table, const float2 (&e)[kTT]) {
    using R = Rows<T, N, P>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float m[NT], l[NT];
    float2 o[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) { m[t] = -INFINITY; l[t] = 0.f; o[t] = make_float2(0.f, 0.f); }
    const int last = min(w.last_memory(), s.bad);
    for (int c = w.first_memory() + warp; c < last; c += kWarps) {
        R rows(a.cache, memory_index(a.cache, a.H, table[c / a.cache.R], w.h, c % a.cache.R), lane);
        float2 u[NT], v[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) u[t] = v[t] = make_float2(0.f, 0.f);
        for (int st = 0; st < R::STEPS; st += R::BATCH) {
            float2 x[R::BATCH];
            rows.load(st, x);
#pragma unroll
            for (int i = 0; i < R::BATCH; ++i) {
                const float* qc = s.qc[R::row(st + i, lane)];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    u[t].x = fmaf(qc[t], x[i].x, u[t].x);
                    u[t].y = fmaf(qc[t], x[i].y, u[t].y);
                    v[t].x = fmaf(qc[kTT + t], x[i].x, v[t].x);
                    v[t].y = fmaf(qc[kTT + t], x[i].y, v[t].y);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float sc = warp_sum(fmaf(u[t].x, e[t].x, u[t].y * e[t].y));
            if (c < s.count[t]) {                     // the row sees this memory (same for the whole warp)
                const float mn = fmaxf(m[t], sc);
                const bool none = mn == -INFINITY;    // only scores of -inf so far: they weigh nothing
                const float al = none ? 1.f : exp2f(m[t] - mn), wt = none ? (sc == sc ? 0.f : sc) : exp2f(sc - mn);
                l[t] = fmaf(l[t], al, wt);
                m[t] = mn;
                if (wt != 0.f) {                      // 0 weight reads nothing, whatever the value is
                    o[t].x = fmaf(o[t].x, al, wt * v[t].x);
                    o[t].y = fmaf(o[t].y, al, wt * v[t].y);
                }
            }
        }
    }
    // a lane's o holds the rows it read: sum over the lanes of the same columns
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int off = P / 2; off < 32; off <<= 1) {
            o[t].x += __shfl_xor_sync(0xffffffffu, o[t].x, off);
            o[t].y += __shfl_xor_sync(0xffffffffu, o[t].y, off);
        }
        if (lane < P / 2) *reinterpret_cast<float2*>(&s.o[warp][t][2 * lane]) = o[t];
        if (lane == 0) { s.m[warp][t] = m[t]; s.l[warp][t] = l[t]; }
    }
}

template <typename T, int N, int P>
__global__ void __launch_bounds__(kThreads) sma_paged_kernel(SmaPagedArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    Smem<N, P>& s = *reinterpret_cast<Smem<N, P>*>(raw);
    const int tid = threadIdx.x, lane = tid & 31;
    build_tiles<kTT, kCap>(a, s.tiles);
    if (tid < 2) piece_header(a.part, blockIdx.x, tid)->state = 0;
    if (s.tiles.n == 0) return;
    const float qscale = kLog2e * rsqrtf((float)N);
    __syncthreads();
    for (Walk w = start_walk(s.tiles, a.H, blockIdx.x, gridDim.x, kLeast); next_piece(w); advance(s.tiles, w, a.H)) {
        const int b = s.tiles.seq[w.k], t0 = s.tiles.t0[w.k], rows = tile_rows(a.cu, b, t0, kTT);
        const int* table = a.cache.table + (size_t)b * a.cache.width;
        __syncthreads();
        const int grp = group_of(w.h, a.H, a.G);
        for (int i = tid; i < kTT * N; i += kThreads) {
            const int t = i / N, n = i % N;
            const bool live = t < rows;
            s.qc[n][t] = live ? qscale * ldf(static_cast<const T*>(a.Q) + ((size_t)(t0 + t) * a.H + w.h) * N + n) : 0.f;
            s.qc[n][kTT + t] = live ? ldf(static_cast<const T*>(a.Cm) + ((size_t)(t0 + t) * a.G + grp) * N + n) : 0.f;
        }
        if (tid < kTT) s.count[tid] = tid < rows ? a.mem_count[t0 + tid] : -1;
        if (tid < 32) {
            const int seen = w.memories();     // the most that a row of the tile sees
            const int bad = first_bad_memory(table, a.cache, seen);
            if (lane == 0) {
                s.bad = bad;
                if (bad < seen) flag_status(a.status, kStatusDevice);
            }
        }
        float2 e[kTT];
#pragma unroll
        for (int t = 0; t < kTT; ++t) {
            e[t] = make_float2(0.f, 0.f);
            if (t < rows) {
                const T* src = static_cast<const T*>(a.E) + ((size_t)(t0 + t) * a.H + w.h) * P + 2 * (lane % (P / 2));
                e[t] = make_float2(ldf(src), ldf(src + 1));
            }
        }
        __syncthreads();
        if (rows == 1) run_piece<T, N, P, 1>(a, s, w, table, e);
        else if (rows <= 4) run_piece<T, N, P, 4>(a, s, w, table, e);
        else run_piece<T, N, P, 8>(a, s, w, table, e);
        __syncthreads();
        // join the warps: a whole item is written out, a part of one kept for the combine kernel
        const int which = w.c > 0 ? 0 : 1;
        if (!w.whole() && tid == 0)
            *piece_header(a.part, blockIdx.x, which) = PieceHeader{w.last == w.units ? 2 : 1, t0, rows, w.h};
        for (int i = tid; i < rows * P; i += kThreads) {
            const int t = i / P, p = i % P;
            float mm = -INFINITY, l = 0.f, o = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) mm = fmaxf(mm, s.m[k][t]);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float f = s.l[k][t] == 0.f ? 0.f : exp2f(s.m[k][t] - mm);
                l = fmaf(s.l[k][t], f, l);
                if (f != 0.f) o = fmaf(s.o[k][t][p], f, o);
            }
            const bool left = s.count[t] < 0 || s.count[t] > s.bad;   // a row that is not to be computed
            if (w.whole()) {
                if (left) continue;
                const size_t at = ((size_t)(t0 + t) * a.H + w.h) * P + p;
                const float r = l == 0.f ? 0.f : o / l;
                a.out[at] = a.y_ssd ? fmaf(a.g, r, a.y_ssd[at]) : r;
            } else {
                float* row = piece_rows<kTT, P>(a.part, blockIdx.x, which) + t * (P + 4);
                if (p == 0) { row[P] = mm; row[P + 1] = left ? -1.f : l; }
                row[p] = o;
            }
        }
    }
}

// Block (i, y) joins ROWS rows, from row ROWS y on, of the item that begins in
// run i and ends in a later one (most blocks find none and leave).  A thread has four columns of one row,
// and where there are fewer rows than threads for them, every n-th of the item's
// pieces: an item of one row may be spread over all runs, and many read it then.
template <int TT, int P, int ROWS>
__global__ void __launch_bounds__(ROWS * P / 4) sma_paged_combine_kernel(SmaPagedArgs a, int runs) {
    constexpr int COLS = P / 4, SUB = ROWS;                  // threads of a row, of a column
    constexpr int AHEAD = 4;                                 // pieces read at a time
    sm100::griddep_wait();
    const PieceHeader hd = *piece_header(a.part, blockIdx.x, 1);
    const int r0 = ROWS * blockIdx.y, rows = min(ROWS, hd.rows - r0);
    if (hd.state != 1 || rows <= 0) return;
    const int lane = threadIdx.x & 31;
    int end = runs;                           // the run that has the item's last piece
    for (int j = blockIdx.x + 1; j < runs && end == runs; j += 32) {
        const unsigned hit = __ballot_sync(0xffffffffu, j + lane < runs && piece_header(a.part, j + lane, 0)->state == 2);
        if (hit) end = j + __ffs(hit) - 1;
    }
    int rp = 1;                               // rows as a power of two
    while (rp < rows) rp *= 2;
    const int groups = SUB / rp, p = 4 * (threadIdx.x % COLS), sub = threadIdx.x / COLS, t = sub % rp, grp = sub / rp;
    __shared__ float sm[SUB], sl[SUB];
    __shared__ float4 so[SUB][COLS];
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float m2, float l2, const float4& o2) {
        if (l2 == 0.f) return;                // saw nothing
        const float mn = fmaxf(m, m2);
        const float f = l == 0.f ? 0.f : exp2f(m - mn), k = exp2f(m2 - mn);
        l = fmaf(l, f, l2 * k);
        o = f == 0.f ? make_float4(o2.x * k, o2.y * k, o2.z * k, o2.w * k)
                     : make_float4(o.x * f + o2.x * k, o.y * f + o2.y * k, o.z * f + o2.z * k, o.w * f + o2.w * k);
        m = mn;
    };
    bool left = false;
    const size_t at = ((size_t)(hd.t0 + r0 + t) * a.H + hd.h) * P + p;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t < rows) {
        const size_t off = (size_t)(r0 + t) * (P + 4);
        const float* own = piece_rows<TT, P>(a.part, blockIdx.x, 1) + off;
        if (grp == 0 && a.y_ssd) y = *reinterpret_cast<const float4*>(a.y_ssd + at);
        left = own[P + 1] < 0.f;              // a row that is not to be computed
        if (grp == 0 && !left) add(own[P], own[P + 1], *reinterpret_cast<const float4*>(own + p));
        for (int j = blockIdx.x + 1 + grp; j <= end && j < runs && !left; j += AHEAD * groups) {
            float m2[AHEAD], l2[AHEAD];
            float4 o2[AHEAD];
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const int k = j + u * groups;
                l2[u] = 0.f;
                if (k <= end && k < runs && piece_header(a.part, k, 0)->state != 0) {
                    const float* r = piece_rows<TT, P>(a.part, k, 0) + off;
                    m2[u] = r[P];
                    l2[u] = r[P + 1];
                    o2[u] = *reinterpret_cast<const float4*>(r + p);
                }
            }
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) add(m2[u], l2[u], o2[u]);
        }
    }
    if (groups > 1) {
        if (p == 0) { sm[sub] = m; sl[sub] = l; }
        so[sub][p / 4] = o;
        __syncthreads();
        if (grp == 0)
            for (int k = 1; k < groups; ++k) add(sm[sub + k * rp], sl[sub + k * rp], so[sub + k * rp][p / 4]);
    }
    if (grp != 0 || t >= rows || left) return;
    const float f = l == 0.f ? 0.f : (a.y_ssd ? a.g : 1.f) / l;
    *reinterpret_cast<float4*>(a.out + at) = make_float4(fmaf(f, o.x, y.x), fmaf(f, o.y, y.y), fmaf(f, o.z, y.z), fmaf(f, o.w, y.w));
}

template <typename T, int N, int P>
cudaError_t run(const SmaPagedArgs& a, cudaStream_t st) {
    auto kern = sma_paged_kernel<T, N, P>;
    const int smem = (int)sizeof(Smem<N, P>), sms = paged_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    static std::atomic<unsigned long long> ready{0};   // devices whose kernel has its shared memory allowed
    cudaError_t e = paged_allow_smem(reinterpret_cast<const void*>(kern), smem, ready);
    if (e != cudaSuccess) return e;
    const int blocks = min(2 * sms, kMaxRuns);
    kern<<<blocks, kThreads, smem, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    count_launches(1);
    return launch_sma_paged_combine(a, blocks, kTT, st);
}

}  // namespace

int paged_sm_count() {
    static std::atomic<int> cache[64];   // threads that race on the first lookup store the same value
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

cudaError_t paged_allow_smem(const void* kernel, int bytes, std::atomic<unsigned long long>& ready) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (ready.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

cudaError_t launch_sma_paged_combine(const SmaPagedArgs& a, int runs, int tt, cudaStream_t st) {
    const int rows = tt < 32 ? 8 : 32;
    auto kern = a.P != 64 ? sma_paged_combine_kernel<8, 16, 8> : tt == 4 ? sma_paged_combine_kernel<4, 64, 8>
                : tt == 8 ? sma_paged_combine_kernel<8, 64, 8>
                : tt == 128 ? sma_paged_combine_kernel<128, 64, 32> : sma_paged_combine_kernel<256, 64, 32>;
    const cudaError_t e = launch_dependent(kern, dim3(runs, (tt + rows - 1) / rows), dim3(rows * a.P / 4), 0, st, 1, a, runs);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

size_t sma_paged_workspace_bytes(int P) {
    static_assert(kMaxTcRuns * 128 >= kMaxRuns * kTT, "rows of the pieces");
    return 2 * (kMaxRuns * sizeof(PieceHeader) + kMaxTcRuns * 128 * sizeof(float) * ((size_t)P + 4));
}
long long sma_paged_tiles(int B, int T) { return B + (long long)T / 4; }   // of 4 rows, the smallest tiles
long long sma_paged_max_tiles() { return kCap; }

cudaError_t launch_sma_paged(const SmaPagedArgs& a, dart_dtype dt, cudaStream_t st) {
    if (sma_paged_tc_applicable(a, dt)) return launch_sma_paged_tc(a, st);
    if (a.P == 64 && (a.cache.mxfp4 || dt == DART_BF16)) return launch_sma_paged_mma(a, dt, st);
    if (a.N == 128 && a.P == 64 && dt == DART_F32) return run<float, 128, 64>(a, st);
    if (a.N == 64 && a.P == 64 && dt == DART_F32) return run<float, 64, 64>(a, st);
    if (a.N == 16 && a.P == 16) return dt == DART_F32 ? run<float, 16, 16>(a, st) : run<__nv_bfloat16, 16, 16>(a, st);
    return cudaErrorInvalidValue;
}

}  // namespace dart
