// sma_paged.cu -- state-memory attention of packed new tokens over paged chunk
// memories, on CUDA cores: float32, and the shape (16, 16).
//
// Per token t, head h and visible memory M_c (N x P):
//   u = Q_t^T M_c,  v = C_t^T M_c,  s = u . E_t / sqrt(N),
//   o = sum_c softmax_c(s) v_c,  out = y_ssd + g o        (o = 0 with none visible).
//
// Every warp is a worker of its own, with its run of units and its ring of stages
// copied ahead over the ends of items (16 rows of a memory each, 32 where two fit:
// up to 400 memories in the case below took 90 us with 8 rows, 72 with 16, 62 with
// 32).  A lane has four columns of every second row, and a value is used for U and
// V of up to 8 tokens, whose Q and C stand in the warp's own shared memory.  What
// bounds runs of several tokens is the issue of multiply-adds and of the shared
// loads that feed them: two tokens of a column share one paired multiply-add, and
// four columns a lane halve the loads of Q and C (32 runs of up to 6 tokens over
// 131 memories, 32 heads: 888 us with two columns and single multiply-adds, 664 so,
// 590 with the cheaper wait of sma_paged.cuh, 540 with the softmax as below, 485 at
// a copy's rate; 64 single tokens 892 us, HBM).  A token's scores are summed into the
// lanes that own it, which alone run its softmax (online, base 2) and pass its two
// weights on (against a warp sum and a softmax in every lane for each token, 19 runs
// of up to 137 tokens over 48 memories of 16 x 16: 60 -> 42 us); v is folded into
// the lane's columns.  (With eight warps to a piece and loads straight from global
// memory, 7 runs of 5 float32 tokens over 45 memories of 8 heads took 32 us; this
// takes 24.)
#include "sm100.cuh"
#include "sma_paged.cuh"

#include <float.h>

namespace dart {
namespace {

using namespace sm100;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTT = 8;        // tokens of a tile
constexpr int kCap = 4096;    // tiles of a call
constexpr int kLeast = 1;     // units below which a run is not cut

using Tiles = TileList<kCap>;
struct Params { SmaPagedArgs a; };

template <typename T, int N, int P>
struct Dense {
    static constexpr int kRows = N == 64 ? 32 : 16, kStages = N == 64 ? 2 : N == 128 ? 3 : 4, kPieces = N / kRows;
    static constexpr uint32_t kStageBytes = kRows * P * sizeof(T);
    static __device__ __forceinline__ void copy(const Params& prm, size_t mem, int piece, uint32_t dst, uint32_t full) {
        bulk_load(dst, static_cast<const T*>(prm.a.cache.pages) + (mem * N + piece * kRows) * P, kStageBytes, full);
    }
};

template <typename M, int N>
struct Smem {
    alignas(16) uint8_t ring[kWarps][M::kStages][M::kStageBytes];
    alignas(16) float qc[kWarps][N][2 * kTT];      // Q (times log2(e) / sqrt(N)) and C of a tile's tokens
    uint64_t full[kWarps][M::kStages];
    int abort_flag;
    Tiles tiles;
};

// Two float32 values side by side, multiplied and added by one instruction.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float x, float y) {
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
    return p;
}
__device__ __forceinline__ void fma2(Pair& d, Pair a, Pair b) { asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b)); }
__device__ __forceinline__ float half_of(Pair p, int i) {
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
    return i ? hi : lo;
}

// U and V of a lane's four columns for NT tokens: a pair is two tokens of a
// column (their Q and C stand side by side), or two columns of a single token.
template <int NT>
struct Sums {
    static constexpr int kPairs = NT == 1 ? 2 : 2 * NT;
    Pair u[kPairs], v[kPairs];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) u[i] = v[i] = 0;
    }
    // adds x (four columns of one row) times that row's Q and C of the tokens at f
    __device__ __forceinline__ void add(const float4& x, const float* f) {
        if constexpr (NT == 1) {
            const Pair q = pair(f[0], f[0]), c = pair(f[kTT], f[kTT]), x01 = pair(x.x, x.y), x23 = pair(x.z, x.w);
            fma2(u[0], q, x01); fma2(u[1], q, x23);
            fma2(v[0], c, x01); fma2(v[1], c, x23);
        } else {
            const Pair xx[4] = {pair(x.x, x.x), pair(x.y, x.y), pair(x.z, x.z), pair(x.w, x.w)};
#pragma unroll
            for (int t = 0; t < NT; t += 4) {
                ulonglong2 q, c;
                if (t + 4 <= NT) {
                    q = *reinterpret_cast<const ulonglong2*>(f + t);
                    c = *reinterpret_cast<const ulonglong2*>(f + kTT + t);
                } else {
                    q.x = *reinterpret_cast<const Pair*>(f + t);
                    c.x = *reinterpret_cast<const Pair*>(f + kTT + t);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    fma2(u[2 * t + i], q.x, xx[i]);
                    fma2(v[2 * t + i], c.x, xx[i]);
                    if (t + 4 <= NT) {
                        fma2(u[2 * t + 4 + i], q.y, xx[i]);
                        fma2(v[2 * t + 4 + i], c.y, xx[i]);
                    }
                }
            }
        }
    }
    static __device__ __forceinline__ float at(const Pair* p, int t, int i) {
        return NT == 1 ? half_of(p[i / 2], i & 1) : half_of(p[t / 2 * 4 + i], t & 1);
    }
};

template <typename T>
__device__ __forceinline__ float4 four_of(const T* p) {
    if constexpr (sizeof(T) == 4) {
        return *reinterpret_cast<const float4*>(p);
    } else {
        const uint2 b = *reinterpret_cast<const uint2*>(p);
        return make_float4(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xffff0000u), __uint_as_float(b.y << 16), __uint_as_float(b.y & 0xffff0000u));
    }
}

// Sums of W values over the warp, the sum of p[lane >> (5 - log2 W)] to each lane:
// a lane keeps half of its values and passes the other half on while it has
// several, so 8 sums take 9 shuffles and not 40.
template <int W>
__device__ __forceinline__ float sum_to_owner(float (&p)[W], int lane) {
    int off = 16;
#pragma unroll
    for (int half = W / 2; half >= 1; half /= 2, off /= 2)
#pragma unroll
        for (int j = 0; j < half; ++j) {
            const bool up = lane & off;
            const float got = __shfl_xor_sync(0xffffffffu, up ? p[j] : p[j + half], off);
            p[j] = (up ? p[j + half] : p[j]) + got;
        }
#pragma unroll
    for (; off >= 1; off /= 2) p[0] += __shfl_xor_sync(0xffffffffu, p[0], off);
    return p[0];
}

// A piece of a run for the first NT tokens of the tile.
template <typename T, int N, int P, int NT, typename M>
__device__ __forceinline__ void run_piece(const Params& prm, Smem<M, N>& s, const Walk& w, int run, int t0, int rows,
                                          Feed<M, Tiles>& feed, int& taken, const WaitCtx& wc, bool& ok) {
    constexpr int LPR = P / 4, RPW = 32 / LPR;      // lanes of a row, rows of the warp at a time
    const SmaPagedArgs& a = prm.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, grp = group_of(w.h, a.H, a.G);
    const float qscale = kLog2e * rsqrtf((float)N);
    float(*qc)[2 * kTT] = s.qc[warp];
    // the softmax of a token belongs to the lanes that its sums end in: lane >> kShift is their token
    constexpr int W = NT == 6 ? 8 : NT, kShift = W == 1 ? 5 : W == 2 ? 4 : W == 4 ? 3 : 2;
    const int mine = lane >> kShift, count = mine < rows ? a.mem_count[t0 + mine] : -1;
    float4 e[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const bool live = t < rows;
        const size_t tok = (size_t)(t0 + t);
        e[t] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (live) e[t] = four_of(static_cast<const T*>(a.E) + (tok * a.H + w.h) * P + 4 * (lane % LPR));
#pragma unroll
        for (int n = lane; n < N; n += 32) {
            qc[n][t] = live ? qscale * ldf(static_cast<const T*>(a.Q) + (tok * a.H + w.h) * N + n) : 0.f;
            qc[n][kTT + t] = live ? ldf(static_cast<const T*>(a.Cm) + (tok * a.G + grp) * N + n) : 0.f;
        }
    }
    const int bad = readable_memories(a.cache.table + (size_t)s.tiles.seq(w.k) * a.cache.width, a.cache, w.first_memory(), w.last_memory());
    __syncwarp();
    float m = -FLT_MAX, l = 0.f, o[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
    const int last = min(w.last_memory(), bad);
    for (int c = w.first_memory(); c < last; ++c) {
        Sums<NT> sums;
        sums.clear();
#pragma unroll 1
        for (int k = 0; k < M::kPieces; ++k) {
            const int st = taken % M::kStages;
            if (ok) ok = wait_warp(smem_u32(&s.full[warp][st]), (uint32_t)(taken / M::kStages) & 1u, wc, 1);
            ++taken;
            if (!ok) continue;
            const T* rows_s = reinterpret_cast<const T*>(s.ring[warp][st]) + (lane / LPR) * P + 4 * (lane % LPR);
#pragma unroll
            for (int r = 0; r < M::kRows / RPW; ++r) sums.add(four_of(rows_s + r * RPW * P), qc[k * M::kRows + r * RPW + lane / LPR]);
            __syncwarp();        // every lane has read the stage
            feed.fill(prm, s.tiles, s.ring[warp], s.full[warp]);
        }
        float p[W];
#pragma unroll
        for (int t = 0; t < W; ++t) {
            if (t < NT) {
                const float u0 = sums.at(sums.u, t, 0), u1 = sums.at(sums.u, t, 1), u2 = sums.at(sums.u, t, 2), u3 = sums.at(sums.u, t, 3);
                p[t] = fmaf(u0, e[t].x, u1 * e[t].y) + fmaf(u2, e[t].z, u3 * e[t].w);
            } else {
                p[t] = 0.f;
            }
        }
        const float sc = sum_to_owner<W>(p, lane);
        float al = 1.f, wt = 0.f;
        if (c < count) {                              // the row sees this memory
            const float mn = fmaxf(m, sc);
            al = exp2f(m - mn);
            wt = exp2f(sc - mn);
            l = fmaf(l, al, wt);
            m = mn;
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float at = __shfl_sync(0xffffffffu, al, t << kShift), wtt = __shfl_sync(0xffffffffu, wt, t << kShift);
            if (wtt != 0.f) {                         // 0 weight reads nothing, whatever the value is
#pragma unroll
                for (int i = 0; i < 4; ++i) o[t][i] = fmaf(o[t][i], at, wtt * sums.at(sums.v, t, i));
            }
        }
    }
    // a whole item is written out, a part of one kept for the combine kernel
    const int which = w.c > 0 ? 0 : 1;
    if (!w.whole() && lane == 0) *piece_header(a.part, run, which) = PieceHeader{w.last == w.units ? 2 : 1, t0, rows, w.h};
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        // a lane's o holds the rows it read: sum over the lanes of the same columns
#pragma unroll
        for (int off = LPR; off < 32; off <<= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[t][i] += __shfl_xor_sync(0xffffffffu, o[t][i], off);
        const float lt = __shfl_sync(0xffffffffu, l, t << kShift), mt = __shfl_sync(0xffffffffu, m, t << kShift);
        const int ct = __shfl_sync(0xffffffffu, count, t << kShift);
        if (t >= rows || lane >= LPR) continue;
        const bool left = ct < 0 || ct > bad;      // a row that is not to be computed
        if (w.whole()) {
            if (left) continue;
            const size_t at = ((size_t)(t0 + t) * a.H + w.h) * P + 4 * lane;
            const float f = lt == 0.f ? 0.f : (a.y_ssd ? a.g : 1.f) / lt;
            const float4 y = a.y_ssd ? *reinterpret_cast<const float4*>(a.y_ssd + at) : make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4*>(a.out + at) = make_float4(fmaf(f, o[t][0], y.x), fmaf(f, o[t][1], y.y), fmaf(f, o[t][2], y.z), fmaf(f, o[t][3], y.w));
        } else {
            float* row = piece_rows<kTT, P>(a.part, run, which) + t * (P + 4);
            *reinterpret_cast<float4*>(row + 4 * lane) = make_float4(o[t][0], o[t][1], o[t][2], o[t][3]);
            if (lane == 0) { row[P] = mt; row[P + 1] = left ? -1.f : lt; }
        }
    }
    __syncwarp();        // qc is read no more
}

template <typename T, int N, int P>
__global__ void __launch_bounds__(kThreads, 1) sma_paged_kernel(const __grid_constant__ Params prm) {
    using M = Dense<T, N, P>;
    extern __shared__ __align__(128) uint8_t raw[];
    Smem<M, N>& s = *reinterpret_cast<Smem<M, N>*>(raw);
    const SmaPagedArgs& a = prm.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < kWarps * M::kStages; ++i) mbar_init(smem_u32(&s.full[0][0] + i), 1);
        s.abort_flag = 0;
        fence_mbar_init();
    }
    // neighbours in the order of units go to different blocks: a few units spread over all of them
    const int runs = gridDim.x * kWarps, run = warp * gridDim.x + blockIdx.x;
    griddep_wait();
    if (lane < 2) piece_header(a.part, run, lane)->state = 0;
    __syncwarp();
    build_tiles<kTT>(a, s.tiles);
    if (s.tiles.n == 0) return;
    const WaitCtx wc{&s.abort_flag, a.status, 12};
    bool ok = true;
    int taken = 0;
    Walk w = start_walk(s.tiles, a.H, run, runs, kLeast);
    Feed<M, Tiles> feed;
    feed.begin(a, s.tiles, w);
    for (int i = 0; i < M::kStages; ++i) feed.fill(prm, s.tiles, s.ring[warp], s.full[warp]);
    for (; next_piece(w); advance(s.tiles, w, a.H)) {
        const int t0 = s.tiles.t0[w.k], rows = s.tiles.rows(w.k);
        if (rows == 1) run_piece<T, N, P, 1>(prm, s, w, run, t0, rows, feed, taken, wc, ok);
        else if (rows == 2) run_piece<T, N, P, 2>(prm, s, w, run, t0, rows, feed, taken, wc, ok);
        else if (rows <= 4) run_piece<T, N, P, 4>(prm, s, w, run, t0, rows, feed, taken, wc, ok);
        else if (rows <= 6) run_piece<T, N, P, 6>(prm, s, w, run, t0, rows, feed, taken, wc, ok);
        else run_piece<T, N, P, 8>(prm, s, w, run, t0, rows, feed, taken, wc, ok);
    }
    if (!ok) feed.drain(s.full[warp]);      // else every copy has been waited for
}

// Block (i, y) joins ROWS rows, from row ROWS y on, of the item that begins in
// run i and ends in a later one (most blocks find none and leave).  A thread has four columns of one row,
// and where there are fewer rows than threads for them, every n-th of the item's
// pieces: an item of one row may be spread over all runs, and many read it then.
template <int TT, int P, int ROWS>
__global__ void __launch_bounds__(ROWS * P / 4, TT >= 128 ? 4 : 1) sma_paged_combine_kernel(SmaPagedArgs a, int runs) {
    constexpr int COLS = P / 4, SUB = ROWS;                  // threads of a row, of a column
    // Pieces read at a time (8 where an item may have dozens: 29 us for the float32 case, 32 with 4).  An item of a
    // large tile has few, and all blocks of its rows fit the machine at once with 32
    // registers a thread (one block an SM and four rounds of them took 12 us behind the prompt pieces)
    constexpr int AHEAD = TT >= 128 ? 1 : 8;
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
    bool left = false;                        // a row that is not to be computed, as some piece says
    auto add = [&](float m2, float l2, const float4& o2) {
        left |= l2 < 0.f;
        if (l2 == 0.f) return;                // saw nothing
        const float mn = fmaxf(m, m2);
        const float f = l == 0.f ? 0.f : exp2f(m - mn), k = exp2f(m2 - mn);
        l = fmaf(l, f, l2 * k);
        o = f == 0.f ? make_float4(o2.x * k, o2.y * k, o2.z * k, o2.w * k)
                     : make_float4(o.x * f + o2.x * k, o.y * f + o2.y * k, o.z * f + o2.z * k, o.w * f + o2.w * k);
        m = mn;
    };
    const size_t at = ((size_t)(hd.t0 + r0 + t) * a.H + hd.h) * P + p;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t < rows) {
        const size_t off = (size_t)(r0 + t) * (P + 4);
        const float* own = piece_rows<TT, P>(a.part, blockIdx.x, 1) + off;
        if (grp == 0 && a.y_ssd) y = *reinterpret_cast<const float4*>(a.y_ssd + at);
        if (grp == 0) add(own[P], own[P + 1], *reinterpret_cast<const float4*>(own + p));
        for (int j = blockIdx.x + 1 + grp; j <= end && j < runs; j += AHEAD * groups) {
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
        if (p == 0) { sm[sub] = m; sl[sub] = left ? -1.f : l; }
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
    constexpr int smem = (int)sizeof(Smem<Dense<T, N, P>, N>);
    static_assert(smem <= 232448, "shared memory");
    const int sms = paged_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    static std::atomic<unsigned long long> ready{0};   // devices whose kernel has its shared memory allowed
    cudaError_t e = paged_allow_smem(reinterpret_cast<const void*>(kern), smem, ready);
    if (e != cudaSuccess) return e;
    const int blocks = min(sms, kMaxRuns / kWarps);
    if ((e = launch_dependent(kern, dim3(blocks), dim3(kThreads), smem, st, 1, Params{a})) != cudaSuccess) return e;
    count_launches(1);
    return launch_sma_paged_combine(a, blocks * kWarps, kTT, st);
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
