// sma_paged_tc.cu -- state-memory attention of long runs of new tokens (pieces of
// a prompt) over paged bfloat16 memories, on tcgen05.
//
// The formulas are sma_paged_mma.cu's; the shape is the prefill kernel's
// (sma_tc.cu): a tile of 128 rows of one (sequence, head) is the M of two MMAs a
// batch of four memories, U = Q_T M and V = C_T M (N = 4 P = 256, K = dstate),
// with the accumulators in TMEM (U in columns 0..255, V in 256..511).  Reading a
// memory once for 128 tokens instead of 8 makes the run compute-bound:
// 4 x 256 tokens over 100 memories took 470 us on warp-level products, where
// every 8 tokens stream all memories through the SM again, and take 79 here (93 with
// nothing in L2).
//
// What differs from prefill: memories come from pages, a tile ends with its
// sequence (rows behind it belong to others and are not written), every row has
// its own count, and items are cut into equal runs of units (sma_paged.cuh), so
// that a few long sequences fill the machine; an item that falls into several
// runs is joined by the combine kernel.
//
// CTA pairs (runs of more than 160 tokens on average): two CTAs of a cluster run
// the two halves of a 256-row tile as M = 256 MMAs (cta_group::2).  Each loads
// its own rows of Q and C and two memories of a batch, so an SM takes in half
// the bytes for each product and its ring holds twice the batches: with single
// CTAs the ring's latency bounds a batch (64 KB for every 2048 cycles of MMA is
// 9 TB/s over all SMs).  CTA 0 issues the MMAs and owns the barriers they wait
// on; the peer's copies complete on them and its epilogue arrives there.
//
// Roles (320 threads): warp 0 issues TMA, warp 1 the MMAs, warps 2-9 are four
// pairs, one for each TMEM lane quadrant (32 rows); a pair splits the 64 value
// columns, exchanges partial scores through shared memory and runs the same
// online softmax.
#include <string.h>

#include "sm100.cuh"
#include "sma_paged.cuh"
#include "tensor_map.h"

namespace dart {
namespace {

using namespace sm100;

constexpr int kP = 64;
constexpr int kRows = 128;         // rows of a CTA (MMA M, or half of it)
constexpr int kCB = 4;             // memories of a batch (MMA N = 256)
constexpr int kCap = 1024;         // tiles of a call
constexpr int kLeast = 8;          // units below which a run is not cut
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr uint32_t kPanel = kRows * 64 * 2;      // 128 rows x 64 bfloat16, one swizzle panel
constexpr uint32_t kTmemCols = 512, kColV = 256;
constexpr int kHalfP = kP / 2;

enum Bar { Q_FULL, Q_FREE, C_FULL, C_FREE, U_FULL, U_EMPTY, V_FULL, V_EMPTY, B_FULL0 };

template <int N, bool kPair>
struct Smem {
    static constexpr int kMem = kPair ? kCB / 2 : kCB;           // memories of a stage (this CTA's of a batch)
    static constexpr int kStages = 8 / kMem * 128 / N;           // 128 KB
    static constexpr uint32_t kMemBytes = N * kP * 2, kStageBytes = kMem * kMemBytes;
    uint8_t q[N / 64 * kPanel], c[N / 64 * kPanel];
    uint8_t ring[kStages * kStageBytes];
    float4 scores[2][2][kRows];                  // [batch parity][half][row]: partial scores of four memories
    uint64_t bars[B_FULL0 + 2 * kStages];
    uint32_t tmem;
    int abort_flag;
    TileList<kCap> tiles;
};

struct Params {
    CUtensorMap map_q, map_c;     // (N, H, T) and (N, G, T), boxes (64, 1, 128)
    CUtensorMap map_m;            // (P, rows of N), boxes of one memory
    SmaPagedArgs a;
};

// v[j] of lane i and v[i] of lane j change places.
__device__ __forceinline__ void transpose32(float* v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
        const bool up = (lane & s) != 0;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if ((i & s) == 0) {
                const float got = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + s], s);
                if (up) v[i] = got;
                else v[i + s] = got;
            }
    }
}

template <int N, bool kPair>
__global__ void __launch_bounds__(kThreads, 1) sma_paged_tc_kernel(const __grid_constant__ Params prm) {
    using S = Smem<N, kPair>;
    constexpr int TT = kPair ? 2 * kRows : kRows;
    extern __shared__ uint8_t raw[];
    S& s = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const SmaPagedArgs& a = prm.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = kPair ? (int)cluster_ctarank() : 0;
    const int run = kPair ? (int)blockIdx.x / 2 : (int)blockIdx.x, runs = kPair ? (int)gridDim.x / 2 : (int)gridDim.x;
    auto bar = [&](int i) { return smem_u32(&s.bars[i]); };
    auto full = [&](int st) { return bar(B_FULL0 + st); };
    auto empty = [&](int st) { return bar(B_FULL0 + S::kStages + st); };
    auto lead = [&](uint32_t b) { return kPair ? mapa_shared(b, 0) : b; };      // the barrier in CTA 0
    if (tid == 0) {
        for (int i = 0; i < B_FULL0 + 2 * S::kStages; ++i) mbar_init(bar(i), i == U_EMPTY || i == V_EMPTY ? kEpiWarps * (kPair ? 2 : 1) : 1);
        s.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        if constexpr (kPair) {
            tmem_alloc_pair(smem_u32(&s.tmem), kTmemCols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_u32(&s.tmem), kTmemCols);
            tmem_relinquish();
        }
    }
    griddep_wait();
    if (tid < 2 && rank == 0) piece_header(a.part, run, tid)->state = 0;
    build_tiles<TT>(a, s.tiles);
    tc_fence_before();
    if (kPair) cluster_sync();                   // both CTAs' barriers exist before any remote arrive or copy
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    const WaitCtx wc{&s.abort_flag, a.status, 11};
    bool ok = true;
    Walk w;
    w.u = w.end = 0;
    if (s.tiles.n > 0) w = start_walk(s.tiles, a.H, run, runs, kLeast);
    auto table_of = [&]() { return a.cache.table + (size_t)s.tiles.seq(w.k) * a.cache.width; };
    if (warp == 0) {
        // ------------------------------------------------------------ TMA
        // the rows that the epilogue starts and ends with, while it is still at the last piece
        auto prefetch_rows = [&]() {
            const int t0 = s.tiles.t0[w.k], rows = s.tiles.rows(w.k);
#pragma unroll
            for (int r = rank * kRows + lane; r < (rank + 1) * kRows; r += 32)
                if (r < rows) {
                    const size_t at = ((size_t)(t0 + r) * a.H + w.h) * kP;
                    prefetch_l2(static_cast<const __nv_bfloat16*>(a.E) + at);
                    if (a.y_ssd && w.whole()) {
                        prefetch_l2(a.y_ssd + at);
                        prefetch_l2(a.y_ssd + at + kP / 2);
                    }
                }
        };
        uint32_t ph = 0;          // of Q_FREE and C_FREE
        int it = 0, q_filled = 0;
        for (; ok && next_piece(w); advance(s.tiles, w, a.H)) {
            const int* table = table_of();
            const int bad = readable_memories(table, a.cache, w.first_memory(), w.last_memory());
            if (bad < w.last_memory() && lane == 0) flag_status(a.status, kStatusDevice);
            const int first = w.first_memory(), last = min(w.last_memory(), bad);
            if (first >= last) continue;
            for (int c0 = first; c0 < last; c0 += kCB, ++it) {
                const int nv = min(kCB, last - c0), st = it % S::kStages;
                // lane i looks up memory i of this CTA's
                const int q0 = S::kMem * rank, mine = max(0, min(S::kMem, nv - q0));
                const int c = c0 + (lane < mine ? q0 + lane : 0);
                const size_t mem = memory_index(a.cache, a.H, table[c / a.cache.R], w.h, c % a.cache.R);
                if (!(ok = wait_warp(empty(st), ((uint32_t)(it / S::kStages) & 1u) ^ 1u, wc, 3))) break;
                if (lane == 0 && rank == 0) mbar_expect_tx(full(st), (uint32_t)nv * S::kMemBytes);
                __syncwarp();
                if (lane < mine) {
                    const uint32_t dst = smem_u32(s.ring + (size_t)st * S::kStageBytes + (size_t)lane * S::kMemBytes);
                    if constexpr (kPair) tma_load_2d_pair(dst, &prm.map_m, lead(full(st)), 0, (int)(mem * N));
                    else tma_load_2d(dst, &prm.map_m, full(st), 0, (int)(mem * N));
                }
                __syncwarp();
                if (c0 == first) {
                    const int t0 = s.tiles.t0[w.k] + rank * kRows, grp = group_of(w.h, a.H, a.G);
                    auto rows = [&](const uint8_t* to, const CUtensorMap* map, int b, int head) {
                        if (rank == 0) mbar_expect_tx(bar(b), (kPair ? 2 : 1) * (N / 64) * kPanel);
#pragma unroll
                        for (int k = 0; k < N / 64; ++k) {
                            if constexpr (kPair) tma_load_3d_pair(smem_u32(to + k * kPanel), map, lead(bar(b)), 64 * k, head, t0);
                            else tma_load_3d(smem_u32(to + k * kPanel), map, bar(b), 64 * k, head, t0);
                        }
                    };
                    if (!(ok = wait_warp(bar(Q_FREE), ph ^ 1u, wc, 1))) break;
                    if (lane == 0) rows(s.q, &prm.map_q, Q_FULL, w.h);
                    ++q_filled;
                    if (!(ok = wait_warp(bar(C_FREE), ph ^ 1u, wc, 2))) break;
                    if (lane == 0) rows(s.c, &prm.map_c, C_FULL, grp);
                    ph ^= 1u;
                    prefetch_rows();
                }
            }
        }
        if (!ok && rank == 0 && lane == 0) {
            // a wait gave up: copies in flight (the peer's complete here too, and it stays until this CTA is done)
            // are waited for, with a limit, before their shared memory goes
            auto drain = [&](uint32_t b, uint32_t parity) { for (int k = 0; k < (1 << 20) && !mbar_try_wait(b, parity); ++k) {} };
            for (int i = max(0, it - S::kStages); i < it; ++i) drain(full(i % S::kStages), (uint32_t)(i / S::kStages) & 1u);
            if (q_filled > 0) {
                drain(bar(Q_FULL), (uint32_t)(q_filled - 1) & 1u);
                drain(bar(C_FULL), (uint32_t)(q_filled - 1) & 1u);
            }
        }
        __syncwarp();
    } else if (warp == 1 && rank == 0) {
        // ------------------------------------------------------------ MMA
        auto commit = [&](uint32_t b) {
            if constexpr (kPair) mma_commit_pair(b);
            else mma_commit(b);
        };
        uint32_t ph = 0;
        int it = 0;
        for (; ok && next_piece(w); advance(s.tiles, w, a.H)) {
            const int first = w.first_memory(), last = min(w.last_memory(), readable_memories(table_of(), a.cache, w.first_memory(), w.last_memory()));
            if (first >= last) continue;
            if (!(ok = wait_warp(bar(Q_FULL), ph, wc, 4))) break;
            for (int c0 = first; c0 < last; c0 += kCB, ++it) {
                const int nv = min(kCB, last - c0), st = it % S::kStages;
                const bool end = c0 + kCB >= last;
                // a pair multiplies all four column blocks (the epilogue reads the valid ones): N splits over the CTAs
                const uint32_t idesc = idesc_bf16_f32(TT, kPair ? kP * kCB : kP * nv, false, true);
                const uint32_t b_base = smem_u32(s.ring + (size_t)st * S::kStageBytes);
                auto product = [&](uint32_t d, const uint8_t* rows) {
#pragma unroll
                    for (int kk = 0; kk < N / 16; ++kk) {
                        const uint64_t ad = smem_desc_sw128(smem_u32(rows) + (uint32_t)(kk >> 2) * kPanel + (uint32_t)(kk & 3) * 32, 16, 1024);
                        const uint64_t bd = smem_desc_sw128(b_base + (uint32_t)kk * 2048, S::kMemBytes, 1024);
                        if constexpr (kPair) mma_f16_ss_pair(d, ad, bd, idesc, kk > 0 ? 1u : 0u);
                        else mma_f16_ss(d, ad, bd, idesc, kk > 0 ? 1u : 0u);
                    }
                };
                if (!(ok = wait_warp(full(st), (uint32_t)(it / S::kStages) & 1u, wc, 5))) break;
                if (!(ok = wait_warp(bar(U_EMPTY), ((uint32_t)it & 1u) ^ 1u, wc, 6))) break;
                tc_fence_after();
                if (lane == 0) {
                    product(tmem, s.q);
                    commit(bar(U_FULL));
                    if (end) commit(bar(Q_FREE));
                }
                __syncwarp();
                if (c0 == first && !(ok = wait_warp(bar(C_FULL), ph, wc, 7))) break;
                if (!(ok = wait_warp(bar(V_EMPTY), ((uint32_t)it & 1u) ^ 1u, wc, 8))) break;
                tc_fence_after();
                if (lane == 0) {
                    product(tmem + kColV, s.c);
                    commit(bar(V_FULL));
                    commit(empty(st));
                    if (end) commit(bar(C_FREE));
                }
                __syncwarp();
            }
            ph ^= 1u;
        }
    } else if (warp >= 2) {
        // ------------------------------------------------------- epilogue
        // The two warps of a pair run the same batches and the same named barrier
        // for each, also after a failed wait (they then skip the work).
        const int quad = warp & 3, half = (warp - 2) >> 2, col0 = half * kHalfP, row = quad * 32 + lane;
        const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16);
        const float sscale = kLog2e * rsqrtf((float)N);
        int it = 0;
        for (; next_piece(w); advance(s.tiles, w, a.H)) {
            const int t0 = s.tiles.t0[w.k], rows = s.tiles.rows(w.k);
            const int tr = rank * kRows + row;         // row of the tile
            const bool live = tr < rows;
            const int count = live ? a.mem_count[t0 + tr] : -1;
            const size_t at = ((size_t)(t0 + tr) * a.H + w.h) * kP + col0;
            float2 e2[kHalfP / 2], o2[kHalfP / 2];
            uint4 er[kHalfP / 8];
#pragma unroll
            for (int q = 0; q < kHalfP / 8; ++q)
                er[q] = live ? __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.E) + at) + q) : make_uint4(0u, 0u, 0u, 0u);
            const int bad = readable_memories(table_of(), a.cache, w.first_memory(), w.last_memory());
            const int first = w.first_memory(), last = min(w.last_memory(), bad);
#pragma unroll
            for (int q = 0; q < kHalfP / 8; ++q) {
                const uint32_t w4[4] = {er[q].x, er[q].y, er[q].z, er[q].w};
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    e2[4 * q + r] = make_float2(__uint_as_float(w4[r] << 16), __uint_as_float(w4[r] & 0xffff0000u));
            }
#pragma unroll
            for (int j = 0; j < kHalfP / 2; ++j) o2[j] = make_float2(0.f, 0.f);
            float m = -INFINITY, l = 0.f;
            for (int c0 = first; c0 < last; c0 += kCB, ++it) {
                const int nv = min(kCB, last - c0);
                const uint32_t ph = (uint32_t)it & 1u;
                float part[kCB] = {0.f, 0.f, 0.f, 0.f};
                if (ok) ok = wait_warp(bar(U_FULL), ph, wc, 9);
                if (ok) {
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < kCB; ++c) {
                        if (c < nv) {
                            float u[kHalfP];
                            tmem_ld_32x32b_x32(t_lane + (uint32_t)(c * kP + col0), u);
                            tmem_ld_wait();
                            float2 a0 = make_float2(0.f, 0.f), a1 = a0;
#pragma unroll
                            for (int q = 0; q < kHalfP / 2; q += 2) {
                                a0 = __ffma2_rn(make_float2(u[2 * q], u[2 * q + 1]), e2[q], a0);
                                a1 = __ffma2_rn(make_float2(u[2 * q + 2], u[2 * q + 3]), e2[q + 1], a1);
                            }
                            part[c] = (a0.x + a1.x) + (a0.y + a1.y);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (kPair) mbar_arrive_cluster(lead(bar(U_EMPTY)));
                        else mbar_arrive(bar(U_EMPTY));
                    }
                }
                // scores: own half and the partner's
                s.scores[it & 1][half][row] = make_float4(part[0], part[1], part[2], part[3]);
                named_bar_sync(2 + quad, 64);
                const float4 pp = s.scores[it & 1][1 - half][row];
                const float other[kCB] = {pp.x, pp.y, pp.z, pp.w};
                float sc[kCB], wt[kCB], mn = m;
#pragma unroll
                for (int c = 0; c < kCB; ++c) {
                    // added in the same order by both warps, whose softmax has to be the same
                    sc[c] = (half ? other[c] + part[c] : part[c] + other[c]) * sscale;
                    if (c >= nv || c0 + c >= count) sc[c] = -INFINITY;     // not a memory this row sees
                    mn = fmaxf(mn, sc[c]);
                }
                const bool none = mn == -INFINITY;     // only scores of -inf so far: they weigh nothing
                const float alpha = none ? 1.f : exp2f(m - mn);
#pragma unroll
                for (int c = 0; c < kCB; ++c) wt[c] = none ? (sc[c] == sc[c] ? 0.f : sc[c]) : exp2f(sc[c] - mn);
                l = l * alpha + (wt[0] + wt[1]) + (wt[2] + wt[3]);
                m = mn;
                const float2 alpha2 = make_float2(alpha, alpha);
#pragma unroll
                for (int q = 0; q < kHalfP / 2; ++q) o2[q] = __fmul2_rn(o2[q], alpha2);
                if (ok) ok = wait_warp(bar(V_FULL), ph, wc, 10);
                if (ok) {
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < kCB; ++c) {
                        if (c < nv) {
                            float v[kHalfP];
                            tmem_ld_32x32b_x32(t_lane + kColV + (uint32_t)(c * kP + col0), v);
                            tmem_ld_wait();
                            if (wt[c] != 0.f) {        // 0 weight reads nothing, whatever the value is
                                const float2 w2 = make_float2(wt[c], wt[c]);
#pragma unroll
                                for (int q = 0; q < kHalfP / 2; ++q)
                                    o2[q] = __ffma2_rn(w2, make_float2(v[2 * q], v[2 * q + 1]), o2[q]);
                            }
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (kPair) mbar_arrive_cluster(lead(bar(V_EMPTY)));
                        else mbar_arrive(bar(V_EMPTY));
                    }
                }
            }
            // a whole item is written out, a part of one kept for the combine kernel
            const bool left = count < 0 || count > bad;      // a row that is not to be computed
            const int which = w.c > 0 ? 0 : 1;
            if (!w.whole() && tid == 64 && rank == 0)
                *piece_header(a.part, run, which) = PieceHeader{w.last == w.units ? 2 : 1, t0, rows, w.h};
            // Rows are written whole: the 32 rows x 32 columns of a warp change places, so that a lane has a column.
            float* v = reinterpret_cast<float*>(o2);
            if (w.whole()) {
                const float f = l == 0.f ? 0.f : (a.y_ssd ? a.g : 1.f) / l;
#pragma unroll
                for (int q = 0; q < kHalfP / 2; ++q) o2[q] = __fmul2_rn(o2[q], make_float2(f, f));
            } else if (live && half == 0) {
                float* to = piece_rows<TT, kP>(a.part, run, which) + tr * (kP + 4);
                to[kP] = m;
                to[kP + 1] = left ? -1.f : l;
            }
            transpose32(v);
            const unsigned mask = __ballot_sync(0xffffffffu, live && !(w.whole() && left));
            const int r0 = rank * kRows + quad * 32;
            if (w.whole()) {
                const size_t base = ((size_t)(t0 + r0) * a.H + w.h) * kP + col0 + lane;
                const size_t stride = (size_t)a.H * kP;
                if (a.y_ssd) {
                    float y[32];      // all loads before the first store: out may be y_ssd itself
#pragma unroll
                    for (int r = 0; r < 32; ++r) y[r] = mask >> r & 1u ? a.y_ssd[base + r * stride] : 0.f;
#pragma unroll
                    for (int r = 0; r < 32; ++r) v[r] += y[r];
                }
#pragma unroll
                for (int r = 0; r < 32; ++r)
                    if (mask >> r & 1u) a.out[base + r * stride] = v[r];
            } else {
                float* to = piece_rows<TT, kP>(a.part, run, which) + (size_t)r0 * (kP + 4) + col0 + lane;
#pragma unroll
                for (int r = 0; r < 32; ++r)
                    if (mask >> r & 1u) to[r * (kP + 4)] = v[r];
            }
        }
    }
    tc_fence_before();
    if (kPair) cluster_sync();   // neither CTA leaves while the other may still reach its memory
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        if constexpr (kPair) tmem_dealloc_pair(tmem, kTmemCols);
        else tmem_dealloc(tmem, kTmemCols);
    }
}

// How many clusters of two can be resident (not every SM need pair up), once per device.
cudaError_t resident_pairs(const void* kern, int sms, int smem, std::atomic<int> (&cache)[64], int& pairs) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    pairs = dev < 64 ? cache[dev].load(std::memory_order_relaxed) : 0;
    if (pairs > 0) return cudaSuccess;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(2 * (unsigned)(sms / 2));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if ((e = cudaOccupancyMaxActiveClusters(&pairs, kern, &cfg)) != cudaSuccess) return e;
    if (pairs <= 0) return cudaErrorInvalidConfiguration;
    if (dev < 64) cache[dev].store(pairs, std::memory_order_relaxed);
    return cudaSuccess;
}

template <int N, bool kPair>
cudaError_t run(const SmaPagedArgs& a, cudaStream_t st) {
    using S = Smem<N, kPair>;
    static_assert(sizeof(S) + 1024 <= 232448, "shared memory");
    auto kern = sma_paged_tc_kernel<N, kPair>;
    const int smem = (int)sizeof(S) + 1024, sms = paged_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    Params p;
    memset(&p, 0, sizeof(p));
    p.a = a;
    const uint32_t box[3] = {64, 1, kRows};
    {
        const uint64_t dims[3] = {N, (uint64_t)a.H, (uint64_t)a.T}, strides[2] = {N * 2, (uint64_t)a.H * N * 2};
        if (!encode_tile_map_bf16(&p.map_q, 3, a.Q, dims, strides, box)) return cudaErrorInvalidValue;
    }
    {
        const uint64_t dims[3] = {N, (uint64_t)a.G, (uint64_t)a.T}, strides[2] = {N * 2, (uint64_t)a.G * N * 2};
        if (!encode_tile_map_bf16(&p.map_c, 3, a.Cm, dims, strides, box)) return cudaErrorInvalidValue;
    }
    {
        const uint64_t rows = (uint64_t)a.cache.npages * a.H * a.cache.R * N;
        if (rows > 0x7fffffffull) return cudaErrorInvalidValue;      // 256 GB and more of memories
        const uint64_t dims[2] = {kP, rows}, strides[1] = {kP * 2};
        const uint32_t mbox[2] = {kP, N};
        if (!encode_tile_map_bf16(&p.map_m, 2, a.cache.pages, dims, strides, mbox)) return cudaErrorInvalidValue;
    }
    static std::atomic<unsigned long long> ready{0};   // devices whose kernel has its shared memory allowed
    cudaError_t e = paged_allow_smem(reinterpret_cast<const void*>(kern), smem, ready);
    if (e != cudaSuccess) return e;
    int runs = sms < kMaxTcRuns ? sms : kMaxTcRuns;
    if constexpr (kPair) {
        static std::atomic<int> cache[64];
        if ((e = resident_pairs(reinterpret_cast<const void*>(kern), sms, smem, cache, runs)) != cudaSuccess) return e;
        if (runs > kMaxTcRuns / 2) runs = kMaxTcRuns / 2;
    }
    if ((e = launch_dependent(kern, dim3(kPair ? 2 * runs : runs), dim3(kThreads), smem, st, kPair ? 2 : 1, p)) != cudaSuccess) return e;
    count_launches(1);
    return launch_sma_paged_combine(a, runs, kPair ? 2 * kRows : kRows, st);
}

}  // namespace

bool sma_paged_tc_applicable(const SmaPagedArgs& a, dart_dtype dt) {
    // More than 8 rows a sequence are two tiles of the warp-level kernel, which then streams the memories
    // twice.  32 sequences over up to 100 memories of 32 heads, warp-level / here: 4 rows on average
    // 188 / 263 us, 6 rows 210 / 289, 9 rows 314 / 316, 12 rows 378 / 282; 4 sequences: 4 rows 41 / 44 us,
    // 6 rows 43 / 43, 9 rows 48 / 44, 15 rows 51 / 44.
    return dt == DART_BF16 && !a.cache.mxfp4 && a.P == kP && (a.N == 128 || a.N == 64) && a.T > 8 * (long long)a.B &&
           a.B + a.T / kRows <= kCap;
}

cudaError_t launch_sma_paged_tc(const SmaPagedArgs& a, cudaStream_t st) {
    // A pair's tile is 256 rows, full or not.  16 sequences, single blocks / pairs: 89 rows on average
    // 189 / 291 us, 112 rows 195 / 283, 134 rows 274 / 293, 195 rows 370 / 302; 4 sequences: 105 rows 50 / 76 us,
    // 161 rows 77 / 79, 201 rows 85 / 79.
    if (a.T > 160 * (long long)a.B) return a.N == 128 ? run<128, true>(a, st) : run<64, true>(a, st);
    return a.N == 128 ? run<128, false>(a, st) : run<64, false>(a, st);
}

}  // namespace dart
