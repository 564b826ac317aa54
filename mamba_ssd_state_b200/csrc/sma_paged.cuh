// sma_paged.cuh -- how the paged attention kernels divide their work.
//
// The packed tokens of a sequence are cut into tiles of TT rows.  An item is a
// tile and a head; it reads the memories its rows may see (up to the largest
// count among them), one unit each, and kItemUnits stand for the item itself.
// The units in the order (tile, head, memory) are cut into equal runs, one for
// every worker (a block, or a warp), whatever the batch looks like.  An item
// that falls into several runs leaves one partial result (running maximum, sum,
// weighted values) per run in the workspace; a run has at most two such pieces,
// the one it begins with and the one it ends with.  sma_paged_combine joins
// them in order.
//
// Every block computes the list itself from cu_tokens and mem_count (they live
// on the device), which costs less than a launch of its own would.
#pragma once

#include "dart_paged.cuh"
#include "sm100.cuh"

namespace dart {

// Workspace: per run a header for its first and its last piece, then the pieces,
// rows of P + 4 floats: the weighted values, the maximum, the sum (-1 for a row
// that is not to be computed) and two that keep rows 16-byte aligned.
struct PieceHeader {
    int state;    // 0: no such piece, 1: more pieces follow, 2: the item ends here
    int t0;       // first token row of the tile
    int rows;
    int h;
};
constexpr int kMaxRuns = 2048;   // runs of any of the kernels
// What starting an item costs a worker, in memories: its loads wait for each
// other while a memory of the ring is there already.  With 1, a batch that held
// a sequence without memories took twice as long as its other items.
constexpr int kItemUnits = 4;

constexpr int kMaxTcRuns = 160;  // of the kernel with 128-row tiles

// Joins the pieces that the runs of a kernel with tiles of tt rows left.
cudaError_t launch_sma_paged_combine(const SmaPagedArgs& a, int runs, int tt, cudaStream_t st);
// sma_paged_mma.cu: bfloat16 and 4-bit memories with P = 64, runs of few tokens.
cudaError_t launch_sma_paged_mma(const SmaPagedArgs& a, dart_dtype dt, cudaStream_t st);
// sma_paged_tc.cu: bfloat16 memories with P = 64, long runs.
bool sma_paged_tc_applicable(const SmaPagedArgs& a, dart_dtype dt);
cudaError_t launch_sma_paged_tc(const SmaPagedArgs& a, cudaStream_t st);

#ifdef __CUDACC__

// What a memory costs a worker, in units: the same for all tiles, unless a kernel
// says otherwise.
struct EvenCost { static __device__ __forceinline__ int of(int) { return 1; } };

// Tiles of the batch in shared memory: tile k covers rows(k) rows of sequence
// seq(k) from row t0[k] on and has pre[k+1] - pre[k] units a head, the cost of a
// memory times (kItemUnits + the memories it reads).
template <int CAP, typename COST = EvenCost>
struct TileList {
    int pre[CAP + 1];
    unsigned tile[CAP];      // sequence, and rows << 16
    int t0[CAP];
    int scan[32];
    int n;
    static_assert(CAP <= 65536, "sequences in 16 bits");
    __device__ __forceinline__ int seq(int k) const { return (int)(tile[k] & 0xffffu); }
    __device__ __forceinline__ int rows(int k) const { return (int)(tile[k] >> 16); }
};

// The count a row may really see: 0 for rows that are not to be computed.
__device__ __forceinline__ int usable_count(int c, long long limit) { return c < 0 || c > limit ? 0 : c; }

// Sum over the block of one value per thread, exclusive; total to all.  scan: 32 ints
// that are not read any more; all threads have passed a barrier since.
__device__ __forceinline__ int block_scan(int v, int* scan, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (int)blockDim.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    if (lane == 31) scan[warp] = s;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    return before + s - v;
}

// Builds the list; all threads of the block.  Ranges that are no ranges or that an
// earlier sequence's may meet and counts beyond the table are flagged, and what they
// name is left out.  (CAP tiles hold every batch the host lets through.)
template <int TT, int CAP, typename COST>
__device__ __forceinline__ void build_tiles(const SmaPagedArgs& a, TileList<CAP, COST>& L) {
    const int threads = blockDim.x, tid = threadIdx.x;
    const long long limit = (long long)a.cache.width * a.cache.R;
    bool bad = false;
    int n = 0;
    for (int b0 = 0; b0 < a.B; b0 += threads) {
        const int b = b0 + tid;
        int t0 = 0, t1 = 0, tiles = 0;
        if (b < a.B) {
            if (token_range(a.cu, b, a.T, t0, t1)) tiles = (t1 - t0 + TT - 1) / TT;
            else bad = true;
        }
        // ranges can only meet where one before them is out of order
        if (__syncthreads_or(bad) && tiles > 0 && rows_taken(a.cu, b, a.T, t0, 0, 1)) {
            bad = true;
            tiles = 0;
        }
        int total;
        const int at = n + block_scan(tiles, L.scan, total);
        for (int j = 0; j < tiles; ++j) {
            if (at + j >= CAP) { bad = true; break; }
            L.tile[at + j] = (unsigned)b | (unsigned)min(TT, t1 - t0 - j * TT) << 16;
            L.t0[at + j] = t0 + j * TT;
        }
        n = min(CAP, n + total);
    }
    __syncthreads();
    // the units of every tile: a thread reads the counts of a small one, a warp those of a large one
    constexpr int BY = TT < 32 ? 1 : 32;
    for (int k = tid / BY; k < n; k += threads / BY) {
        const int t0 = L.t0[k], rows = L.rows(k);
        int most = 0;
#pragma unroll 8
        for (int r = tid % BY; r < rows; r += BY) {
            const int c = a.mem_count[t0 + r];
            bad |= c < -1 || c > limit;
            most = max(most, usable_count(c, limit));
        }
        if (BY == 32) most = __reduce_max_sync(0xffffffffu, most);
        if (tid % BY == 0) L.pre[k] = (most + kItemUnits) * COST::of(rows);
    }
    __syncthreads();
    int sum = 0;
    for (int k0 = 0; k0 < n; k0 += threads) {
        const int k = k0 + tid;
        if (k0 > 0) __syncthreads();       // the last scan has been read
        int total;
        const int at = sum + block_scan(k < n ? L.pre[k] : 0, L.scan, total);
        if (k < n) L.pre[k] = at;
        sum += total;
    }
    if (tid == 0) { L.pre[n] = sum; L.n = n; }
    if (bad && blockIdx.x == 0) flag_status(a.status, kStatusDevice);
    __syncthreads();
}

// A run of units, and the walk over its pieces.
struct Walk {
    long long u, end;    // next unit, end of the run
    int k, h, c;         // tile, head, unit of the item at u
    int units, cost;     // units of the item, and of a memory
    int last;            // the piece: units [c, last) of the item, and the memories that begin there
    __device__ __forceinline__ int memories() const { return units / cost - kItemUnits; }   // of the item
    __device__ __forceinline__ int first_memory() const { return max((c + cost - 1) / cost - kItemUnits, 0); }
    __device__ __forceinline__ int last_memory() const { return (last + cost - 1) / cost - kItemUnits; }
    __device__ __forceinline__ bool whole() const { return last - c == units; }
};

// The tile of unit u.
template <typename List>
__device__ __forceinline__ int tile_of(const List& L, int H, long long u) {
    int lo = 0, hi = L.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if ((long long)L.pre[mid] * H <= u) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// a / b for a >= 0, b > 0, in 32 bits where they do (a 64-bit division takes about
// a hundred instructions, and every worker starts with a few).
__device__ __forceinline__ long long quick_div(long long a, long long b) {
    if ((unsigned long long)(a | b) < (1ull << 32)) return (unsigned)a / (unsigned)b;
    return a / b;
}

// Run i of `runs`; runs of fewer than `least` units are not cut smaller, and a
// cut that would leave a run with an item but none of its memories goes before it.
template <int CAP, typename COST>
__device__ __forceinline__ Walk start_walk(const TileList<CAP, COST>& L, int H, int i, int runs, int least) {
    const long long W = (long long)L.pre[L.n] * H;
    const long long G = W < (long long)runs * least ? quick_div(W + least - 1, least) : runs;
    Walk w;
    auto cut = [&](long long u) {      // leaves w at the cut
        w.u = u;
        w.h = w.c = 0;
        w.units = w.cost = 1;
        if (u >= W) return;
        w.k = tile_of(L, H, u);
        w.units = L.pre[w.k + 1] - L.pre[w.k];
        w.cost = COST::of(L.rows(w.k));
        const long long r = u - (long long)L.pre[w.k] * H;
        w.h = (int)quick_div(r, w.units);
        w.c = (int)(r - (long long)w.h * w.units);
        if (w.c <= kItemUnits * w.cost) {  // no memory before the cut
            w.u -= w.c;
            w.c = 0;
        }
    };
    w.k = 0;
    if (i >= G) {
        cut(W);
        w.end = W;
        return w;
    }
    const long long each = quick_div(W, G), more = W - each * G;      // the first `more` runs have one unit more
    cut((i + 1) * each + min((long long)i + 1, more));
    w.end = w.u;
    cut(i * each + min((long long)i, more));
    return w;
}
// The next piece; false at the end of the run.
__device__ __forceinline__ bool next_piece(Walk& w) {
    if (w.u >= w.end) return false;
    w.last = (int)min((long long)w.units, w.c + (w.end - w.u));
    return true;
}
template <int CAP, typename COST>
__device__ __forceinline__ void advance(const TileList<CAP, COST>& L, Walk& w, int H) {
    w.u += w.last - w.c;
    w.c = 0;
    if (++w.h == H) {
        w.h = 0;
        ++w.k;
        if (w.k < L.n) {
            w.units = L.pre[w.k + 1] - L.pre[w.k];
            w.cost = COST::of(L.rows(w.k));
        }
    }
}

// Header and rows of a run's piece in the workspace: which = 0 for the piece
// that it begins with when the item began earlier, 1 for an item that begins in
// it and does not end there.
__device__ __forceinline__ PieceHeader* piece_header(float* part, int run, int which) {
    return reinterpret_cast<PieceHeader*>(part) + 2 * run + which;
}
template <int TT, int P>
__device__ __forceinline__ float* piece_rows(float* part, int run, int which) {
    return part + 2 * kMaxRuns * (sizeof(PieceHeader) / sizeof(float)) + (size_t)(2 * run + which) * TT * (P + 4);
}

// How many of a sequence's memories a row may see as far as the piece with
// memories [first, last) can tell: up to the first of its pages that is no page,
// all of the table if there is none.  A row that sees more is not computed; the
// pieces of an item look at their own pages, the join at what each found.  All
// lanes of a warp.
__device__ __forceinline__ int readable_memories(const int* table, const PagedCache& c, int first, int last) {
    const int lane = threadIdx.x & 31;
    if (first < last)
        for (int k = first / c.R, end = (last - 1) / c.R; k <= end; k += 32) {
            const int page = k + lane <= end ? table[k + lane] : 0;
            const unsigned m = __ballot_sync(0xffffffffu, page < 0 || page >= c.npages);
            if (m) return (k + __ffs(m) - 1) * c.R;
        }
    return c.width * c.R;
}

// A warp's wait that costs little when the phase is over already, as it mostly is
// in these rings: every lane looks for itself and the warp votes; else the
// bounded wait.  With that wait alone, in which lane 0 polls and tells the
// others, float32 runs of drafts took 663 us instead of 590, 4-bit ones 134
// instead of 131 and prompt pieces 90 instead of 80.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const sm100::WaitCtx& wc, int site) {
    return __all_sync(0xffffffffu, sm100::mbar_try_wait(bar, parity)) || sm100::mbar_wait_warp(bar, parity, wc, site);
}

// What a warp that works by itself copies: the memories of its run, piece by
// piece, into the stages of its ring, ahead of what it multiplies and over the
// ends of items.  M says how a memory is kept: kStages, kStageBytes, kPieces
// pieces of a memory, and copy(params, memory, piece, shared address, barrier).
template <typename M, typename List>
struct Feed {
    Walk w;
    const int* table;        // the sequence's
    int c, last, piece;      // next memory and piece of it, end of the memories of this part of the run
    int slot, idx;           // where memory c is: slot of the page table[idx]
    int page, ahead;         // table[idx] and, loaded long before it is needed, the next entry
    int issued;              // stages filled
    bool more;

    __device__ __forceinline__ void begin(const SmaPagedArgs& a, const List& L, const Walk& walk) {
        w = walk;
        issued = 0;
        start(a, L);
    }
    __device__ __forceinline__ void look_ahead(int R) { ahead = (idx + 1) * R < last ? table[idx + 1] : 0; }
    __device__ __forceinline__ void start(const SmaPagedArgs& a, const List& L) {
        // to the next part of the run that has memories to copy
        while ((more = next_piece(w))) {
            table = a.cache.table + (size_t)L.seq(w.k) * a.cache.width;
            c = w.first_memory();
            last = w.last_memory();
            piece = 0;
            if (c < last) {
                idx = c / a.cache.R;
                slot = c - idx * a.cache.R;
                page = table[idx];
                look_ahead(a.cache.R);
            }
            const int bad = readable_memories(table, a.cache, c, last);
            if (bad < last && (threadIdx.x & 31) == 0) flag_status(a.status, kStatusDevice);
            last = min(last, bad);
            if (c < last) return;
            advance(L, w, a.H);
        }
    }
    template <typename Params, typename Stage>
    __device__ __forceinline__ void fill(const Params& prm, const List& L, Stage* ring, uint64_t* full) {
        if (!more) return;
        const SmaPagedArgs& a = prm.a;
        const int st = issued % M::kStages;
        if ((threadIdx.x & 31) == 0) {
            const uint32_t bar = sm100::smem_u32(full + st);
            sm100::mbar_expect_tx(bar, M::kStageBytes);
            M::copy(prm, memory_index(a.cache, a.H, page, w.h, slot), piece, sm100::smem_u32(ring + st), bar);
        }
        ++issued;
        if (++piece == M::kPieces) {
            piece = 0;
            if (++c == last) {
                advance(L, w, a.H);
                start(a, L);
            } else if (++slot == a.cache.R) {
                slot = 0;
                page = ahead;
                ++idx;
                look_ahead(a.cache.R);
            }
        }
    }
    // After a wait gave up: what is in flight is waited for (with a limit) before its shared memory goes.
    __device__ __forceinline__ void drain(uint64_t* full) const {
        if ((threadIdx.x & 31) != 0) return;
        for (int i = max(0, issued - M::kStages); i < issued; ++i)
            for (int k = 0; k < (1 << 20) && !sm100::mbar_try_wait(sm100::smem_u32(full + i % M::kStages), (uint32_t)(i / M::kStages) & 1u); ++k) {}
    }
};

#endif

}  // namespace dart
