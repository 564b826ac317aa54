// dart_abi.cu -- the extern "C" surface declared in include/dart.h:
// host-side validation, workspace sizing, dispatch to the kernel families and
// the device status word.
#include <atomic>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include "dart_backward.cuh"
#include "dart_paged.cuh"

namespace dart {
// [0]: status flags; [1]: (kernel id << 8 | wait site) of the first bounded
// wait that gave up, 0 if none.
__device__ int g_status[2] = {0, 0};

namespace {
std::atomic<unsigned long long> g_launches{0};
}  // namespace

void count_launches(int n) { g_launches.fetch_add((unsigned long long)n, std::memory_order_relaxed); }
}  // namespace dart

namespace {

// Device address of the status word on the current device, looked up once
// per device.  Threads that race on the first lookup store the same value.
int* status_word() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    static std::atomic<int*> cache[64];
    int* w = cache[dev].load(std::memory_order_relaxed);
    if (!w) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, dart::g_status) != cudaSuccess) return nullptr;
        w = static_cast<int*>(p);
        cache[dev].store(w, std::memory_order_relaxed);
    }
    return w;
}

thread_local char t_err[512] = "";

dart_status fail(dart_status st, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(t_err, sizeof(t_err), fmt, ap);
    va_end(ap);
    return st;
}

dart_status cuda_fail(cudaError_t e, const char* where) {
    return fail(DART_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Workspace of the scan: per-chunk decay sums (float), padded to 256 bytes,
// followed on the tensor-core path by the bf16 state entering each chunk.
size_t scan_asum_bytes(size_t bhc) { return (bhc * sizeof(float) + 255) & ~size_t(255); }

#define DART_REQUIRE_PTR(p)                                                           \
    do {                                                                              \
        if (!(p)) return fail(DART_ERR_INVALID_ARG, "%s: null pointer", #p);          \
        if (!aligned16(p)) return fail(DART_ERR_INVALID_ARG, "%s: not 16-byte aligned", #p); \
    } while (0)

#define DART_OPTIONAL_PTR(p)                                                          \
    do {                                                                              \
        if ((p) && !aligned16(p))                                                     \
            return fail(DART_ERR_INVALID_ARG, "%s: not 16-byte aligned", #p);         \
    } while (0)

// int32 vectors (tables, ranges, counters) may be slices: their own alignment is enough
#define DART_REQUIRE_INTS(p)                                                          \
    do {                                                                              \
        if (!(p)) return fail(DART_ERR_INVALID_ARG, "%s: null pointer", #p);          \
        if (reinterpret_cast<uintptr_t>(p) & 3u)                                      \
            return fail(DART_ERR_INVALID_ARG, "%s: not 4-byte aligned", #p);          \
    } while (0)

dart_status check_common(const dart_dims* d, dart_dtype dt, bool need_seqlen) {
    if (!d) return fail(DART_ERR_INVALID_ARG, "dims: null pointer");
    if (dt != DART_F32 && dt != DART_BF16) return fail(DART_ERR_INVALID_ARG, "dtype: unknown value %d", (int)dt);
    if (d->batch < 1 || d->nheads < 1 || d->headdim < 1 || d->dstate < 1 || d->chunk < 1)
        return fail(DART_ERR_INVALID_ARG, "dims: batch, nheads, headdim, dstate and chunk must be >= 1");
    if (d->ngroups < 1 || d->nheads % d->ngroups != 0)
        return fail(DART_ERR_INVALID_ARG, "ngroups = %d: must be >= 1 and divide nheads = %d", d->ngroups, d->nheads);
    if (need_seqlen) {
        if (d->seqlen < 1) return fail(DART_ERR_INVALID_ARG, "dims: seqlen must be >= 1");
    }
    if (d->batch > 65535 || d->nheads > 65535)
        return fail(DART_ERR_UNSUPPORTED, "batch and nheads must be <= 65535");
    return DART_OK;
}

// A tensor of a call, for the check that results have memory of their own: blocks read
// their inputs at their own time, while others write.
struct Span {
    const char* name;
    const void* p;
    size_t bytes;
    int onto = -1;     // of a result: the input that it may also lie right on
};

bool overlap(const Span& a, const Span& b) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.p), q = reinterpret_cast<uintptr_t>(b.p);
    return a.bytes && b.bytes && p < q + b.bytes && q < p + a.bytes;
}

// No result on an input or on another result.
template <int R, int I>
dart_status check_apart(const char* call, const Span (&results)[R], const Span (&inputs)[I]) {
    for (int i = 0; i < R; ++i) {
        for (int j = 0; j < I; ++j)
            if (overlap(results[i], inputs[j]) && !(j == results[i].onto && inputs[j].p == results[i].p))
                return fail(DART_ERR_INVALID_ARG, "%s: %s overlaps %s", call, results[i].name, inputs[j].name);
        for (int j = i + 1; j < R; ++j)
            if (overlap(results[i], results[j]))
                return fail(DART_ERR_INVALID_ARG, "%s: %s overlaps %s", call, results[i].name, results[j].name);
    }
    return DART_OK;
}

// The paged cache's own fields, and the memory shape it is asked to hold.
dart_status check_paged(const char* call, const dart_dims* d, const dart_paged_cache* c, dart::PagedCache* out) {
    if (!c) return fail(DART_ERR_INVALID_ARG, "%s: cache: null pointer", call);
    if (c->format != DART_CACHE_DTYPE && c->format != DART_CACHE_MXFP4)
        return fail(DART_ERR_INVALID_ARG, "%s: cache format: unknown value %d", call, (int)c->format);
    const int mxfp4 = c->format == DART_CACHE_MXFP4;
    if (!dart::paged_supported(d->dstate, d->headdim, mxfp4))
        return fail(DART_ERR_UNSUPPORTED, "%s: (N=%d, P=%d) not compiled for this cache format", call, d->dstate,
                    d->headdim);
    if (c->npages < 1 || c->page_size < 1 || c->table_width < 1)
        return fail(DART_ERR_INVALID_ARG, "%s: npages, page_size and table_width must be >= 1", call);
    if ((long long)c->page_size * c->table_width > dart::kPagedMaxMemories ||
        (long long)c->npages * c->page_size * d->nheads > 0x7fffffffLL)
        return fail(DART_ERR_UNSUPPORTED, "%s: at most %lld memories a sequence and 2^31 - 1 in the pool", call,
                    dart::kPagedMaxMemories);
    const void *pages = c->pages, *table = c->table, *scales = c->scales;
    DART_REQUIRE_PTR(pages); DART_REQUIRE_INTS(table);
    if (mxfp4) DART_REQUIRE_PTR(scales);
    *out = dart::PagedCache{mxfp4, c->npages, c->page_size, c->table_width, c->pages, c->scales, c->table};
    return DART_OK;
}

Span pages_span(const dart_dims* d, dart_dtype dtype, const dart::PagedCache& c) {
    const size_t values = (size_t)c.npages * c.R * d->nheads * d->dstate * d->headdim;
    return {"pages", c.pages, c.mxfp4 ? values / 2 : values * (dtype == DART_F32 ? 4 : 2)};
}
Span scales_span(const dart_dims* d, const dart::PagedCache& c) {
    return {"scales", c.scales, c.mxfp4 ? (size_t)c.npages * c.R * d->nheads * d->dstate * d->headdim / 32 : 0};
}
Span table_span(const dart_dims* d, const dart::PagedCache& c) {
    return {"table", c.table, (size_t)d->batch * c.width * sizeof(int)};
}

}  // namespace

extern "C" {

int dart_abi_version(void) { return 4; }

unsigned long long dart_launch_count(void) { return dart::g_launches.load(std::memory_order_relaxed); }

const char* dart_last_error(void) { return t_err; }

int dart_supported(int dstate, int headdim, int chunk, dart_dtype dtype) {
    if (dtype != DART_F32 && dtype != DART_BF16) return 0;
    return dart::ssd_scan_supported(dstate, headdim, chunk, dtype) &&
           dart::sma_supported(dstate, headdim, chunk, dtype) &&
           dart::decode_supported(dstate, headdim, chunk, dtype);
}

const char* dart_sma_impl(int dstate, int headdim, int chunk, dart_dtype dtype) {
    if ((dtype != DART_F32 && dtype != DART_BF16) || !dart::sma_supported(dstate, headdim, chunk, dtype))
        return "";
    return dart::sma_impl_name(dstate, headdim, chunk, dtype);
}

size_t dart_ssd_chunk_scan_workspace_bytes(const dart_dims* d, dart_dtype dtype) {
    if (!d || d->chunk < 1) return 0;
    const size_t C = (size_t)((d->seqlen + d->chunk - 1) / d->chunk);
    const size_t bhc = (size_t)d->batch * (size_t)d->nheads * C;
    size_t bytes = scan_asum_bytes(bhc);
    if (dart::ssd_scan_tc_applicable(d->dstate, d->headdim, d->chunk, dtype)) {
        bytes += bhc * (size_t)d->dstate * (size_t)d->headdim * 2;  // bf16 state entering each chunk
        bytes += 3 * bhc * (size_t)d->chunk * sizeof(float);         // per-token decay terms
    }
    return bytes;
}

dart_status dart_ssd_chunk_scan(const dart_dims* d, dart_dtype dtype, const void* x, const float* dt,
                                const float* A, const void* Bm, const void* Cm, const float* init_state,
                                float* y_ssd, void* dH, float* states, void* workspace,
                                size_t workspace_bytes, void* stream) {
    t_err[0] = 0;
    dart_status st = check_common(d, dtype, true);
    if (st != DART_OK) return st;
    if (!dart::ssd_scan_supported(d->dstate, d->headdim, d->chunk, dtype))
        return fail(DART_ERR_UNSUPPORTED, "dart_ssd_chunk_scan: (N=%d, P=%d, S=%d) not compiled",
                    d->dstate, d->headdim, d->chunk);
    DART_REQUIRE_PTR(x); DART_REQUIRE_PTR(dt); DART_REQUIRE_PTR(A); DART_REQUIRE_PTR(Bm);
    DART_REQUIRE_PTR(Cm); DART_OPTIONAL_PTR(init_state); DART_REQUIRE_PTR(y_ssd);
    DART_REQUIRE_PTR(dH); DART_REQUIRE_PTR(states); DART_REQUIRE_PTR(workspace);
    if (workspace_bytes < dart_ssd_chunk_scan_workspace_bytes(d, dtype))
        return fail(DART_ERR_INVALID_ARG, "workspace: %zu bytes, need %zu", workspace_bytes,
                    dart_ssd_chunk_scan_workspace_bytes(d, dtype));
    const size_t bhc = (size_t)d->batch * (size_t)d->nheads * (size_t)((d->seqlen + d->chunk - 1) / d->chunk);
    char* hin = static_cast<char*>(workspace) + scan_asum_bytes(bhc);
    float* decay = reinterpret_cast<float*>(hin + bhc * (size_t)d->dstate * (size_t)d->headdim * 2);
    dart::ScanArgs a{d->batch, d->seqlen, d->nheads, d->headdim, d->dstate, d->chunk, d->ngroups,
                     x, dt, A, Bm, Cm, init_state, y_ssd, dH, states, static_cast<float*>(workspace),
                     hin, decay, status_word()};
    if (!a.status) return fail(DART_ERR_CUDA, "dart_ssd_chunk_scan: no device status word");
    cudaError_t e = dart::launch_ssd_scan(a, dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "dart_ssd_chunk_scan launch");
    return DART_OK;
}

dart_status dart_sma_forward(const dart_dims* d, dart_dtype dtype, const void* Q, const void* E,
                             const void* Cm, const void* dH, float g, const float* y_ssd, float* out,
                             void* stream) {
    t_err[0] = 0;
    dart_status st = check_common(d, dtype, true);
    if (st != DART_OK) return st;
    if (!dart::sma_supported(d->dstate, d->headdim, d->chunk, dtype))
        return fail(DART_ERR_UNSUPPORTED, "dart_sma_forward: (N=%d, P=%d, S=%d) not compiled",
                    d->dstate, d->headdim, d->chunk);
    DART_REQUIRE_PTR(Q); DART_REQUIRE_PTR(E); DART_REQUIRE_PTR(Cm); DART_REQUIRE_PTR(dH);
    DART_OPTIONAL_PTR(y_ssd); DART_REQUIRE_PTR(out);
    if (y_ssd && y_ssd != out) {
        const size_t bytes = (size_t)d->batch * d->seqlen * d->nheads * d->headdim * sizeof(float);
        const uintptr_t ya = reinterpret_cast<uintptr_t>(y_ssd), oa = reinterpret_cast<uintptr_t>(out);
        if (ya < oa + bytes && oa < ya + bytes)
            return fail(DART_ERR_INVALID_ARG, "dart_sma_forward: out overlaps y_ssd without being the same pointer");
    }
    dart::SmaArgs a{d->batch, d->seqlen, d->nheads, d->headdim, d->dstate, d->chunk, d->ngroups,
                    Q, E, Cm, dH, g, y_ssd, out, status_word()};
    if (!a.status) return fail(DART_ERR_CUDA, "dart_sma_forward: no device status word");
    cudaError_t e = dart::launch_sma(a, dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "dart_sma_forward launch");
    return DART_OK;
}

size_t dart_sma_decayed_workspace_bytes(const dart_dims* d) {
    if (!d) return 0;
    return dart::sma_decay_workspace_bytes(d->batch, d->seqlen, d->nheads, d->chunk);
}

dart_status dart_sma_forward_decayed(const dart_dims* d, dart_dtype dtype, const void* Q, const void* E,
                                     const void* Cm, const void* dH, const float* dt, const float* A, float g,
                                     const float* y_ssd, float* out, void* workspace, size_t workspace_bytes,
                                     void* stream) {
    t_err[0] = 0;
    dart_status st = check_common(d, dtype, true);
    if (st != DART_OK) return st;
    if (!dart::sma_supported(d->dstate, d->headdim, d->chunk, dtype))
        return fail(DART_ERR_UNSUPPORTED, "dart_sma_forward_decayed: (N=%d, P=%d, S=%d) not compiled",
                    d->dstate, d->headdim, d->chunk);
    DART_REQUIRE_PTR(Q); DART_REQUIRE_PTR(E); DART_REQUIRE_PTR(Cm); DART_REQUIRE_PTR(dH);
    DART_REQUIRE_PTR(dt); DART_REQUIRE_PTR(A);
    DART_OPTIONAL_PTR(y_ssd); DART_REQUIRE_PTR(out); DART_REQUIRE_PTR(workspace);
    if (reinterpret_cast<uintptr_t>(workspace) % 16 != 0)
        return fail(DART_ERR_INVALID_ARG, "dart_sma_forward_decayed: workspace not 16-byte aligned");
    const size_t need = dart_sma_decayed_workspace_bytes(d);
    if (workspace_bytes < need)
        return fail(DART_ERR_INVALID_ARG, "workspace: %zu bytes, need %zu", workspace_bytes, need);
    if (y_ssd && y_ssd != out) {
        const size_t bytes = (size_t)d->batch * d->seqlen * d->nheads * d->headdim * sizeof(float);
        const uintptr_t ya = reinterpret_cast<uintptr_t>(y_ssd), oa = reinterpret_cast<uintptr_t>(out);
        if (ya < oa + bytes && oa < ya + bytes)
            return fail(DART_ERR_INVALID_ARG,
                        "dart_sma_forward_decayed: out overlaps y_ssd without being the same pointer");
    }
    const int C = (d->seqlen + d->chunk - 1) / d->chunk;
    float* la2 = static_cast<float*>(workspace);
    const size_t la2_bytes = ((sizeof(float) * (size_t)d->batch * d->nheads * C * d->chunk) + 255) & ~size_t(255);
    double* gpre = reinterpret_cast<double*>(static_cast<uint8_t*>(workspace) + la2_bytes);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = dart::launch_sma_decay_terms(d->batch, d->seqlen, d->nheads, d->chunk, dt, A, la2, gpre, s);
    if (e != cudaSuccess) return cuda_fail(e, "dart_sma_forward_decayed: decay terms");
    dart::SmaArgs a{d->batch, d->seqlen, d->nheads, d->headdim, d->dstate, d->chunk, d->ngroups,
                    Q, E, Cm, dH, g, y_ssd, out, status_word(), la2, gpre};
    if (!a.status) return fail(DART_ERR_CUDA, "dart_sma_forward_decayed: no device status word");
    e = dart::launch_sma(a, dtype, s);
    if (e != cudaSuccess) return cuda_fail(e, "dart_sma_forward_decayed launch");
    return DART_OK;
}

size_t dart_ssd_scan_backward_workspace_bytes(const dart_dims* d) {
    if (!d) return 0;
    return dart::scan_bwd_workspace_bytes(d->batch, d->seqlen, d->nheads, d->dstate, d->headdim, d->chunk);
}

dart_status dart_ssd_scan_backward(const dart_dims* d, dart_dtype dtype, const void* x, const float* dt,
                                   const float* A, const void* Bm, const void* Cm, const float* init_state,
                                   const float* states, const float* dy, const float* ddH, const float* dCm_add,
                                   float* dx, float* ddt, float* dA, float* dBm, float* dCm, float* dinit_state,
                                   void* workspace, size_t workspace_bytes, void* stream) {
    t_err[0] = 0;
    dart_status st = check_common(d, dtype, true);
    if (st != DART_OK) return st;
    if (!dart::scan_bwd_supported(d->dstate, d->headdim, d->chunk))
        return fail(DART_ERR_UNSUPPORTED, "dart_ssd_scan_backward: (N=%d, P=%d, S=%d) not compiled", d->dstate,
                    d->headdim, d->chunk);
    DART_REQUIRE_PTR(x); DART_REQUIRE_PTR(dt); DART_REQUIRE_PTR(A); DART_REQUIRE_PTR(Bm); DART_REQUIRE_PTR(Cm);
    DART_OPTIONAL_PTR(init_state); DART_REQUIRE_PTR(states); DART_REQUIRE_PTR(dy); DART_OPTIONAL_PTR(ddH);
    DART_OPTIONAL_PTR(dCm_add); DART_REQUIRE_PTR(dx); DART_REQUIRE_PTR(ddt); DART_REQUIRE_PTR(dA); DART_REQUIRE_PTR(dBm); DART_REQUIRE_PTR(dCm);
    DART_OPTIONAL_PTR(dinit_state); DART_REQUIRE_PTR(workspace);
    const size_t need = dart_ssd_scan_backward_workspace_bytes(d);
    if (workspace_bytes < need)
        return fail(DART_ERR_INVALID_ARG, "workspace: %zu bytes, need %zu", workspace_bytes, need);
    dart::ScanBwdArgs a{d->batch, d->seqlen, d->nheads, d->headdim, d->dstate, d->chunk, d->ngroups, x, dt, A, Bm, Cm,
                        init_state, states, dy, ddH, dCm_add, dx, ddt, dA, dBm, dCm, dinit_state, status_word()};
    if (!a.status) return fail(DART_ERR_CUDA, "dart_ssd_scan_backward: no device status word");
    cudaError_t e = dart::launch_ssd_scan_bwd(a, workspace, dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "dart_ssd_scan_backward launch");
    return DART_OK;
}

size_t dart_sma_backward_workspace_bytes(const dart_dims* d) {
    if (!d) return 0;
    return dart::sma_bwd_workspace_bytes(d->batch, d->seqlen, d->nheads, d->dstate, d->chunk);
}

dart_status dart_sma_backward(const dart_dims* d, dart_dtype dtype, const void* Q, const void* E, const void* Cm,
                              const void* dH, float g, const float* dy, float* dQ, float* dE, float* dCm,
                              float* ddH, float* dg, void* workspace, size_t workspace_bytes, void* stream) {
    t_err[0] = 0;
    dart_status st = check_common(d, dtype, true);
    if (st != DART_OK) return st;
    if (!dart::sma_supported(d->dstate, d->headdim, d->chunk, dtype))
        return fail(DART_ERR_UNSUPPORTED, "dart_sma_backward: (N=%d, P=%d, S=%d) not compiled", d->dstate,
                    d->headdim, d->chunk);
    DART_REQUIRE_PTR(Q); DART_REQUIRE_PTR(E); DART_REQUIRE_PTR(Cm); DART_REQUIRE_PTR(dH); DART_REQUIRE_PTR(dy);
    DART_REQUIRE_PTR(dQ); DART_REQUIRE_PTR(dE); DART_REQUIRE_PTR(dCm); DART_REQUIRE_PTR(ddH); DART_REQUIRE_PTR(dg);
    DART_REQUIRE_PTR(workspace);
    const size_t need = dart_sma_backward_workspace_bytes(d);
    if (workspace_bytes < need)
        return fail(DART_ERR_INVALID_ARG, "workspace: %zu bytes, need %zu", workspace_bytes, need);
    dart::SmaBwdArgs a{d->batch, d->seqlen, d->nheads, d->headdim, d->dstate, d->chunk, d->ngroups, Q, E, Cm, dH, g, dy,
                       dQ, dE, dCm, ddH, dg, status_word()};
    if (!a.status) return fail(DART_ERR_CUDA, "dart_sma_backward: no device status word");
    cudaError_t e = dart::launch_sma_bwd(a, workspace, dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "dart_sma_backward launch");
    return DART_OK;
}

size_t dart_decode_step_workspace_bytes(const dart_dims* d, dart_dtype, int cmax) {
    if (!d || cmax < 0 || cmax > dart::kDecodeMaxCmax) return 0;
    const size_t ns = (size_t)dart::decode_num_splits(d->batch, d->nheads, cmax);
    return sizeof(float) * (size_t)d->batch * (size_t)d->nheads * ns * (2 + 2 * (size_t)d->headdim);
}

dart_status dart_decode_step(const dart_dims* d, dart_dtype dtype, const void* x_t, const float* dt_t,
                             const float* A, const void* B_t, const void* C_t, const void* Q_t,
                             const void* E_t, float g, float* state, float* dH_cur, void* dH_cache,
                             int cmax, int* n_chunks, int* pos, float* y, void* workspace,
                             size_t workspace_bytes, void* stream) {
    t_err[0] = 0;
    dart_status st = check_common(d, dtype, false);
    if (st != DART_OK) return st;
    if (!dart::decode_supported(d->dstate, d->headdim, d->chunk, dtype))
        return fail(DART_ERR_UNSUPPORTED, "dart_decode_step: (N=%d, P=%d) not compiled", d->dstate, d->headdim);
    if (cmax < 1 || cmax > dart::kDecodeMaxCmax)
        return fail(DART_ERR_INVALID_ARG, "cmax = %d outside [1, %d]", cmax, dart::kDecodeMaxCmax);
    DART_REQUIRE_PTR(x_t); DART_REQUIRE_PTR(dt_t); DART_REQUIRE_PTR(A); DART_REQUIRE_PTR(B_t);
    DART_REQUIRE_PTR(C_t); DART_REQUIRE_PTR(Q_t); DART_REQUIRE_PTR(E_t); DART_REQUIRE_PTR(state);
    DART_REQUIRE_PTR(dH_cur); DART_REQUIRE_PTR(dH_cache); DART_REQUIRE_PTR(n_chunks);
    DART_REQUIRE_PTR(pos); DART_REQUIRE_PTR(y); DART_REQUIRE_PTR(workspace);
    if (workspace_bytes < dart_decode_step_workspace_bytes(d, dtype, cmax))
        return fail(DART_ERR_INVALID_ARG, "workspace: %zu bytes, need %zu", workspace_bytes,
                    dart_decode_step_workspace_bytes(d, dtype, cmax));
    dart::DecodeArgs a{d->batch, d->nheads, d->headdim, d->dstate, d->chunk, d->ngroups, cmax,
                       dart::decode_num_splits(d->batch, d->nheads, cmax),
                       x_t, dt_t, A, B_t, C_t, Q_t, E_t, g, state, dH_cur, dH_cache,
                       n_chunks, pos, y, static_cast<float*>(workspace), status_word()};
    if (!a.status) return fail(DART_ERR_CUDA, "dart_decode_step: no device status word");
    cudaError_t e = dart::launch_decode(a, dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "dart_decode_step launch");
    return DART_OK;
}

dart_status dart_decode_step_decayed(const dart_dims* d, dart_dtype dtype, const void* x_t, const float* dt_t,
                                     const float* A, const void* B_t, const void* C_t, const void* Q_t,
                                     const void* E_t, float g, float* state, float* dH_cur, void* dH_cache,
                                     int cmax, int* n_chunks, int* pos, float* mem_logdecay, float* y,
                                     void* workspace, size_t workspace_bytes, void* stream) {
    t_err[0] = 0;
    dart_status st = check_common(d, dtype, false);
    if (st != DART_OK) return st;
    if (!dart::decode_supported(d->dstate, d->headdim, d->chunk, dtype))
        return fail(DART_ERR_UNSUPPORTED, "dart_decode_step_decayed: (N=%d, P=%d) not compiled", d->dstate,
                    d->headdim);
    if (cmax < 1 || cmax > dart::kDecodeMaxCmax)
        return fail(DART_ERR_INVALID_ARG, "cmax = %d outside [1, %d]", cmax, dart::kDecodeMaxCmax);
    DART_REQUIRE_PTR(x_t); DART_REQUIRE_PTR(dt_t); DART_REQUIRE_PTR(A); DART_REQUIRE_PTR(B_t);
    DART_REQUIRE_PTR(C_t); DART_REQUIRE_PTR(Q_t); DART_REQUIRE_PTR(E_t); DART_REQUIRE_PTR(state);
    DART_REQUIRE_PTR(dH_cur); DART_REQUIRE_PTR(dH_cache); DART_REQUIRE_PTR(n_chunks);
    DART_REQUIRE_PTR(pos); DART_REQUIRE_PTR(mem_logdecay); DART_REQUIRE_PTR(y); DART_REQUIRE_PTR(workspace);
    if (workspace_bytes < dart_decode_step_workspace_bytes(d, dtype, cmax))
        return fail(DART_ERR_INVALID_ARG, "workspace: %zu bytes, need %zu", workspace_bytes,
                    dart_decode_step_workspace_bytes(d, dtype, cmax));
    dart::DecodeArgs a{d->batch, d->nheads, d->headdim, d->dstate, d->chunk, d->ngroups, cmax,
                       dart::decode_num_splits(d->batch, d->nheads, cmax),
                       x_t, dt_t, A, B_t, C_t, Q_t, E_t, g, state, dH_cur, dH_cache,
                       n_chunks, pos, y, static_cast<float*>(workspace), status_word(), mem_logdecay};
    if (!a.status) return fail(DART_ERR_CUDA, "dart_decode_step_decayed: no device status word");
    cudaError_t e = dart::launch_decode(a, dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "dart_decode_step_decayed launch");
    return DART_OK;
}

dart_status dart_decode_step_e4m3(const dart_dims* d, dart_dtype dtype, const void* x_t, const float* dt_t,
                                  const float* A, const void* B_t, const void* C_t, const void* Q_t,
                                  const void* E_t, float g, float* state, float* dH_cur, unsigned char* cache,
                                  signed char* cache_exp, int cmax, int* n_chunks, int* pos, float* mem_logdecay,
                                  float* y, void* workspace, size_t workspace_bytes, void* stream) {
    t_err[0] = 0;
    dart_status st = check_common(d, dtype, false);
    if (st != DART_OK) return st;
    if (!dart::decode_e4m3_supported(d->dstate, d->headdim))
        return fail(DART_ERR_UNSUPPORTED, "dart_decode_step_e4m3: (N=%d, P=%d) not compiled (P = 64, N = 64 or 128)",
                    d->dstate, d->headdim);
    if (cmax < 1 || cmax > dart::kDecodeMaxCmax)
        return fail(DART_ERR_INVALID_ARG, "cmax = %d outside [1, %d]", cmax, dart::kDecodeMaxCmax);
    DART_REQUIRE_PTR(x_t); DART_REQUIRE_PTR(dt_t); DART_REQUIRE_PTR(A); DART_REQUIRE_PTR(B_t);
    DART_REQUIRE_PTR(C_t); DART_REQUIRE_PTR(Q_t); DART_REQUIRE_PTR(E_t); DART_REQUIRE_PTR(state);
    DART_REQUIRE_PTR(dH_cur); DART_REQUIRE_PTR(cache); DART_REQUIRE_PTR(cache_exp); DART_REQUIRE_PTR(n_chunks);
    DART_REQUIRE_PTR(pos); DART_OPTIONAL_PTR(mem_logdecay); DART_REQUIRE_PTR(y); DART_REQUIRE_PTR(workspace);
    if (workspace_bytes < dart_decode_step_workspace_bytes(d, dtype, cmax))
        return fail(DART_ERR_INVALID_ARG, "workspace: %zu bytes, need %zu", workspace_bytes,
                    dart_decode_step_workspace_bytes(d, dtype, cmax));
    dart::DecodeArgs a{d->batch, d->nheads, d->headdim, d->dstate, d->chunk, d->ngroups, cmax,
                       dart::decode_num_splits(d->batch, d->nheads, cmax),
                       x_t, dt_t, A, B_t, C_t, Q_t, E_t, g, state, dH_cur, cache,
                       n_chunks, pos, y, static_cast<float*>(workspace), status_word(), mem_logdecay, cache_exp};
    if (!a.status) return fail(DART_ERR_CUDA, "dart_decode_step_e4m3: no device status word");
    cudaError_t e = dart::launch_decode_e4m3(a, dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "dart_decode_step_e4m3 launch");
    return DART_OK;
}

dart_status dart_cache_quantize_e4m3(const dart_dims* d, dart_dtype dtype, const void* dH, int nmem,
                                     unsigned char* cache, signed char* cache_exp, int cmax, void* stream) {
    t_err[0] = 0;
    dart_status st = check_common(d, dtype, true);
    if (st != DART_OK) return st;
    if (!dart::decode_e4m3_supported(d->dstate, d->headdim))
        return fail(DART_ERR_UNSUPPORTED, "dart_cache_quantize_e4m3: (N=%d, P=%d) not compiled", d->dstate,
                    d->headdim);
    const int C = (d->seqlen + d->chunk - 1) / d->chunk;
    if (nmem < 0 || nmem > C || nmem > cmax)
        return fail(DART_ERR_INVALID_ARG, "dart_cache_quantize_e4m3: nmem = %d outside [0, min(C = %d, cmax = %d)]",
                    nmem, C, cmax);
    DART_REQUIRE_PTR(dH); DART_REQUIRE_PTR(cache); DART_REQUIRE_PTR(cache_exp);
    cudaError_t e = dart::launch_cache_quantize_e4m3(d->batch, d->nheads, C, d->dstate, d->headdim, nmem, cmax, dH,
                                                     dtype, cache, cache_exp, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "dart_cache_quantize_e4m3 launch");
    return DART_OK;
}

dart_status dart_decode_memlog_init(const dart_dims* d, const float* dt, const float* A, float* mem_logdecay,
                                    int cmax, void* stream) {
    t_err[0] = 0;
    if (!d) return fail(DART_ERR_INVALID_ARG, "dims is NULL");
    if (d->batch < 1 || d->seqlen < 1 || d->nheads < 1 || d->chunk < 1)
        return fail(DART_ERR_INVALID_ARG, "dart_decode_memlog_init: batch, seqlen, nheads and chunk must be >= 1");
    if (cmax < 1 || d->seqlen / d->chunk > cmax)
        return fail(DART_ERR_INVALID_ARG, "dart_decode_memlog_init: %d completed chunks do not fit cmax = %d",
                    d->seqlen / d->chunk, cmax);
    DART_REQUIRE_PTR(dt); DART_REQUIRE_PTR(A); DART_REQUIRE_PTR(mem_logdecay);
    cudaError_t e = dart::launch_decode_memlog_init(d->batch, d->seqlen, d->nheads, d->chunk, cmax, dt, A,
                                                    mem_logdecay, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "dart_decode_memlog_init launch");
    return DART_OK;
}

// The decode step for callers that cannot allocate device memory: the split
// partials go to the library's fixed static scratch (decode.cu) instead of a
// caller workspace.  Validation matches dart_decode_step, plus the scratch
// size limit; no allocation of any kind happens here.
dart_status dart_decode_step_noalloc(const dart_dims* d, dart_dtype dtype, const void* x_t, const float* dt_t,
                                     const float* A, const void* B_t, const void* C_t, const void* Q_t,
                                     const void* E_t, float g, float* state, float* dH_cur, void* dH_cache,
                                     int cmax, int* n_chunks, int* pos, float* y, void* stream) {
    t_err[0] = 0;
    dart_status st = check_common(d, dtype, false);
    if (st != DART_OK) return st;
    if (!dart::decode_supported(d->dstate, d->headdim, d->chunk, dtype))
        return fail(DART_ERR_UNSUPPORTED, "dart_decode_step_noalloc: (N=%d, P=%d) not compiled", d->dstate,
                    d->headdim);
    if (cmax < 1 || cmax > dart::kDecodeMaxCmax)
        return fail(DART_ERR_INVALID_ARG, "cmax = %d outside [1, %d]", cmax, dart::kDecodeMaxCmax);
    DART_REQUIRE_PTR(x_t); DART_REQUIRE_PTR(dt_t); DART_REQUIRE_PTR(A); DART_REQUIRE_PTR(B_t);
    DART_REQUIRE_PTR(C_t); DART_REQUIRE_PTR(Q_t); DART_REQUIRE_PTR(E_t); DART_REQUIRE_PTR(state);
    DART_REQUIRE_PTR(dH_cur); DART_REQUIRE_PTR(dH_cache); DART_REQUIRE_PTR(n_chunks);
    DART_REQUIRE_PTR(pos); DART_REQUIRE_PTR(y);
    const size_t need = dart_decode_step_workspace_bytes(d, dtype, cmax);
    if (need > dart::kNoAllocScratchBytes)
        return fail(DART_ERR_UNSUPPORTED,
                    "dart_decode_step_noalloc: this batch needs %zu bytes of scratch, more than the fixed %zu; "
                    "use dart_decode_step with a workspace or fewer sequences / a smaller cmax",
                    need, dart::kNoAllocScratchBytes);
    void* scratch = nullptr;
    cudaError_t e = dart::noalloc_scratch(&scratch);
    if (e != cudaSuccess) return cuda_fail(e, "dart_decode_step_noalloc: static scratch address");
    dart::DecodeArgs a{d->batch, d->nheads, d->headdim, d->dstate, d->chunk, d->ngroups, cmax,
                       dart::decode_num_splits(d->batch, d->nheads, cmax),
                       x_t, dt_t, A, B_t, C_t, Q_t, E_t, g, state, dH_cur, dH_cache,
                       n_chunks, pos, y, static_cast<float*>(scratch), status_word()};
    if (!a.status) return fail(DART_ERR_CUDA, "dart_decode_step_noalloc: no device status word");
    e = dart::launch_decode(a, dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "dart_decode_step_noalloc launch");
    return DART_OK;
}

static dart_status cache_copy(const char* call, bool write, const dart_dims* d, dart_dtype dtype, void* dH, int nmem,
                              const int* first, const int* count, const dart_paged_cache* cache, void* stream) {
    t_err[0] = 0;
    dart_status st = check_common(d, dtype, false);
    if (st != DART_OK) return st;
    dart::CacheCopyArgs a{};
    if ((st = check_paged(call, d, cache, &a.cache)) != DART_OK) return st;
    if (nmem < 1) return fail(DART_ERR_INVALID_ARG, "%s: nmem = %d: must be >= 1", call, nmem);
    DART_REQUIRE_PTR(dH); DART_REQUIRE_INTS(first); DART_REQUIRE_INTS(count);
    a.B = d->batch; a.C = nmem; a.H = d->nheads; a.P = d->headdim; a.N = d->dstate;
    a.dH = dH; a.first = first; a.count = count; a.status = status_word();
    const size_t ints = (size_t)d->batch * sizeof(int);
    const Span in[3] = {{"first", first, ints}, {"count", count, ints}, table_span(d, a.cache)};
    const Span dense = {"dH", dH, (size_t)d->batch * d->nheads * nmem * d->dstate * d->headdim * (dtype == DART_F32 ? 4 : 2)};
    const Span to_pages[2] = {pages_span(d, dtype, a.cache), scales_span(d, a.cache)}, to_dense[1] = {dense};
    if ((st = write ? check_apart(call, to_pages, in) : check_apart(call, to_dense, in)) != DART_OK) return st;
    if (!a.status) return fail(DART_ERR_CUDA, "%s: no device status word", call);
    cudaError_t e = write ? dart::launch_cache_write(a, dtype, static_cast<cudaStream_t>(stream))
                          : dart::launch_cache_read(a, dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, call);
    return DART_OK;
}

dart_status dart_cache_write_paged(const dart_dims* d, dart_dtype dtype, const void* dH, int nmem, const int* first,
                                   const int* count, const dart_paged_cache* cache, void* stream) {
    return cache_copy("dart_cache_write_paged", true, d, dtype, const_cast<void*>(dH), nmem, first, count, cache, stream);
}

dart_status dart_cache_read_paged(const dart_dims* d, dart_dtype dtype, const dart_paged_cache* cache, const int* first,
                                  const int* count, void* dH, int nmem, void* stream) {
    return cache_copy("dart_cache_read_paged", false, d, dtype, dH, nmem, first, count, cache, stream);
}

dart_status dart_ssd_extend(const dart_dims* d, dart_dtype dtype, const void* x, const float* dt, const float* A,
                            const void* Bm, const void* Cm, const int* cu_tokens, const float* state, float* state_out,
                            const float* dH_cur, float* dH_cur_out, const dart_paged_cache* cache, const int* n_chunks,
                            const int* pos, int* n_chunks_out, int* pos_out, float* y, int* mem_count, void* stream) {
    t_err[0] = 0;
    dart_status st = check_common(d, dtype, false);
    if (st != DART_OK) return st;
    dart::ExtendArgs a{};
    if ((st = check_paged("dart_ssd_extend", d, cache, &a.cache)) != DART_OK) return st;
    if (d->seqlen < 0) return fail(DART_ERR_INVALID_ARG, "dart_ssd_extend: seqlen (packed token rows) must be >= 0");
    if (d->seqlen > 0) {
        DART_REQUIRE_PTR(x); DART_REQUIRE_PTR(dt); DART_REQUIRE_PTR(Bm); DART_REQUIRE_PTR(Cm);
        DART_REQUIRE_PTR(y); DART_REQUIRE_INTS(mem_count);
    }
    DART_REQUIRE_PTR(A); DART_REQUIRE_INTS(cu_tokens); DART_REQUIRE_PTR(state); DART_REQUIRE_PTR(state_out);
    DART_REQUIRE_PTR(dH_cur); DART_REQUIRE_PTR(dH_cur_out); DART_REQUIRE_INTS(n_chunks); DART_REQUIRE_INTS(pos);
    DART_REQUIRE_INTS(n_chunks_out); DART_REQUIRE_INTS(pos_out);
    const size_t T = d->seqlen, H = d->nheads, item = dtype == DART_F32 ? 4 : 2, ints = (size_t)d->batch * sizeof(int);
    const size_t tokens = T * H * d->headdim, bc = T * d->ngroups * d->dstate * item, matrices = d->batch * H * d->dstate * d->headdim * 4;
    const Span in[11] = {{"x", x, tokens * item}, {"dt", dt, T * H * 4}, {"A", A, H * 4}, {"Bm", Bm, bc}, {"Cm", Cm, bc},
                         {"cu_tokens", cu_tokens, ints + sizeof(int)}, {"state", state, matrices}, {"dH_cur", dH_cur, matrices},
                         {"n_chunks", n_chunks, ints}, {"pos", pos, ints}, table_span(d, a.cache)};
    const Span out[8] = {{"y", y, tokens * 4}, {"mem_count", mem_count, T * sizeof(int)}, {"n_chunks_out", n_chunks_out, ints},
                         {"pos_out", pos_out, ints}, {"state_out", state_out, matrices, 6}, {"dH_cur_out", dH_cur_out, matrices, 7},
                         pages_span(d, dtype, a.cache), scales_span(d, a.cache)};
    if ((st = check_apart("dart_ssd_extend", out, in)) != DART_OK) return st;
    a.B = d->batch; a.T = d->seqlen; a.H = d->nheads; a.P = d->headdim; a.N = d->dstate; a.S = d->chunk; a.G = d->ngroups;
    a.x = x; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.cu = cu_tokens;
    a.state = state; a.state_out = state_out; a.cur = dH_cur; a.cur_out = dH_cur_out;
    a.nchunks = n_chunks; a.pos = pos; a.nchunks_out = n_chunks_out; a.pos_out = pos_out;
    a.y = y; a.mem_count = mem_count; a.status = status_word();
    if (!a.status) return fail(DART_ERR_CUDA, "dart_ssd_extend: no device status word");
    cudaError_t e = dart::launch_ssd_extend(a, dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "dart_ssd_extend launch");
    return DART_OK;
}

size_t dart_sma_paged_workspace_bytes(const dart_dims* d) {
    return d && d->headdim > 0 ? dart::sma_paged_workspace_bytes(d->headdim) : 0;
}

dart_status dart_sma_paged(const dart_dims* d, dart_dtype dtype, const void* Q, const void* E, const void* Cm,
                           const int* cu_tokens, const dart_paged_cache* cache, const int* mem_count, float g,
                           const float* y_ssd, float* out, void* workspace, size_t workspace_bytes, void* stream) {
    t_err[0] = 0;
    dart_status st = check_common(d, dtype, false);
    if (st != DART_OK) return st;
    dart::SmaPagedArgs a{};
    if ((st = check_paged("dart_sma_paged", d, cache, &a.cache)) != DART_OK) return st;
    if (d->seqlen < 0) return fail(DART_ERR_INVALID_ARG, "dart_sma_paged: seqlen (packed token rows) must be >= 0");
    if (d->seqlen == 0) return DART_OK;
    DART_REQUIRE_PTR(Q); DART_REQUIRE_PTR(E); DART_REQUIRE_PTR(Cm); DART_REQUIRE_INTS(cu_tokens);
    DART_REQUIRE_INTS(mem_count); DART_OPTIONAL_PTR(y_ssd); DART_REQUIRE_PTR(out); DART_REQUIRE_PTR(workspace);
    if (dart::sma_paged_tiles(d->batch, d->seqlen) > dart::sma_paged_max_tiles())
        return fail(DART_ERR_UNSUPPORTED, "dart_sma_paged: %d sequences and %d tokens are too many for one call "
                    "(batch + seqlen / 4 must be <= %lld)", d->batch, d->seqlen, dart::sma_paged_max_tiles());
    const size_t need = dart_sma_paged_workspace_bytes(d);
    if (workspace_bytes < need)
        return fail(DART_ERR_INVALID_ARG, "workspace: %zu bytes, need %zu", workspace_bytes, need);
    const size_t T = d->seqlen, item = dtype == DART_F32 ? 4 : 2, tokens = T * d->nheads * d->headdim;
    const Span in[9] = {{"Q", Q, T * d->nheads * d->dstate * item}, {"E", E, tokens * item}, {"Cm", Cm, T * d->ngroups * d->dstate * item},
                        {"y_ssd", y_ssd, y_ssd ? tokens * 4 : 0}, {"cu_tokens", cu_tokens, (d->batch + (size_t)1) * sizeof(int)},
                        {"mem_count", mem_count, T * sizeof(int)}, table_span(d, a.cache), pages_span(d, dtype, a.cache), scales_span(d, a.cache)};
    const Span results[2] = {{"out", out, tokens * 4, 3}, {"workspace", workspace, need}};
    if ((st = check_apart("dart_sma_paged", results, in)) != DART_OK) return st;
    a.B = d->batch; a.T = d->seqlen; a.H = d->nheads; a.P = d->headdim; a.N = d->dstate; a.G = d->ngroups;
    a.Q = Q; a.E = E; a.Cm = Cm; a.cu = cu_tokens; a.mem_count = mem_count; a.g = g; a.y_ssd = y_ssd; a.out = out;
    a.part = static_cast<float*>(workspace); a.status = status_word();
    if (!a.status) return fail(DART_ERR_CUDA, "dart_sma_paged: no device status word");
    cudaError_t e = dart::launch_sma_paged(a, dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "dart_sma_paged launch");
    return DART_OK;
}

dart_status dart_selftest_wait_timeout(unsigned int limit_us, void* stream) {
    t_err[0] = 0;
    if (limit_us < 1 || limit_us > 2000000)
        return fail(DART_ERR_INVALID_ARG, "dart_selftest_wait_timeout: limit_us = %u outside [1, 2000000]", limit_us);
    int* status = status_word();
    if (!status) return fail(DART_ERR_CUDA, "dart_selftest_wait_timeout: no device status word");
    cudaError_t e = dart::launch_wait_drill(status, 1000ull * limit_us, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "dart_selftest_wait_timeout launch");
    dart::count_launches(1);
    return DART_OK;
}

dart_status dart_sync_status(void* stream) {
    t_err[0] = 0;
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "dart_sync_status: stream synchronize");
    int words[2] = {0, 0};
    e = cudaMemcpyFromSymbol(words, dart::g_status, sizeof(words));
    if (e != cudaSuccess) return cuda_fail(e, "dart_sync_status: read status");
    if (words[0] || words[1]) {
        const int zero[2] = {0, 0};
        e = cudaMemcpyToSymbol(dart::g_status, zero, sizeof(zero));
        if (e != cudaSuccess) return cuda_fail(e, "dart_sync_status: clear status");
    }
    if (words[0] & dart::kStatusTimeout)
        return fail(DART_ERR_TIMEOUT, "a bounded device wait gave up (kernel %d, wait site %d)", words[1] >> 8,
                    words[1] & 0xff);
    if (words[0] & dart::kStatusDevice)
        return fail(DART_ERR_DEVICE, "device flagged bad state (decode or paged-cache counters, ranges or pages out of range, or cache full)");
    return DART_OK;
}

}  // extern "C"
