// C ABI of the library (declared in include/gdn.h): argument validation,
// error reporting and dispatch to the kernels. Host code only, apart from the
// small cu_seqlens validation kernel.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <mutex>
#include <string>
#include <vector>

#include <nvtx3/nvToolsExt.h>

#include "common.cuh"
#include "kernels.h"

namespace {

thread_local char g_msg[512] = "";

gdn_status fail(gdn_status s, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
    va_end(ap);
    return s;
}

gdn_status ok() {
    g_msg[0] = '\0';
    return GDN_OK;
}

gdn_status cuda_fail(cudaError_t e, const char *what) {
    return fail(GDN_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

bool misaligned(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

constexpr size_t kErrWordBytes = 256;  // error word, padded to keep later regions 256-byte aligned

// ---- optional per-kernel timing (gdn_profile_*): CUDA events recorded on the
// launching stream around each kernel the entry points launch.
struct ProfRec {
    const char *name;
    cudaEvent_t start, stop;
};
struct Prof {
    std::mutex mu;
    bool on = false;
    std::vector<ProfRec> recs;
    std::vector<cudaEvent_t> pool;
} g_prof;

cudaEvent_t prof_event() {
    if (!g_prof.pool.empty()) {
        cudaEvent_t e = g_prof.pool.back();
        g_prof.pool.pop_back();
        return e;
    }
    cudaEvent_t e = nullptr;
    cudaEventCreate(&e);
    return e;
}

// RAII: records a start event now and a stop event (plus the record) at scope exit.
struct ProfScope {
    const char *name;
    cudaStream_t st;
    cudaEvent_t start = nullptr;
    ProfScope(const char *n, cudaStream_t s) : name(n), st(s) {
        std::lock_guard<std::mutex> lk(g_prof.mu);
        if (g_prof.on) {
            start = prof_event();
            cudaEventRecord(start, st);
        }
    }
    ~ProfScope() {
        if (!start) return;
        std::lock_guard<std::mutex> lk(g_prof.mu);
        cudaEvent_t stop = prof_event();
        cudaEventRecord(stop, st);
        g_prof.recs.push_back({name, start, stop});
    }
};

gdn_status check_common(const void *q, const void *k, const void *v, const float *g, const float *beta,
                        const void *o, int T_tot, int H, int dk, int dv, int dtype) {
    if (dtype != GDN_F32 && dtype != GDN_BF16) return fail(GDN_ERR_DTYPE, "dtype %d is not GDN_F32 or GDN_BF16", dtype);
    if (H < 1 || T_tot < 0) return fail(GDN_ERR_SHAPE, "H=%d T=%d out of range", H, T_tot);
    if (dk != dv || (dk != 64 && dk != 128))
        return fail(GDN_ERR_SHAPE, "head sizes dk=%d dv=%d unsupported (need dk == dv in {64, 128})", dk, dv);
    if (T_tot > 0 && (!q || !k || !v || !g || !beta || !o)) return fail(GDN_ERR_NULL, "q, k, v, g, beta and o are required");
    const void *ptrs[] = {q, k, v, o};
    for (const void *p : ptrs)
        if (misaligned(p)) return fail(GDN_ERR_ALIGN, "tensor pointer %p is not 16-byte aligned", p);
    if ((reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(beta)) & 3u)
        return fail(GDN_ERR_ALIGN, "g and beta must be 4-byte aligned");
    if ((double)T_tot * H * dk >= 9.0e18) return fail(GDN_ERR_SHAPE, "sizes overflow");
    return GDN_OK;
}

}  // namespace

namespace gdn {

__global__ void k_validate_seqlens(const int32_t *__restrict__ cu, int N, int T_tot, uint32_t *__restrict__ err) {
    // One warp: err = ERRBIT_SEQLENS unless cu[0] == 0, cu non-decreasing, cu[N] == T_tot.
    bool bad = false;
    if (cu) {
        for (int n = threadIdx.x; n < N; n += 32) bad |= cu[n + 1] < cu[n];
        if (threadIdx.x == 0) bad |= (cu[0] != 0) || (cu[N] != T_tot);
    }
    bad = __any_sync(0xffffffffu, bad);
    if (threadIdx.x == 0) *err = bad ? ERRBIT_SEQLENS : 0u;
}

cudaError_t launch_validate_seqlens(const int32_t *cu, int N, int T_tot, uint32_t *err, cudaStream_t st) {
    k_validate_seqlens<<<1, 32, 0, st>>>(cu, N, T_tot, err);
    return cudaGetLastError();
}

struct ProfHandle {
    const char *name;
    cudaStream_t st;
    cudaEvent_t start;
};

// Every launch site brackets its kernel with these: an NVTX range named after the kernel (seen by
// Nsight tools when one is attached; a few nanoseconds otherwise) and, while profiling is enabled,
// a pair of CUDA events on the launch stream.
void *prof_start(const char *name, cudaStream_t st) {
    nvtxRangePushA(name);
    std::lock_guard<std::mutex> lk(g_prof.mu);
    if (!g_prof.on) return nullptr;
    ProfHandle *hd = new ProfHandle{name, st, prof_event()};
    cudaEventRecord(hd->start, st);
    return hd;
}

void prof_stop(void *handle) {
    nvtxRangePop();
    if (!handle) return;
    ProfHandle *hd = static_cast<ProfHandle *>(handle);
    std::lock_guard<std::mutex> lk(g_prof.mu);
    cudaEvent_t stop = prof_event();
    cudaEventRecord(stop, hd->st);
    g_prof.recs.push_back({hd->name, hd->start, stop});
    delete hd;
}

std::atomic<int> g_inject_kind{0};
std::atomic<unsigned long long> g_inject_wait_ns{0};

Inject inject_settings() {
    const int kind = g_inject_kind.load(std::memory_order_relaxed);
    const uint64_t ns = g_inject_wait_ns.load();
    if (kind == GDN_INJECT_WITHHOLD_LINK) return Inject{true, ns, 0, 0};
    if (kind == GDN_INJECT_WITHHOLD_KEYS) return Inject{false, 0, 2, ns};
    if (kind == GDN_INJECT_WITHHOLD_VALUES) return Inject{false, 0, 3, ns};
    return Inject{};
}

// Sets the calling thread's last-error message (for entry points defined in other files).
gdn_status record_error(gdn_status s, const char *msg) { return fail(s, "%s", msg); }

}  // namespace gdn

extern "C" {

int gdn_version(void) { return 100; }

const char *gdn_last_error(void) { return g_msg; }

size_t gdn_chunk_fwd_workspace_size(int N, int T_tot, int H, int dk, int dv, gdn_dtype dtype) {
    if (dtype == GDN_BF16 && dk == 128 && dv == 128 && N >= 1 && H >= 1 && T_tot >= 0)
        // (the plan differs with and without cu_seqlens; the larger workspace covers both)
        return std::max({kErrWordBytes, gdn::chunk_ws_workspace(N, T_tot, H, gdn::chunk_ws_seg_chunks(N, T_tot, H, false)),
                         gdn::chunk_ws_workspace(N, T_tot, H, gdn::chunk_ws_seg_chunks(N, T_tot, H, true))});
    return kErrWordBytes;
}

static gdn_status chunk_fwd_impl(const void *q, const void *k, const void *v, const float *g, const float *beta,
                                 const float *S0, const int32_t *cu_seqlens, int N, int T_tot, int H, int dk, int dv,
                                 gdn_dtype dtype, void *o, float *S_T, void *workspace, size_t ws_bytes, void *stream,
                                 bool raw) {
    gdn_status s = check_common(q, k, v, g, beta, o, T_tot, H, dk, dv, dtype);
    if (s != GDN_OK) return s;
    if (N < 1) return fail(GDN_ERR_SHAPE, "N=%d must be >= 1", N);
    if (!S_T) return fail(GDN_ERR_NULL, "S_T is required");
    if (misaligned(S0) || misaligned(S_T) || misaligned(cu_seqlens))
        return fail(GDN_ERR_ALIGN, "S0, S_T and cu_seqlens must be 16-byte aligned");
    if (!cu_seqlens && T_tot % N != 0)
        return fail(GDN_ERR_SEQLENS, "cu_seqlens is NULL and T_tot=%d is not a multiple of N=%d", T_tot, N);
    if (!workspace || ws_bytes < kErrWordBytes)
        return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes given, at least %zu needed", workspace ? ws_bytes : 0,
                    kErrWordBytes);
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return fail(GDN_ERR_ALIGN, "workspace must be 256-byte aligned");

    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint32_t *err = static_cast<uint32_t *>(workspace);
    cudaError_t e;
    if (dtype == GDN_BF16 && dk == 128) {
        const char *stage = "";
        // The pipelined path needs room for one prep record per (chunk, head) (and, split into
        // segments, the published segment states); with less workspace the single-kernel path runs.
        const int seg = gdn::chunk_ws_seg_chunks(N, T_tot, H, cu_seqlens != nullptr);
        const int use_seg = ws_bytes >= gdn::chunk_ws_workspace(N, T_tot, H, seg) ? seg : 0;
        if (ws_bytes >= gdn::chunk_ws_workspace(N, T_tot, H, use_seg)) {
            e = gdn::launch_chunk_ws(static_cast<const __nv_bfloat16 *>(q), static_cast<const __nv_bfloat16 *>(k),
                                     static_cast<const __nv_bfloat16 *>(v), g, beta, S0, cu_seqlens, N, T_tot, H,
                                     static_cast<__nv_bfloat16 *>(o), S_T, workspace, use_seg, st, &stage, raw);
            if (e != cudaSuccess) return cuda_fail(e, stage);
            return ok();
        }
        if (raw)
            return fail(GDN_ERR_WORKSPACE,
                        "raw inputs need the pipelined path: workspace of %zu bytes given, at least %zu needed",
                        ws_bytes, gdn::chunk_ws_workspace(N, T_tot, H, 0));
        e = gdn::launch_chunk_tc(static_cast<const __nv_bfloat16 *>(q), static_cast<const __nv_bfloat16 *>(k),
                                 static_cast<const __nv_bfloat16 *>(v), g, beta, S0, cu_seqlens, N, T_tot, H,
                                 static_cast<__nv_bfloat16 *>(o), S_T, workspace, ws_bytes, st, &stage);
        if (e != cudaSuccess) return cuda_fail(e, stage);
        return ok();
    }
    {
        ProfScope ps("validate_seqlens", st);
        e = gdn::launch_validate_seqlens(cu_seqlens, N, T_tot, err, st);
    }
    if (e != cudaSuccess) return cuda_fail(e, "cu_seqlens validation launch");
    ProfScope ps("chunk_simt", st);
    if (dtype == GDN_F32) {
        const float *qf = static_cast<const float *>(q), *kf = static_cast<const float *>(k),
                    *vf = static_cast<const float *>(v);
        float *of = static_cast<float *>(o);
        e = (dk == 64) ? gdn::launch_chunk_simt<float, 64>(qf, kf, vf, g, beta, S0, cu_seqlens, N, T_tot, H, of, S_T, err, st, raw)
                       : gdn::launch_chunk_simt<float, 128>(qf, kf, vf, g, beta, S0, cu_seqlens, N, T_tot, H, of, S_T, err, st, raw);
    } else {
        const __nv_bfloat16 *qb = static_cast<const __nv_bfloat16 *>(q), *kb = static_cast<const __nv_bfloat16 *>(k),
                            *vb = static_cast<const __nv_bfloat16 *>(v);
        __nv_bfloat16 *ob = static_cast<__nv_bfloat16 *>(o);
        e = (dk == 64)
                ? gdn::launch_chunk_simt<__nv_bfloat16, 64>(qb, kb, vb, g, beta, S0, cu_seqlens, N, T_tot, H, ob, S_T, err, st, raw)
                : gdn::launch_chunk_simt<__nv_bfloat16, 128>(qb, kb, vb, g, beta, S0, cu_seqlens, N, T_tot, H, ob, S_T, err, st, raw);
    }
    if (e != cudaSuccess) return cuda_fail(e, "chunked forward launch");
    return ok();
}

gdn_status gdn_chunk_fwd(const void *q, const void *k, const void *v, const float *g, const float *beta,
                         const float *S0, const int32_t *cu_seqlens, int N, int T_tot, int H, int dk, int dv,
                         gdn_dtype dtype, void *o, float *S_T, void *workspace, size_t ws_bytes, void *stream) {
    return chunk_fwd_impl(q, k, v, g, beta, S0, cu_seqlens, N, T_tot, H, dk, dv, dtype, o, S_T, workspace, ws_bytes,
                          stream, false);
}

gdn_status gdn_chunk_fwd_raw(const void *q_raw, const void *k_raw, const void *v, const float *a, const float *b,
                             const float *S0, const int32_t *cu_seqlens, int N, int T_tot, int H, int dk, int dv,
                             gdn_dtype dtype, void *o, float *S_T, void *workspace, size_t ws_bytes, void *stream) {
    return chunk_fwd_impl(q_raw, k_raw, v, a, b, S0, cu_seqlens, N, T_tot, H, dk, dv, dtype, o, S_T, workspace,
                          ws_bytes, stream, true);
}

gdn_status gdn_chunk_fwd_check(const void *workspace, size_t ws_bytes, void *stream) {
    if (!workspace || ws_bytes < sizeof(uint32_t)) return fail(GDN_ERR_WORKSPACE, "workspace missing");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // the error word, then (pipelined path) where the first timed-out wait was: the barrier's
    // shared-memory address + 1 or bit 30 + a flag's word offset, the block, the thread and parity
    uint32_t w[4] = {0, 0, 0, 0};
    const size_t n = ws_bytes >= sizeof(w) ? sizeof(w) : sizeof(uint32_t);
    cudaError_t e = cudaMemcpyAsync(w, workspace, n, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return cuda_fail(e, "reading the device error word");
    const uint32_t word = w[0];
    if (word & gdn::ERRBIT_SEQLENS) return fail(GDN_ERR_SEQLENS, "cu_seqlens is not 0 = c0 <= c1 <= ... <= cN = T_tot");
    if (word & gdn::ERRBIT_TIMEOUT) {
        if (w[1] & (1u << 30))
            return fail(GDN_ERR_TIMEOUT, "a bounded device-side wait gave up (first: flag word %u, block (%u, %u), thread %u)",
                        w[1] & 0x3FFFFFFFu, w[2] & 0xFFFFu, w[2] >> 16, w[3] & 0xFFFFu);
        if (w[1])
            return fail(GDN_ERR_TIMEOUT,
                        "a bounded device-side wait gave up (first: mbarrier at shared address %u, parity %u, block "
                        "(%u, %u), thread %u)",
                        w[1] - 1u, w[3] >> 16, w[2] & 0xFFFFu, w[2] >> 16, w[3] & 0xFFFFu);
        return fail(GDN_ERR_TIMEOUT, "a bounded device-side wait gave up");
    }
    if (word & gdn::ERRBIT_INTERNAL) return fail(GDN_ERR_CUDA, "internal: misaligned shared-memory base, nothing written");
    if (word & gdn::ERRBIT_PAGES)
        return fail(GDN_ERR_PAGES, "a slot, page number or cached length is outside the cache");
    if (word & gdn::ERRBIT_BOUNDS)
        return fail(GDN_ERR_BOUNDS, "a device-side index check failed (GDN_DEBUG_CHECKS build): an index into the "
                                    "workspace or an output was out of range and was redirected to 0");
    return ok();
}

static gdn_status decode_step_impl(const void *q, const void *k, const void *v, const float *g, const float *beta,
                                   float *S, int B, int H, int dk, int dv, gdn_dtype dtype, void *o, void *stream,
                                   bool raw) {
    if (B < 1) return fail(GDN_ERR_SHAPE, "B=%d must be >= 1", B);
    gdn_status s = check_common(q, k, v, g, beta, o, B, H, dk, dv, dtype);
    if (s != GDN_OK) return s;
    if (!S) return fail(GDN_ERR_NULL, "S is required");
    if (misaligned(S)) return fail(GDN_ERR_ALIGN, "S must be 16-byte aligned");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    ProfScope ps("decode_step", st);
    if (dtype == GDN_F32) {
        const float *qf = static_cast<const float *>(q), *kf = static_cast<const float *>(k),
                    *vf = static_cast<const float *>(v);
        float *of = static_cast<float *>(o);
        e = (dk == 64) ? gdn::launch_decode_step<float, 64>(qf, kf, vf, g, beta, S, B, H, of, st, raw)
                       : gdn::launch_decode_step<float, 128>(qf, kf, vf, g, beta, S, B, H, of, st, raw);
    } else {
        const __nv_bfloat16 *qb = static_cast<const __nv_bfloat16 *>(q), *kb = static_cast<const __nv_bfloat16 *>(k),
                            *vb = static_cast<const __nv_bfloat16 *>(v);
        __nv_bfloat16 *ob = static_cast<__nv_bfloat16 *>(o);
        e = (dk == 64) ? gdn::launch_decode_step<__nv_bfloat16, 64>(qb, kb, vb, g, beta, S, B, H, ob, st, raw)
                       : gdn::launch_decode_step<__nv_bfloat16, 128>(qb, kb, vb, g, beta, S, B, H, ob, st, raw);
    }
    if (e != cudaSuccess) return cuda_fail(e, "decode step launch");
    return ok();
}

gdn_status gdn_decode_step(const void *q, const void *k, const void *v, const float *g, const float *beta, float *S,
                           int B, int H, int dk, int dv, gdn_dtype dtype, void *o, void *stream) {
    return decode_step_impl(q, k, v, g, beta, S, B, H, dk, dv, dtype, o, stream, false);
}

gdn_status gdn_decode_step_raw(const void *q_raw, const void *k_raw, const void *v, const float *a, const float *b,
                               float *S, int B, int H, int dk, int dv, gdn_dtype dtype, void *o, void *stream) {
    return decode_step_impl(q_raw, k_raw, v, a, b, S, B, H, dk, dv, dtype, o, stream, true);
}

gdn_status gdn_seq_scan(const void *q, const void *k, const void *v, const float *g, const float *beta,
                        const float *S0, const int32_t *cu_seqlens, int N, int T_tot, int H, int dk, int dv,
                        gdn_dtype dtype, void *o, float *S_T, void *stream) {
    gdn_status s = check_common(q, k, v, g, beta, o, T_tot, H, dk, dv, dtype);
    if (s != GDN_OK) return s;
    if (N < 1) return fail(GDN_ERR_SHAPE, "N=%d must be >= 1", N);
    if (!S_T) return fail(GDN_ERR_NULL, "S_T is required");
    if (misaligned(S0) || misaligned(S_T) || misaligned(cu_seqlens))
        return fail(GDN_ERR_ALIGN, "S0, S_T and cu_seqlens must be 16-byte aligned");
    if (!cu_seqlens && T_tot % N != 0)
        return fail(GDN_ERR_SEQLENS, "cu_seqlens is NULL and T_tot=%d is not a multiple of N=%d", T_tot, N);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    ProfScope ps("seq_scan", st);
    if (dtype == GDN_F32) {
        const float *qf = static_cast<const float *>(q), *kf = static_cast<const float *>(k),
                    *vf = static_cast<const float *>(v);
        float *of = static_cast<float *>(o);
        e = (dk == 64) ? gdn::launch_seq_scan<float, 64>(qf, kf, vf, g, beta, S0, cu_seqlens, N, T_tot, H, of, S_T, st)
                       : gdn::launch_seq_scan<float, 128>(qf, kf, vf, g, beta, S0, cu_seqlens, N, T_tot, H, of, S_T, st);
    } else {
        const __nv_bfloat16 *qb = static_cast<const __nv_bfloat16 *>(q), *kb = static_cast<const __nv_bfloat16 *>(k),
                            *vb = static_cast<const __nv_bfloat16 *>(v);
        __nv_bfloat16 *ob = static_cast<__nv_bfloat16 *>(o);
        e = (dk == 64) ? gdn::launch_seq_scan<__nv_bfloat16, 64>(qb, kb, vb, g, beta, S0, cu_seqlens, N, T_tot, H, ob, S_T, st)
                       : gdn::launch_seq_scan<__nv_bfloat16, 128>(qb, kb, vb, g, beta, S0, cu_seqlens, N, T_tot, H, ob, S_T, st);
    }
    if (e != cudaSuccess) return cuda_fail(e, "sequential scan launch");
    return ok();
}

gdn_status gdn_proj_w8(const void *x, const int8_t *w, const float *scale, int T, int D, int H, int dk, int dv,
                       void *q_raw, void *k_raw, void *v, float *a, float *b, void *workspace, size_t ws_bytes,
                       void *stream) {
    if (T < 0 || D < 64 || D % 64 != 0 || H < 1 || dk < 1 || dv < 1 || (H * dk) % 8 != 0 || (H * dv) % 8 != 0)
        return fail(GDN_ERR_SHAPE, "T=%d D=%d H=%d dk=%d dv=%d unsupported (D a positive multiple of 64, H dk and "
                    "H dv multiples of 8)", T, D, H, dk, dv);
    if ((double)T * D >= 2.0e9 || (double)H * (2 * dk + dv) >= 1.0e6) return fail(GDN_ERR_SHAPE, "sizes overflow");
    if (T > 0 && (!x || !w || !scale || !q_raw || !k_raw || !v || !a || !b))
        return fail(GDN_ERR_NULL, "x, w, scale and every output are required");
    const void *p16[] = {x, w, scale, q_raw, k_raw, v};
    for (const void *p : p16)
        if (misaligned(p)) return fail(GDN_ERR_ALIGN, "pointer %p is not 16-byte aligned", p);
    if ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & 3u)
        return fail(GDN_ERR_ALIGN, "a and b must be 4-byte aligned");
    if (!workspace || ws_bytes < kErrWordBytes)
        return fail(GDN_ERR_WORKSPACE, "workspace of at least %zu bytes (the error word) needed", kErrWordBytes);
    const char *stage = "";
    const cudaError_t e = gdn::launch_proj_w8(
        static_cast<const __nv_bfloat16 *>(x), w, scale, T, D, H, dk, dv, static_cast<__nv_bfloat16 *>(q_raw),
        static_cast<__nv_bfloat16 *>(k_raw), static_cast<__nv_bfloat16 *>(v), a, b, static_cast<uint32_t *>(workspace),
        static_cast<cudaStream_t>(stream), &stage);
    if (e != cudaSuccess) return cuda_fail(e, stage);
    return ok();
}

gdn_status gdn_attn_fwd(const void *q, const void *k, const void *v, const int32_t *cu_seqlens, int N, int T_tot,
                        int H, int d, int max_len, float scale, gdn_dtype dtype, void *o, void *workspace,
                        size_t ws_bytes, void *stream) {
    if (dtype != GDN_BF16) return fail(GDN_ERR_DTYPE, "attention takes bf16 inputs only");
    if (d != 128) return fail(GDN_ERR_SHAPE, "attention head size d=%d unsupported (128)", d);
    if (N < 1 || H < 1 || T_tot < 0) return fail(GDN_ERR_SHAPE, "N=%d H=%d T=%d out of range", N, H, T_tot);
    if (!cu_seqlens && T_tot % N != 0)
        return fail(GDN_ERR_SEQLENS, "cu_seqlens is NULL and T_tot=%d is not a multiple of N=%d", T_tot, N);
    if (!cu_seqlens) max_len = T_tot / N;
    if (max_len < 0 || max_len > T_tot) return fail(GDN_ERR_SHAPE, "max_len=%d outside 0 .. T_tot", max_len);
    if ((double)T_tot * H * d >= 9.0e18 || (double)((max_len + 127) / 128) * H * N >= 2.0e9)
        return fail(GDN_ERR_SHAPE, "sizes overflow");
    if (T_tot > 0 && (!q || !k || !v || !o)) return fail(GDN_ERR_NULL, "q, k, v and o are required");
    const void *ptrs[] = {q, k, v, o, cu_seqlens};
    for (const void *p : ptrs)
        if (misaligned(p)) return fail(GDN_ERR_ALIGN, "pointer %p is not 16-byte aligned", p);
    if (!workspace || ws_bytes < kErrWordBytes)
        return fail(GDN_ERR_WORKSPACE, "workspace of at least %zu bytes (the error word) needed", kErrWordBytes);
    if (!(scale > 0.f)) scale = 1.f / sqrtf((float)d);
    const char *stage = "";
    const cudaError_t e = gdn::launch_attn_fwd(
        static_cast<const __nv_bfloat16 *>(q), static_cast<const __nv_bfloat16 *>(k),
        static_cast<const __nv_bfloat16 *>(v), cu_seqlens, N, T_tot, H, max_len, scale,
        static_cast<__nv_bfloat16 *>(o), static_cast<uint32_t *>(workspace), static_cast<cudaStream_t>(stream), &stage);
    if (e != cudaSuccess) return cuda_fail(e, stage);
    return ok();
}

// Token stride of a [T][H][d] tensor whose rows may lie inside a wider one (a fused projection's
// output): at least one token's elements, and tokens 16-byte aligned like the base.
static bool stride_ok(int64_t stride, int T, int H, int d, int esize) {
    return (T <= 1 || stride >= (int64_t)H * d) && stride >= 0 && (stride * esize) % 16 == 0 &&
           (double)stride * std::max(T, 1) < 4.0e18 / esize;
}
// Whether a contiguous output of T tokens of Ho heads overlaps a [T][H][d] input; `in_place`: other than as the
// whole of it, token for token.
static bool overlaps(const void *out, int Ho, const void *in, int64_t stride, int H, int T, int d, int esize, bool in_place) {
    if (!out || !in || T < 1) return false;
    if (in_place && out == in && Ho == H && (T == 1 || stride == (int64_t)H * d)) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(out), b = reinterpret_cast<uintptr_t>(in);
    const uintptr_t an = (uintptr_t)T * Ho * d * esize, bn = ((uintptr_t)(T - 1) * stride + (uintptr_t)H * d) * esize;
    return a < b + bn && b < a + an;
}
static bool page_size_ok(int p) { return p == 16 || p == 32 || p == 64 || p == 128; }

gdn_status gdn_qk_norm_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                            int64_t v_stride, const float *wq, const float *wk, float eps, const int32_t *positions,
                            int T, int Hq, int Hkv, int d, int rot, double base, gdn_dtype dtype, void *q_out,
                            void *k_out, void *k_cache, void *v_cache, const int32_t *slots, int num_pages,
                            int page_size, void *workspace, size_t ws_bytes, void *stream) {
    if (dtype != GDN_F32 && dtype != GDN_BF16) return fail(GDN_ERR_DTYPE, "dtype %d is not GDN_F32 or GDN_BF16", dtype);
    if (d != 64 && d != 128) return fail(GDN_ERR_SHAPE, "head size d=%d unsupported (64 or 128)", d);
    if (T < 0 || Hq < 1 || Hkv < 1 || Hq > 65536 || Hkv > 65536)
        return fail(GDN_ERR_SHAPE, "T=%d Hq=%d Hkv=%d out of range", T, Hq, Hkv);
    if (rot != 0 && (rot < 16 || rot > d || (rot & (rot - 1)) != 0))
        return fail(GDN_ERR_SHAPE, "rot=%d unsupported (0, or a power of two from 16 to d)", rot);
    if (rot != 0 && !(base > 1.0 && isfinite(base))) return fail(GDN_ERR_SHAPE, "base must be finite and above 1");
    if (!(eps >= 0.f) || !isfinite(eps)) return fail(GDN_ERR_SHAPE, "eps must be finite and not negative");
    const int es = dtype == GDN_F32 ? 4 : 2;
    if (!stride_ok(q_stride, T, Hq, d, es) || !stride_ok(k_stride, T, Hkv, d, es) ||
        (slots && !stride_ok(v_stride, T, Hkv, d, es)))
        return fail(GDN_ERR_SHAPE, "token strides must cover a token's heads and be multiples of 16 bytes");
    if (T > 0 && (!q || !k || !q_out || (rot && !positions)))
        return fail(GDN_ERR_NULL, "q, k, q_out and (with rot) positions are required");
    if (T > 0 && !k_out && !slots) return fail(GDN_ERR_NULL, "k_out or slots is required: the keys would go nowhere");
    if (slots && (!v || !k_cache || !v_cache)) return fail(GDN_ERR_NULL, "slots needs v, k_cache and v_cache");
    if (!slots && (k_cache || v_cache) && T > 0) return fail(GDN_ERR_NULL, "k_cache and v_cache need slots");
    if (slots && (!page_size_ok(page_size) || num_pages < 1 || (int64_t)num_pages * page_size > INT32_MAX))
        return fail(GDN_ERR_SHAPE, "num_pages=%d page_size=%d unsupported (page_size 16, 32, 64 or 128; at most 2^31-1 "
                    "slots)", num_pages, page_size);
    const void *ptrs[] = {q, k, slots ? v : nullptr, wq, wk, q_out, k_out, k_cache, v_cache};
    for (const void *p : ptrs)
        if (misaligned(p)) return fail(GDN_ERR_ALIGN, "tensor pointer %p is not 16-byte aligned", p);
    if ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(slots)) & 3u)
        return fail(GDN_ERR_ALIGN, "positions and slots must be 4-byte aligned");
    if (!workspace || ws_bytes < kErrWordBytes)
        return fail(GDN_ERR_WORKSPACE, "workspace of at least %zu bytes (the error word) needed", kErrWordBytes);
    if ((reinterpret_cast<uintptr_t>(workspace) & 3u) != 0) return fail(GDN_ERR_ALIGN, "workspace must be 4-byte aligned");
    if (overlaps(q_out, Hq, q, q_stride, Hq, T, d, es, true) || overlaps(q_out, Hq, k, k_stride, Hkv, T, d, es, false) ||
        overlaps(k_out, Hkv, k, k_stride, Hkv, T, d, es, true) || overlaps(k_out, Hkv, q, q_stride, Hq, T, d, es, false) ||
        overlaps(k_out, Hkv, q_out, (int64_t)Hq * d, Hq, T, d, es, false) ||
        (slots && (overlaps(q_out, Hq, v, v_stride, Hkv, T, d, es, false) ||
                   overlaps(k_out, Hkv, v, v_stride, Hkv, T, d, es, false))))
        return fail(GDN_ERR_SHAPE, "q_out and k_out may be contiguous q and k themselves, but not overlap the inputs or each "
                    "other otherwise");
    const gdn::NormRope a{q, k, v, q_stride, k_stride, v_stride, wq, wk, eps, positions, T, Hq, Hkv, rot, base,
                          q_out, k_out, k_cache, v_cache, slots, num_pages, page_size, static_cast<uint32_t *>(workspace)};
    const cudaError_t e = gdn::launch_norm_rope(a, d, dtype == GDN_BF16, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "qk_norm_rope launch");
    return ok();
}

gdn_status gdn_attn_prefill(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                            int64_t v_stride, const int32_t *cu_seqlens, int N, int T_tot, int Hq, int Hkv, int d,
                            int max_len, float scale, gdn_dtype dtype, void *o, void *workspace, size_t ws_bytes,
                            void *stream) {
    if (dtype != GDN_BF16) return fail(GDN_ERR_DTYPE, "attention takes bf16 inputs only");
    if (d != 64 && d != 128) return fail(GDN_ERR_SHAPE, "head size d=%d unsupported (64 or 128)", d);
    if (N < 1 || T_tot < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq / Hkv > 16)
        return fail(GDN_ERR_SHAPE, "N=%d T=%d Hq=%d Hkv=%d unsupported (Hq a multiple of Hkv, at most 16 times it)", N,
                    T_tot, Hq, Hkv);
    if (!cu_seqlens && T_tot % N != 0)
        return fail(GDN_ERR_SEQLENS, "cu_seqlens is NULL and T_tot=%d is not a multiple of N=%d", T_tot, N);
    if (!cu_seqlens) max_len = T_tot / N;
    if (max_len < 0 || max_len > T_tot || (int64_t)max_len * N < T_tot)
        return fail(GDN_ERR_SHAPE, "max_len=%d cannot bound %d sequences of %d tokens together", max_len, N, T_tot);
    if (!stride_ok(q_stride, T_tot, Hq, d, 2) || !stride_ok(k_stride, T_tot, Hkv, d, 2) ||
        !stride_ok(v_stride, T_tot, Hkv, d, 2))
        return fail(GDN_ERR_SHAPE, "token strides must cover a token's heads and be multiples of 16 bytes");
    // TMA strides are below 2^40 bytes; the grid has a block per query tile, key head and sequence
    const int64_t pos = 128 / (Hq / Hkv);
    if (std::max({q_stride, k_stride, v_stride}) >= ((int64_t)1 << 39) ||
        (double)std::min((max_len + pos - 1) / pos * N, gdn::attn_prefill_tiles(T_tot, N, (int)pos)) * Hkv >= 5.0e8)
        return fail(GDN_ERR_SHAPE, "sizes overflow");
    if (T_tot > 0 && (!q || !k || !v || !o)) return fail(GDN_ERR_NULL, "q, k, v and o are required");
    const void *ptrs[] = {q, k, v, o};
    for (const void *p : ptrs)
        if (misaligned(p)) return fail(GDN_ERR_ALIGN, "pointer %p is not 16-byte aligned", p);
    if ((reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0) return fail(GDN_ERR_ALIGN, "cu_seqlens must be 4-byte aligned");
    if (!workspace || ws_bytes < kErrWordBytes)
        return fail(GDN_ERR_WORKSPACE, "workspace of at least %zu bytes (the error word) needed", kErrWordBytes);
    if ((reinterpret_cast<uintptr_t>(workspace) & 3u) != 0) return fail(GDN_ERR_ALIGN, "workspace must be 4-byte aligned");
    if (overlaps(o, Hq, q, q_stride, Hq, T_tot, d, 2, false) || overlaps(o, Hq, k, k_stride, Hkv, T_tot, d, 2, false) ||
        overlaps(o, Hq, v, v_stride, Hkv, T_tot, d, 2, false))
        return fail(GDN_ERR_SHAPE, "o overlaps q, k or v");
    if (!(scale > 0.f)) scale = 1.f / sqrtf((float)d);
    gdn::AttnPrefill a{};
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k = static_cast<const __nv_bfloat16 *>(k);
    a.v = static_cast<const __nv_bfloat16 *>(v);
    a.q_stride = T_tot > 1 ? q_stride : (int64_t)Hq * d;  // (of one token any is good)
    a.k_stride = T_tot > 1 ? k_stride : (int64_t)Hkv * d;
    a.v_stride = T_tot > 1 ? v_stride : (int64_t)Hkv * d;
    a.cu = cu_seqlens;
    a.N = N;
    a.T_tot = T_tot;
    a.max_len = max_len;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.o = static_cast<__nv_bfloat16 *>(o);
    a.err = static_cast<uint32_t *>(workspace);
    const char *stage = "";
    const cudaError_t e = gdn::launch_attn_prefill(a, d, static_cast<cudaStream_t>(stream), &stage);
    if (e != cudaSuccess) return cuda_fail(e, stage);
    return ok();
}

// Regions of gdn_attn_decode's workspace, each 256-byte aligned.
struct DecodeWs {
    size_t bad, slot_o, slot_ml, part_o, part_ml, total;
    DecodeWs(int B, int Hq, int Hkv, int d, int prefix_len) {
        const size_t slots = gdn::attn_decode_slots(B, Hq, Hkv, prefix_len);
        const size_t parts = (size_t)gdn::attn_decode_splits(B, Hq, Hkv, prefix_len) * B * Hq;
        auto up = [](size_t n) { return (n + 255) / 256 * 256; };
        bad = kErrWordBytes;
        slot_o = bad + up(gdn::kDecodeCtas * sizeof(uint32_t));
        slot_ml = slot_o + up(slots * d * sizeof(float));
        part_o = slot_ml + up(slots * sizeof(float2));
        part_ml = part_o + up(parts * d * sizeof(float));
        total = part_ml + up(parts * sizeof(float2));
    }
};
static bool decode_sizes_ok(int B, int Hq, int Hkv, int d, int prefix_len) {
    return B >= 1 && Hq >= 1 && Hkv >= 1 && Hq % Hkv == 0 && Hq / Hkv <= 16 && (d == 64 || d == 128) && prefix_len >= 0 &&
           prefix_len <= 1 << 30 && (double)B * Hq < 2.0e9;
}

size_t gdn_attn_decode_workspace_size(int B, int Hq, int Hkv, int d, int prefix_len) {
    return decode_sizes_ok(B, Hq, Hkv, d, prefix_len) ? DecodeWs(B, Hq, Hkv, d, prefix_len).total : kErrWordBytes;
}

gdn_status gdn_attn_decode(const void *q, const void *k_cache, const void *v_cache, int num_pages, int page_size,
                           const int32_t *page_table, int max_pages, const int32_t *lens, const int32_t *prefix_pages,
                           int prefix_len, int B, int Hq, int Hkv, int d, float scale, gdn_dtype dtype, void *o,
                           void *workspace, size_t ws_bytes, void *stream) {
    if (dtype != GDN_BF16) return fail(GDN_ERR_DTYPE, "attention takes bf16 inputs only");
    if (!decode_sizes_ok(B, Hq, Hkv, d, prefix_len))
        return fail(GDN_ERR_SHAPE, "B=%d Hq=%d Hkv=%d d=%d prefix_len=%d unsupported (d 64 or 128, Hq a multiple of Hkv, at "
                    "most 16 times it, a prefix of at most 2^30 keys)", B, Hq, Hkv, d, prefix_len);
    if (!page_size_ok(page_size) || num_pages < 1 || (int64_t)num_pages * page_size > INT32_MAX ||
        ((int64_t)num_pages + 1) * Hkv > INT32_MAX)
        return fail(GDN_ERR_SHAPE, "num_pages=%d page_size=%d unsupported (page_size 16, 32, 64 or 128; at most 2^31-1 "
                    "slots)", num_pages, page_size);
    if (max_pages < 1 || (int64_t)max_pages * page_size > 1 << 30)
        return fail(GDN_ERR_SHAPE, "max_pages=%d out of range (at least 1, at most 2^30 keys a sequence)", max_pages);
    if ((double)B * Hkv * max_pages * page_size >= 16.0 * INT32_MAX - 16.0 * B * Hkv)
        return fail(GDN_ERR_SHAPE, "B=%d Hkv=%d max_pages=%d: more than 2^31 steps of 16 keys", B, Hkv, max_pages);
    if (!q || !k_cache || !v_cache || !page_table || !lens || !o || (prefix_len > 0 && !prefix_pages))
        return fail(GDN_ERR_NULL, "q, k_cache, v_cache, page_table, lens, o and (with prefix_len) prefix_pages are required");
    const void *ptrs[] = {q, k_cache, v_cache, o};
    for (const void *p : ptrs)
        if (misaligned(p)) return fail(GDN_ERR_ALIGN, "pointer %p is not 16-byte aligned", p);
    if ((reinterpret_cast<uintptr_t>(page_table) | reinterpret_cast<uintptr_t>(lens) |
         reinterpret_cast<uintptr_t>(prefix_pages)) & 3u)
        return fail(GDN_ERR_ALIGN, "page_table, lens and prefix_pages must be 4-byte aligned");
    if (overlaps(o, Hq, q, (int64_t)Hq * d, Hq, B, d, 2, false)) return fail(GDN_ERR_SHAPE, "o overlaps q");
    const DecodeWs w(B, Hq, Hkv, d, prefix_len);
    if (!workspace || ws_bytes < w.total)
        return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", workspace ? ws_bytes : 0, w.total);
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return fail(GDN_ERR_ALIGN, "workspace must be 256-byte aligned");
    if (!(scale > 0.f)) scale = 1.f / sqrtf((float)d);
    char *ws = static_cast<char *>(workspace);
    gdn::AttnDecode a{};
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k_cache = static_cast<const __nv_bfloat16 *>(k_cache);
    a.v_cache = static_cast<const __nv_bfloat16 *>(v_cache);
    a.table = page_table;
    a.lens = lens;
    a.prefix_pages = prefix_pages;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    while ((1 << a.page_log) < page_size) ++a.page_log;
    a.prefix_len = prefix_len;
    a.splits = gdn::attn_decode_splits(B, Hq, Hkv, prefix_len);
    a.scale_log2 = scale * 1.4426950408889634f;
    a.o = static_cast<__nv_bfloat16 *>(o);
    a.err = reinterpret_cast<uint32_t *>(ws);
    a.slot_o = reinterpret_cast<float *>(ws + w.slot_o);
    a.slot_ml = reinterpret_cast<float2 *>(ws + w.slot_ml);
    a.part_o = reinterpret_cast<float *>(ws + w.part_o);
    a.part_ml = reinterpret_cast<float2 *>(ws + w.part_ml);
    a.bad = reinterpret_cast<uint32_t *>(ws + w.bad);
    const char *stage = "";
    const cudaError_t e = gdn::launch_attn_decode(a, d, static_cast<cudaStream_t>(stream), &stage);
    if (e != cudaSuccess) return cuda_fail(e, stage);
    return ok();
}

gdn_status gdn_debug_inject(int kind, unsigned wait_us) {
    if (kind < GDN_INJECT_NONE || kind > GDN_INJECT_WITHHOLD_VALUES)
        return fail(GDN_ERR_SHAPE, "unknown injection kind %d", kind);
    if (kind != GDN_INJECT_NONE && (wait_us == 0 || wait_us > 1000000u))
        return fail(GDN_ERR_SHAPE, "wait_us=%u outside 1 .. 1000000", wait_us);
    gdn::g_inject_wait_ns.store((unsigned long long)wait_us * 1000ull);
    gdn::g_inject_kind.store(kind);
    return ok();
}

void gdn_profile_enable(int on) {
    std::lock_guard<std::mutex> lk(g_prof.mu);
    g_prof.on = on != 0;
}

int gdn_profile_read(char *names, size_t names_len, float *ms, int *counts, int max_kernels) {
    std::lock_guard<std::mutex> lk(g_prof.mu);
    std::vector<std::string> keys;
    std::vector<float> tot;
    std::vector<int> cnt;
    for (const ProfRec &r : g_prof.recs) {
        float t = 0.f;
        if (cudaEventSynchronize(r.stop) != cudaSuccess || cudaEventElapsedTime(&t, r.start, r.stop) != cudaSuccess)
            t = -1.f;
        size_t i = 0;
        while (i < keys.size() && keys[i] != r.name) ++i;
        if (i == keys.size()) {
            keys.push_back(r.name);
            tot.push_back(0.f);
            cnt.push_back(0);
        }
        tot[i] += t;
        cnt[i] += 1;
        g_prof.pool.push_back(r.start);
        g_prof.pool.push_back(r.stop);
    }
    g_prof.recs.clear();
    std::string joined;
    int n = 0;
    for (size_t i = 0; i < keys.size() && n < max_kernels; ++i, ++n) {
        if (ms) ms[n] = tot[i];
        if (counts) counts[n] = cnt[i];
        joined += keys[i];
        joined += '\n';
    }
    if (names && names_len) {
        strncpy(names, joined.c_str(), names_len - 1);
        names[names_len - 1] = '\0';
    }
    return n;
}

}  // extern "C"
