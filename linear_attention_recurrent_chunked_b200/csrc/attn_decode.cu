// Attention of one new token per sequence over the paged cache, with an optional prefix that the
// whole batch shares.
//
//     o = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),   s_j = q . k_j scale log2(e)
//
// over the prefix's keys and the sequence's own. Both sums are taken piecewise: a piece gives its
// reference maximum m, l = sum 2^(s - m) and O = sum 2^(s - m) v, and pieces join as
// M = max m, o = sum 2^(m - M) O / sum 2^(m - M) l, in fp32 and in a fixed order, so that equal calls
// give equal bits.
//
// Own keys (k_attn_decode). Bound: HBM, each key and value row is read once for the G query heads of
// its key head (G <= 16: at most 16 flops a byte). The work is cut into steps of 16 keys of one (sequence,
// key head), numbered sequence by sequence; each warp of one resident grid takes an equal run of
// consecutive steps whatever the lengths are, so ragged batches and single long sequences alike fill the
// GPU, and a warp never waits for another while keys are left. A step's rows (8 KB for d = 128) come by
// TMA, four 2 KB boxes, into a ring of the warp's own that runs ahead across (sequence, head) borders
// (by 16-byte asynchronous copies a step took 750 cycles to ask for, as long as all of its arithmetic). The
// products are S^T = K Q^T and O^T = V^T P^T on m16n8k16 tensor instructions: the 16 keys (or 16 of the d
// columns) are the rows and the heads the 8 columns, so a group of up to 8 heads wastes nothing on padding
// rows, which a 128-row tile would; at these few flops a byte the memory stays the bound. A run cuts at most
// its first and last (sequence, head) short: those pieces are joined over the CTA's warps once at the end, and
// what even the CTA's run cuts short goes to the CTA's two slots.
//
// The prefix runs in the prompt kernel (attn_prefill.cu) without a mask, all sequences' query heads of a
// key head as rows of one tile, so its keys are read once per 128 rows and not once per sequence.
//
// k_attn_combine joins the pieces; it is launched to start while the kernel before it drains.
//
// 64 sequences of 512 to 10,240 keys, 16/4 heads, d = 128 (427 MB): 76 us with the combine kernel, 5.6 TB/s. Three
// sequences of 10,240 to 40,960, 16/2 heads (61 MB): 20 us. One of 2,048: 8.5 us, of which 4.8 remain with no key
// at all (two launches, the lengths). 64 sequences behind a prefix of 10,230: 27 us, of which the prefix 15: 37 splits
// of it fill two CTAs per SM with 4 or 5 steps of 64 keys each, whose results are 19 MB (half the splits, twice
// the steps: 27 us too).
#include <algorithm>

#include "attn_common.cuh"
#include "chunk_common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

using bf16 = __nv_bfloat16;
using attn::Ctl;
using attn::grid_launch_dependents;
using attn::grid_wait;
constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kStep = 16;                // keys of a step
constexpr int kRuns = kDecodeCtas * kWarps;
constexpr float kRescale = 8.f;          // log2 units: how far the true maximum may run ahead of the reference

template <int D, int NT>
struct Smem {
    static constexpr int NST = (NT == 1 ? 3 : 2) * 128 / D;  // ring stages of a warp
    static constexpr uint32_t HALF = kStep * D * 2;          // K, then V, of a stage
    static constexpr uint32_t RING = NST * 2 * HALF;         // per warp
    static constexpr int LD = D + 4;                         // padded row of a piece
    static constexpr uint32_t PIECE = NT * 8 * LD * 4;       // O of a piece (a warp's last one goes over its ring)
    static constexpr uint32_t OFF_FIRST = kWarps * RING;
    static constexpr uint32_t OFF_ML = OFF_FIRST + kWarps * PIECE;
    static constexpr uint32_t TOTAL = OFF_ML + kWarps * 2 * NT * 8 * 8;
    static_assert(PIECE <= RING && kWarps * PIECE >= kThreads * 8, "");
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ int length_of(const AttnDecode &a, int b) {
    return min(max(a.lens[b], 0), a.max_pages << a.page_log);  // max_pages << page_log is at most 2^30
}
__device__ __forceinline__ int steps_of(int len) { return (len + kStep - 1) / kStep; }

// The run of steps of warp w of the grid is [first_step(w), first_step(w + 1)). With fewer steps than warps
// each of the first warps has one, so that the pieces of a (sequence, head) always lie in consecutive CTAs.
__device__ __forceinline__ int first_step(int steps, int w) {  // (steps are below 2^31, which the call checks)
    return steps < kRuns ? min(w, steps) : (int)((uint64_t)steps * (uint32_t)w / kRuns);
}
// The CTA whose warps' runs hold step x.
__device__ __forceinline__ int cta_of(int steps, int x) {
    if (steps < kRuns) return x / kWarps;
    int w = (int)((float)x / (float)steps * kRuns);  // about
    w = min(max(w, 0), kRuns - 1);
    while (first_step(steps, w) > x) --w;
    while (first_step(steps, w + 1) <= x) ++w;
    return w / kWarps;
}

// Q^T as the second operand of S^T = K Q^T: of head g (lane / 4) of the group at q, words lane % 4 of each
// 8-column chunk. Loaded as whole chunks, 16 bytes a lane, and transposed within the four lanes of a head: as
// words, the many warps that start on one head together would ask L2 for its sectors 8 times as often.
template <int N>
__device__ __forceinline__ void load_q(const bf16 *q, int g, int G, uint32_t (&f)[N][2]) {
    const int j = threadIdx.x & 3;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (g < G) v = *reinterpret_cast<const uint4 *>(q + (int64_t)g * (N * 16) + (4 * i + j) * 8);
        uint32_t x[4] = {v.x, v.y, v.z, v.w};  // words 0 .. 3 of chunk 4 i + j
#pragma unroll
        for (int d = 1; d < 4; d <<= 1)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (!(k & d)) {
                    const uint32_t y = __shfl_xor_sync(0xffffffffu, j & d ? x[k] : x[k + d], d);
                    if (j & d) x[k] = y; else x[k + d] = y;
                }
        f[2 * i][0] = x[0];  // now word j of chunks 4 i .. 4 i + 3
        f[2 * i][1] = x[1];
        f[2 * i + 1][0] = x[2];
        f[2 * i + 1][1] = x[3];
    }
}

// A place in a run: step `chunk` of the `n` steps of (sequence b, key head h).
struct Place {
    int b, h, chunk, n, len;
    // To the run's next step, which there must be; by a converged warp. Empty sequences are passed 32 at a time (one by
    // one a batch of 4,096 in which only the first has keys took 513 us and not 91).
    __device__ __forceinline__ void next(const AttnDecode &a) {
        if (++chunk < n) return;
        chunk = 0;
        if (++h < a.Hkv) return;
        h = 0;
        for (++b; b < a.B; b += 32) {
            const int i = b + (threadIdx.x & 31), own = i < a.B ? length_of(a, i) : 0;
            const uint32_t some = __ballot_sync(0xffffffffu, own > 0);
            if (some) {
                const int first = __ffs(some) - 1;
                b += first;
                len = __shfl_sync(0xffffffffu, own, first);
                n = steps_of(len);
                return;
            }
        }
    }
};

// What the CTA's warps leave for the end: up to two pieces each.
struct PieceTable {
    int seg[2 * kWarps];   // b Hkv + h, or -1
    int ends[2 * kWarps];  // whether it comes to that one's end
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_decode(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ AttnDecode a) {
    using S = Smem<D, NT>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t ring = tc::smem_u32(smem) + warp * S::RING;
    float2 *const piece_ml = reinterpret_cast<float2 *>(smem + S::OFF_ML);  // [2 warp + (0 first, 1 last)][heads]
    __shared__ int warp_sum[kWarps];
    // steps of one key head before each thread's stretch of sequences, where pieces will be once all have read it
    int *const stretch = reinterpret_cast<int *>(smem + S::OFF_FIRST);
    int *const lens_of = reinterpret_cast<int *>(stretch + kThreads);  // and the lengths, with a sequence a thread
    __shared__ PieceTable pieces;
    __shared__ uint64_t bars[kWarps][S::NST];  // a stage has landed
    __shared__ Ctl ctl;
    bool bad = false, timed_out = false;  // a length or page number outside its range; a wait that gave up
    if (lane == 0) {
        for (int i = 0; i < S::NST; ++i) tc::mbar_init(&bars[warp][i], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid == 0) {
        ctl.abort = 0;
        ctl.wait_ns = a.wait_ns;
    }
    // with a prefix its kernel comes before, whose CTAs have all waited already and whose results nothing here reads
    if (!a.prefix_len) grid_wait();
    grid_launch_dependents();

    if (ring & 1023u) {  // the boxes' swizzle counts on it
        if (tid == 0) a.bad[blockIdx.x] = ERRBIT_INTERNAL;
        if (a.prefix_len) grid_wait();
        return;
    }

    // ---- the runs: a scan of the sequences' step counts, a stretch of sequences per thread
    const int per = (a.B + kThreads - 1) / kThreads;
    int mine = 0;
    for (int b = tid * per; b < min(a.B, (tid + 1) * per); ++b) {
        const int len = length_of(a, b);
        bad |= len != a.lens[b];
        mine += steps_of(len);
        if (per == 1) lens_of[tid] = len;
    }
    int upto = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, m);
        if (lane >= m) upto += x;
    }
    if (lane == 31) warp_sum[warp] = upto;
    if (tid < 2 * kWarps) pieces.seg[tid] = -1;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) upto += warp_sum[w];
        total += warp_sum[w];
    }
    const int steps = total * a.Hkv;
    const int run0 = blockIdx.x * kWarps;
    stretch[tid] = upto - mine;
    __syncthreads();
    const int u0 = first_step(steps, run0 + warp), u1 = first_step(steps, run0 + warp + 1);

    Place at{};
    if (u0 < u1) {
        // the last stretch that starts at or before u0, and the sequence in it
        int last = -1;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i)
            last += __popc(__ballot_sync(0xffffffffu, stretch[i * 32 + lane] * a.Hkv <= u0));
        int in = u0 - stretch[last] * a.Hkv;
        for (at.b = last * per;; ++at.b) {
            at.len = per == 1 ? lens_of[at.b] : length_of(a, at.b);
            at.n = steps_of(at.len);
            if (in < at.n * a.Hkv) break;
            in -= at.n * a.Hkv;
        }
        at.h = (int)((uint32_t)in / (uint32_t)at.n);
        at.chunk = in - at.h * at.n;
    }
    __syncthreads();

    if (u0 < u1) {
        // ---- loads: a lane holds the page number of one of 32 consecutive steps of a sequence (any of its heads)
        Place ld = at;
        int ld_u = u0;
        int ids = -1, ids_at = 0;  // of steps ids_at + lane
        auto fetch_ids = [&]() {
            ids_at = ld.chunk;
            if (ld.chunk + lane < ld.n)
                ids = a.table[(int64_t)ld.b * a.max_pages + ((int64_t)(ld.chunk + lane) * kStep >> a.page_log)];
        };
        fetch_ids();
        int ld_st = 0;
        auto load = [&]() {
            if (ld_u < u1) {
                const int page = __shfl_sync(0xffffffffu, ids, ld.chunk - ids_at);
                const bool there = page >= 0 && page < a.num_pages;
                bad |= !there;
                uint64_t *bar = &bars[warp][ld_st];
                const bool withheld = a.withhold && blockIdx.x == 0 && ld_u == u0 + 1;  // (tests of the give-up path)
                if (lane == 0 && !withheld) tc::mbar_arrive_expect_tx(bar, 2 * S::HALF);
                __syncwarp();
                if (lane < 2 * (D / 64) && !withheld) {  // K's and V's 64-column halves; a page that is none reads as zeros
                    const int kv = lane / (D / 64), hf = lane % (D / 64);
                    tc::tma_load_3d(ring + ld_st * 2 * S::HALF + kv * S::HALF + hf * (kStep * 128), kv ? &tm_v : &tm_k, bar, hf * 64,
                                    ld.chunk * kStep & ((1 << a.page_log) - 1), (there ? page : a.num_pages) * a.Hkv + ld.h);
                }
                if (++ld_u < u1) {
                    const int b = ld.b;
                    ld.next(a);
                    if (ld.b != b || ld.chunk < ids_at || ld.chunk >= ids_at + 32) fetch_ids();
                }
            }
            ld_st = ld_st + 1 == S::NST ? 0 : ld_st + 1;
        };

        uint32_t qf[NT][D / 16][2];
        float o[NT][D / 16][4], m[NT][2], l[NT][2];
        bool started_before = at.chunk > 0, fresh = true;
        int st = 0, phase = 0;
        for (int u = u0 - (S::NST - 1); u < u1; ++u) {
            __syncwarp();
            load();  // NST - 1 steps ahead, into the stage that was read one step ago
            if (u < u0) continue;
            if (fresh) {
                fresh = false;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    load_q(a.q + ((int64_t)at.b * a.Hq + at.h * a.G) * D, t * 8 + (lane >> 2), a.G, qf[t]);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) o[t][kk][0] = o[t][kk][1] = o[t][kk][2] = o[t][kk][3] = 0.f;
                    m[t][0] = m[t][1] = -INFINITY;
                    l[t][0] = l[t][1] = 0.f;
                }
            }
            if (!attn::wait_bar_w(&bars[warp][st], phase, &ctl, nullptr)) {
                // gave up (or another warp did, and then this step's copy too may be under way): its own copies still
                // have to land before the CTA may end
                timed_out = true;
                for (int i = 0; i < S::NST; ++i) {
                    if (lane == 0 && u + i < ld_u) attn::drain_bar(&bars[warp][st], phase, &ctl);
                    st = st + 1 == S::NST ? 0 : st + 1;
                    phase ^= st == 0;
                }
                __syncwarp();
                break;
            }
            const int n = at.len - at.chunk * kStep;  // keys of the step, at least 1; 16 or more: all
            const uint32_t kb = ring + st * 2 * S::HALF, vb = kb + S::HALF;
            if (n < kStep) {
                // places past the end: whatever stale slots hold; K's scores are masked, V's rows become zeros
                for (int i = n * (D / 8) + lane; i < kStep * (D / 8); i += 32) {
                    const int r = i / (D / 8), c = i % (D / 8);
                    chunk::st_shared_v4(vb + (c >> 3) * (kStep * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4), 0, 0, 0, 0);
                }
                tc::fence_smem_to_async();  // before TMA writes here again
                __syncwarp();
            }
            float s[NT][4], s2[NT][4];  // two sums: a chain of half the length
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[t][i] = s2[t][i] = 0.f;
            const int kr = lane & 15, kc = lane >> 4;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t f[4];
                ldmatrix4(kb + (kk >> 2) * (kStep * 128) + kr * 128 + (((2 * (kk & 3) + kc) ^ (kr & 7)) << 4), f);
#pragma unroll
                for (int t = 0; t < NT; ++t) mma16816(kk & 1 ? s2[t] : s[t], f, qf[t][kk][0], qf[t][kk][1]);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[t][i] += s2[t][i];
            // this lane: keys lane / 4 and lane / 4 + 8, heads 2 (lane % 4) and one more
            const bool in0 = (lane >> 2) < n, in1 = (lane >> 2) + 8 < n;
            uint32_t pf[NT][2], pl[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float mt[2], alpha[2];
                bool grow = false;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    s[t][i] = in0 ? s[t][i] * a.scale_log2 : -INFINITY;
                    s[t][i + 2] = in1 ? s[t][i + 2] * a.scale_log2 : -INFINITY;
                    mt[i] = fmaxf(s[t][i], s[t][i + 2]);
                    mt[i] = fmaxf(mt[i], __shfl_xor_sync(0xffffffffu, mt[i], 4));
                    mt[i] = fmaxf(mt[i], __shfl_xor_sync(0xffffffffu, mt[i], 8));
                    mt[i] = fmaxf(mt[i], __shfl_xor_sync(0xffffffffu, mt[i], 16));
                    alpha[i] = 1.f;
                    if (mt[i] > m[t][i] + kRescale) {
                        alpha[i] = exp2f(m[t][i] - mt[i]);  // 0 at first
                        m[t][i] = mt[i];
                        grow = true;
                    }
                    // (no finite score yet, m = -inf: those weights are zero too, and -inf - -inf would be NaN)
                    const float ref = m[t][i] == -INFINITY ? 0.f : m[t][i];
                    const float p0 = chunk::ex2(s[t][i] - ref), p1 = chunk::ex2(s[t][i + 2] - ref);
                    l[t][i] = l[t][i] * alpha[i] + p0 + p1;
                    s[t][i] = p0;
                    s[t][i + 2] = p1;
                }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[t][kk][i] *= alpha[i & 1];
                }
                // the weights enter the second product as the sum of two bf16 values (within 2^-17 of each): the tensor
                // pipe is idle here, and one value alone would add as much error as the output's own rounding has
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t hi = tc::pack_bf16x2(s[t][2 * i], s[t][2 * i + 1]);
                    pf[t][i] = transpose8(hi);
                    pl[t][i] = transpose8(tc::pack_bf16x2(s[t][2 * i] - __uint_as_float(hi << 16),
                                                          s[t][2 * i + 1] - __uint_as_float(hi & 0xFFFF0000u)));
                }
            }
            const int vr = (lane & 7) + ((lane >> 4) << 3), vc = (lane >> 3) & 1;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t f[4];
                ldmatrix4_t(vb + (kk >> 2) * (kStep * 128) + vr * 128 + (((2 * (kk & 3) + vc) ^ (vr & 7)) << 4), f);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    mma16816(o[t][kk], f, pf[t][0], pf[t][1]);
                    mma16816(o[t][kk], f, pl[t][0], pl[t][1]);
                }
            }
            st = st + 1 == S::NST ? 0 : st + 1;
            phase ^= st == 0;

            const bool ends = at.chunk + 1 == at.n;
            if (ends || u + 1 == u1) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float x = l[t][i];
                        x += __shfl_xor_sync(0xffffffffu, x, 4);
                        x += __shfl_xor_sync(0xffffffffu, x, 8);
                        l[t][i] = x + __shfl_xor_sync(0xffffffffu, x, 16);
                    }
                const int c = (lane & 3) * 2, r = lane >> 2;  // this lane: heads c, c + 1 (of 8), columns r, r + 8 (of 16)
                if (ends && !started_before) {
                    // the whole (sequence, head) in this run
                    if (a.prefix_len) {
                        const int64_t row = (2 * (int64_t)kDecodeCtas + (int64_t)at.b * a.Hkv + at.h) * a.G;
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int g = t * 8 + c + i;
                                if (g >= a.G) continue;
                                if (r == 0) a.slot_ml[row + g] = make_float2(m[t][i], l[t][i]);
#pragma unroll
                                for (int kk = 0; kk < D / 16; ++kk) {
                                    a.slot_o[(row + g) * D + kk * 16 + r] = o[t][kk][i];
                                    a.slot_o[(row + g) * D + kk * 16 + r + 8] = o[t][kk][i + 2];
                                }
                            }
                    } else {
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const float i0 = 1.f / l[t][0], i1 = 1.f / l[t][1];
                            const int g = t * 8 + r;  // transposed: head r, columns c, c + 1 of 8
                            bf16 *dst = a.o + ((int64_t)at.b * a.Hq + at.h * a.G + g) * D + c;
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint32_t lo = transpose8(tc::pack_bf16x2(o[t][kk][0] * i0, o[t][kk][1] * i1));
                                const uint32_t hi = transpose8(tc::pack_bf16x2(o[t][kk][2] * i0, o[t][kk][3] * i1));
                                if (g < a.G) {
                                    *reinterpret_cast<uint32_t *>(dst + kk * 16) = lo;
                                    *reinterpret_cast<uint32_t *>(dst + kk * 16 + 8) = hi;
                                }
                            }
                        }
                    }
                } else {
                    // a piece: the run's first, kept beside the ring, or its last, over the ring, which is done with
                    const int which = started_before ? 0 : 1;
                    __syncwarp();
                    float *po = reinterpret_cast<float *>(smem + (which ? warp * S::RING : S::OFF_FIRST + warp * S::PIECE));
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int g = t * 8 + c + i;
                            if (r == 0) piece_ml[(2 * warp + which) * NT * 8 + g] = make_float2(m[t][i], l[t][i]);
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                po[g * S::LD + kk * 16 + r] = o[t][kk][i];
                                po[g * S::LD + kk * 16 + r + 8] = o[t][kk][i + 2];
                            }
                        }
                    if (lane == 0) {
                        pieces.seg[2 * warp + which] = at.b * a.Hkv + at.h;
                        pieces.ends[2 * warp + which] = ends;
                    }
                }
                fresh = true;
                started_before = false;
            }
            if (u + 1 < u1) at.next(a);
        }
    }

    // ---- join the warps' pieces: those of a (sequence, head) stand next to each other
    const bool any = __syncthreads_or(bad || timed_out);
    if (!any) {
        if (tid == 0) a.bad[blockIdx.x] = 0u;
    } else {
        const bool pages = __syncthreads_or(bad), late = __syncthreads_or(timed_out);
        if (tid == 0) a.bad[blockIdx.x] = (pages ? ERRBIT_PAGES : 0u) | (late ? ERRBIT_TIMEOUT : 0u);
    }
    static_assert(2 * kWarps <= 32, "");
    const int my_seg = lane < 2 * kWarps ? pieces.seg[lane] : -1;
    const uint32_t ending = __ballot_sync(0xffffffffu, lane < 2 * kWarps && pieces.ends[lane]);
    const uint32_t same = __match_any_sync(0xffffffffu, my_seg);
    uint32_t leaders = __ballot_sync(0xffffffffu, my_seg >= 0 && (same & ((1u << lane) - 1)) == 0);
    for (int item = 0; leaders; leaders &= leaders - 1) {
        const int first = __ffs(leaders) - 1;
        const int seg = __shfl_sync(0xffffffffu, my_seg, first);
        const uint32_t members = __shfl_sync(0xffffffffu, same, first);
        // what the CTA's run starts in the middle of (its first piece) goes to slot 0, what it cuts off to slot 1
        const bool before = first == 0, whole = !before && (ending >> (31 - __clz(members)) & 1);
        const int b = seg / a.Hkv, h = seg - b * a.Hkv;
        const int64_t row = (whole ? 2 * (int64_t)kDecodeCtas + seg : 2 * (int64_t)blockIdx.x + (before ? 0 : 1)) * a.G;
        for (int g = 0; g < a.G; ++g, ++item) {  // a warp takes every eighth head
            if ((item & (kWarps - 1)) != warp) continue;
            float2 ml = make_float2(-INFINITY, 0.f);
            if (members >> lane & 1) ml = piece_ml[lane * NT * 8 + g];
            float top = ml.x;
#pragma unroll
            for (int i = 16; i; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
            const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - top);
            float sum = f * ml.y;
#pragma unroll
            for (int i = 16; i; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
            const int d = (lane & (D / 4 - 1)) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            for (uint32_t left = members; left; left &= left - 1) {
                const int p = __ffs(left) - 1;
                const float fp = __shfl_sync(0xffffffffu, f, p);
                const float4 y = *reinterpret_cast<const float4 *>(
                    smem + ((p & 1) ? (p >> 1) * S::RING : S::OFF_FIRST + (p >> 1) * S::PIECE) + (g * S::LD + d) * 4);
                x.x += fp * y.x;
                x.y += fp * y.y;
                x.z += fp * y.z;
                x.w += fp * y.w;
            }
            if (lane >= D / 4) continue;
            if (whole && !a.prefix_len) {
                const float inv = 1.f / sum;
                *reinterpret_cast<uint2 *>(a.o + ((int64_t)b * a.Hq + h * a.G + g) * D + d) =
                    make_uint2(tc::pack_bf16x2(x.x * inv, x.y * inv), tc::pack_bf16x2(x.z * inv, x.w * inv));
            } else {
                *reinterpret_cast<float4 *>(a.slot_o + (row + g) * D + d) = x;
                if (d == 0) a.slot_ml[row + g] = make_float2(top, sum);
            }
        }
    }
    if (a.prefix_len) grid_wait();  // this kernel's end then means the prefix kernel's too
}

// One CTA per sequence and a.rows of its query heads: joins each one's pieces of its own keys with those of the
// prefix. A row that the decode kernel finished is left alone; one without any keys is zero.
constexpr int kMostPieces = kDecodeCtas + kPromptCtas;  // a piece per CTA and per split of the prefix at most
constexpr int kCombineCtas = 148 * 9;  // that run at once, by registers
template <int D>
__global__ void __launch_bounds__(128) k_attn_combine(const __grid_constant__ AttnDecode a) {
    constexpr int LPR = D / 4, SUBS = 128 / LPR, AHEAD = 4;  // lanes per row; pieces read together; and ahead
    const int per = (a.Hq + a.rows - 1) / a.rows, b = blockIdx.x / per, hq0 = (blockIdx.x - b * per) * a.rows;
    const int tid = threadIdx.x, sub = tid / LPR, d = tid % LPR * 4;
    __shared__ int sums[2][4];
    __shared__ float weight[kMostPieces], red[2][4];
    __shared__ float4 part[SUBS][LPR];
    int before = 0, total = 0;
    for (int i = tid; i < a.B; i += 128) {
        const int n = steps_of(length_of(a, i));
        total += n;
        if (i < b) before += n;
    }
    const int n = steps_of(length_of(a, b));
    before = __reduce_add_sync(0xffffffffu, before);
    total = __reduce_add_sync(0xffffffffu, total);
    if ((tid & 31) == 0) {
        sums[0][tid >> 5] = before;
        sums[1][tid >> 5] = total;
    }
    bool bad = false;
    if (blockIdx.x == 0) {
        const int np = (int)(((int64_t)a.prefix_len + (1 << a.page_log) - 1) >> a.page_log);
        for (int i = tid; i < np; i += 128) bad |= a.prefix_pages[i] < 0 || a.prefix_pages[i] >= a.num_pages;
    }
    __syncthreads();
    const int steps = (sums[1][0] + sums[1][1] + sums[1][2] + sums[1][3]) * a.Hkv;
    const int x_seq = (sums[0][0] + sums[0][1] + sums[0][2] + sums[0][3]) * a.Hkv;
    int row, h, g, c0, own, all;  // the row, the first CTA with a piece of it, its own pieces and all
    auto set_row = [&](int hq) {
        row = b * a.Hq + hq;
        h = hq / a.G;
        g = hq - h * a.G;
        c0 = own = 0;
        if (n) {
            c0 = cta_of(steps, x_seq + h * n);
            own = cta_of(steps, x_seq + h * n + n - 1) - c0 + 1;
        }
        all = own + (a.prefix_len ? a.splits : 0);
    };
    set_row(hq0);
    // piece i: a row of the slots, or of the prefix kernel's results
    auto place = [&](int i, const float *&po, const float2 *&ml) {
        const bool mine = i < own;
        const int64_t r = !mine ? (int64_t)(i - own) * a.B * a.Hq + row
                                : (own == 1 ? 2 * (int64_t)kDecodeCtas + (int64_t)b * a.Hkv + h
                                            : 2 * (int64_t)(c0 + i) + (i == 0 ? 1 : 0)) * a.G + g;
        po = (mine ? a.slot_o : a.part_o) + r * D + d;
        ml = (mine ? a.slot_ml : a.part_ml) + r;
    };

    grid_wait();  // also where nothing is left to do: this kernel's end means the one before it has ended
    if (blockIdx.x == 0) {
        // the error word, from what the decode kernel's CTAs found (the prefix kernel has set it up already)
        uint32_t found = bad ? ERRBIT_PAGES : 0u;
        for (int i = tid; i < kDecodeCtas; i += 128) found |= a.bad[i];
        const bool pages = __syncthreads_or(found & ERRBIT_PAGES), late = __syncthreads_or(found & ERRBIT_TIMEOUT),
                   internal = __syncthreads_or(found & ERRBIT_INTERNAL);
        if (tid == 1) a.err[1] = 0u;
        if (tid == 0)
            *a.err = (a.prefix_len ? *a.err : 0u) | (pages ? ERRBIT_PAGES : 0u) | (late ? ERRBIT_TIMEOUT : 0u) |
                     (internal ? ERRBIT_INTERNAL : 0u);
    }
    for (int hq = hq0;;) {
        const bool pieces = own != 1 || a.prefix_len;
        if (pieces) {
            // the first pieces set out while the weights are worked out
            float4 y[AHEAD];
            const float *po;
            const float2 *pml;
            auto fetch = [&](int i0) {
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    const int i = i0 + k * SUBS;
                    y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (i < all) {
                        place(i, po, pml);
                        y[k] = *reinterpret_cast<const float4 *>(po);
                    }
                }
            };
            fetch(sub);
            float2 ml[(kMostPieces + 127) / 128];
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < (kMostPieces + 127) / 128; ++k) {
                ml[k] = make_float2(-INFINITY, 0.f);
                if (k * 128 + tid < all) {
                    place(k * 128 + tid, po, pml);
                    ml[k] = *pml;
                }
                top = fmaxf(top, ml[k].x);
            }
#pragma unroll
            for (int i = 16; i; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
            if ((tid & 31) == 0) red[0][tid >> 5] = top;
            __syncthreads();
            top = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < (kMostPieces + 127) / 128; ++k) {
                const float f = ml[k].x == -INFINITY ? 0.f : exp2f(ml[k].x - top);
                if (k * 128 + tid < all) weight[k * 128 + tid] = f;
                sum += f * ml[k].y;
            }
#pragma unroll
            for (int i = 16; i; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
            if ((tid & 31) == 0) red[1][tid >> 5] = sum;
            __syncthreads();
            sum = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i0 = sub; i0 < all; i0 += AHEAD * SUBS) {
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    const float f = i0 + k * SUBS < all ? weight[i0 + k * SUBS] : 0.f;
                    x.x += f * y[k].x;
                    x.y += f * y[k].y;
                    x.z += f * y[k].z;
                    x.w += f * y[k].w;
                }
                if (i0 + AHEAD * SUBS < all) fetch(i0 + AHEAD * SUBS);
            }
            part[sub][tid % LPR] = x;
            __syncthreads();
            if (!sub) {
#pragma unroll
                for (int i = 1; i < SUBS; ++i) {
                    const float4 z = part[i][tid % LPR];
                    x.x += z.x;
                    x.y += z.y;
                    x.z += z.z;
                    x.w += z.w;
                }
                const float inv = all ? 1.f / sum : 0.f;
                *reinterpret_cast<uint2 *>(a.o + (int64_t)row * D + d) =
                    make_uint2(tc::pack_bf16x2(x.x * inv, x.y * inv), tc::pack_bf16x2(x.z * inv, x.w * inv));
            }
        }
        hq = pieces ? hq + 1 : (h + 1) * a.G;  // (whole for one query head of a group is whole for all)
        if (hq >= min(hq0 + a.rows, a.Hq)) break;
        if (pieces) __syncthreads();  // the row's shared values have been read
        set_row(hq);
    }
}

template <int D, int NT>
cudaError_t launch(AttnDecode a, cudaStream_t st, const char **stage) {
    cudaError_t e;
    CUtensorMap tm_k, tm_v;
    *stage = "TMA descriptor encoding";
    const uint64_t page = 1u << a.page_log, n = (uint64_t)a.num_pages * a.Hkv;
    if ((e = attn::make_map(&tm_k, a.k_cache, D, page, n, D, page * D, kStep, 1)) != cudaSuccess) return e;
    if ((e = attn::make_map(&tm_v, a.v_cache, D, page, n, D, page * D, kStep, 1)) != cudaSuccess) return e;
    *stage = "attn_decode";
    auto kern = k_attn_decode<D, NT>;
    constexpr size_t smem = Smem<D, NT>::TOTAL;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess) return e;
    void *pr = prof_start("attn_decode", st);
    e = attn::launch_early(kern, kDecodeCtas, kThreads, smem, st, tm_k, tm_v, a);
    prof_stop(pr);
    if (e != cudaSuccess) return e;
    *stage = "attn_combine";
    pr = prof_start("attn_combine", st);
    // One row per CTA while all of those run at once; beyond, several, since each CTA reads all of the lengths. With one
    // row for each CTA 4,096 sequences of 100 keys and 16 heads take 353 us and not 192, 1,600 of 500 keys 316 and not 283.
    a.rows = (int)std::min<int64_t>(a.Hq, ((int64_t)a.B * a.Hq + kCombineCtas - 1) / kCombineCtas);
    e = attn::launch_early(k_attn_combine<D>, (unsigned)(a.B * ((a.Hq + a.rows - 1) / a.rows)), 128, 0, st, a);
    prof_stop(pr);
    return e;
}

}  // namespace

int attn_decode_splits(int B, int Hq, int Hkv, int prefix_len) {
    if (prefix_len <= 0) return 0;
    // as many splits of the prefix's steps of 64 keys as the GPU holds at once
    const int64_t pos = 128 / (Hq / Hkv), blocks = (B + pos - 1) / pos * Hkv;
    const int64_t steps = ((int64_t)prefix_len + 63) / 64;
    return (int)std::max<int64_t>(1, std::min<int64_t>(steps, kPromptCtas / blocks));
}

size_t attn_decode_slots(int B, int Hq, int Hkv, int prefix_len) {
    return (size_t)(Hq / Hkv) * 2 * kDecodeCtas + (prefix_len > 0 ? (size_t)B * Hq : 0);
}

cudaError_t launch_attn_decode(AttnDecode a, int d, cudaStream_t st, const char **stage) {
    const Inject inj = inject_settings();
    a.wait_ns = inj.wait_ns ? inj.wait_ns : attn::kWaitNs;
    a.withhold = inj.withhold_tile;
    if (a.prefix_len > 0) {
        AttnPrefill p{};
        p.q = a.q;
        p.k = a.k_cache;
        p.v = a.v_cache;
        p.N = 1;
        p.T_tot = a.B;
        p.Hq = a.Hq;
        p.Hkv = a.Hkv;
        p.G = a.G;
        p.scale_log2 = a.scale_log2;
        p.err = a.err;
        p.pages = a.prefix_pages;
        p.num_pages = a.num_pages;
        p.page_log = a.page_log;
        p.prefix_len = a.prefix_len;
        p.splits = a.splits;
        p.part_o = a.part_o;
        p.part_ml = a.part_ml;
        p.wait_ns = a.wait_ns;
        p.withhold = a.withhold;
        const cudaError_t e = launch_attn_prefix(p, d, st, stage);
        if (e != cudaSuccess) return e;
    }
    // groups of more than 8 heads take two tiles of 8 columns
    if (d == 64) return a.G <= 8 ? launch<64, 1>(a, st, stage) : launch<64, 2>(a, st, stage);
    return a.G <= 8 ? launch<128, 1>(a, st, stage) : launch<128, 2>(a, st, stage);
}

}  // namespace gdn
