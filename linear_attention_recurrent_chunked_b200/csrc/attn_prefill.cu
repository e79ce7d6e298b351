// Causal attention with grouped heads over packed prompts, and the same kernel without the mask over
// a cached prefix that a whole decode batch shares, on the sm_100a tensor cores.
//
//     o_t = sum_{j <= t} softmax_j(scale q_t . k_j) v_j,     key head = query head / G, G = Hq / Hkv
//
// A tile of 128 query rows packs P = floor(128 / G) consecutive positions times the G query heads of
// one key head, position-major, which is the order in which one TMA box {64 columns, G heads,
// P positions} lands. All rows of a tile then share their key and value tiles whatever G is, and a
// tile's causal edge is P positions long. Per step of 64 keys
//
//     S = Q K^T (tensor memory)  ->  P = 2^(S c - m) (bf16, tensor memory)  ->  O += P V (tensor memory)
//
// with c = scale log2(e) and m a running row maximum that moves only when the true one has grown by
// more than 8, so P <= 2^8 and O and the row sum l are seldom rescaled; o = O / l. P is rounded to
// bf16 for the tensor core (at most 2^-8 of each weight); l sums the unrounded weights in fp32.
//
// One CTA holds one tile and goes through the keys in steps of 64. Its steps are a chain (S -> maximum ->
// weights -> O), so two CTAs share an SM and one's softmax runs beside the other's products. Roles:
//   softmax  (4 warps)  one query row per thread: no exchange between lanes
//   loader   (1 warp)   TMA: Q once, then K and V tiles of 64 keys, by turns, through one ring of five
//   S        (1 warp)   S = Q K^T as soon as the softmax has S of the step before in registers
//   O        (1 warp)   O += P V as soon as the weights are written
// Weights have their own tensor memory beside S, so that the next S does not wait for O += P V; with O that
// is 224 of the CTA's 256 columns, and the last 32 hold 64 of Q's columns: those products of S take one operand
// from shared memory instead of two (32 cycles of 128x64x16 against 48 at 128 bytes a cycle).
// Bound: tensor pipe and power. One sequence of 10,240 tokens, 16/4 heads, d = 128: 345 us in short runs, 400 over
// seconds, at 990 W and 1.50 GHz: 1,245 and 1,075 TFLOP/s, against 1,656 and 1,385 of a library bf16 product of the same
// kind of machine. A step then takes 812 cycles of an SM, of which its products need 576 (8 of 128x64x16, 4 of 128x128x16).
// At 4,096 tokens: 68.4 us, exponentials (MUFU) 57 %, issue slots 38 %. The same long prompt on the way here, in short
// runs: two tiles in one CTA, whose softmax warps fall into lockstep, 361 us (with two threads per row 403, with steps
// of 128 keys, where P lies over S, 391); one tile per CTA 349, with a quarter of the exponentials as polynomials on
// the FMA pipe 353, with Q's columns in tensor memory 345. The maximum off the softmax's path (weights against the
// last reference, once more where it moves): 342, but 3 % more for short prompts and prefixes, where it always moves.
// Key tiles are counted from the sequence's start (or the prefix split's), so a tile may reach past
// the end into another sequence's rows or stale cache slots; their weights are zero, and their V rows
// are overwritten with zeros in shared memory before the product, so that a NaN there stays there.
// Every wait is bounded in time; a timeout sets the error word and all roles leave their loops.
#include <math.h>

#include <algorithm>

#include "attn_common.cuh"
#include "chunk_common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

using attn::Ctl;
using attn::wait_bar_w;
using bf16 = __nv_bfloat16;

constexpr int TQ = 128, STEP = 64;  // query rows of a tile, keys of a step and of a K or V tile in the ring
constexpr float kRescale = 8.f;     // log2 units
constexpr int NTHREADS = 224;       // four softmax warps, the loader, S and O
constexpr int W_LOAD = 4, W_S = 5;  // and O's

template <int D>
struct Layout {
    static constexpr uint32_t QTILE = TQ * D * 2;   // D / 64 column blocks of 128 rows x 128 bytes
    static constexpr uint32_t KTILE = STEP * D * 2; // D / 64 column blocks of 64 rows x 128 bytes
    static constexpr uint32_t QBLOCK = TQ * 128, KBLOCK = STEP * 128;
    static constexpr int NST = 5;                   // K and V tiles in the ring: K of step j is tile 2 j, V tile 2 j + 1
    static constexpr uint32_t OFF_Q = 0, OFF_KV = QTILE, OFF_BAR = OFF_KV + NST * KTILE;
    // barriers: Q landed, ring full / empty, S complete, S read, P written, O += P V done, Q in tensor memory; all
    // products done
    static constexpr int QFULL = 0, FULL = 1, EMPTY = FULL + NST, SFULL = EMPTY + NST, SFREE = SFULL + 1, PREADY = SFREE + 1,
                         QT = PREADY + 1, PVD = QT + 1, FIN = PVD + 1, NBAR = FIN + 1;
    static constexpr uint32_t OFF_CTL = OFF_BAR + 8 * NBAR;
    static constexpr uint32_t OFF_FIND = OFF_CTL + 16;  // find_tile's scratch (static memory would cost a whole 1024 bytes)
    static constexpr uint32_t SMEM = OFF_FIND + 4 * (NTHREADS / 32 + 2);
    static_assert(2 * (SMEM + 1024) <= 228 * 1024, "two CTAs per SM");
    // tensor memory columns, 256 of them: S, P, 64 columns of Q, O
    static constexpr uint32_t TM_S = 0, TM_P = 64, TM_Q = 96, TM_O = 128;
};

// What a CTA works on: query positions [pos0, pos0 + P) of a sequence of `len` from token t0 on, `ns` steps
// over the keys from k0 on, `keys` of them there.
struct Item {
    int t0, len, pos0, head, k0, keys, ns, split;
};

// cu_seqlens malformed: the same answer from every thread of the CTA.
__device__ __forceinline__ bool seqlens_bad(const AttnPrefill &a) {
    bool bad = false;
    for (int n = threadIdx.x; n < a.N; n += NTHREADS) {
        const int x = a.cu[n], y = a.cu[n + 1];
        bad |= y < x || y - x > a.max_len || x < 0 || y > a.T_tot;
    }
    if (threadIdx.x == 0) bad |= a.cu[0] != 0 || a.cu[a.N] != a.T_tot;
    return __syncthreads_or(bad);
}

// The sequence and its query tile's first position (longest tiles first) that x is when tiles are numbered
// sequence by sequence: -1 beyond the last one, -2 if cu_seqlens is malformed. (Not inlined: its registers would
// cost the softmax 5 % of its speed.)
__device__ __noinline__ int2 find_tile(const int32_t *cu, int N, int T_tot, int max_len, int P, int x, int *scratch) {
    uint32_t *const sums = reinterpret_cast<uint32_t *>(scratch);  // a word per warp
    int *const found = scratch + NTHREADS / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = (N + NTHREADS - 1) / NTHREADS, n1 = min((tid + 1) * per, N);
    bool bad = tid == 0 && (cu[0] != 0 || cu[N] != T_tot);
    auto tiles = [&](int i) { return (uint32_t)(cu[i + 1] - cu[i] + P - 1) / (uint32_t)P; };
    uint32_t mine = 0;
    for (int i = tid * per; i < n1; ++i) {
        const int u = cu[i], v = cu[i + 1];
        bad |= v < u || v - u > max_len || u < 0 || v > T_tot;
        mine += tiles(i);
    }
    uint32_t upto = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, upto, m);
        if (lane >= m) upto += y;
    }
    if (lane == 31) sums[warp] = upto;
    if (tid == 0) found[0] = -1;
    if (__syncthreads_or(bad)) return make_int2(-2, 0);
    for (int w = 0; w < warp; ++w) upto += sums[w];
    uint32_t left = (uint32_t)x - (upto - mine);
    if ((uint32_t)x < upto && (uint32_t)x >= upto - mine) {
        int i = tid * per;
        for (; left >= tiles(i); ++i) left -= tiles(i);
        found[0] = i;
        found[1] = (int)(tiles(i) - 1 - left) * P;
    }
    __syncthreads();
    return make_int2(found[0], found[1]);
}

// A warp waits only for the ring tiles that it uses, K or V, each freed by the commit of its product. A wait by
// parity then is good only because the tile before in the same stage (of the other kind) has certainly landed: it
// follows the wait that shows it, as said at each.
template <int D>
__device__ __forceinline__ bool ring_full(uint64_t *bar, int c, Ctl *ctl, uint32_t *err) {
    using L = Layout<D>;
    return wait_bar_w(&bar[L::FULL + c % L::NST], (uint32_t)((c / L::NST) & 1), ctl, err);
}

template <int D>
__device__ __forceinline__ void s_loop(int ns, uint32_t tm, uint32_t sb, uint64_t *bar, Ctl *ctl, uint32_t *err) {
    using L = Layout<D>;
    const uint32_t id_s = tc::make_idesc_bf16(TQ, STEP, 0, 0);  // both operands K-major
    const tc::Desc dq = tc::split_desc(tc::make_desc_sw128(sb + L::OFF_Q, 16, 1024));
    const tc::Desc dk = tc::split_desc(tc::make_desc_sw128(sb + L::OFF_KV, 16, 1024));
    bool ok = wait_bar_w(&bar[L::QFULL], 0, ctl, err) && wait_bar_w(&bar[L::QT], 0, ctl, err);
    for (int j = 0; ok && j < ns; ++j) {
        // S of step j - 1 read: the weights of step j - 2 are written, so O has taken V of step j - 3, ring tile 2 j - 5
        if (!(ok = (j == 0 || wait_bar_w(&bar[L::SFREE], (uint32_t)((j - 1) & 1), ctl, err)) && ring_full<D>(bar, 2 * j, ctl, err)))
            break;
        tc::fence_after_sync();
        const uint32_t kb = (uint32_t)(2 * j % L::NST) * L::KTILE;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t q = (kk >> 2) * L::QBLOCK + (kk & 3) * 32, k = kb + (kk >> 2) * L::KBLOCK + (kk & 3) * 32;
            if (kk < 4)
                tc::mma_bf16_ts_off_w(tm + L::TM_S, tm + L::TM_Q + 8 * kk, dk, k, id_s, kk > 0);
            else
                tc::mma_bf16_off_w(tm + L::TM_S, dq, q, dk, k, id_s, kk > 0);
        }
        tc::mma_commit_w(&bar[L::SFULL]);
        tc::mma_commit_w(&bar[L::EMPTY + 2 * j % L::NST]);
    }
}

template <int D>
__device__ __forceinline__ void o_loop(int ns, uint32_t tm, uint32_t sb, uint64_t *bar, Ctl *ctl, uint32_t *err) {
    using L = Layout<D>;
    const uint32_t id_o = tc::make_idesc_bf16(TQ, D, 0, 1);  // V MN-major
    const tc::Desc dv = tc::split_desc(tc::make_desc_sw128(sb + L::OFF_KV, L::KBLOCK, 1024));
    bool ok = true;
    for (int j = 0; ok && j < ns; ++j) {
        const int c = 2 * j + 1;
        // the weights of step j written: its S has taken K of step j - 2, ring tile 2 j - 4, long ago
        if (!(ok = wait_bar_w(&bar[L::PREADY], (uint32_t)(j & 1), ctl, err) && ring_full<D>(bar, c, ctl, err))) break;
        tc::fence_after_sync();
        const uint32_t vb = (uint32_t)(c % L::NST) * L::KTILE;
#pragma unroll
        for (int kk = 0; kk < STEP / 16; ++kk)
            tc::mma_bf16_ts_off_w(tm + L::TM_O, tm + L::TM_P + 8 * kk, dv, vb + kk * 2048, id_o, (j > 0 || kk > 0) ? 1u : 0u);
        tc::mma_commit_w(&bar[L::PVD]);
        tc::mma_commit_w(&bar[L::EMPTY + c % L::NST]);
    }
}

enum Mode { PROMPTS, DENSE, PREFIX };  // DENSE: prompts whose query tiles are numbered sequence by sequence
template <int D, Mode MODE>
__global__ void __launch_bounds__(NTHREADS, 2)
    k_attn_prefill(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ AttnPrefill a) {
    using L = Layout<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sb = tc::smem_u32(smem);
    // (a shuffle, so that the compiler knows the roles' branches to be warp-uniform and keeps the product
    // warps' operands in uniform registers)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int P = a.P;

    attn::grid_wait();
    attn::grid_launch_dependents();  // the kernel of the own keys needs nothing of a prefix's
    Item it;
    if (MODE == PREFIX) {
        if (blockIdx.x == 0 && tid < 2) a.err[tid] = 0u;
        const int b = blockIdx.x, rb = b / (a.Hkv * a.splits), rem = b - rb * a.Hkv * a.splits;
        it.head = rem / a.splits;
        it.split = rem - it.head * a.splits;
        it.t0 = 0;
        it.len = a.T_tot;
        it.pos0 = rb * P;
        // steps spread over the splits as evenly as they go
        const int steps = (a.prefix_len + STEP - 1) / STEP;
        const int k0 = (int)((int64_t)steps * it.split / a.splits), k1 = (int)((int64_t)steps * (it.split + 1) / a.splits);
        it.k0 = k0 * STEP;
        it.keys = a.prefix_len - it.k0;
        it.ns = k1 - k0;
    } else {
        it.split = 0;
        int n;
        bool bad = false;
        if (MODE == DENSE) {
            const int x = blockIdx.x / a.Hkv;
            it.head = blockIdx.x - x * a.Hkv;
            const int2 y = find_tile(a.cu, a.N, a.T_tot, a.max_len, P, x, reinterpret_cast<int *>(smem + L::OFF_FIND));
            n = __reduce_max_sync(0xffffffffu, y.x);  // (to uniform registers, where block numbers are)
            it.pos0 = __reduce_max_sync(0xffffffffu, y.y);
            bad = n == -2;
        } else {
            // blocks are numbered so that the query tiles with the most key tiles come first
            const int per = a.Hkv * a.N, r = blockIdx.x / per, rem = blockIdx.x - r * per;
            it.head = rem / a.N;
            n = rem - it.head * a.N;
            it.pos0 = (a.blocks - 1 - r) * P;
            if (a.cu) bad = seqlens_bad(a);
        }
        // the error word, and the word that may say where a wait gave up
        if (blockIdx.x == 0 && tid < 2) a.err[tid] = bad && tid == 0 ? ERRBIT_SEQLENS : 0u;
        if (bad || n < 0) return;
        int t1;
        seq_bounds(a.cu, n, a.N, a.T_tot, it.t0, t1);
        it.len = t1 - it.t0;
        if (it.pos0 >= it.len) return;
        it.k0 = it.t0;
        it.keys = it.len;
        it.ns = (min(it.pos0 + P, it.len) + STEP - 1) / STEP;
    }
    if (sb & 1023u) {  // the operand tiles' swizzle counts on it
        if (tid == 0) atomicOr(a.err, ERRBIT_INTERNAL);
        return;
    }

    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + L::OFF_BAR);
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + L::OFF_CTL);
    if (warp == W_S) tc::tmem_alloc(&ctl->tmem, 256);
    if (tid == W_LOAD * 32) {
        for (int i = 0; i < L::NBAR; ++i) tc::mbar_init(&bar[i], (i >= L::SFREE && i < L::PVD) ? 4u : i == L::FIN ? 2u : 1u);
        ctl->abort = 0;
        ctl->wait_ns = a.wait_ns;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = __shfl_sync(0xffffffffu, ctl->tmem, 0);

    if (warp == W_LOAD) {
        if (lane == 0) {
            tc::mbar_arrive_expect_tx(&bar[L::QFULL], (uint32_t)(a.G * P) * 128u * (D / 64));
#pragma unroll
            for (int hf = 0; hf < D / 64; ++hf)
                tc::tma_load_3d(sb + L::OFF_Q + hf * L::QBLOCK, &tm_q, &bar[L::QFULL], 64 * hf, it.head * a.G, it.t0 + it.pos0);
        }
        __syncwarp();
        // paged: lane i brings box i of a tile (a page's rows, 64 of them at most), whose page number it fetched a
        // tile ahead
        const int box_log = min(a.page_log, 6), boxes = MODE == PREFIX ? STEP >> box_log : 1, rows = STEP / boxes;
        const int npages = MODE == PREFIX ? (a.prefix_len + (1 << a.page_log) - 1) >> a.page_log : 0;
        auto page_of = [&](int j) {
            const int i = (it.k0 + j * STEP + (lane << box_log)) >> a.page_log;
            int p = a.num_pages;  // beyond the tensor: reads as zero
            if (lane < boxes && i < npages) {
                const int x = a.pages[i];
                if (x >= 0 && x < a.num_pages) p = x;
            }
            return p;
        };
        int page = MODE == PREFIX ? page_of(0) : 0;
        bool ok = true;
        int c = 0;  // tiles brought
        for (int j = 0; ok && j < it.ns; ++j) {
            for (int kv = 0; kv < 2; ++kv, ++c) {
                const int st = c % L::NST;
                if (c >= L::NST && !(ok = wait_bar_w(&bar[L::EMPTY + st], (uint32_t)((c / L::NST - 1) & 1), ctl, a.err))) break;
                const bool withheld = a.withhold && c == a.withhold && blockIdx.x == 0;  // (tests of the give-up path)
                if (lane == 0 && !withheld) tc::mbar_arrive_expect_tx(&bar[L::FULL + st], L::KTILE);
                __syncwarp();
                const CUtensorMap *map = kv ? &tm_v : &tm_k;
                const uint32_t dst = sb + L::OFF_KV + st * L::KTILE + lane * rows * 128;
                if (lane < boxes && !withheld) {
#pragma unroll
                    for (int hf = 0; hf < D / 64; ++hf) {
                        if (MODE == PREFIX)
                            tc::tma_load_3d(dst + hf * L::KBLOCK, map, &bar[L::FULL + st], 64 * hf,
                                            (it.k0 + j * STEP + (lane << box_log)) & ((1 << a.page_log) - 1), page * a.Hkv + it.head);
                        else
                            tc::tma_load_3d(dst + hf * L::KBLOCK, map, &bar[L::FULL + st], 64 * hf, it.head, it.k0 + j * STEP);
                    }
                }
            }
            if (MODE == PREFIX && j + 1 < it.ns) page = page_of(j + 1);
        }
        if (lane == 0) {
            attn::drain_bar(&bar[L::QFULL], 0, ctl);
            for (int i = std::max(c - L::NST, 0); i < c; ++i) attn::drain_bar(&bar[L::FULL + i % L::NST], (i / L::NST) & 1, ctl);
        }
        __syncwarp();
    } else if (warp >= W_S) {
        if (warp == W_S)
            s_loop<D>(it.ns, tm, sb, bar, ctl, a.err);
        else
            o_loop<D>(it.ns, tm, sb, bar, ctl, a.err);
        // tensor memory may go once every product is done
        tc::mma_commit_w(&bar[L::FIN]);
        if (lane == 0) attn::drain_bar(&bar[L::FIN], 0, ctl);
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- softmax (one query row per thread)
        const int r = tid;
        const uint32_t tl = tm + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t to = tl + L::TM_O;
        const int pos = it.pos0 + r / a.G;  // position within the sequence
        const float sc = a.scale_log2;
        float m_ref = -INFINITY, l = 0.f;
        bool ok = true;
        // this row's first 64 columns of Q to tensor memory
        if ((ok = wait_bar_w(&bar[L::QFULL], 0, ctl, a.err))) {
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint4 x = *reinterpret_cast<const uint4 *>(smem + L::OFF_Q + r * 128 + ((i ^ (r & 7)) << 4));
                w[4 * i] = x.x;
                w[4 * i + 1] = x.y;
                w[4 * i + 2] = x.z;
                w[4 * i + 3] = x.w;
            }
            tc::tmem_st32(tl + L::TM_Q, w);
            tc::tmem_st_wait();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bar[L::QT]);
        }
        for (int j = 0; ok && j < it.ns; ++j) {
            if (!(ok = wait_bar_w(&bar[L::SFULL], (uint32_t)(j & 1), ctl, a.err))) break;
            tc::fence_after_sync();
            uint32_t s[2][32];
            attn::tmem_ld32x(tl + L::TM_S, s[0]);
            attn::tmem_ld32x(tl + L::TM_S + 32, s[1]);
            tc::tmem_wait_ld(s[0]);
            tc::tmem_wait_ld(s[1]);
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bar[L::SFREE]);  // the next S may overwrite these
            // keys beyond this row's position, or beyond the prefix, are masked
            if (MODE == PREFIX ? it.keys - j * STEP < STEP : it.pos0 - j * STEP < STEP - 1) {
                const int lim = (MODE == PREFIX ? it.keys - 1 : pos) - j * STEP;
#pragma unroll
                for (int i = 0; i < STEP; ++i)
                    if (i > lim) s[i >> 5][i & 31] = 0xFF800000u;  // -inf
            }
            auto S = [&](int i) { return __uint_as_float(s[i >> 5][i & 31]); };
            float pm[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) pm[i] = fmaxf(S(2 * i), S(2 * i + 1));
#pragma unroll
            for (int i = 8; i < STEP; i += 2) pm[(i >> 1) & 3] = attn::max3(pm[(i >> 1) & 3], S(i), S(i + 1));
            const float mt = attn::max3(fmaxf(pm[0], pm[1]), pm[2], pm[3]) * sc;
            // lazy rescale: a new reference maximum only when this step's exceeds it by more than kRescale
            float alpha = 1.f;
            const bool grow = mt > m_ref + kRescale;
            if (grow) {
                alpha = (m_ref == -INFINITY) ? 0.f : exp2f(m_ref - mt);
                m_ref = mt;
                l *= alpha;
            }
            if (j > 0 && __any_sync(0xffffffffu, grow)) {
                if (!(ok = wait_bar_w(&bar[L::PVD], (uint32_t)((j - 1) & 1), ctl, a.err))) break;
                tc::fence_after_sync();
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t w[32];
                    attn::tmem_ld32x(to + c0, w);
                    tc::tmem_wait_ld(w);
#pragma unroll
                    for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * alpha);
                    tc::tmem_st32(to + c0, w);
                }
            }
            // the weights as bf16 pairs
            uint64_t ps[2] = {0, 0};
            // (no finite score yet, m_ref = -inf: those weights are zero too, and -inf - -inf would be NaN)
            const float m0 = m_ref == -INFINITY ? 0.f : -m_ref;
            const uint64_t sc2 = attn::pack2(sc, sc), mm2 = attn::pack2(m0, m0);
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const uint64_t x = attn::fma2(attn::pack2(S(2 * i), S(2 * i + 1)), sc2, mm2);
                float p0, p1;
                attn::unpack2(x, p0, p1);
                p0 = chunk::ex2(p0);
                p1 = chunk::ex2(p1);
                ps[i & 1] = attn::add2(ps[i & 1], attn::pack2(p0, p1));
                w[i] = tc::pack_bf16x2(p0, p1);
            }
            if (j >= 1) {  // the last weights have been read
                if (!(ok = wait_bar_w(&bar[L::PVD], (uint32_t)((j - 1) & 1), ctl, a.err))) break;
                tc::fence_after_sync();
            }
            tc::tmem_st32(tl + L::TM_P, w);
            float a0, a1;
            attn::unpack2(attn::add2(ps[0], ps[1]), a0, a1);
            l += a0 + a1;
            if (it.keys - j * STEP < STEP) {
                // rows of V beyond the sequence or the prefix: another sequence's values or stale slots
                const int c = 2 * j + 1, st = c % L::NST, n = it.keys - j * STEP;
                if (!(ok = wait_bar_w(&bar[L::FULL + st], (uint32_t)((c / L::NST) & 1), ctl, a.err))) {
                    tc::tmem_st_wait();  // the weights' store must end before the tensor memory goes
                    break;
                }
                if (r >= n && r < STEP) {
#pragma unroll
                    for (int hf = 0; hf < D / 64; ++hf)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            chunk::st_shared_v4(sb + L::OFF_KV + st * L::KTILE + hf * L::KBLOCK + r * 128 + i * 16, 0, 0, 0, 0);
                }
                tc::fence_smem_to_async();
            }
            tc::tmem_st_wait();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bar[L::PREADY]);
        }
        if (ok)
            ok = wait_bar_w(&bar[L::PVD], (uint32_t)((it.ns - 1) & 1), ctl, a.err);
        if (ok) {
            tc::fence_after_sync();
            const bool valid = r < a.G * P && pos < it.len;
            const int64_t row = (int64_t)(it.t0 + pos) * a.Hq + it.head * a.G + r % a.G;
            if (MODE == PREFIX) {
                // unnormalised, with the reference maximum (log2 units) and the sum
                const int64_t prow = (int64_t)it.split * a.T_tot * a.Hq + row;
                if (valid) a.part_ml[prow] = make_float2(m_ref, l);
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    float x[32];
                    tc::tmem_ld32(to + c0, x);
                    if (valid) {
#pragma unroll
                        for (int i = 0; i < 32; i += 8) attn::st_global8(a.part_o + prow * D + c0 + i, x + i);
                    }
                }
            } else {
                const float inv = 1.f / l;
                bf16 *dst = a.o + row * D;
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    float x[32];
                    tc::tmem_ld32(to + c0, x);
                    if (valid) {
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            *reinterpret_cast<uint4 *>(dst + c0 + i) = make_uint4(
                                tc::pack_bf16x2(x[i] * inv, x[i + 1] * inv), tc::pack_bf16x2(x[i + 2] * inv, x[i + 3] * inv),
                                tc::pack_bf16x2(x[i + 4] * inv, x[i + 5] * inv), tc::pack_bf16x2(x[i + 6] * inv, x[i + 7] * inv));
                    }
                }
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == W_S) tc::tmem_dealloc(tm, 256);
}

template <int D>
cudaError_t launch_prompt(AttnPrefill a, cudaStream_t st, const char **stage) {
    cudaError_t e;
    a.P = TQ / a.G;
    a.blocks = (a.max_len + a.P - 1) / a.P;
    // With as many blocks for every sequence as for the longest, the longest tiles of all sequences start first and
    // a block knows its tile from its number, but those without a tile take their turn too. Numbered sequence by
    // sequence no block is empty, and each takes 0.7 us more to find its tile. 16/4 heads, d = 128: one prompt of
    // 8,192 among 255 of 32 tokens 2,273 us against 255; 4,096 and 15 of 256 117
    // against 77; 8 of 600 to 4,096, with 2.2 blocks a tile, 165 against 159; but 300 of 16 tokens 31 against 36, and
    // six of up to 200, whose blocks all run at once, 6.6 against 7.4.
    const int64_t tiles = attn_prefill_tiles(a.T_tot, a.N, a.P), each = (int64_t)a.blocks * a.N;
    a.dense = a.cu && each > tiles + tiles / 2 && each * a.Hkv > kPromptCtas;
    CUtensorMap tm_q, tm_k, tm_v;
    *stage = "TMA descriptor encoding";
    if ((e = attn::make_map(&tm_q, a.q, D, a.Hq, a.T_tot, D, a.q_stride, a.G, a.P)) != cudaSuccess) return e;
    if ((e = attn::make_map(&tm_k, a.k, D, a.Hkv, a.T_tot, D, a.k_stride, 1, STEP)) != cudaSuccess) return e;
    if ((e = attn::make_map(&tm_v, a.v, D, a.Hkv, a.T_tot, D, a.v_stride, 1, STEP)) != cudaSuccess) return e;
    *stage = "attn_prefill";
    auto kern = a.dense ? k_attn_prefill<D, DENSE> : k_attn_prefill<D, PROMPTS>;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<D>::SMEM)) != cudaSuccess)
        return e;
    void *pr = prof_start("attn_prefill", st);
    e = attn::launch_early(kern, (unsigned)((a.dense ? tiles : each) * a.Hkv), NTHREADS, Layout<D>::SMEM, st, tm_q, tm_k, tm_v, a);
    prof_stop(pr);
    return e;
}

template <int D>
cudaError_t launch_prefix(AttnPrefill a, cudaStream_t st, const char **stage) {
    cudaError_t e;
    a.P = TQ / a.G;
    a.blocks = (a.T_tot + a.P - 1) / a.P;
    CUtensorMap tm_q, tm_k, tm_v;
    *stage = "TMA descriptor encoding";
    const uint64_t page = 1u << a.page_log, n = (uint64_t)a.num_pages * a.Hkv;
    if ((e = attn::make_map(&tm_q, a.q, D, a.Hq, a.T_tot, D, (uint64_t)a.Hq * D, a.G, a.P)) != cudaSuccess) return e;
    if ((e = attn::make_map(&tm_k, a.k, D, page, n, D, page * D, (uint32_t)std::min<uint64_t>(page, 64), 1)) != cudaSuccess) return e;
    if ((e = attn::make_map(&tm_v, a.v, D, page, n, D, page * D, (uint32_t)std::min<uint64_t>(page, 64), 1)) != cudaSuccess) return e;
    *stage = "attn_prefix";
    auto kern = k_attn_prefill<D, PREFIX>;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<D>::SMEM)) != cudaSuccess)
        return e;
    void *pr = prof_start("attn_prefix", st);
    e = attn::launch_early(kern, (unsigned)(a.blocks * a.Hkv * a.splits), NTHREADS, Layout<D>::SMEM, st, tm_q, tm_k, tm_v, a);
    prof_stop(pr);
    return e;
}

}  // namespace

int64_t attn_prefill_tiles(int T_tot, int N, int P) { return (T_tot + (int64_t)N * (P - 1)) / P; }

cudaError_t launch_attn_prefix(const AttnPrefill &a, int d, cudaStream_t st, const char **stage) {
    return d == 64 ? launch_prefix<64>(a, st, stage) : launch_prefix<128>(a, st, stage);
}

cudaError_t launch_attn_prefill(AttnPrefill a, int d, cudaStream_t st, const char **stage) {
    const Inject inj = inject_settings();
    a.wait_ns = inj.wait_ns ? inj.wait_ns : attn::kWaitNs;
    a.withhold = inj.withhold_tile;
    if (a.T_tot == 0 || a.max_len == 0) {
        // nothing to compute: only the error word (cu_seqlens must then be all zeros)
        *stage = "error word";
        return launch_validate_seqlens(a.cu, a.N, a.T_tot, a.err, st);
    }
    return d == 64 ? launch_prompt<64>(a, st, stage) : launch_prompt<128>(a, st, stage);
}

}  // namespace gdn
