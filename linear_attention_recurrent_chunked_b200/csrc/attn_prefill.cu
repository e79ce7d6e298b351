// Causal attention with grouped heads over packed prompts, and the same kernel without the mask over
// a cached prefix that a whole decode batch shares, on the sm_100a tensor cores.
//
//     o_t = sum_{j <= t} softmax_j(scale q_t . k_j) v_j,     key head = query head / G, G = Hq / Hkv
//
// A tile of 128 query rows packs P = floor(128 / G) consecutive positions times the G query heads of
// one key head, position-major, which is the order in which one TMA box {64 columns, G heads,
// P positions} lands. All rows of a tile then share their key and value tiles whatever G is, and a
// tile's causal edge is P positions long. Per key tile of 128 keys
//
//     S = Q K^T (tensor memory)  ->  P = 2^(S c - m) (bf16, over S)  ->  O += P V (tensor memory)
//
// with c = scale log2(e) and m a running row maximum that moves only when the true one has grown by
// more than 8, so P <= 2^8 and O and the row sum l are seldom rescaled; o = O / l. P is rounded to
// bf16 for the tensor core (at most 2^-8 of each weight); l sums the unrounded weights in fp32.
//
// One CTA holds two tiles (256 rows), and S comes in steps of 64 keys with two buffers per tile: the
// softmax of one step of a tile runs while the tensor core computes the tile's next S and the other
// tile's products. Roles:
//   softmax  (2 x 4 warps)  one query row per thread
//   loader   (1 warp)       TMA: Q once, then K and V tiles of 128 keys through one ring
//   MMA      (1 warp)       per step and query tile: O += P V; then, one product later, the S two steps on
//                           into the buffer that P was in, once that product has read P (a later
//                           tcgen05.mma is not ordered after an earlier one's tensor-memory operand reads)
// Bound: the tensor pipe. A step of a tile costs 8 products M=128 N=64 K=16 for S, whose operands both
// come from shared memory (6 KB each at 128 bytes a cycle: 48 cycles, against 32 of arithmetic), and
// 4 products M=128 N=128 K=16 for O (64 cycles each, V alone from shared memory): 640 cycles. With steps
// of 128 keys S would run at its arithmetic rate (1024 cycles for twice the keys), but tensor memory then
// holds one S buffer per tile beside O, and the chain S -> maximum -> weights -> O -> next S (4,250
// cycles measured, half of it barrier and tensor-memory latencies) sets the pace instead.
// Key tiles are counted from the sequence's start (or the prefix split's), so a tile may reach past
// the end into another sequence's rows or stale cache slots; their weights are zero, and their V rows
// are overwritten with zeros in shared memory before the product, so that a NaN there stays there.
// Every wait is bounded in time; a timeout sets the error word and all roles leave their loops.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "attn_common.cuh"
#include "chunk_common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

using attn::Ctl;
using attn::wait_bar;
using attn::wait_bar_w;
using bf16 = __nv_bfloat16;

constexpr int TQ = 128, TK = 128;   // query rows of a tile, keys of a K or V tile in the ring
constexpr int STEP = 64;            // keys of a step: half a ring tile
constexpr float kRescale = 8.f;  // log2 units
constexpr int NTHREADS = 416;
constexpr int W_LOAD = 8, W_MMA = 9;

template <int D>
struct Layout {
    static constexpr uint32_t TILE = 128 * D * 2;      // D / 64 column blocks of 128 rows x 128 bytes
    static constexpr int NST = D == 128 ? 5 : 8;       // K and V tiles in the ring
    static constexpr uint32_t OFF_Q = 0, OFF_KV = 2 * TILE, OFF_BAR = OFF_KV + NST * TILE;
    // barriers: Q landed, ring full / empty, per query tile: S complete, S read, P written, O += P V done, Q in
    // tensor memory; the first weights of tile 0; all products done
    static constexpr int QFULL = 0, FULL = 1, EMPTY = FULL + NST, SFULL = EMPTY + NST, SFREE = SFULL + 2,
                         PREADY = SFREE + 2, QT = PREADY + 2, START = QT + 2, PVD = START + 1, FIN = PVD + 2, NBAR = FIN + 1;
    static constexpr uint32_t OFF_CTL = OFF_BAR + 8 * NBAR;
    static constexpr uint32_t SMEM = OFF_CTL + 16 + 1024;
    // tensor memory columns: S of tile u at u * 64, P at 128 + u * 32, Q of the first QT_TILES tiles, O at 256 + u * D
    static constexpr uint32_t TM_S = 0, TM_P = 128, TM_Q = 192, TM_O = 256;
    static constexpr int QT_TILES = 128 / D;
    static constexpr int POLY = D == 64 ? 2 : 0;       // of every 8 weights, those that the FMA pipe computes: see the softmax
};

// What a CTA works on: query positions [pos0, pos0 + 2 P) of a sequence of `len` from token t0 on, ns0 and
// ns1 steps of its two query tiles (ns1 is 0 or at least ns0) over the keys from k0 on, `keys` of them there.
struct Item {
    int t0, len, pos0, head, k0, keys, ns0, ns1, split;
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

// The ring holds K of steps 2 t and 2 t + 1 as tile 2 t, V of them as tile 2 t + 1. A tile is freed by two
// arrivals, one for each query tile: the commit of that query tile's last product on it, or the loader's own
// where it has none. A warp waits only for the tiles that it uses, K or V: a parity wait then is good only
// because the tile before in the same stage (of the other kind) has certainly landed, as the same query
// tile's earlier products read it.
template <int D>
__device__ __forceinline__ bool ring_full(uint64_t *bar, int c, Ctl *ctl, uint32_t *err) {
    using L = Layout<D>;
    return wait_bar_w(&bar[L::FULL + c % L::NST], (uint32_t)((c / L::NST) & 1), ctl, err);
}

// S of query tile U, issued by a warp of its own. The second tile starts when the first has its first
// weights, which keeps the two tiles about half a step apart: in step they would wait for the MUFU and the
// tensor core together and leave both idle together (10k prompt: 391 us in step, 352 us apart).
template <int D, int U>
__device__ __forceinline__ void s_loop(std::integral_constant<int, U> u, int myns, uint32_t tm, uint32_t sb,
                                       uint64_t *bar, Ctl *ctl, uint32_t *err) {
    using L = Layout<D>;
    const uint32_t id_s = tc::make_idesc_bf16(TQ, STEP, 0, 0);  // both operands K-major
    const tc::Desc dq = tc::split_desc(tc::make_desc_sw128(sb + L::OFF_Q + u * L::TILE, 16, 1024));
    const tc::Desc dk = tc::split_desc(tc::make_desc_sw128(sb + L::OFF_KV, 16, 1024));
    constexpr bool TS = U < L::QT_TILES;
    bool ok = myns == 0 || wait_bar_w(&bar[TS ? L::QT + U : L::QFULL], 0, ctl, err);
    if (ok && U == 1 && myns > 0) ok = wait_bar_w(&bar[L::START], 0, ctl, err);
    for (int j = 0; ok && j < myns; ++j) {
        const int c = j & ~1;
        if (!(ok = ((j & 1) || ring_full<D>(bar, c, ctl, err)) &&
                   (j == 0 || wait_bar_w(&bar[L::SFREE + u], (uint32_t)((j - 1) & 1), ctl, err))))
            break;
        tc::fence_after_sync();
        const uint32_t kb = (uint32_t)(c % L::NST) * L::TILE + (j & 1) * (STEP * 128);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
            if (TS)
                tc::mma_bf16_ts_off_w(tm + L::TM_S + u * 64, tm + L::TM_Q + u * (D / 2) + 8 * kk, dk, kb + off, id_s, kk > 0);
            else
                tc::mma_bf16_off_w(tm + L::TM_S + u * 64, dq, off, dk, kb + off, id_s, kk > 0);
        }
        tc::mma_commit_w(&bar[L::SFULL + u]);
        if ((j & 1) || j + 1 == myns) tc::mma_commit_w(&bar[L::EMPTY + c % L::NST]);
    }
}

// O of query tile u, issued by a warp of its own.
template <int D, int U>
__device__ __forceinline__ void pv_loop(std::integral_constant<int, U> u, int myns, uint32_t tm, uint32_t sb,
                                        uint64_t *bar, Ctl *ctl, uint32_t *err) {
    using L = Layout<D>;
    const uint32_t id_o = tc::make_idesc_bf16(TQ, D, 0, 1);  // V MN-major
    const tc::Desc dv = tc::split_desc(tc::make_desc_sw128(sb + L::OFF_KV, 16384, 1024));
    bool ok = true;
    for (int j = 0; ok && j < myns; ++j) {
        const int b = j & 1, c = j | 1;
        if (!(ok = (b || ring_full<D>(bar, c, ctl, err)) &&
                   wait_bar_w(&bar[L::PREADY + u], (uint32_t)(j & 1), ctl, err)))
            break;
        tc::fence_after_sync();
        const uint32_t vb = (uint32_t)(c % L::NST) * L::TILE + b * (STEP * 128);
#pragma unroll
        for (int kk = 0; kk < STEP / 16; ++kk)
            tc::mma_bf16_ts_off_w(tm + L::TM_O + u * D, tm + L::TM_P + u * 32 + 8 * kk, dv, vb + kk * 2048, id_o,
                                  (j > 0 || kk > 0) ? 1u : 0u);
        tc::mma_commit_w(&bar[L::PVD + u]);
        if (b || j + 1 == myns) tc::mma_commit_w(&bar[L::EMPTY + c % L::NST]);
    }
}

template <int D, bool PREFIX>
__global__ void __launch_bounds__(NTHREADS, 1)
    k_attn_prefill(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ AttnPrefill a) {
    using L = Layout<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = tc::smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw_base & 1023u)) & 1023u);
    const uint32_t sb = tc::smem_u32(smem);
    // (a shuffle, so that the compiler knows the roles' branches to be warp-uniform and keeps the product
    // warps' operands in uniform registers)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int P = a.P;

    attn::grid_wait();
    attn::grid_launch_dependents();  // the kernel of the own keys needs nothing of a prefix's
    Item it;
    if (PREFIX) {
        if (blockIdx.x == 0 && tid < 2) a.err[tid] = 0u;
        const int b = blockIdx.x, rb = b / (a.Hkv * a.splits), rem = b - rb * a.Hkv * a.splits;
        it.head = rem / a.splits;
        it.split = rem - it.head * a.splits;
        it.t0 = 0;
        it.len = a.T_tot;
        it.pos0 = rb * 2 * P;
        // steps spread over the splits as evenly as they go
        const int steps = (a.prefix_len + STEP - 1) / STEP;
        const int k0 = (int)((int64_t)steps * it.split / a.splits), k1 = (int)((int64_t)steps * (it.split + 1) / a.splits);
        it.k0 = k0 * STEP;
        it.keys = a.prefix_len - it.k0;
        it.ns0 = k1 - k0;
        it.ns1 = it.pos0 + P < it.len ? it.ns0 : 0;
    } else {
        // blocks are numbered so that the query tiles with the most key tiles come first
        const int per = a.Hkv * a.N, r = blockIdx.x / per, rem = blockIdx.x - r * per;
        it.head = rem / a.N;
        const int n = rem - it.head * a.N;
        it.split = 0;
        if (a.cu) {
            const bool bad = seqlens_bad(a);
            if (blockIdx.x == 0 && tid < 2) a.err[tid] = bad && tid == 0 ? ERRBIT_SEQLENS : 0u;
            if (bad) return;
        } else if (blockIdx.x == 0 && tid < 2) {
            a.err[tid] = 0u;  // and the word that may say where a wait gave up
        }
        int t1;
        seq_bounds(a.cu, n, a.N, a.T_tot, it.t0, t1);
        it.len = t1 - it.t0;
        it.pos0 = (a.blocks - 1 - r) * 2 * P;
        if (it.pos0 >= it.len) return;
        it.k0 = it.t0;
        it.keys = it.len;
        const int e0 = min(it.pos0 + P, it.len), e1 = min(it.pos0 + 2 * P, it.len);
        it.ns0 = (e0 + STEP - 1) / STEP;
        it.ns1 = e1 > it.pos0 + P ? (e1 + STEP - 1) / STEP : 0;
    }
    const int ns = max(it.ns0, it.ns1), nk = (ns + 1) / 2;  // steps, ring tiles

    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + L::OFF_BAR);
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + L::OFF_CTL);
    if (warp == W_MMA) tc::tmem_alloc(&ctl->tmem, 512);
    if (tid == W_LOAD * 32) {
        for (int i = 0; i < L::NBAR; ++i) tc::mbar_init(&bar[i], (i >= L::SFREE && i < L::PVD) ? 4u : i == L::FIN ? 4u : (i >= L::EMPTY && i < L::SFULL) ? 2u : 1u);
        ctl->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = __shfl_sync(0xffffffffu, ctl->tmem, 0);

    if (warp == W_LOAD) {
        if (lane == 0) {
            const uint32_t bytes = (uint32_t)(a.G * P) * 128u * (D / 64);
            tc::mbar_arrive_expect_tx(&bar[L::QFULL], it.ns1 ? 2 * bytes : bytes);
            for (int u = 0; u < (it.ns1 ? 2 : 1); ++u)
#pragma unroll
                for (int hf = 0; hf < D / 64; ++hf)
                    tc::tma_load_3d(sb + L::OFF_Q + u * L::TILE + hf * 16384, &tm_q, &bar[L::QFULL], 64 * hf, it.head * a.G,
                                    it.t0 + it.pos0 + u * P);
        }
        __syncwarp();
        // paged: lane i brings box i of a tile (a page's rows, 64 of them at most), whose page number it fetched a
        // tile ahead
        const int box_log = min(a.page_log, 6), boxes = PREFIX ? TK >> box_log : 1, rows = TK / boxes;
        const int npages = PREFIX ? (a.prefix_len + (1 << a.page_log) - 1) >> a.page_log : 0;
        auto page_of = [&](int j) {
            const int i = (it.k0 + j * TK + (lane << box_log)) >> a.page_log;
            int p = a.num_pages;  // beyond the tensor: reads as zero
            if (lane < boxes && i < npages) {
                const int x = a.pages[i];
                if (x >= 0 && x < a.num_pages) p = x;
            }
            return p;
        };
        int page = PREFIX ? page_of(0) : 0;
        bool ok = true;
        int c = 0;  // tiles brought
        for (int j = 0; ok && j < nk; ++j) {
            for (int kv = 0; kv < 2; ++kv, ++c) {
                const int st = c % L::NST;
                if (c >= L::NST && !(ok = wait_bar_w(&bar[L::EMPTY + st], (uint32_t)((c / L::NST - 1) & 1), ctl, a.err))) break;
                if (lane == 0) {
                    if (2 * j >= it.ns0) tc::mbar_arrive(&bar[L::EMPTY + st]);  // a query tile that does not use it
                    if (2 * j >= it.ns1) tc::mbar_arrive(&bar[L::EMPTY + st]);
                    tc::mbar_arrive_expect_tx(&bar[L::FULL + st], L::TILE);
                }
                __syncwarp();
                const CUtensorMap *map = kv ? &tm_v : &tm_k;
                const uint32_t dst = sb + L::OFF_KV + st * L::TILE + lane * rows * 128;
                if (lane < boxes) {
#pragma unroll
                    for (int hf = 0; hf < D / 64; ++hf) {
                        if (PREFIX)
                            tc::tma_load_3d(dst + hf * 16384, map, &bar[L::FULL + st], 64 * hf,
                                            (it.k0 + j * TK + (lane << box_log)) & ((1 << a.page_log) - 1), page * a.Hkv + it.head);
                        else
                            tc::tma_load_3d(dst + hf * 16384, map, &bar[L::FULL + st], 64 * hf, it.head, it.k0 + j * TK);
                    }
                }
            }
            if (PREFIX && j + 1 < nk) page = page_of(j + 1);
        }
        if (lane == 0) {
            attn::drain_bar(&bar[L::QFULL], 0);
            for (int i = std::max(c - L::NST, 0); i < c; ++i) attn::drain_bar(&bar[L::FULL + i % L::NST], (i / L::NST) & 1);
        }
        __syncwarp();
    } else if (warp >= W_MMA) {
        if (warp == W_MMA)
            s_loop<D>(std::integral_constant<int, 0>(), it.ns0, tm, sb, bar, ctl, a.err);
        else if (warp == W_MMA + 1)
            s_loop<D>(std::integral_constant<int, 1>(), it.ns1, tm, sb, bar, ctl, a.err);
        else if (warp == W_MMA + 2)
            pv_loop<D>(std::integral_constant<int, 0>(), it.ns0, tm, sb, bar, ctl, a.err);
        else
            pv_loop<D>(std::integral_constant<int, 1>(), it.ns1, tm, sb, bar, ctl, a.err);
        // tensor memory may go once every product is done
        tc::mma_commit_w(&bar[L::FIN]);
        if (lane == 0) attn::drain_bar(&bar[L::FIN], 0);
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- softmax (one query row per thread)
        const int u = warp >> 2, r = tid & 127;
        const uint32_t tl = tm + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t to = tl + L::TM_O + u * D;
        const int myns = u ? it.ns1 : it.ns0;
        const int pos = it.pos0 + u * P + r / a.G;  // position within the sequence
        const int first = it.pos0 + u * P;          // the tile's first position
        const float sc = a.scale_log2;
        float m_ref = -INFINITY, l = 0.f;
        bool ok = true;
        if (u < L::QT_TILES && myns) {
            // this row of Q to tensor memory, where the products for S read it without shared memory
            ok = wait_bar_w(&bar[L::QFULL], 0, ctl, a.err);
            if (ok) {
#pragma unroll
                for (int hf = 0; hf < D / 64; ++hf) {
                    uint32_t w[32];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(smem + L::OFF_Q + u * L::TILE + hf * 16384 + r * 128 + ((i ^ (r & 7)) << 4));
                        w[4 * i] = x.x;
                        w[4 * i + 1] = x.y;
                        w[4 * i + 2] = x.z;
                        w[4 * i + 3] = x.w;
                    }
                    tc::tmem_st32(tl + L::TM_Q + u * (D / 2) + hf * 32, w);
                }
                tc::tmem_st_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bar[L::QT + u]);
            }
        }
        for (int j = 0; ok && j < myns; ++j) {
            const uint32_t ts = tl + L::TM_S + u * 64;
            if (!(ok = wait_bar_w(&bar[L::SFULL + u], (uint32_t)(j & 1), ctl, a.err))) break;
            tc::fence_after_sync();
            // keys beyond this row's position, or beyond the prefix, are masked
            uint32_t s[2][32];
            attn::tmem_ld32x(ts, s[0]);
            attn::tmem_ld32x(ts + 32, s[1]);
            tc::tmem_wait_ld(s[0]);
            tc::tmem_wait_ld(s[1]);
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bar[L::SFREE + u]);  // the next S may overwrite these
            if (PREFIX ? it.keys - j * STEP < STEP : first - j * STEP < STEP - 1) {
                const int lim = (PREFIX ? it.keys - 1 : pos) - j * STEP;
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
            // lazy rescale: a new reference maximum only when this step's exceeds it by more than kRescale. (A step
            // may be masked whole for a row, mt = -inf, but never the first one.)
            float alpha = 1.f;
            const bool grow = mt > m_ref + kRescale;
            if (grow) {
                alpha = (m_ref == -INFINITY) ? 0.f : exp2f(m_ref - mt);
                m_ref = mt;
                l *= alpha;
            }
            if (j > 0 && __any_sync(0xffffffffu, grow)) {
                if (!(ok = wait_bar_w(&bar[L::PVD + u], (uint32_t)((j - 1) & 1), ctl, a.err))) break;
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
            // the weights as bf16 pairs over the first 32 columns of the buffer. For D = 64, where the products take
            // half the time, the MUFU (8 cycles a warp's exponential) would be the bound, and the FMA pipe takes a quarter
            uint64_t ps[2] = {0, 0};
            const uint64_t sc2 = attn::pack2(sc, sc), mm2 = attn::pack2(-m_ref, -m_ref);
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const uint64_t x = attn::fma2(attn::pack2(S(2 * i), S(2 * i + 1)), sc2, mm2);
                float p0, p1;
                if ((i & 3) >= 4 - L::POLY / 2) {
                    attn::exp2_poly(x, p0, p1);
                } else {
                    attn::unpack2(x, p0, p1);
                    p0 = chunk::ex2(p0);
                    p1 = chunk::ex2(p1);
                }
                ps[i & 1] = attn::add2(ps[i & 1], attn::pack2(p0, p1));
                w[i] = tc::pack_bf16x2(p0, p1);
            }
            if (j >= 1) {  // the last weights have been read
                if (!(ok = wait_bar_w(&bar[L::PVD + u], (uint32_t)((j - 1) & 1), ctl, a.err))) break;
                tc::fence_after_sync();
            }
            tc::tmem_st32(tl + L::TM_P + u * 32, w);
            float a0, a1;
            attn::unpack2(attn::add2(ps[0], ps[1]), a0, a1);
            l += a0 + a1;
            if (it.keys - j * STEP < STEP) {
                // rows of V beyond the sequence or the prefix: another sequence's values or stale slots
                const int c = j | 1, st = c % L::NST, n = it.keys - j * STEP;
                if (!(ok = wait_bar_w(&bar[L::FULL + st], (uint32_t)((c / L::NST) & 1), ctl, a.err))) break;
                if (r >= n && r < STEP) {
#pragma unroll
                    for (int hf = 0; hf < D / 64; ++hf)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            chunk::st_shared_v4(sb + L::OFF_KV + st * L::TILE + hf * 16384 + ((j & 1) * STEP + r) * 128 + i * 16, 0, 0,
                                                0, 0);
                }
                tc::fence_smem_to_async();
            }
            tc::tmem_st_wait();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(&bar[L::PREADY + u]);
                if (u == 0 && j == 0) tc::mbar_arrive(&bar[L::START]);  // (PREADY's phases come round; this one's does not)
            }
        }
        if (ok && myns)
            ok = wait_bar_w(&bar[L::PVD + u], (uint32_t)((myns - 1) & 1), ctl, a.err);
        if (ok && myns) {
            tc::fence_after_sync();
            const bool valid = r < a.G * P && pos < it.len;
            const int64_t row = (int64_t)(it.t0 + pos) * a.Hq + it.head * a.G + r % a.G;
            if (PREFIX) {
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
    if (warp == W_MMA) tc::tmem_dealloc(tm, 512);
}

template <int D>
cudaError_t launch_prompt(AttnPrefill a, cudaStream_t st, const char **stage) {
    cudaError_t e;
    a.P = TQ / a.G;
    a.blocks = (a.max_len + 2 * a.P - 1) / (2 * a.P);
    CUtensorMap tm_q, tm_k, tm_v;
    *stage = "TMA descriptor encoding";
    if ((e = attn::make_map(&tm_q, a.q, D, a.Hq, a.T_tot, D, a.q_stride, a.G, a.P)) != cudaSuccess) return e;
    if ((e = attn::make_map(&tm_k, a.k, D, a.Hkv, a.T_tot, D, a.k_stride, 1, TK)) != cudaSuccess) return e;
    if ((e = attn::make_map(&tm_v, a.v, D, a.Hkv, a.T_tot, D, a.v_stride, 1, TK)) != cudaSuccess) return e;
    *stage = "attn_prefill";
    auto kern = k_attn_prefill<D, false>;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<D>::SMEM)) != cudaSuccess)
        return e;
    void *pr = prof_start("attn_prefill", st);
    e = attn::launch_early(kern, (unsigned)(a.blocks * a.Hkv * a.N), NTHREADS, Layout<D>::SMEM, st, tm_q, tm_k, tm_v, a);
    prof_stop(pr);
    return e;
}

template <int D>
cudaError_t launch_prefix(AttnPrefill a, cudaStream_t st, const char **stage) {
    cudaError_t e;
    a.P = TQ / a.G;
    a.blocks = (a.T_tot + 2 * a.P - 1) / (2 * a.P);
    CUtensorMap tm_q, tm_k, tm_v;
    *stage = "TMA descriptor encoding";
    const uint64_t page = 1u << a.page_log, n = (uint64_t)a.num_pages * a.Hkv;
    if ((e = attn::make_map(&tm_q, a.q, D, a.Hq, a.T_tot, D, (uint64_t)a.Hq * D, a.G, a.P)) != cudaSuccess) return e;
    if ((e = attn::make_map(&tm_k, a.k, D, page, n, D, page * D, (uint32_t)std::min<uint64_t>(page, 64), 1)) != cudaSuccess) return e;
    if ((e = attn::make_map(&tm_v, a.v, D, page, n, D, page * D, (uint32_t)std::min<uint64_t>(page, 64), 1)) != cudaSuccess) return e;
    *stage = "attn_prefix";
    auto kern = k_attn_prefill<D, true>;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<D>::SMEM)) != cudaSuccess)
        return e;
    void *pr = prof_start("attn_prefix", st);
    e = attn::launch_early(kern, (unsigned)(a.blocks * a.Hkv * a.splits), NTHREADS, Layout<D>::SMEM, st, tm_q, tm_k, tm_v, a);
    prof_stop(pr);
    return e;
}

}  // namespace

cudaError_t launch_attn_prefix(const AttnPrefill &a, int d, cudaStream_t st, const char **stage) {
    return d == 64 ? launch_prefix<64>(a, st, stage) : launch_prefix<128>(a, st, stage);
}

cudaError_t launch_attn_prefill(const AttnPrefill &a, int d, cudaStream_t st, const char **stage) {
    if (a.T_tot == 0 || a.max_len == 0) {
        // nothing to compute: only the error word (cu_seqlens must then be all zeros)
        *stage = "error word";
        return launch_validate_seqlens(a.cu, a.N, a.T_tot, a.err, st);
    }
    return d == 64 ? launch_prompt<64>(a, st, stage) : launch_prompt<128>(a, st, stage);
}

}  // namespace gdn
