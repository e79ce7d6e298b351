// Norms of queries and keys for each head with the position rotation in the same pass, and the
// write of keys and values into the pages of the layer's cache: what an attention layer of the
// hybrid backbone does between its projection and its attention (page 1, abstract: the backbone
// interleaves recurrent layers with causal attention layers; the pages print neither step).
//
//     x^ = x w / sqrt(mean(x^2) + eps)                       per (token, head) row of d elements
//     y_i       = x^_i cos(a_i) - x^_{i+r/2} sin(a_i)        i < r/2, a_i = pos base^(-2i/r)
//     y_{i+r/2} = x^_{i+r/2} cos(a_i) + x^_i sin(a_i)        elements from r on: y = x^
//
// all in fp32 and rounded once, when y is stored. The angle is formed in turns, pos f_i with f_i =
// base^(-2i/r) / (2 pi), as a 64-bit binary fraction that wraps by itself: pos times 2^64 f_i modulo 2^64.
// The frequencies come from a chain of up to 63 rounded products, which puts 2^64 f_i off by 30 at most (up to 3.7
// found, for bases near 1), 2^-28 turns at any int32 position, where an fp32 product would be off by 0.06 radians at
// position 10^6 already. The fraction's upper 32 bits, 2^-32 less at most, then become a signed fp32 value within
// 2^-26: together less than 2^-25 turns, 2e-7 radians.
//
// Bound: HBM (each row is read once and written once), as long as few enough instructions are spent on
// an element. A lane holds two 16-byte runs of a row: a run of first elements of pairs and the run of their
// partners r/2 elements on (or, beyond r, two runs next to each other), so that only the sum of squares
// takes shuffles and nothing passes through shared memory. With w folded into the cosines and sines an
// element costs one product, one multiply-add and one more product,
//     y = (x (w c) + x' (w' s)) / sqrt(mean(x^2) + eps),       x' the partner, w' its weight,
// in packed pairs. The rows of all tokens are cut evenly over the warps of one resident grid, whatever T
// is: with few tokens (a decode step) each warp has one group of rows; with many a warp walks through
// tokens, computes a token's sines and cosines once for all of its heads there (a lane keeps the same
// columns for every row), loads the next rows while it works on these and asks L2 for those a token on.
// 10240 tokens, 16 + 4 heads of 128 in bf16, keys and values cached: 136 MB in 27.5 us (4.96 TB/s; a plain
// copy of as many bytes takes 23.4 us), issue slots 58 % busy. One run a lane with shuffled partners, a token a
// warp: 40 us; at 29.5 us, without the L2 prefetch 33; with 3 CTAs per SM 30.1, with 5 (two row groups no longer
// fit the registers) 32.7; at 28.0, with the prefetch two tokens ahead 30.3, and 27.5 once the loads were hinted as
// first out of L2. A decode step's 64 tokens: 2.7 us, a launch.
#include <math.h>

#include <algorithm>

#include "attn_common.cuh"
#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

constexpr int kWarps = 4;     // per CTA
constexpr int kResident = 4;  // CTAs per SM
constexpr int kUnroll = 2;    // row groups whose loads are in flight together

struct Freq {
    uint64_t f[64];  // 2^64 turns per position of pair i
};

struct Args {
    NormRope a;
    int gq, gk, gv;  // groups of rows that a warp holds at a time: of queries, keys, values (when cached)
    int64_t warps;   // over which the T (gq + gk + gv) groups are cut
    int page_log;
};

template <typename T>
struct Run;  // 16 bytes of T, as pairs of fp32 values
template <>
struct Run<float> {
    static constexpr int E = 4;
    // sine and cosine of t turns, |t| <= 1/2
    static __device__ __forceinline__ void turn(float t, float &s, float &c) { sincospif(2.f * t, &s, &c); }
    static __device__ __forceinline__ void unpack(const uint4 &u, uint64_t (&x)[2]) {
        x[0] = attn::pack2(__uint_as_float(u.x), __uint_as_float(u.y));
        x[1] = attn::pack2(__uint_as_float(u.z), __uint_as_float(u.w));
    }
    static __device__ __forceinline__ uint4 pack(const uint64_t (&x)[2]) {
        float a, b, c, d;
        attn::unpack2(x[0], a, b);
        attn::unpack2(x[1], c, d);
        return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
    }
};
template <>
struct Run<__nv_bfloat16> {
    static constexpr int E = 8;
    // (within 2^-21 for these arguments: nothing beside the 2^-8 of a bf16 result)
    static __device__ __forceinline__ void turn(float t, float &s, float &c) { __sincosf(6.283185307f * t, &s, &c); }
    static __device__ __forceinline__ void unpack(const uint4 &u, uint64_t (&x)[4]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = attn::pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint4 pack(const uint64_t (&x)[4]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            attn::unpack2(x[i], a, b);
            w[i] = tc::pack_bf16x2(a, b);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// The first CTA checks every slot and alone writes the error word, so that no call has to clear it first.
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32, kResident) k_norm_rope(const __grid_constant__ Args p, const __grid_constant__ Freq fr) {
    constexpr int E = Run<T>::E, LPR = D / (2 * E), RPW = 32 / LPR;  // elements of a run, lanes per row, rows per group
    const NormRope &a = p.a;
    __shared__ uint64_t freq[64];
    if (threadIdx.x < a.rot / 2) freq[threadIdx.x] = fr.f[threadIdx.x];
    attn::grid_wait();
    attn::grid_launch_dependents();
    if (blockIdx.x == 0) {
        bool bad = false;
        if (a.slots) {
            const int64_t lim = (int64_t)a.num_pages << p.page_log;
#pragma unroll 8
            for (int t = threadIdx.x; t < a.T; t += kWarps * 32) bad |= a.slots[t] < -1 || a.slots[t] >= lim;
        }
        bad = __syncthreads_or(bad);
        if (threadIdx.x < 2) a.err[threadIdx.x] = bad && threadIdx.x == 0 ? ERRBIT_PAGES : 0u;
        return;
    }
    __syncthreads();
    const int64_t w = (int64_t)(blockIdx.x - 1) * kWarps + (threadIdx.x >> 5);
    if (w >= p.warps) return;
    const int lane = threadIdx.x & 31, part = lane % LPR, sub = lane / LPR;
    const int half = a.rot >> 1;
    const bool turned = part * E < half;                                              // pairs, or columns beyond rot
    const int col = turned ? part * E : a.rot + (part - half / E) * 2 * E;            // first run
    const int to_b = turned ? half : E;                                               // from it to the second
    const int groups = p.gq + p.gk + p.gv;
    // this warp's groups: the queries', then keys', then values' of a token, token after token
    const int64_t all = (int64_t)a.T * groups, first = all * w / p.warps, end = all * (w + 1) / p.warps;

    // A batch: up to kUnroll groups (head h0 + i RPW + sub in group i) of the queries, keys or values of one token, its
    // position and slot. Batches do not straddle, so that a batch has one address and fixed distances from it.
    constexpr int STEP = RPW * D;  // elements from a group to the next
    uint4 next[kUnroll][2];
    int next_t = (int)(first / groups), next_g = (int)(first - (int64_t)next_t * groups), next_n = 0, next_slot = -1;
    int64_t next_pos = 0, left = end - first;
    auto load = [&]() {
        const bool is_q = next_g < p.gq, is_k = next_g < p.gq + p.gk;
        const int seg_end = is_q ? p.gq : is_k ? p.gq + p.gk : groups, g0 = next_g - (is_q ? 0 : is_k ? p.gq : p.gq + p.gk);
        next_n = (int)min((int64_t)min(kUnroll, seg_end - next_g), left);
        const int heads = (is_q ? a.Hq : a.Hkv) - g0 * RPW - sub;  // still there for this lane
        const int64_t stride = is_q ? a.q_stride : is_k ? a.k_stride : a.v_stride;
        const T *src = static_cast<const T *>(is_q ? a.q : is_k ? a.k : a.v) + next_t * stride + (g0 * RPW + sub) * D + col;
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            next[i][0] = next[i][1] = make_uint4(0, 0, 0, 0);
            if (i < next_n && i * RPW < heads) {
                // (first out of L2: nothing here reads them again)
                next[i][0] = __ldcs(reinterpret_cast<const uint4 *>(src + i * STEP));
                next[i][1] = __ldcs(reinterpret_cast<const uint4 *>(src + i * STEP + to_b));
                if (left > groups) {  // the next token's, on their way to L2
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(src + i * STEP + stride));
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(src + i * STEP + to_b + stride));
                }
            }
        }
        if (a.rot) next_pos = a.positions[next_t];
        if (a.slots) next_slot = a.slots[next_t];
    };
    load();

    const int64_t head_step = (int64_t)RPW * D << p.page_log;  // in the cache from a group to the next
    float c[E], s[E];  // cosines and sines of this lane's pairs; beyond rot 1 and 0
    uint64_t wc[2][E / 2], ws[2][E / 2];  // w c and signed w' s of the two runs, for the queries or the keys
    auto fold = [&](const float *wt) {
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            const float2 one = make_float2(1.f, 1.f);
            const float2 x = wt ? *reinterpret_cast<const float2 *>(wt + col + i) : one;
            const float2 y = wt ? *reinterpret_cast<const float2 *>(wt + col + to_b + i) : one;
            wc[0][i / 2] = attn::pack2(c[i] * x.x, c[i + 1] * x.y);
            wc[1][i / 2] = attn::pack2(c[i] * y.x, c[i + 1] * y.y);
            ws[0][i / 2] = attn::pack2(-s[i] * y.x, -s[i + 1] * y.y);
            ws[1][i / 2] = attn::pack2(s[i] * x.x, s[i + 1] * x.y);
        }
    };
    int token = -1, folded = -1;
    int64_t cache = -1;  // element offset of (page, head 0, offset in page) of the token's slot
    while (left > 0) {
        const int t = next_t, n = next_n, kind = next_g < p.gq ? 0 : next_g < p.gq + p.gk ? 1 : 2;
        const int h0 = (next_g - (kind == 0 ? 0 : kind == 1 ? p.gq : p.gq + p.gk)) * RPW + sub;
        uint4 u[kUnroll][2];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            u[i][0] = next[i][0];
            u[i][1] = next[i][1];
        }
        if (t != token) {
            token = t;
            folded = -1;
            cache = -1;
            if (next_slot >= 0 && next_slot < ((int64_t)a.num_pages << p.page_log))
                cache = ((((int64_t)(next_slot >> p.page_log) * a.Hkv) << p.page_log) + (next_slot & ((1 << p.page_log) - 1))) * D + col;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                c[i] = 1.f;
                s[i] = 0.f;
            }
            if (turned && kind < 2) {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const int32_t turns = (int32_t)((uint64_t)next_pos * freq[col + i] >> 32);
                    Run<T>::turn((float)turns * 0x1p-32f, s[i], c[i]);
                }
            }
        }
        left -= n;
        next_g += n;
        if (next_g == groups) {
            next_g = 0;
            ++next_t;
        }
        if (left > 0) load();

        const int heads = (kind ? a.Hkv : a.Hq) - h0;  // still there for this lane
        T *const in_cache = static_cast<T *>(kind == 2 ? a.v_cache : a.k_cache) + cache + (int64_t)h0 * (head_step / RPW);
        if (kind == 2) {
#pragma unroll
            for (int i = 0; i < kUnroll; ++i)
                if (i < n && i * RPW < heads && cache >= 0) {
                    *reinterpret_cast<uint4 *>(in_cache + i * head_step) = u[i][0];
                    *reinterpret_cast<uint4 *>(in_cache + i * head_step + to_b) = u[i][1];
                }
            continue;
        }
        if (folded != kind) {
            folded = kind;
            fold(kind ? a.wk : a.wq);
        }
        T *const out = kind == 0 ? static_cast<T *>(a.q_out) + ((int64_t)t * a.Hq + h0) * D + col
                                 : static_cast<T *>(a.k_out) + ((int64_t)t * a.Hkv + h0) * D + col;
        const bool to_out = kind == 0 || a.k_out, to_cache = kind == 1 && cache >= 0;
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            if (i >= n) break;  // the whole warp
            uint64_t x[E / 2], z[E / 2];
            Run<T>::unpack(u[i][0], x);
            Run<T>::unpack(u[i][1], z);
            uint64_t sq = 0, sz = 0;
#pragma unroll
            for (int e = 0; e < E / 2; ++e) {
                sq = attn::fma2(x[e], x[e], sq);
                sz = attn::fma2(z[e], z[e], sz);
            }
            float ss, s1;
            attn::unpack2(attn::add2(sq, sz), ss, s1);
            ss += s1;
#pragma unroll
            for (int m = 1; m < LPR; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
            const float inv = rsqrtf(ss * (1.f / D) + a.eps);
            const uint64_t inv2 = attn::pack2(inv, inv);
#pragma unroll
            for (int e = 0; e < E / 2; ++e) {
                const uint64_t ya = attn::mul2(attn::fma2(z[e], ws[0][e], attn::mul2(x[e], wc[0][e])), inv2);
                z[e] = attn::mul2(attn::fma2(x[e], ws[1][e], attn::mul2(z[e], wc[1][e])), inv2);
                x[e] = ya;
            }
            const uint4 ya = Run<T>::pack(x), yb = Run<T>::pack(z);
            if (i * RPW < heads) {
                if (to_out) {
                    *reinterpret_cast<uint4 *>(out + i * STEP) = ya;
                    *reinterpret_cast<uint4 *>(out + i * STEP + to_b) = yb;
                }
                if (to_cache) {
                    *reinterpret_cast<uint4 *>(in_cache + i * head_step) = ya;
                    *reinterpret_cast<uint4 *>(in_cache + i * head_step + to_b) = yb;
                }
            }
        }
    }
}

template <typename T, int D>
cudaError_t launch(const NormRope &a, cudaStream_t st) {
    constexpr int RPW = 32 / (D / (2 * Run<T>::E));
    Args p;
    p.a = a;
    p.gq = (a.Hq + RPW - 1) / RPW;
    p.gk = (a.Hkv + RPW - 1) / RPW;
    p.gv = a.slots ? p.gk : 0;
    p.page_log = 0;
    while (a.slots && (1 << p.page_log) < a.page_size) ++p.page_log;
    p.warps = std::min<int64_t>((int64_t)a.T * (p.gq + p.gk + p.gv), (148 * kResident - 1) * kWarps);  // one CTA checks
    Freq fr;
    // (extended precision throughout; what the chain of products loses is said above)
    const long double step = a.rot ? powl(a.base, -2.0L / a.rot) : 1.0L;
    long double f = 0x1p64L / 6.283185307179586476925287L;
    for (int i = 0; i < a.rot / 2; ++i, f *= step) fr.f[i] = (uint64_t)(f + 0.5L);
    const unsigned grid = (unsigned)((p.warps + kWarps - 1) / kWarps) + 1;
    void *pr = prof_start("qk_norm_rope", st);
    const cudaError_t e = attn::launch_early(k_norm_rope<T, D>, grid, kWarps * 32, 0, st, p, fr);
    prof_stop(pr);
    return e;
}

}  // namespace

cudaError_t launch_norm_rope(const NormRope &a, int d, bool bf16, cudaStream_t st) {
    if (bf16) return d == 64 ? launch<__nv_bfloat16, 64>(a, st) : launch<__nv_bfloat16, 128>(a, st);
    return d == 64 ? launch<float, 64>(a, st) : launch<float, 128>(a, st);
}

}  // namespace gdn
