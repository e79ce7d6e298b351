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
// base^(-2i/r) / (2 pi) in fp64, and only the fraction of a turn is rounded to fp32: at position 10^6
// an fp32 product would be off by up to 2^-24 10^6 = 0.06 radians, this one by little more than 2^-26
// turns at any int32 position.
//
// Bound: HBM (each row is read once and written once, about 7 flops an element). A row is held by
// the d sizeof(T) / 16 lanes that load it as 16-byte runs, so the sum of squares and the pair partner
// (r/2 elements away: a whole number of lanes) come by shuffles and nothing passes through shared
// memory. A lane keeps the same columns for every row of its warp, so a warp that takes all rows of a
// token computes the sines and cosines once for all of its heads. With few tokens (a decode step) a
// token's rows are split over up to all the warps that they can fill instead, which shortens the
// chain of dependent loads.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

constexpr int kWarps = 4;   // per CTA
constexpr int kUnroll = 4;  // row groups whose loads are in flight together

struct Freq {
    double f[64];  // turns per position of pair i
};

struct Args {
    NormRope a;
    int rows;     // per token: Hq + Hkv, and Hkv more when v is cached
    int chunks;   // warps per token
    int per;      // rows per warp (a multiple of the rows a warp holds at a time)
    int page_log;
};

template <typename T>
struct Run;  // 16 bytes of T
template <>
struct Run<float> {
    static constexpr int E = 4;
    static __device__ __forceinline__ void unpack(const uint4 &u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
template <>
struct Run<__nv_bfloat16> {
    static constexpr int E = 8;
    static __device__ __forceinline__ void unpack(const uint4 &u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Row `row` of token t: 0 .. Hq-1 the queries, then the keys, then (v cached) the values.
// The last CTA checks every slot and alone writes the error word, so that no call has to clear it first.
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) k_norm_rope(const __grid_constant__ Args p, const __grid_constant__ Freq fr) {
    constexpr int E = Run<T>::E, LPR = D / E, RPW = 32 / LPR;  // elements and lanes per row, rows per warp
    const NormRope &a = p.a;
    if (blockIdx.x == gridDim.x - 1) {
        bool bad = false;
        if (a.slots) {
            const int64_t lim = (int64_t)a.num_pages << p.page_log;
            for (int t = threadIdx.x; t < a.T; t += kWarps * 32) bad |= a.slots[t] < -1 || a.slots[t] >= lim;
        }
        bad = __syncthreads_or(bad);
        if (threadIdx.x == 0) *a.err = bad ? ERRBIT_PAGES : 0u;
        return;
    }
    __shared__ double freq[64];
    if (threadIdx.x < a.rot / 2) freq[threadIdx.x] = fr.f[threadIdx.x];
    __syncthreads();
    const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int t = (int)(w / p.chunks), chunk = (int)(w - (int64_t)t * p.chunks);
    if (t >= a.T) return;
    const int lane = threadIdx.x & 31, col = (lane % LPR) * E, sub = lane / LPR;
    const int row_end = min(p.rows, (chunk + 1) * p.per);

    // where this token goes in the cache, if anywhere
    int64_t cache = -1;  // element offset of (page, head 0, offset in page)
    if (a.slots) {
        const int slot = a.slots[t];
        if (slot >= 0 && slot < ((int64_t)a.num_pages << p.page_log))
            cache = ((((int64_t)(slot >> p.page_log) * a.Hkv) << p.page_log) + (slot & ((1 << p.page_log) - 1))) * D;
    }
    const int64_t head_step = (int64_t)D << p.page_log;  // from one head of a page to the next

    // cosines and sines of this lane's columns; beyond rot: 1 and 0
    float c[E], s[E];
    const bool turned = col < a.rot;
    const int half = a.rot >> 1;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        c[i] = 1.f;
        s[i] = 0.f;
    }
    if (turned && chunk * p.per < a.Hq + a.Hkv) {
        const double pos = (double)a.positions[t];
        const int i0 = col & (half - 1);
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const double turns = pos * freq[i0 + i];
            sincospif(2.f * (float)(turns - rint(turns)), &s[i], &c[i]);
        }
        if (col < half) {
#pragma unroll
            for (int i = 0; i < E; ++i) s[i] = -s[i];
        }
    }
    float wq[E], wk[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        wq[i] = a.wq ? a.wq[col + i] : 1.f;
        wk[i] = a.wk ? a.wk[col + i] : 1.f;
    }

    const T *q = static_cast<const T *>(a.q) + (int64_t)t * a.q_stride;
    const T *k = static_cast<const T *>(a.k) + (int64_t)t * a.k_stride;
    const T *v = static_cast<const T *>(a.v) + (int64_t)t * a.v_stride;
    T *q_out = static_cast<T *>(a.q_out) + (int64_t)t * a.Hq * D;
    T *k_out = static_cast<T *>(a.k_out) + (int64_t)t * a.Hkv * D;
    for (int r0 = chunk * p.per; r0 < row_end; r0 += kUnroll * RPW) {
        uint4 u[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int r = r0 + i * RPW + sub;
            u[i] = make_uint4(0, 0, 0, 0);
            if (r < row_end) {
                const T *src = r < a.Hq ? q + (int64_t)r * D
                                        : r < a.Hq + a.Hkv ? k + (int64_t)(r - a.Hq) * D : v + (int64_t)(r - a.Hq - a.Hkv) * D;
                u[i] = *reinterpret_cast<const uint4 *>(src + col);
            }
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int r = r0 + i * RPW + sub;
            const bool is_q = r < a.Hq, is_v = r >= a.Hq + a.Hkv;
            if (r0 + i * RPW >= row_end) break;  // the whole warp
            uint4 y = u[i];
            if (r0 + i * RPW < a.Hq + a.Hkv) {  // at least one row of the warp is a query or a key
                float x[E];
                Run<T>::unpack(u[i], x);
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
                for (int m = 1; m < LPR; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
                const float inv = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
                for (int e = 0; e < E; ++e) x[e] *= inv * (is_q ? wq[e] : wk[e]);
                if (half) {
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float other = __shfl_xor_sync(0xffffffffu, x[e], (half / E) & 31);
                        x[e] = turned ? fmaf(other, s[e], x[e] * c[e]) : x[e];
                    }
                }
                if (!is_v) y = Run<T>::pack(x);
            }
            if (r >= row_end) continue;
            if (is_q) {
                *reinterpret_cast<uint4 *>(q_out + (int64_t)r * D + col) = y;
            } else if (!is_v) {
                const int h = r - a.Hq;
                if (a.k_out) *reinterpret_cast<uint4 *>(k_out + (int64_t)h * D + col) = y;
                if (cache >= 0)
                    *reinterpret_cast<uint4 *>(static_cast<T *>(a.k_cache) + cache + h * head_step + col) = y;
            } else if (cache >= 0) {
                *reinterpret_cast<uint4 *>(static_cast<T *>(a.v_cache) + cache + (r - a.Hq - a.Hkv) * head_step + col) = y;
            }
        }
    }
}

template <typename T, int D>
cudaError_t launch(const NormRope &a, cudaStream_t st) {
    constexpr int RPW = 32 / (D / Run<T>::E);
    Args p;
    p.a = a;
    p.rows = a.Hq + a.Hkv + (a.slots ? a.Hkv : 0);
    p.page_log = 0;
    while (a.slots && (1 << p.page_log) < a.page_size) ++p.page_log;
    // Few tokens: split each token's rows over warps until about 16 warps per SM are busy.
    const int groups = (p.rows + RPW - 1) / RPW;
    const int64_t want = 148 * 16;
    const int chunks = (int)std::min<int64_t>(groups, std::max<int64_t>(1, want / std::max(a.T, 1)));
    p.per = (groups + chunks - 1) / chunks * RPW;
    p.chunks = (p.rows + p.per - 1) / p.per;
    Freq fr;
    // extended precision, so that the chain of products costs nothing against a double's 2^-53
    const long double step = a.rot ? powl(a.base, -2.0L / a.rot) : 1.0L;
    long double f = 1.0L / 6.283185307179586476925287L;
    for (int i = 0; i < a.rot / 2; ++i, f *= step) fr.f[i] = (double)f;
    const int64_t warps = (int64_t)a.T * p.chunks;
    const unsigned grid = (unsigned)((warps + kWarps - 1) / kWarps) + 1;
    void *pr = prof_start("qk_norm_rope", st);
    k_norm_rope<T, D><<<grid, kWarps * 32, 0, st>>>(p, fr);
    prof_stop(pr);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRope &a, int d, bool bf16, cudaStream_t st) {
    if (bf16) return d == 64 ? launch<__nv_bfloat16, 64>(a, st) : launch<__nv_bfloat16, 128>(a, st);
    return d == 64 ? launch<float, 64>(a, st) : launch<float, 128>(a, st);
}

}  // namespace gdn
