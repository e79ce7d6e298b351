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
// its key head (G <= 16: at most 16 flops a byte). The work is cut into units of 128 keys of one
// (sequence, key head), numbered sequence by sequence; each CTA takes an equal run of consecutive units
// whatever the lengths are, so ragged batches and single long sequences alike fill the GPU. A run cuts
// at most its first and last (sequence, head) short; those pieces go to two slots of the CTA, all
// others are finished in place. In a unit a warp owns 16 keys, brought by 16-byte asynchronous copies into
// a ring of its own that runs ahead across (sequence, head) borders. The products are
// S^T = K Q^T and O^T = V^T P^T on m16n8k16 tensor instructions: the 16 keys (or 16 of the d columns)
// are the rows and the heads the 8 columns, so a group of up to 8 heads wastes nothing on padding rows,
// which a 128-row tile would; at these few flops a byte the memory stays the bound.
//
// The prefix runs in the prompt kernel (attn_prefill.cu) without a mask, all sequences' query heads of a
// key head as rows of one tile, so its keys are read once per 256 rows and not once per sequence.
//
// k_attn_combine joins the pieces; it is launched to start while the kernel before it drains.
#include <algorithm>

#include "attn_common.cuh"
#include "chunk_common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kStep = 16;                // keys of a warp in a unit
constexpr int kUnit = kWarps * kStep;    // keys of a unit
constexpr float kRescale = 8.f;          // log2 units: how far the true maximum may run ahead of the reference

template <int D>
struct Smem {
    static constexpr int NST = 3 * 128 / D;              // ring stages of a warp
    static constexpr uint32_t HALF = kStep * D * 2;      // K, then V, of a stage
    static constexpr uint32_t RING = NST * 2 * HALF;     // per warp
    static constexpr int LD = D + 4;                     // padded row of the merge buffer
    static constexpr uint32_t OFF_MRG = kWarps * RING;
    static constexpr uint32_t OFF_ML = OFF_MRG + kWarps * 8 * LD * 4;
    static constexpr uint32_t TOTAL = OFF_ML + kWarps * 8 * 8;
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
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ int length_of(const AttnDecode &a, int b) {
    return min(max(a.lens[b], 0), a.max_pages << a.page_log);  // max_pages << page_log is at most 2^30
}
__device__ __forceinline__ int units_of(int len) { return (len + kUnit - 1) / kUnit; }

// The run of units of CTA c is [first_unit(c), first_unit(c + 1)). With fewer units than CTAs each of the
// first `units` CTAs has one, so that the pieces of a (sequence, head) always lie in consecutive CTAs.
__device__ __forceinline__ int64_t first_unit(int64_t units, int c) {
    return units < kDecodeCtas ? min((int64_t)c, units) : units * c / kDecodeCtas;
}
// The CTA whose run holds unit x.
__device__ __forceinline__ int cta_of(int64_t units, int64_t x) {
    if (units < kDecodeCtas) return (int)x;
    int c = (int)(x * kDecodeCtas / units);
    while (c > 0 && first_unit(units, c) > x) --c;
    while (first_unit(units, c + 1) <= x) ++c;
    return c;
}

// A place in a CTA's run: unit `chunk` of the `n` units of (sequence b, key head h).
struct Place {
    int b, h, chunk, n, len;
    __device__ __forceinline__ void next(const AttnDecode &a) {
        if (++chunk < n) return;
        chunk = 0;
        if (++h < a.Hkv) return;
        h = 0;
        for (n = 0; n == 0 && ++b < a.B;) {
            len = length_of(a, b);
            n = units_of(len);
        }
    }
};

// The CTA behind the last run checks lengths and page numbers and alone writes the error word.
__device__ __forceinline__ void check_pages(const AttnDecode &a) {
    bool bad = false;
    const int page_size = 1 << a.page_log;
    const int64_t most = (int64_t)a.max_pages << a.page_log;
    for (int b = threadIdx.x >> 5; b < a.B; b += kWarps) {
        const int len = a.lens[b];
        bad |= len < 0 || len > most;
        const int n = (int)min((int64_t)a.max_pages, ((int64_t)max(len, 0) + page_size - 1) >> a.page_log);
        for (int i = threadIdx.x & 31; i < n; i += 32) {
            const int p = a.table[(int64_t)b * a.max_pages + i];
            bad |= p < 0 || p >= a.num_pages;
        }
    }
    for (int i = threadIdx.x; i < (a.prefix_len + page_size - 1) >> a.page_log; i += kThreads)
        bad |= a.prefix_pages[i] < 0 || a.prefix_pages[i] >= a.num_pages;
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        if (a.prefix_len) {  // the prefix kernel cleared the word and may have set a bit
            grid_wait();
            if (bad) atomicOr(a.err, ERRBIT_PAGES);
        } else {
            *a.err = bad ? ERRBIT_PAGES : 0u;
        }
    }
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 1) k_attn_decode(const __grid_constant__ AttnDecode a) {
    using S = Smem<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    grid_launch_dependents();
    if (blockIdx.x == kDecodeCtas) {
        check_pages(a);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t ring = tc::smem_u32(smem) + warp * S::RING;
    float *mrg = reinterpret_cast<float *>(smem + S::OFF_MRG);
    float2 *mrg_ml = reinterpret_cast<float2 *>(smem + S::OFF_ML);

    // ---- this CTA's run: a scan of the sequences' unit counts, a run of sequences per thread
    __shared__ int64_t warp_sum[kWarps];
    __shared__ int64_t found[3];  // sequence, units before it, total
    const int per = (a.B + kThreads - 1) / kThreads;
    int64_t mine = 0;
    for (int b = tid * per; b < min(a.B, (tid + 1) * per); ++b) mine += units_of(length_of(a, b));
    int64_t upto = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, m);
        if (lane >= m) upto += x;
    }
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) upto += warp_sum[w];
        total += warp_sum[w];
    }
    const int64_t units = total * a.Hkv;
    const int64_t u0 = first_unit(units, blockIdx.x), u1 = first_unit(units, blockIdx.x + 1);
    if (u0 == u1) {
        // nothing to read; sequences without keys are written by the combine kernel
        if (a.prefix_len) grid_wait();
        return;
    }
    if (u0 >= (upto - mine) * a.Hkv && u0 < upto * a.Hkv) {
        int64_t before = upto - mine;
        int b = tid * per;
        for (;; ++b) {
            const int n = units_of(length_of(a, b));
            if (u0 < (before + n) * a.Hkv) break;
            before += n;
        }
        found[0] = b;
        found[1] = before;
    }
    __syncthreads();
    Place at;
    at.b = (int)found[0];
    at.len = length_of(a, at.b);
    at.n = units_of(at.len);
    {
        const int64_t in = u0 - found[1] * a.Hkv;
        at.h = (int)(in / at.n);
        at.chunk = (int)(in - (int64_t)at.h * at.n);
    }

    // ---- loads: the page number is fetched one unit ahead of the copies
    Place ld = at;
    int64_t ld_u = u0;
    auto page_of = [&](const Place &p) {
        const int key = p.chunk * kUnit + warp * kStep;
        return key < p.len ? a.table[(int64_t)p.b * a.max_pages + (key >> a.page_log)] : -1;
    };
    int page = page_of(ld);
    int ld_st = 0;
    auto load = [&]() {
        if (ld_u < u1) {
            const int key = ld.chunk * kUnit + warp * kStep, n = min(ld.len - key, kStep);
            if (n > 0) {
                const bool there = page >= 0 && page < a.num_pages;
                const int64_t row = there ? ((((int64_t)page * a.Hkv + ld.h) << a.page_log) | (key & ((1 << a.page_log) - 1))) : 0;
                const bf16 *k = a.k_cache + row * D, *v = a.v_cache + row * D;
                const uint32_t dst = ring + ld_st * 2 * S::HALF;
#pragma unroll
                for (int i = 0; i < kStep * D / 8 / 32; ++i) {
                    const int id = i * 32 + lane, r = id / (D / 8), c = id % (D / 8);
                    const bool in = there && r < n;  // places past the end are filled with zeros
                    const uint32_t off = r * (D * 2) + ((c ^ (r & 7)) << 4);
                    const int64_t src = in ? r * D + c * 8 : 0;
                    chunk::cp_async16(dst + off, k + src, in ? 16u : 0u);
                    chunk::cp_async16(dst + S::HALF + off, v + src, in ? 16u : 0u);
                }
            }
            ld.next(a);
            if (++ld_u < u1) page = page_of(ld);
        }
        chunk::cp_async_commit();
        ld_st = ld_st + 1 == S::NST ? 0 : ld_st + 1;
    };
#pragma unroll
    for (int i = 0; i < S::NST - 1; ++i) load();

    uint32_t qf[NT][D / 16][2];
    float o[NT][D / 16][4], m[NT][2], l[NT][2];
    const bool starts_before = at.chunk > 0;  // the first piece's head lies in an earlier CTA
    bool fresh = true, first_piece = true;
    int st = 0;
    for (int64_t u = u0; u < u1; ++u) {
        if (fresh) {
            fresh = false;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int g = t * 8 + (lane >> 2);
                const bf16 *q = a.q + ((int64_t)at.b * a.Hq + at.h * a.G + min(g, a.G - 1)) * D + (lane & 3) * 2;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    qf[t][kk][0] = g < a.G ? *reinterpret_cast<const uint32_t *>(q + kk * 16) : 0u;
                    qf[t][kk][1] = g < a.G ? *reinterpret_cast<const uint32_t *>(q + kk * 16 + 8) : 0u;
                    o[t][kk][0] = o[t][kk][1] = o[t][kk][2] = o[t][kk][3] = 0.f;
                }
                m[t][0] = m[t][1] = -INFINITY;
                l[t][0] = l[t][1] = 0.f;
            }
        }
        cp_async_wait<S::NST - 2>();
        __syncwarp();
        load();  // into the stage that was read one unit ago
        const int n = min(at.len - at.chunk * kUnit - warp * kStep, kStep);
        if (n > 0) {
            const uint32_t kb = ring + st * 2 * S::HALF, vb = kb + S::HALF;
            float s[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
            const int kr = lane & 15, kc = lane >> 4;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t f[4];
                ldmatrix4(kb + kr * (D * 2) + (((2 * kk + kc) ^ (kr & 7)) << 4), f);
#pragma unroll
                for (int t = 0; t < NT; ++t) mma16816(s[t], f, qf[t][kk][0], qf[t][kk][1]);
            }
            // this lane: keys lane / 4 and lane / 4 + 8, heads 2 (lane % 4) and one more
            const bool in0 = (lane >> 2) < n, in1 = (lane >> 2) + 8 < n;
            uint32_t pf[NT][2];
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
                    const float p0 = chunk::ex2(s[t][i] - m[t][i]), p1 = chunk::ex2(s[t][i + 2] - m[t][i]);
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
                // the weights enter the second product as bf16 (at most 2^-8 of each); l sums them unrounded
                pf[t][0] = transpose8(tc::pack_bf16x2(s[t][0], s[t][1]));
                pf[t][1] = transpose8(tc::pack_bf16x2(s[t][2], s[t][3]));
            }
            const int vr = (lane & 7) + ((lane >> 4) << 3), vc = (lane >> 3) & 1;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t f[4];
                ldmatrix4_t(vb + vr * (D * 2) + (((2 * kk + vc) ^ (vr & 7)) << 4), f);
#pragma unroll
                for (int t = 0; t < NT; ++t) mma16816(o[t][kk], f, pf[t][0], pf[t][1]);
            }
        }
        st = st + 1 == S::NST ? 0 : st + 1;

        const bool piece_ends = at.chunk + 1 == at.n || u + 1 == u1;
        if (piece_ends) {
            // ---- join the warps' pieces of this (sequence, head)
            const bool whole = at.chunk + 1 == at.n && !(first_piece && starts_before);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int heads = min(a.G - t * 8, 8);
                if (heads <= 0) break;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float x = l[t][i];
                    x += __shfl_xor_sync(0xffffffffu, x, 4);
                    x += __shfl_xor_sync(0xffffffffu, x, 8);
                    x += __shfl_xor_sync(0xffffffffu, x, 16);
                    if (lane < 4) mrg_ml[warp * 8 + 2 * lane + i] = make_float2(m[t][i], x);
                }
                float *mine_o = mrg + (warp * 8 + (lane & 3) * 2) * S::LD + (lane >> 2);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int i = 0; i < 4; ++i) mine_o[(i & 1) * S::LD + kk * 16 + (i >> 1) * 8] = o[t][kk][i];
                __syncthreads();
                for (int e = tid; e < heads * (D / 4); e += kThreads) {
                    const int g = e / (D / 4), d = e % (D / 4) * 4;
                    float top = -INFINITY;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, mrg_ml[w * 8 + g].x);
                    float sum = 0.f;
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float2 ml = mrg_ml[w * 8 + g];
                        const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - top);
                        const float4 y = *reinterpret_cast<const float4 *>(mrg + (w * 8 + g) * S::LD + d);
                        sum += f * ml.y;
                        x.x += f * y.x;
                        x.y += f * y.y;
                        x.z += f * y.z;
                        x.w += f * y.w;
                    }
                    const int head = t * 8 + g;
                    if (whole && !a.prefix_len) {
                        const float inv = 1.f / sum;
                        *reinterpret_cast<uint2 *>(a.o + ((int64_t)at.b * a.Hq + at.h * a.G + head) * D + d) =
                            make_uint2(tc::pack_bf16x2(x.x * inv, x.y * inv), tc::pack_bf16x2(x.z * inv, x.w * inv));
                    } else {
                        const int64_t row = (whole ? 2 * (int64_t)kDecodeCtas + (int64_t)at.b * a.Hkv + at.h
                                                   : 2 * (int64_t)blockIdx.x + (first_piece && starts_before ? 0 : 1)) * a.G + head;
                        *reinterpret_cast<float4 *>(a.slot_o + row * D + d) = x;
                        if (d == 0) a.slot_ml[row] = make_float2(top, sum);
                    }
                }
                __syncthreads();
            }
            fresh = true;
            first_piece = false;
        }
        at.next(a);
    }
    cp_async_wait<0>();
    if (a.prefix_len) grid_wait();  // this kernel's end then means the prefix kernel's too
}

// One CTA per (sequence, query head): joins the pieces of its own keys with those of the prefix. A row
// that the decode kernel finished is left alone; one without any keys is zero.
template <int D>
__global__ void __launch_bounds__(128) k_attn_combine(const __grid_constant__ AttnDecode a) {
    constexpr int LPR = D / 4, SUBS = 128 / LPR;  // lanes per row; pieces in flight
    const int row = blockIdx.x, b = row / a.Hq, hq = row - b * a.Hq, h = hq / a.G, g = hq - h * a.G;
    const int tid = threadIdx.x, sub = tid / LPR, d = tid % LPR * 4;
    __shared__ int64_t sums[2];
    __shared__ float4 part[SUBS][LPR];
    __shared__ float2 part_ml[SUBS];
    if (tid < 2) sums[tid] = 0;
    __syncthreads();
    int64_t before = 0, total = 0;
    for (int i = tid; i < a.B; i += 128) {
        const int n = units_of(length_of(a, i));
        total += n;
        if (i < b) before += n;
    }
#pragma unroll
    for (int m = 16; m; m >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, m);
        total += __shfl_xor_sync(0xffffffffu, total, m);
    }
    if ((tid & 31) == 0) {
        atomicAdd(reinterpret_cast<unsigned long long *>(&sums[0]), (unsigned long long)before);
        atomicAdd(reinterpret_cast<unsigned long long *>(&sums[1]), (unsigned long long)total);
    }
    __syncthreads();
    const int64_t units = sums[1] * a.Hkv;
    const int n = units_of(length_of(a, b));
    const int64_t x0 = sums[0] * a.Hkv + (int64_t)h * n;
    int c0 = 0, own = 0;  // first CTA with a piece, number of pieces
    if (n) {
        c0 = cta_of(units, x0);
        own = cta_of(units, x0 + n - 1) - c0 + 1;
    }
    grid_wait();  // also where nothing is left to do: this kernel's end means the one before it has ended
    if (own == 1 && !a.prefix_len) return;
    const int splits = a.prefix_len ? a.splits : 0;
    float top = -INFINITY, sum = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = sub; i < own + splits; i += SUBS) {
        const float *po;
        float2 ml;
        if (i < own) {
            const int64_t slot = (own == 1 ? 2 * (int64_t)kDecodeCtas + (int64_t)b * a.Hkv + h
                                           : 2 * (int64_t)(c0 + i) + (i == 0 ? 1 : 0)) * a.G + g;
            po = a.slot_o + slot * D;
            ml = a.slot_ml[slot];
        } else {
            const int64_t r = (int64_t)(i - own) * a.B * a.Hq + row;
            po = a.part_o + r * D;
            ml = a.part_ml[r];
        }
        const float4 y = *reinterpret_cast<const float4 *>(po + d);
        const float t = fmaxf(top, ml.x);
        const float fo = top == -INFINITY ? 0.f : exp2f(top - t), fn = ml.x == -INFINITY ? 0.f : exp2f(ml.x - t);
        x.x = x.x * fo + y.x * fn;
        x.y = x.y * fo + y.y * fn;
        x.z = x.z * fo + y.z * fn;
        x.w = x.w * fo + y.w * fn;
        sum = sum * fo + ml.y * fn;
        top = t;
    }
    part[sub][tid % LPR] = x;
    if (d == 0) part_ml[sub] = make_float2(top, sum);
    __syncthreads();
    if (sub) return;
    for (int i = 0; i < SUBS; ++i) top = fmaxf(top, part_ml[i].x);
    sum = 0.f;
    x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < SUBS; ++i) {
        const float2 ml = part_ml[i];
        const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - top);
        const float4 y = part[i][tid % LPR];
        x.x += f * y.x;
        x.y += f * y.y;
        x.z += f * y.z;
        x.w += f * y.w;
        sum += f * ml.y;
    }
    const float inv = own + splits ? 1.f / sum : 0.f;
    *reinterpret_cast<uint2 *>(a.o + (int64_t)row * D + d) =
        make_uint2(tc::pack_bf16x2(x.x * inv, x.y * inv), tc::pack_bf16x2(x.z * inv, x.w * inv));
}

template <typename K>
cudaError_t launch_pdl(K kern, unsigned grid, unsigned threads, size_t smem, cudaStream_t st, bool early, const AttnDecode &a) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int D, int NT>
cudaError_t launch(AttnDecode a, cudaStream_t st, const char **stage) {
    cudaError_t e;
    *stage = "attn_decode";
    auto kern = k_attn_decode<D, NT>;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Smem<D>::TOTAL)) != cudaSuccess) return e;
    void *pr = prof_start("attn_decode", st);
    e = launch_pdl(kern, kDecodeCtas + 1, kThreads, Smem<D>::TOTAL, st, a.prefix_len > 0, a);
    prof_stop(pr);
    if (e != cudaSuccess) return e;
    *stage = "attn_combine";
    pr = prof_start("attn_combine", st);
    e = launch_pdl(k_attn_combine<D>, (unsigned)((int64_t)a.B * a.Hq), 128, 0, st, true, a);
    prof_stop(pr);
    return e;
}

}  // namespace

int attn_decode_splits(int B, int Hq, int Hkv, int prefix_len) {
    if (prefix_len <= 0) return 0;
    // as many splits of the prefix's key tiles as fill the SMs once
    const int64_t pos = 2 * (128 / (Hq / Hkv)), blocks = (B + pos - 1) / pos * Hkv;
    const int64_t tiles = ((int64_t)prefix_len + 127) / 128;
    return (int)std::max<int64_t>(1, std::min<int64_t>(tiles, kDecodeCtas / blocks));
}

size_t attn_decode_slots(int B, int Hq, int Hkv, int prefix_len) {
    return (size_t)(Hq / Hkv) * 2 * kDecodeCtas + (prefix_len > 0 ? (size_t)B * Hq : 0);
}

cudaError_t launch_attn_decode(const AttnDecode &a, int d, cudaStream_t st, const char **stage) {
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
        const cudaError_t e = launch_attn_prefix(p, d, st, stage);
        if (e != cudaSuccess) return e;
    }
    if (d == 64) return a.G <= 8 ? launch<64, 1>(a, st, stage) : launch<64, 2>(a, st, stage);
    return a.G <= 8 ? launch<128, 1>(a, st, stage) : launch<128, 2>(a, st, stage);
}

}  // namespace gdn
