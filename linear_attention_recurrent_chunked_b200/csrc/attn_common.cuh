// Helpers of the grouped-head attention kernels (attn_prefill.cu, attn_decode.cu): bounded barrier
// waits with a CTA-wide abort, and TMA descriptors of 3-D bf16 tensors.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "common.cuh"
#include "tc.cuh"

namespace gdn {
namespace attn {

constexpr uint64_t kWaitNs = 1000000000ull;  // of a wait, but for tests of the give-up path (gdn_debug_inject)
constexpr float kLog2e = 1.4426950408889634f;

struct Ctl {
    uint32_t tmem, abort;
    uint64_t wait_ns;  // how long a wait may last
};

// Bounded wait for the phase `parity` of an mbarrier; gives up when another role has aborted, or
// after ctl->wait_ns (the error word is set and the CTA's other roles leave their loops too). The first
// test is inlined, the polling loop is a call.
__device__ __noinline__ inline bool wait_bar_poll(uint64_t *bar, uint32_t parity, Ctl *ctl, uint32_t *err) {
    const uint64_t t0 = tc::globaltimer();
    for (uint32_t i = 1;; ++i) {
        if (tc::mbar_try_wait(bar, parity)) return true;
        if ((i & 15u) == 0) {
            if (*reinterpret_cast<volatile uint32_t *>(&ctl->abort)) return false;
            if (tc::globaltimer() - t0 > ctl->wait_ns) {
                if (err) atomicOr(err, ERRBIT_TIMEOUT);
                *reinterpret_cast<volatile uint32_t *>(&ctl->abort) = 1u;
                return false;
            }
        }
    }
}
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, Ctl *ctl, uint32_t *err) {
    return tc::mbar_try_wait(bar, parity) || wait_bar_poll(bar, parity, ctl, err);
}
// The same by all lanes of a converged warp, which stays converged.
__device__ __forceinline__ bool wait_bar_w(uint64_t *bar, uint32_t parity, Ctl *ctl, uint32_t *err) {
    return __all_sync(0xffffffffu, wait_bar(bar, parity, ctl, err));
}
// Before a CTA that gave up may end: its own copies and products in flight (bounded too).
__device__ __noinline__ inline void drain_bar(uint64_t *bar, uint32_t parity, const Ctl *ctl) {
    const uint64_t t0 = tc::globaltimer();
    while (!tc::mbar_try_wait(bar, parity))
        if (tc::globaltimer() - t0 > ctl->wait_ns) return;
}

// Every kernel here is launched to start while the one before it in the stream drains (launch_early): it sets
// up what is its own, then waits here for that one's end before it touches global memory. Two read some of their inputs
// before: the decode kernel behind a prefix, and the joining kernel (its lengths and pages). They start only after every
// CTA of their call's first kernel has passed this wait, so whatever wrote those inputs before the call has ended.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel may start. (Its own wait still waits for this kernel's end.)
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename K, typename... A>
inline cudaError_t launch_early(K kern, unsigned grid, unsigned threads, size_t smem, cudaStream_t st, const A &...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Two fp32 values in one 64-bit register pair, for the packed fp32 instructions.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t x, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Eight fp32 values to a 32-byte aligned place: a whole sector from one thread.
__device__ __forceinline__ void st_global8(float *p, const float *x) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(__float_as_uint(x[0])),
                 "r"(__float_as_uint(x[1])), "r"(__float_as_uint(x[2])), "r"(__float_as_uint(x[3])), "r"(__float_as_uint(x[4])),
                 "r"(__float_as_uint(x[5])), "r"(__float_as_uint(x[6])), "r"(__float_as_uint(x[7]))
                 : "memory");
}

// TMEM -> registers, 32 columns, without the wait (see tc::tmem_wait_ld).
__device__ __forceinline__ void tmem_ld32x(uint32_t taddr, uint32_t (&u)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
          "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]),
          "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]),
          "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(taddr)
        : "memory");
}
// TMA descriptor of a bf16 tensor [n2][n1][n0] with n0 contiguous and the given strides (elements,
// multiples of 8); boxes of 64 x b1 x b2 elements written with the 128-byte swizzle, places outside
// the tensor reading as zero.
inline cudaError_t make_map(CUtensorMap *map, const void *base, uint64_t n0, uint64_t n1, uint64_t n2, uint64_t s1,
                            uint64_t s2, uint32_t b1, uint32_t b2) {
    static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {n0, n1, n2};
    const cuuint64_t strides[2] = {s1 * 2, s2 * 2};
    const cuuint32_t box[3] = {64, b1, b2};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
                              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace attn
}  // namespace gdn
