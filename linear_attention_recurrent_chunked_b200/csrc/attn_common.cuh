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

constexpr uint64_t kWaitNs = 1000000000ull;
constexpr float kLog2e = 1.4426950408889634f;

struct Ctl {
    uint32_t tmem, abort;
};

// Bounded wait for the phase `parity` of an mbarrier; gives up when another role has aborted, or
// after kWaitNs (the error word is set and the CTA's other roles leave their loops too). The first
// test is inlined, the polling loop is a call.
__device__ __noinline__ inline bool wait_bar_poll(uint64_t *bar, uint32_t parity, Ctl *ctl, uint32_t *err) {
    const uint64_t t0 = tc::globaltimer();
    for (uint32_t i = 1;; ++i) {
        if (tc::mbar_try_wait(bar, parity)) return true;
        if ((i & 15u) == 0) {
            if (*reinterpret_cast<volatile uint32_t *>(&ctl->abort)) return false;
            if (tc::globaltimer() - t0 > kWaitNs) {
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
__device__ __noinline__ inline void drain_bar(uint64_t *bar, uint32_t parity) {
    const uint64_t t0 = tc::globaltimer();
    while (!tc::mbar_try_wait(bar, parity))
        if (tc::globaltimer() - t0 > kWaitNs) return;
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
