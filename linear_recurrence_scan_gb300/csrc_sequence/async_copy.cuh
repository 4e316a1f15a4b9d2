// async_copy.cuh -- waits with a limit, tensor maps and the copies that go
// through them, for the kernels of the token policy's layers.
#pragma once

#include "sequence.cuh"

#include <cuda.h>

namespace rlscan {
namespace seq {

// ---- waits -----------------------------------------------------------------------
// A wait that runs out sets the block's flag.  The block then goes on to its end
// through the same barriers of all its threads, but a thread whose wait was in
// vain asks for no copy and arrives at no mbarrier, whose counts no longer fit.
// One whose waits pass goes on meanwhile, on phases that others completed before
// they gave up, until one does not.  The block's results are void, and it sets its
// file's device flag.
constexpr uint64_t kWaitNs = 4'000'000'000ull;

__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Waits for phase `parity`, at most `limit`; then, or once another thread of
// the block has given up, false.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int *gave_up, uint64_t limit = kWaitNs)
{
    if (try_wait(bar, parity)) return true;
    const uint64_t start = ptx::globaltimer_ns();
    while (!try_wait(bar, parity)) {
        if (*gave_up != 0) return false;
        if (ptx::globaltimer_ns() - start > limit) {
            *gave_up = 1;
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ bool has_given_up(const int *gave_up) { return *const_cast<const volatile int *>(gave_up) != 0; }

// The same by a warp, in front of what its lanes do together (votes, exchanges,
// loads of tensor memory): one answer for all of them.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, int *gave_up, uint64_t limit = kWaitNs)
{
    return __all_sync(0xffffffffu, wait(bar, parity, gave_up, limit)) != 0;
}

// At the end of a block, by all its threads: any that has seen the flag tells
// the host, and stays until what is in flight (which takes microseconds) has ended.
__device__ __forceinline__ void leave(const int *gave_up, unsigned int *device_flag)
{
    if (!has_given_up(gave_up)) return;
    atomicExch(device_flag, 1u);
    const uint64_t start = ptx::globaltimer_ns();
    while (ptx::globaltimer_ns() - start < 1'000'000) {
    }
}

// Whether a kernel of a file has given up on the current device since the last
// question (`flag`: the file's device flag).
template <class S>
inline rlscan_status take_flag(const S &flag, cudaStream_t s)
{
    unsigned int seen = 0;
    const unsigned int none = 0;
    if (!ok(cudaMemcpyFromSymbolAsync(&seen, flag, sizeof seen, 0, cudaMemcpyDeviceToHost, s)) || !ok(cudaStreamSynchronize(s)))
        return RLSCAN_ERR_CUDA;
    if (seen == 0) return RLSCAN_OK;
    if (!ok(cudaMemcpyToSymbolAsync(flag, &none, sizeof none, 0, cudaMemcpyHostToDevice, s)) || !ok(cudaStreamSynchronize(s)))
        return RLSCAN_ERR_CUDA;
    return RLSCAN_ERR_TIMEOUT;
}

// ---- tensor maps --------------------------------------------------------------------
// `dims` extents, innermost first, with the strides in bytes of all but the
// first, copied in boxes; what lies outside reads 0 and is not written.
inline bool encode_map(CUtensorMap *map, const void *p, bool bf16_type, int dims, const int64_t *extents, const int64_t *strides,
                       const uint32_t *box, bool swizzle128)
{
    using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode call = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (!ok(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found)) ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    if (call == nullptr) return false;
    cuuint64_t size[3], stride[2];
    cuuint32_t boxes[3];
    const cuuint32_t step[3] = {1, 1, 1};
    for (int i = 0; i < dims; ++i) {
        size[i] = static_cast<cuuint64_t>(extents[i]);
        boxes[i] = box[i];
        if (i > 0) stride[i - 1] = static_cast<cuuint64_t>(strides[i - 1]);
    }
    auto encode = [&] {
        return call(map, bf16_type ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, dims, const_cast<void *>(p), size,
                    stride, boxes, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    swizzle128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (encode()) return true;
    // A thread that has made no runtime call of its own yet (autograd's, say)
    // has no context for the driver's: setting its device gives it one.
    const int device = current_device();
    return device >= 0 && ok(cudaSetDevice(device)) && encode();
}

// A box into this block's shared memory, its bytes counted on `bar`
__device__ __forceinline__ void load_box3(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
// A box out of this block's shared memory (written before a fence of the
// asynchronous proxy), as a group of the calling thread
__device__ __forceinline__ void store_box3(const CUtensorMap *map, int x, int y, int z, uint32_t src)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x), "r"(y),
                 "r"(z), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void stores_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// until the shared memory of the thread's stores has been read
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

}  // namespace seq
}  // namespace rlscan
