// prefill.cuh -- what the prompts' attention kernels (mla_prefill.cu, gqa_prefill.cu) share: rings, the take-over of
// CTAs that have not started, tensor maps.
#pragma once

#include "encode_tiled.cuh"
#include "mla_units.cuh"
#include "tcgen05.cuh"

namespace coli {

namespace {

constexpr uint32_t kBlk = kRows * 128;   // 128 rows x 64 bf16, 128-byte swizzle
constexpr float kGrow = 8.f;             // log2 of the weight that moves the reference
constexpr float kNone = -3e38f;          // reference of a row that has seen no key

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// A place in a ring of n buffers and the parity of its use.
struct Ring {
    int slot, par;
    __device__ __forceinline__ void step(int by, int n) {
        slot += by;
        if (slot >= n) {
            slot -= n;
            par ^= 1;
        }
    }
};

// The same values, all from lane 0: the compiler then keeps them, and the operands of MMAs and copies that derive from
// them, in uniform registers.
__device__ __forceinline__ Unit uniform(Unit u) {
    for (int *p : {&u.head, &u.q0, &u.nq, &u.nk, &u.qrow, &u.krow, &u.nt[0], &u.nt[1], &u.n}) *p = __shfl_sync(0xffffffffu, *p, 0);
    return u;
}

// Asks for the work of a CTA that has not started yet, in its stead; the answer (16 bytes) comes to `next`.
template <class S>
__device__ __forceinline__ void ask_next(S &s) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(smem_addr(s.next)),
                 "r"(smem_addr(&s.next_full))
                 : "memory");
}
// That CTA's index; -1: all have started, and no further request may be made.
template <class S>
__device__ __forceinline__ int read_next(S &s) {
    int i;
    asm volatile(
        "{\n .reg .b128 r;\n .reg .pred p;\n mov.s32 %0, -1;\n ld.shared.b128 r, [%1];\n"
        " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n"
        " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n"
        " fence.proxy.async.shared::cta;\n}\n"
        : "=&r"(i)
        : "r"(smem_addr(s.next))
        : "memory");
    return i;
}

cudaError_t matrix_map(const void *p, long long cols, long long rows, long long stride, int box_rows, CUtensorMap *out) {
    const PFN_cuTensorMapEncodeTiled_v12000 fn = encode_tiled();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, estr[2] = {1, 1};
    return fn(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

}  // namespace coli
