// encode_tiled.cuh -- the driver's encoder of tensor maps, looked up once.
#pragma once

#include <cudaTypedefs.h>
#include <cuda_runtime.h>

namespace coli {
namespace {

// NULL where the driver has none.
PFN_cuTensorMapEncodeTiled_v12000 encode_tiled() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return (PFN_cuTensorMapEncodeTiled_v12000)f;
    }();
    return fn;
}

}  // namespace
}  // namespace coli
