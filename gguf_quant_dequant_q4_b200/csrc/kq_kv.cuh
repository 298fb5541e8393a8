// Shared by the KV-cache kernels (plan, append, attention).
//
// A pool is [n_pages, n_kv_heads, page_size, row] bytes, row = head_dim / 32
// q4_0 wire blocks of 18 bytes, so the rows of one head in one page are one
// contiguous run; page_size is a multiple of 16, so every run of 16 tokens
// starts on a 16-byte boundary and is a multiple of 16 bytes (288 * blocks).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kq_device.cuh"
#include "kq_launch.h"

namespace kq {

// Programmatic dependent launch: a kernel may start while the one before it
// on the stream still runs; nothing is read or written before this wait.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class K, class... A>
int launch_pdl(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = use_pdl() ? 1 : 0;
    return record_cuda(cudaLaunchKernelEx(&cfg, kernel, args...));
}

}  // namespace kq
