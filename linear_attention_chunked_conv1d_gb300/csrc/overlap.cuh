// Launches whose start overlaps the end of the kernel before them in the stream: the blocks are set up
// while that kernel's last ones write back, and wait for it where they say so. Between short kernels in a
// stream this takes 1.5 to 3 us off each (4-bit products 1 x 4096 x 8192 in a row: 10.3 us each without, 7.4 with;
// in a captured graph 7.5 and 7.1).
#pragma once
#include <cuda_runtime.h>

#include <utility>

namespace la {

// Waits until what was launched before in the stream is complete and its writes can be seen. Every thread of
// a kernel that launch_overlapped starts calls it before it touches global memory (but see start_beside).
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Lets the next kernel of the stream that waits so start its blocks where they fit beside this one's.
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Two kernels of one call side by side, the second in the places that the first leaves empty. The second reads global memory
// without having waited itself, which is in order under these conditions alone:
//  - the kernel launched directly ahead of it in the stream is the call's first, and every block of that one lets it start
//    by wait_and_let_beside(): what was launched before the call is then complete and its writes are in global memory;
//  - neither kernel reads or writes what the other writes;
//  - every thread of the second calls start_beside() before it touches global memory, and end_beside() when it is done.
// What a wait makes visible, it makes visible to the grid that waits. So the first kernel's fence passes that on before its
// signal, and the second's fence, behind its start, keeps its loads from finding older values in its SM's L1; a thread that
// copies by TMA puts beside_tma() between that fence and its first copy. (777 x 5001 x 2048 with bias, GELU and residual
// 22.8 us without the fences and 22.9 with them, 1030 x 8192 x 2048 28.6 and 29.1; in one kernel 29.7 and 32.3, with the
// second kernel waiting for the first 32.0 and 36.3.)
__device__ __forceinline__ void fence_gpu() { asm volatile("fence.acq_rel.gpu;" ::: "memory"); }
__device__ __forceinline__ void wait_and_let_beside() {
    wait_for_previous();
    if (threadIdx.x == 0) {  // one thread's signal is its block's
        fence_gpu();
        launch_next();
    }
}
__device__ __forceinline__ void start_beside() { fence_gpu(); }
__device__ __forceinline__ void beside_tma() { asm volatile("fence.proxy.async;" ::: "memory"); }
// Who waits for the second kernel waits for the first one too.
__device__ __forceinline__ void end_beside() { wait_for_previous(); }

// cluster: a cluster's blocks, or cluster.x = 0.
template <class... Params, class... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, dim3 cluster, cudaStream_t st,
                              Args &&...args) {
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster.x;
    attr[1].val.clusterDim.y = cluster.y;
    attr[1].val.clusterDim.z = cluster.z;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = cluster.x ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// cluster: blocks of a cluster along x, or 0.
template <class... Params, class... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t st,
                              Args &&...args) {
    return launch_overlapped(kernel, grid, block, smem, dim3(cluster, 1, 1), st, std::forward<Args>(args)...);
}

}  // namespace la
