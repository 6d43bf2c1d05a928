// Launches in which a kernel's start overlaps the end of the one before it in
// the stream (programmatic dependent launch).
//
// The kernel's blocks may be set up as soon as every block of the kernel
// before has ended; what would otherwise come in between is the wait until
// its writes are visible, and the launch.  Calls one after another, no graph:
// 14.4 -> 9.9 us for a step of the e4m3 attention (two kernels, 1001 tokens),
// and two to three us for a launch in general.  Letting the next kernel in
// earlier, while blocks still run, was 0.7 us slower: its blocks are in the
// way.
//
// The order of the stream holds because every thread of a kernel that is
// launched so calls await_previous() before it touches global memory: it
// returns when the kernel before has completed and its writes are visible.
// That is needed in every block, also in one that has nothing to do, or a
// kernel could complete before the one it follows, and the next one, which
// waits for it alone, begin too early.
//
// Such a kernel is there before what it reads is written, so it reads with
// plain loads: ld.global.nc (__ldg) is for memory that stays as it is for as
// long as the kernel lives, and is not held behind the wait.
#pragma once

#include <cuda_runtime.h>

namespace attn {

__device__ __forceinline__ void await_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, const A &...args)
{
    cudaLaunchAttribute overlap = {};
    overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    overlap.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    c.attrs = &overlap;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, args...);
}

}  // namespace attn
