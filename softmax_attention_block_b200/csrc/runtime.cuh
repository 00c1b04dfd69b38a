// Host-side diagnostics of the library: a process-wide count of kernel
// launches and optional per-stage timing with CUDA events on the stage's own
// stream (used by the benchmark to time one stage inside a full step).
#pragma once
#include <cuda_runtime.h>

namespace path {

void count_launches(int n = 1);

// path_test_withhold_kv_load's setting (0 or 1).
int withhold_kv_load();

// Streaming multiprocessors of the current device (cached per device; 148 if
// the query fails).
int sm_count();

// Brackets one stage of an entry point with events when profiling is on.
class Stage {
  public:
    Stage(const char *name, cudaStream_t st);
    ~Stage();
    Stage(const Stage &) = delete;
    Stage &operator=(const Stage &) = delete;

  private:
    const char *name_;
    cudaStream_t st_;
    cudaEvent_t e0_ = nullptr;
};

// Launches a kernel that may start while the one before it on the stream still runs, once all of
// that one's blocks have called release_next() or left. It reads what that kernel writes only
// after wait_previous(), and at least one of its threads calls that, so that the kernels of a
// call complete in order.
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args)
{
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = grid;
    c.blockDim = block;
    c.dynamicSmemBytes = smem;
    c.stream = st;
    c.attrs = &at;
    c.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
    count_launches();
    return e;
}

__device__ __forceinline__ void release_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace path
