// Host-side helpers shared by the library's translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdarg.h>
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>

#include "common.cuh"

namespace fgm {

// Defined in fgm.cu: the calling thread's error message, the device check and
// the bound of every wait inside a kernel.
int host_fail(int code, const char *msg);
int host_device_ready(int *sms);
long long host_wait_limit_ns();
int host_rows64_map(CUtensorMap *map, const void *base, uint64_t rows, uint32_t box_rows);
int host_lm_logits(const uint16_t *emb, int64_t V, const uint16_t *h, int M, float *z, void *ws, void *stream);
int host_hidden_map(CUtensorMap *map, const void *base, uint64_t rows, uint32_t box_rows, uint32_t slices);

inline int failf(int code, const char *fmt, ...)
{
    char buf[400];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return host_fail(code, buf);
}

#define FGM_HOST_TRY(expr)         \
    do {                           \
        int rc_ = (expr);          \
        if (rc_ != FGM_OK)         \
            return rc_;            \
    } while (0)

#define FGM_HOST_CUDA(call)                                                                     \
    do {                                                                                        \
        cudaError_t e_ = (call);                                                                \
        if (e_ != cudaSuccess)                                                                  \
            return failf(FGM_ERR_CUDA, "%s failed: %s", #call, cudaGetErrorString(e_));         \
    } while (0)

inline bool is_aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Launches a kernel that may start while the one before it in the stream ends:
// it waits for that end itself (griddepcontrol.wait) before it touches memory.
// What the one before may write is therefore not constant while the kernel lives,
// and is never read by the read-only path (__ldg), which asks for that.
template <typename... P, typename... A>
int launch_overlapped(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    FGM_HOST_CUDA(cudaLaunchKernelEx(&cfg, kernel, args...));
    return FGM_OK;
}

// A workspace of at least `need` bytes.
inline int host_check_ws(const void *ws, size_t ws_bytes, size_t need)
{
    if (!ws)
        return failf(FGM_ERR_WORKSPACE, "workspace is NULL");
    if (!is_aligned(ws, 256))
        return failf(FGM_ERR_WORKSPACE, "workspace is not 256-byte aligned");
    if (ws_bytes < need)
        return failf(FGM_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", ws_bytes, need);
    return FGM_OK;
}

}  // namespace fgm
