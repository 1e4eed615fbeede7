// Shared by the stand-alone serving operators (sampling rows, paged cache, prompt attention).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <atomic>

#include "../../include/mfs.h"

namespace mfs {
void set_thread_error(const char* msg);  // defined with mfs_last_error

inline int op_fail(int code, const char* op, const char* msg)
{
    char buf[200];
    snprintf(buf, sizeof buf, "%s: %s", op, msg);
    set_thread_error(buf);
    return code;
}

inline int op_launched(const char* op, cudaError_t e)
{
    return e == cudaSuccess ? MFS_OK : op_fail(MFS_E_CUDA, op, cudaGetErrorString(e));
}

// What a kernel's launches need to know of each device: its SMs, and that its shared memory limit has been raised there.
struct PerDevice {
    std::atomic<int> sms[64];
};

// SMs of the current device; on the first call there, `kernel` (if any) is allowed `smem` bytes of dynamic shared memory.
inline cudaError_t op_device(PerDevice& known, const void* kernel, int smem, int* sms)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (*sms = known.sms[dev].load(std::memory_order_acquire)) > 0) return cudaSuccess;
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && kernel) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && dev < 64) known.sms[dev].store(*sms, std::memory_order_release);
    return e;
}

// Pointer and token stride of a [tokens][heads][head_dim] array: 16-byte steps, heads dense.
inline bool rows_ok(const void* p, long long stride, int heads, int head_dim, int elem)
{
    return ((uintptr_t)p & 15u) == 0 && stride >= (long long)heads * head_dim && (stride * elem) % 16 == 0;
}

// nullptr if the descriptor is sound, else what is wrong with it.
inline const char* paged_kv_problem(const mfs_paged_kv* c)
{
    if (!c) return "null cache";
    if (!c->k || !c->v || !c->table) return "null cache pointer";
    if (c->dtype != MFS_DTYPE_F32 && c->dtype != MFS_DTYPE_BF16) return "cache dtype must be fp32 or bf16";
    if (c->head_dim != 64 && c->head_dim != 128) return "head_dim must be 64 or 128";
    if (c->n_pages < 1 || c->n_kv_heads < 1 || c->table_width < 1 || c->table_stride < 0)
        return "need n_pages, n_kv_heads and table_width >= 1, table_stride >= 0";
    if (c->n_kv_heads > MFS_MAX_HEADS) return "more than 65535 kv heads";
    if (c->page_size < 1 || c->page_size > MFS_MAX_PAGE_SIZE) return "page_size outside [1, 65536]";
    const int elem = c->dtype == MFS_DTYPE_BF16 ? 2 : 4;
    if (c->page_stride < 0 || c->head_stride < 0 || c->row_stride < 0) return "negative cache stride";
    if ((((uintptr_t)c->k | (uintptr_t)c->v) & 15u) || (c->page_stride * elem) % 16 || (c->head_stride * elem) % 16 ||
        (c->row_stride * elem) % 16)
        return "cache pointers and strides must be multiples of 16 bytes";
    return nullptr;
}

}  // namespace mfs
