// Shared by the stand-alone serving operators (sampling rows, paged cache, prompt attention).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
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
inline const char* paged_kv_problem(const mfs_paged_kv* c, bool quant = false)
{
    if (!c) return "null cache";
    if (!c->k || !c->v || !c->table) return "null cache pointer";
    if (quant && c->dtype != MFS_DTYPE_E4M3) return "cache dtype must be e4m3";
    if (!quant && c->dtype != MFS_DTYPE_F32 && c->dtype != MFS_DTYPE_BF16) return "cache dtype must be fp32 or bf16";
    if (c->head_dim != 64 && c->head_dim != 128) return "head_dim must be 64 or 128";
    if (c->n_pages < 1 || c->n_kv_heads < 1 || c->table_width < 1 || c->table_stride < 0)
        return "need n_pages, n_kv_heads and table_width >= 1, table_stride >= 0";
    if (c->n_kv_heads > MFS_MAX_HEADS) return "more than 65535 kv heads";
    if (c->page_size < 1 || c->page_size > MFS_MAX_PAGE_SIZE) return "page_size outside [1, 65536]";
    const int elem = quant ? 1 : c->dtype == MFS_DTYPE_BF16 ? 2 : 4;
    if (c->page_stride < 0 || c->head_stride < 0 || c->row_stride < 0) return "negative cache stride";
    if ((((uintptr_t)c->k | (uintptr_t)c->v) & 15u) || (c->page_stride * elem) % 16 || (c->head_stride * elem) % 16 ||
        (c->row_stride * elem) % 16)
        return "cache pointers and strides must be multiples of 16 bytes";
    return nullptr;
}

inline const char* quant_kv_problem(const mfs_quant_kv* c)
{
    if (!c) return "null cache";
    if (const char* why = paged_kv_problem(&c->kv, true)) return why;
    if (!c->k_exp || !c->v_exp) return "null cache pointer";
    if (c->exp_page_stride < 0 || c->exp_head_stride < 0 || c->exp_row_stride < 0) return "negative cache stride";
    return nullptr;
}

// nullptr if the rotation (NULL: none) suits heads of head_dim, else what is wrong with it.
inline const char* rope_problem(const mfs_rope* r, int head_dim)
{
    if (!r || r->layout == MFS_ROPE_NONE) return nullptr;
    if (r->layout != MFS_ROPE_INTERLEAVED && r->layout != MFS_ROPE_HALF) return "unknown rotation layout";
    if (r->dims && (r->dims < 16 || r->dims > head_dim || r->dims % 16)) return "rotated dims must be a multiple of 16, at most head_dim";
    if (!(r->theta > 0.0 && r->theta <= 1e300)) return "theta must be positive and finite";
    if (!(r->factor > 0.0 && r->factor <= 1e300)) return "the rotation's factor must be positive and finite";
    if (!(r->magnitude > 0.0 && r->magnitude <= 1e30)) return "the rotation's magnitude must be positive and finite";
    if (!(r->original >= 0.0 && r->original <= 1e300)) return "the rotation's original length must be finite and not negative";
    if (r->original > 0.0 && !(r->low >= 0.0 && r->high > r->low && r->high <= 1e300)) return "need 0 <= low < high, finite";
    return nullptr;
}

}  // namespace mfs
