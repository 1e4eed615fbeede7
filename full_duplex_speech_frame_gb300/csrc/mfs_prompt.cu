// mfs_prompt_attention: causal attention over packed prompts.
#include "mfs_ops.cuh"

namespace {

using bf16 = __nv_bfloat16;
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(bf16* p, float x) { *p = __float2bfloat16_rn(x); }

// One warp per (token, query head): a running maximum and sum over the row's keys, HD / 32 elements per lane.
template <typename T, int HD>
__global__ void __launch_bounds__(128) prompt_rows_kernel(int n_tokens, int n_seqs, const int32_t* __restrict__ cu,
                                                          const T* __restrict__ q, long long q_stride, int hq,
                                                          const T* __restrict__ k, long long k_stride, const T* __restrict__ v,
                                                          long long v_stride, int hkv, T* out, long long out_stride, float scale,
                                                          int window)
{
    constexpr int E = HD / 32;
    const int t = blockIdx.x, h = blockIdx.y * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (h >= hq) return;
    int lo = 0, hi = n_seqs;
    while (hi - lo > 1) {
        const int m = (lo + hi) / 2;
        if (__ldg(cu + m) <= t) lo = m; else hi = m;
    }
    int b = max(0, __ldg(cu + lo));
    if (t < b || t >= __ldg(cu + lo + 1)) return;
    if (window > 0) b = max(b, t - window + 1);
    const int kvh = h / (hq / hkv);
    float qf[E], o[E], m = -INFINITY, l = 0.f;
    for (int e = 0; e < E; ++e) {
        qf[e] = to_f(q[(long long)t * q_stride + h * HD + lane * E + e]) * scale;
        o[e] = 0.f;
    }
    for (int j = b; j <= t; ++j) {
        const T* kr = k + (long long)j * k_stride + kvh * HD + lane * E;
        const T* vr = v + (long long)j * v_stride + kvh * HD + lane * E;
        float a = 0.f;
        for (int e = 0; e < E; ++e) a = fmaf(qf[e], to_f(kr[e]), a);
        for (int x = 16; x; x >>= 1) a += __shfl_xor_sync(0xffffffffu, a, x);
        const float mn = fmaxf(m, a), c = m == mn ? 1.f : expf(m - mn), p = a == mn ? 1.f : expf(a - mn);
        l = l * c + p;
        for (int e = 0; e < E; ++e) o[e] = o[e] * c + p * to_f(vr[e]);
        m = mn;
    }
    for (int e = 0; e < E; ++e) put(out + (long long)t * out_stride + h * HD + lane * E + e, o[e] / l);
}

template <typename T, int HD>
int run(int n_tokens, int n_seqs, const int32_t* cu, const void* q, long long q_stride, int hq, const void* k, long long k_stride,
        const void* v, long long v_stride, int hkv, void* out, long long out_stride, float scale, int window, cudaStream_t st)
{
    prompt_rows_kernel<T, HD><<<dim3((unsigned)n_tokens, (unsigned)((hq + 3) / 4)), 128, 0, st>>>(
        n_tokens, n_seqs, cu, (const T*)q, q_stride, hq, (const T*)k, k_stride, (const T*)v, v_stride, hkv, (T*)out, out_stride,
        scale, window);
    return mfs::op_launched("prompt_attention", cudaGetLastError());
}

}  // namespace

extern "C" int mfs_prompt_attention(int dtype, int n_tokens, int n_seqs, const int32_t* cu, const void* q, long long q_stride,
                                    int n_q_heads, const void* k, long long k_stride, const void* v, long long v_stride,
                                    int n_kv_heads, int head_dim, void* out, long long out_stride, float scale, int window,
                                    void* cuda_stream)
{
    const char* op = "prompt_attention";
    if (dtype != MFS_DTYPE_F32 && dtype != MFS_DTYPE_BF16) return mfs::op_fail(MFS_E_ARG, op, "dtype must be fp32 or bf16");
    if (head_dim != 64 && head_dim != 128) return mfs::op_fail(MFS_E_ARG, op, "head_dim must be 64 or 128");
    if (n_tokens < 0 || n_seqs < 0 || window < 0) return mfs::op_fail(MFS_E_ARG, op, "need n_tokens, n_seqs and window >= 0");
    if (n_kv_heads < 1 || n_q_heads < 1 || n_q_heads % n_kv_heads || n_q_heads > 65535)
        return mfs::op_fail(MFS_E_ARG, op, "n_q_heads must be a multiple of n_kv_heads, at most 65535");
    if (!(scale > 0.f && scale <= 1e30f)) return mfs::op_fail(MFS_E_ARG, op, "scale must be positive and finite");
    if (n_tokens == 0 || n_seqs == 0) return MFS_OK;
    if (!cu || !q || !k || !v || !out) return mfs::op_fail(MFS_E_ARG, op, "null cu, q, k, v or out");
    const int elem = dtype == MFS_DTYPE_BF16 ? 2 : 4;
    if (!mfs::rows_ok(q, q_stride, n_q_heads, head_dim, elem) || !mfs::rows_ok(k, k_stride, n_kv_heads, head_dim, elem) ||
        !mfs::rows_ok(v, v_stride, n_kv_heads, head_dim, elem) || !mfs::rows_ok(out, out_stride, n_q_heads, head_dim, elem))
        return mfs::op_fail(MFS_E_ARG, op, "pointers and token strides must be multiples of 16 bytes, a stride at least heads x head_dim");
    cudaStream_t st = (cudaStream_t)cuda_stream;
    auto fn = dtype == MFS_DTYPE_BF16 ? (head_dim == 128 ? run<bf16, 128> : run<bf16, 64>)
                                      : (head_dim == 128 ? run<float, 128> : run<float, 64>);
    return fn(n_tokens, n_seqs, cu, q, q_stride, n_q_heads, k, k_stride, v, v_stride, n_kv_heads, out, out_stride, scale, window, st);
}
