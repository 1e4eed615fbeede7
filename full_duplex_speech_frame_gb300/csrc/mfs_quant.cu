// mfs_quant_attention: one new token per sequence over the 8-bit cache.
#include "mfs_quant.cuh"

extern "C" size_t mfs_quant_attention_workspace(const mfs_quant_kv* cache, int dtype, int n_q_heads)
{
    (void)n_q_heads;
    if (mfs::quant_kv_problem(cache) || (dtype != MFS_DTYPE_F32 && dtype != MFS_DTYPE_BF16)) return 0;
    return quant_workspace(cache->kv.head_dim);
}

extern "C" int mfs_quant_attention(const mfs_quant_kv* cache, int dtype, int n_seqs, const int32_t* kv_len, const void* q,
                                   long long q_stride, int n_q_heads, void* out, long long out_stride, float scale, int window,
                                   void* workspace, size_t workspace_bytes, void* cuda_stream)
{
    const char* op = "paged_attention";
    if (const char* why = mfs::quant_kv_problem(cache)) return mfs::op_fail(MFS_E_ARG, op, why);
    PaArgs A = quant_args(cache);
    const int hd = cache->kv.head_dim;
    if (const int rc = pa_checked(op, A, dtype, hd, n_seqs, kv_len, q, q_stride, n_q_heads, out, out_stride, scale, window, workspace,
                                  workspace_bytes, mfs_quant_attention_workspace(cache, dtype, n_q_heads)))
        return rc < 0 ? rc : MFS_OK;
    cudaStream_t st = (cudaStream_t)cuda_stream;
    char* ws = (char*)workspace;
    // bf16: blocks of eight or sixteen query heads; the second reads the cache once for groups of nine and more
    auto fn = dtype == MFS_DTYPE_F32 ? (hd == 128 ? attention<PaKindE4m3<float, 128, 1>> : attention<PaKindE4m3<float, 64, 1>>)
              : A.g <= 8             ? (hd == 128 ? attention<PaKindE4m3<bf16, 128, 1>> : attention<PaKindE4m3<bf16, 64, 1>>)
                                     : (hd == 128 ? attention<PaKindE4m3<bf16, 128, 2>> : attention<PaKindE4m3<bf16, 64, 2>>);
    return fn(A, ws, st, op);
}
