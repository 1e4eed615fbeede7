// Paged key/value cache: mfs_kv_append (rotate and write new tokens) and
// mfs_paged_attention (one new token per sequence).
#include "mfs_ops.cuh"

namespace {

using bf16 = __nv_bfloat16;

struct Cache {
    char* k;
    char* v;
    const int32_t* table;
    int table_width, n_pages, page_size, n_kv_heads;
    long long table_stride, page_stride, head_stride, row_stride;  // elements
};

Cache cache_of(const mfs_paged_kv* c)
{
    return {(char*)c->k, (char*)c->v, c->table, c->table_width, c->n_pages, c->page_size, c->n_kv_heads,
            c->table_stride, c->page_stride, c->head_stride, c->row_stride};
}

// Element offset of head 0 of position p of sequence s, or -1 where the table has no valid page for it.
__device__ __forceinline__ long long row_offset(const Cache& C, int s, int p)
{
    const int j = p / C.page_size;
    if (p < 0 || j >= C.table_width) return -1;
    const int page = __ldg(C.table + s * C.table_stride + j);
    if (page < 0 || page >= C.n_pages) return -1;
    return (long long)page * C.page_stride + (long long)(p - j * C.page_size) * C.row_stride;
}

// ------------------------------------------------------------------ append

struct Turns {
    double f[64];  // turns per position of pair i: theta^(-2 i / head_dim) / (2 pi)
};

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f(float x) { return x; }
template <>
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f(float x) { return x; }
template <>
__device__ __forceinline__ bf16 from_f(float x) { return __float2bfloat16_rn(x); }

constexpr int AP_THREADS = 256;

// One block per token: its position's cosines and sines once, then a pair of elements per thread and step.
template <typename T>
__global__ void __launch_bounds__(AP_THREADS) append_kernel(Cache C, int n_seqs, int n_tokens, const int32_t* __restrict__ cu,
                                                            const int32_t* __restrict__ kv_len, const T* q, long long q_stride,
                                                            int hq, T* q_out, long long q_out_stride, const T* k,
                                                            long long k_stride, T* k_out, long long k_out_stride, const T* v,
                                                            long long v_stride, int hd, int rope,
                                                            const __grid_constant__ Turns turns)
{
    __shared__ float sc[64], ss[64];
    __shared__ long long s_row;
    const int t = blockIdx.x, half = hd / 2;
    // the sequence: the last s with cu[s] <= t
    int lo = 0, hi = n_seqs;
    while (hi - lo > 1) {
        const int m = (lo + hi) / 2;
        if (__ldg(cu + m) <= t) lo = m; else hi = m;
    }
    const int end = __ldg(cu + lo + 1);
    if (t < __ldg(cu) || t >= end) return;  // a row of no sequence
    const long long pos = (long long)__ldg(kv_len + lo) - end + t;
    if (threadIdx.x < half) {
        const double a = (double)pos * turns.f[threadIdx.x];
        float s = 0.f, c = 1.f;
        if (rope) sincospif(2.f * (float)(a - rint(a)), &s, &c);
        sc[threadIdx.x] = c;
        ss[threadIdx.x] = s;
    }
    if (threadIdx.x == AP_THREADS - 1) s_row = pos < 0 || pos > 0x7fffffff ? -1 : row_offset(C, lo, (int)pos);
    __syncthreads();
    const long long row = s_row;
    T* kc = reinterpret_cast<T*>(C.k);
    T* vc = reinterpret_cast<T*>(C.v);
    const int hkv = C.n_kv_heads;
    for (int i = threadIdx.x; i < (hq + hkv) * half; i += AP_THREADS) {
        const int h = i / half, e = i % half;
        const int e0 = rope == MFS_ROPE_HALF ? e : 2 * e, e1 = rope == MFS_ROPE_HALF ? e + half : 2 * e + 1;
        const bool is_q = h < hq;
        const int hh = is_q ? h : h - hq;
        const T* src = (is_q ? q + (long long)t * q_stride : k + (long long)t * k_stride) + hh * hd;
        const float a = to_f(src[e0]), b = to_f(src[e1]);
        T x = src[e0], y = src[e1];
        if (rope) {
            x = from_f<T>(a * sc[e] - b * ss[e]);
            y = from_f<T>(a * ss[e] + b * sc[e]);
        }
        if (is_q) {
            T* dst = q_out + (long long)t * q_out_stride + hh * hd;
            dst[e0] = x;
            dst[e1] = y;
        } else {
            if (k_out) {
                T* dst = k_out + (long long)t * k_out_stride + hh * hd;
                dst[e0] = x;
                dst[e1] = y;
            }
            if (row >= 0) {
                T* dst = kc + row + (long long)hh * C.head_stride;
                dst[e0] = x;
                dst[e1] = y;
            }
        }
    }
    if (row < 0) return;
    for (int i = threadIdx.x; i < hkv * hd; i += AP_THREADS)
        vc[row + (long long)(i / hd) * C.head_stride + i % hd] = v[(long long)t * v_stride + i];
}

template <typename T>
int append(const Cache& C, int n_tokens, int n_seqs, const int32_t* cu, const int32_t* kv_len, const void* q, long long q_stride,
           int hq, void* q_out, long long q_out_stride, const void* k, long long k_stride, void* k_out, long long k_out_stride,
           const void* v, long long v_stride, int hd, int rope, const Turns& turns, cudaStream_t st)
{
    append_kernel<T><<<n_tokens, AP_THREADS, 0, st>>>(C, n_seqs, n_tokens, cu, kv_len, (const T*)q, q_stride, hq, (T*)q_out,
                                                     q_out_stride, (const T*)k, k_stride, (T*)k_out, k_out_stride,
                                                     (const T*)v, v_stride, hd, rope, turns);
    return mfs::op_launched("kv_append", cudaGetLastError());
}

// --------------------------------------------------------------- attention

// One warp per (sequence, query head): a running maximum and sum over the keys, HD / 32 elements per lane.
template <typename T, int HD>
__global__ void __launch_bounds__(128) paged_attention_kernel(Cache C, int n_seqs, const int32_t* __restrict__ kv_len,
                                                              const T* q, long long q_stride, int hq, T* out,
                                                              long long out_stride, float scale, int window)
{
    constexpr int E = HD / 32;
    const int w = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (w >= n_seqs * hq) return;
    const int s = w / hq, h = w % hq, kvh = h / (hq / C.n_kv_heads);
    const int len = __ldg(kv_len + s);
    float qf[E], o[E], m = -INFINITY, l = 0.f;
    for (int e = 0; e < E; ++e) {
        qf[e] = to_f(q[(long long)s * q_stride + h * HD + lane * E + e]) * scale;
        o[e] = 0.f;
    }
    bool bad = false;
    for (int p = window > 0 && len > window ? len - window : 0; p < len; ++p) {
        const long long row = row_offset(C, s, p);
        if (row < 0) { bad = true; break; }
        const T* kr = reinterpret_cast<const T*>(C.k) + row + (long long)kvh * C.head_stride + lane * E;
        const T* vr = reinterpret_cast<const T*>(C.v) + row + (long long)kvh * C.head_stride + lane * E;
        float a = 0.f;
        for (int e = 0; e < E; ++e) a = fmaf(qf[e], to_f(kr[e]), a);
        for (int x = 16; x; x >>= 1) a += __shfl_xor_sync(0xffffffffu, a, x);
        const float mn = fmaxf(m, a), c = m == mn ? 1.f : expf(m - mn), pr = a == mn ? 1.f : expf(a - mn);
        l = l * c + pr;
        for (int e = 0; e < E; ++e) o[e] = o[e] * c + pr * to_f(vr[e]);
        m = mn;
    }
    for (int e = 0; e < E; ++e)
        out[(long long)s * out_stride + h * HD + lane * E + e] = from_f<T>(bad ? NAN : len > 0 ? o[e] / l : 0.f);
}

template <typename T, int HD>
int attention(const Cache& C, int n_seqs, const int32_t* kv_len, const void* q, long long q_stride, int hq, void* out,
              long long out_stride, float scale, int window, cudaStream_t st)
{
    const long long warps = (long long)n_seqs * hq;
    paged_attention_kernel<T, HD><<<(unsigned)((warps + 3) / 4), 128, 0, st>>>(C, n_seqs, kv_len, (const T*)q, q_stride, hq,
                                                                             (T*)out, out_stride, scale, window);
    return mfs::op_launched("paged_attention", cudaGetLastError());
}

}  // namespace

extern "C" int mfs_kv_append(const mfs_paged_kv* cache, int n_tokens, int n_seqs, const int32_t* cu, const int32_t* kv_len,
                             const void* q, long long q_stride, int n_q_heads, void* q_out, long long q_out_stride,
                             const void* k, long long k_stride, void* k_out, long long k_out_stride, const void* v,
                             long long v_stride, int rope, double theta, void* cuda_stream)
{
    const char* op = "kv_append";
    if (const char* why = mfs::paged_kv_problem(cache)) return mfs::op_fail(MFS_E_ARG, op, why);
    if (n_tokens < 0 || n_seqs < 0) return mfs::op_fail(MFS_E_ARG, op, "need n_tokens >= 0 and n_seqs >= 0");
    if (rope != MFS_ROPE_NONE && rope != MFS_ROPE_INTERLEAVED && rope != MFS_ROPE_HALF)
        return mfs::op_fail(MFS_E_ARG, op, "unknown rotation layout");
    if (rope != MFS_ROPE_NONE && !(theta > 0.0 && theta <= 1e300)) return mfs::op_fail(MFS_E_ARG, op, "theta must be positive and finite");
    if (n_tokens == 0 || n_seqs == 0) return MFS_OK;
    const int hd = cache->head_dim, elem = cache->dtype == MFS_DTYPE_BF16 ? 2 : 4;
    if (!cu || !kv_len || !k || !v) return mfs::op_fail(MFS_E_ARG, op, "null cu, kv_len, k or v");
    if ((q != nullptr) != (q_out != nullptr)) return mfs::op_fail(MFS_E_ARG, op, "q and q_out go together");
    if (q && n_q_heads < 1) return mfs::op_fail(MFS_E_ARG, op, "need n_q_heads >= 1");
    if (!mfs::rows_ok(k, k_stride, cache->n_kv_heads, hd, elem) || !mfs::rows_ok(v, v_stride, cache->n_kv_heads, hd, elem) ||
        (k_out && !mfs::rows_ok(k_out, k_out_stride, cache->n_kv_heads, hd, elem)) ||
        (q && (!mfs::rows_ok(q, q_stride, n_q_heads, hd, elem) || !mfs::rows_ok(q_out, q_out_stride, n_q_heads, hd, elem))))
        return mfs::op_fail(MFS_E_ARG, op, "pointers and token strides must be multiples of 16 bytes, a stride at least heads x head_dim");
    Turns turns = {};
    if (rope)
        for (int i = 0; i < hd / 2; ++i) turns.f[i] = pow(theta, -2.0 * i / hd) / 6.283185307179586476925;
    const Cache C = cache_of(cache);
    const int hq = q ? n_q_heads : 0;
    cudaStream_t st = (cudaStream_t)cuda_stream;
    return cache->dtype == MFS_DTYPE_BF16
               ? append<bf16>(C, n_tokens, n_seqs, cu, kv_len, q, q_stride, hq, q_out, q_out_stride, k, k_stride, k_out,
                              k_out_stride, v, v_stride, hd, rope, turns, st)
               : append<float>(C, n_tokens, n_seqs, cu, kv_len, q, q_stride, hq, q_out, q_out_stride, k, k_stride, k_out,
                               k_out_stride, v, v_stride, hd, rope, turns, st);
}

extern "C" size_t mfs_paged_attention_workspace(const mfs_paged_kv* cache, int n_q_heads)
{
    (void)cache;
    (void)n_q_heads;
    return 16;
}

extern "C" int mfs_paged_attention(const mfs_paged_kv* cache, int n_seqs, const int32_t* kv_len, const void* q,
                                   long long q_stride, int n_q_heads, void* out, long long out_stride, float scale, int window,
                                   void* workspace, size_t workspace_bytes, void* cuda_stream)
{
    const char* op = "paged_attention";
    if (const char* why = mfs::paged_kv_problem(cache)) return mfs::op_fail(MFS_E_ARG, op, why);
    if (n_seqs < 0 || window < 0) return mfs::op_fail(MFS_E_ARG, op, "need n_seqs >= 0 and window >= 0");
    if (n_q_heads < 1 || n_q_heads % cache->n_kv_heads) return mfs::op_fail(MFS_E_ARG, op, "n_q_heads must be a multiple of n_kv_heads");
    if (!(scale > 0.f && scale <= 1e30f)) return mfs::op_fail(MFS_E_ARG, op, "scale must be positive and finite");
    if (n_seqs == 0) return MFS_OK;
    if (!kv_len || !q || !out || !workspace) return mfs::op_fail(MFS_E_ARG, op, "null kv_len, q, out or workspace");
    const int hd = cache->head_dim, elem = cache->dtype == MFS_DTYPE_BF16 ? 2 : 4;
    if (!mfs::rows_ok(q, q_stride, n_q_heads, hd, elem) || !mfs::rows_ok(out, out_stride, n_q_heads, hd, elem))
        return mfs::op_fail(MFS_E_ARG, op, "pointers and token strides must be multiples of 16 bytes, a stride at least heads x head_dim");
    if (((uintptr_t)workspace & 15u) || workspace_bytes < mfs_paged_attention_workspace(cache, n_q_heads))
        return mfs::op_fail(MFS_E_ARG, op, "workspace too small or not 16-byte aligned");
    if ((long long)n_seqs * n_q_heads > 0x7fffffffLL) return mfs::op_fail(MFS_E_ARG, op, "too many sequences x heads");
    const Cache C = cache_of(cache);
    cudaStream_t st = (cudaStream_t)cuda_stream;
    if (cache->dtype == MFS_DTYPE_BF16)
        return hd == 128 ? attention<bf16, 128>(C, n_seqs, kv_len, q, q_stride, n_q_heads, out, out_stride, scale, window, st)
                         : attention<bf16, 64>(C, n_seqs, kv_len, q, q_stride, n_q_heads, out, out_stride, scale, window, st);
    return hd == 128 ? attention<float, 128>(C, n_seqs, kv_len, q, q_stride, n_q_heads, out, out_stride, scale, window, st)
                     : attention<float, 64>(C, n_seqs, kv_len, q, q_stride, n_q_heads, out, out_stride, scale, window, st);
}
