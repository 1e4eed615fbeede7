// Paged key/value cache: mfs_kv_append (rotate and write new tokens) and
// mfs_paged_attention (one new token per sequence).
#include <string.h>
#include <type_traits>

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

// A block takes a few tokens: one warp per token finds its sequence, position and row in the cache, and the cosines and
// sines of its angles; the block's threads then move items of two 16-byte vectors that hold whole pairs (neighbours for
// interleaved pairs, half a head apart for split ones), the next one on its way while one is rotated, the first while
// the angles are found.  What bounds it is memory: each input is read and each output written once.  8192 tokens of 32 + 8
// heads of 128 bf16: 39 us, 0.83 of the measured copy rate; blocks of 256 threads and 4 tokens 40 us, three items on
// their way per thread (fewer blocks on an SM) 45 us, 8 tokens 45 us.  The same in fp32: 77 us, 0.84.
constexpr int AP_THREADS = 128;
// Tokens per block; 1 up to 8 blocks per SM (4 tokens of 16 heads: 3.9 us, 5.5 us by twos; 1200 of 32 + 8 heads 8.7 and
// 9.3; 1800 14.2 and 13.1; 8192 40.3 and 38.5).
constexpr int AP_TOKENS = 2;

template <typename T>
struct ApArgs {
    Cache C;
    const int32_t *cu, *kv_len;
    const T *q, *k, *v;
    T *q_out, *k_out;
    long long q_stride, q_out_stride, k_stride, k_out_stride, v_stride;
    int n_tokens, n_seqs, hq, rope;
    Turns turns;
};

template <typename T>
struct Vec2 {
    uint4 a, b;
};

template <typename T, int HD, int TT>
__global__ void __launch_bounds__(AP_THREADS) append_kernel(const __grid_constant__ ApArgs<T> A)
{
    constexpr int VE = 16 / sizeof(T);        // elements per vector
    constexpr int IPH = HD / (2 * VE);        // items per head
    constexpr int HALF = HD / 2;
    __shared__ float2 cs[TT][HALF];
    __shared__ long long row[TT];             // element offset of the token's row (head 0) in the cache; -1: none; -2: no token
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int t0 = blockIdx.x * TT, nt = min(TT, A.n_tokens - t0);
    const int hkv = A.C.n_kv_heads, heads = A.hq + 2 * hkv, items = nt * heads * IPH;
    const bool split = A.rope == MFS_ROPE_HALF;

    // item i: token, head (queries, keys, values), place within the head
    auto where = [&](int i, int& t, int& h, int& e) {
        const int hh = i / IPH;
        e = i % IPH;
        t = TT == 1 ? 0 : hh / heads;
        h = TT == 1 ? hh : hh - t * heads;
    };
    auto source = [&](int i) {
        int t, h, e;
        where(i, t, h, e);
        const long long tok = t0 + t;
        const T* p = h < A.hq ? A.q + tok * A.q_stride + h * HD : h < A.hq + hkv ? A.k + tok * A.k_stride + (h - A.hq) * HD
                                                                              : A.v + tok * A.v_stride + (h - A.hq - hkv) * HD;
        const int first = split ? e * VE : 2 * e * VE, second = split ? first + HALF : first + VE;
        // plain loads: the queries and keys may be their own outputs
        return Vec2<T>{*reinterpret_cast<const uint4*>(p + first), *reinterpret_cast<const uint4*>(p + second)};
    };
    Vec2<T> x;
    if (tid < items) x = source(tid);

    if (warp < nt) {
        // the sequence: the last s with cu[s] <= token, 32 places at a time
        const int t = t0 + warp;
        int lo = 0, size = A.n_seqs;
        while (size > 1) {
            const int step = (size + 31) / 32, at = lane * step;
            const unsigned m = __ballot_sync(0xffffffffu, at < size && __ldg(A.cu + lo + at) <= t);
            const int c = max(0, 31 - __clz(m));  // the last probe that is not past the token
            lo += c * step;
            size = min(step, size - c * step);
        }
        const int begin = __ldg(A.cu + lo), end = __ldg(A.cu + lo + 1);
        const long long pos = (long long)__ldg(A.kv_len + lo) - end + t;
        if (lane == 0) row[warp] = t < begin || t >= end ? -2 : pos < 0 || pos > 0x7fffffff ? -1 : row_offset(A.C, lo, (int)pos);
        if (A.rope)
            for (int i = lane; i < HALF; i += 32) {
                // turns in 64 bits; what is left of one, up to half, in fp32: off by 2^-26 of a turn, 1e-7 in the cosine
                const double a = (double)pos * A.turns.f[i];
                float s, c;
                sincospif(2.f * (float)(a - rint(a)), &s, &c);
                cs[warp][i] = make_float2(c, s);
            }
    }
    __syncthreads();

    auto finish = [&](int i, Vec2<T> y) {
        int t, h, e;
        where(i, t, h, e);
        const long long r = row[t];
        if (r == -2) return;
        const long long tok = t0 + t;
        const int first = split ? e * VE : 2 * e * VE, second = split ? first + HALF : first + VE;
        if (h < A.hq + hkv && A.rope) {
            T in[2 * VE], out[2 * VE];
            memcpy(in, &y, 32);
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                // pair j of the item: elements (j, j + VE) of the two vectors for split pairs, (2 j, 2 j + 1) for neighbours
                const float2 c = cs[t][e * VE + j];
                const float u = to_f(split ? in[j] : in[2 * j]), w = to_f(split ? in[j + VE] : in[2 * j + 1]);
                const T a = from_f<T>(u * c.x - w * c.y), b = from_f<T>(u * c.y + w * c.x);
                if (split) { out[j] = a; out[j + VE] = b; }
                else { out[2 * j] = a; out[2 * j + 1] = b; }
            }
            memcpy(&y, out, 32);
        }
        auto put = [&](T* p) {
            *reinterpret_cast<uint4*>(p + first) = y.a;
            *reinterpret_cast<uint4*>(p + second) = y.b;
        };
        if (h < A.hq) {
            put(A.q_out + tok * A.q_out_stride + h * HD);
        } else if (h < A.hq + hkv) {
            if (A.k_out) put(A.k_out + tok * A.k_out_stride + (h - A.hq) * HD);
            if (r >= 0) put(reinterpret_cast<T*>(A.C.k) + r + (long long)(h - A.hq) * A.C.head_stride);
        } else if (r >= 0) {
            put(reinterpret_cast<T*>(A.C.v) + r + (long long)(h - A.hq - hkv) * A.C.head_stride);
        }
    };
    for (int i = tid; i < items; i += AP_THREADS) {
        const Vec2<T> y = x;
        if (i + AP_THREADS < items) x = source(i + AP_THREADS);
        finish(i, y);
    }
}

template <typename T, int HD>
int append(const ApArgs<T>& A, cudaStream_t st)
{
    int sms = 0;
    static mfs::PerDevice ready;
    cudaError_t e = mfs::op_device(ready, nullptr, 0, &sms);
    if (e == cudaSuccess) {
        if (A.n_tokens <= 8 * sms) append_kernel<T, HD, 1><<<A.n_tokens, AP_THREADS, 0, st>>>(A);
        else append_kernel<T, HD, AP_TOKENS><<<(A.n_tokens + AP_TOKENS - 1) / AP_TOKENS, AP_THREADS, 0, st>>>(A);
        e = cudaGetLastError();
    }
    return mfs::op_launched("kv_append", e);
}

template <typename T>
int append_typed(const Cache& C, int n_tokens, int n_seqs, const int32_t* cu, const int32_t* kv_len, const void* q, long long q_stride,
                 int hq, void* q_out, long long q_out_stride, const void* k, long long k_stride, void* k_out,
                 long long k_out_stride, const void* v, long long v_stride, int hd, int rope, const Turns& turns, cudaStream_t st)
{
    const ApArgs<T> A = {C, cu, kv_len, (const T*)q, (const T*)k, (const T*)v, (T*)q_out, (T*)k_out, q_stride, q_out_stride, k_stride,
                         k_out_stride, v_stride, n_tokens, n_seqs, hq, rope, turns};
    return hd == 128 ? append<T, 128>(A, st) : append<T, 64>(A, st);
}

// --------------------------------------------------------------- attention
//
// The keys of every (sequence, kv head, block of GM query heads), an item, are cut into tiles of 8 KB of
// keys and values (16 positions of 128 bf16).  All tiles of the call, laid end to end with a little room
// at each item's start for what it costs beside them, are cut into equal shares, one per warp of a grid
// that fills the GPU once: a warp walks through its share whatever sequences it crosses, so ragged lengths
// and few long sequences load every SM alike.  An item that lies in one share is finished by its warp.
// The pieces of the others meet in shared memory once, when the CTA's warps are done; what still crosses
// CTAs goes to the workspace (at most two pieces per CTA) and a second kernel, whose launch overlaps the
// first one's run, joins it in share order.
//
// A warp keeps its own running maximum, sum and output, so no warp waits for another before the end;
// it feeds itself through a ring of stages with 16-byte asynchronous copies (rows past the length are
// filled with zeros and never read), with the page of the next stage's rows looked up a stage ahead.
//
// What bounds it is memory: each key and value is read once.  bf16, 8 kv heads of 128: 4 sequences of up
// to 131072, 64 query heads, 202 us = 6.6 TB/s, 0.98 of the measured copy rate; 32 of up to 8192, 32
// query heads, pages of 16, 91 us = 6.1 TB/s; the rest is the start, the join and two launches, which
// is most of one sequence of 3000 positions and 32 kv heads: 17.3 us, 7.3 us of it memory.  The matrix
// instructions (a tile's 16 rows are the group's query heads, zero rows for those it lacks) keep the
// tensor pipe 17 % busy there, so the wide forms of them would gain nothing.

constexpr int PA_WARPS = 4;
constexpr int PA_MAX_CTAS = 304;  // 2 per SM
// What an item costs beside its tiles (its start, its end, its queries), in tiles: shares are cut over both.  64 ragged
// sequences of up to 1000, 24 + 8 heads of 128: 44.3 us with 0, 35.7 with 1, 35.9 with 2, 35.6 with 4; 256 of up to 300,
// 32 + 8 heads: 53.9, 44.0, 43.0, 44.3, fp32 139, 85, 81, 82; 64 of up to 100, 8 + 8 heads: 13.7, 12.7, 13.0, 14.1.
constexpr int PA_ITEM = 2;
constexpr int PA_STAGES = 2;      // 16 KB per warp; 3 stages measured 5 % slower on long contexts

// Query heads per block: the 16 rows of an mma tile for bf16.  fp32, on the CUDA cores, pays for every head of the
// block, so it has three widths, 1, 4 and 8: 8 sequences of 8192, 8 kv heads of 128, groups of 1, 2, 4 and 8 take 87,
// 111, 113 and 167 us, with 8 alone 164, 164, 166 and 167 us (537 MB: 79 us at the measured copy rate).  What bounds the
// wider ones is not the products (9.5 TFLOP/s) but shared memory and the two warps per scheduler: every product's operands
// and a shuffle per key and head go through its data path, 49 % busy for groups of 4 and 56 % for 8; issue 44 and 47 %.
template <typename T>
constexpr int PA_GM_MAX = sizeof(T) == 2 ? 16 : 8;

__device__ __forceinline__ unsigned su32(const void* p) { return (unsigned)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void copy16(unsigned dst, const void* src, bool full)
{
    const int n = full ? 16 : 0;
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const unsigned (&a)[4], unsigned b0, unsigned b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldm4(unsigned addr, unsigned (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}

__device__ __forceinline__ void ldm4t(unsigned addr, unsigned (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}

__device__ __forceinline__ unsigned pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const unsigned*>(&v);
}

template <typename T, int HD>
constexpr int PA_ROWS = 4096 / (HD * (int)sizeof(T));  // positions per tile: 4 KB of keys, 4 KB of values

// Where element x (row x / HD) of a piece lies: 8 rows of a store meet different banks.
template <int HD>
__device__ __forceinline__ int pa_at(int x) { return x ^ (((x / HD) & 7) << 3); }

__device__ __forceinline__ void put4(float* p, float4 v, float by)
{
    *reinterpret_cast<float4*>(p) = make_float4(v.x * by, v.y * by, v.z * by, v.w * by);
}
__device__ __forceinline__ void put4(bf16* p, float4 v, float by)
{
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v.x * by, v.y * by), pack_bf16(v.z * by, v.w * by));
}

struct PaArgs {
    Cache C;
    const int32_t* kv_len;
    const char* q;
    char* out;
    long long q_stride, out_stride;
    int n_seqs, hq, g, nhb, window;
    float c;          // scale * log2(e)
    float* part_o;    // [CTA][2][GM][HD]
    float2* part_ml;  // [CTA][2][GM] running maximum (raw score) and sum
    int join_rows;    // log2 of the query heads per block of the join: 0 or 1
    int4* rec;        // [CTA] {sequence or -1, head block, last CTA of the item, 0}
};

// Where a walk through the tiles stands.
struct PaWalk {
    int s, hb, tile, ntiles, lo, len;
};

template <int ROWS>
__device__ __forceinline__ void pa_sequence(const PaArgs& A, PaWalk& w)
{
    w.len = __ldg(A.kv_len + w.s);
    w.lo = A.window > 0 && w.len > A.window ? w.len - A.window : 0;
    w.ntiles = w.len > w.lo ? (int)(((long long)w.len - w.lo + ROWS - 1) / ROWS) : 0;
}

template <int ROWS>
__device__ __forceinline__ void pa_next(const PaArgs& A, PaWalk& w)
{
    if (++w.tile < w.ntiles) return;
    w.tile = 0;
    if (++w.hb < A.C.n_kv_heads * A.nhb) return;
    w.hb = 0;
    do {
        ++w.s;
        if (w.s >= A.n_seqs) return;
        pa_sequence<ROWS>(A, w);
    } while (w.ntiles == 0);
}

// Element offset of this lane's row (lane mod ROWS) of the tile, or -1.
template <int ROWS>
__device__ __forceinline__ long long pa_offset(const PaArgs& A, const PaWalk& w, bool& bad)
{
    const int p = w.lo + w.tile * ROWS + (threadIdx.x & (ROWS - 1));
    if ((unsigned)p >= (unsigned)w.len) return -1;  // a last tile may reach past 2^31 - 1
    const long long off = row_offset(A.C, w.s, p);
    if (off < 0) { bad = true; return -1; }
    return off + (long long)(w.hb / A.nhb) * A.C.head_stride;
}

template <typename T, int HD>
__device__ __forceinline__ void pa_issue(const PaArgs& A, unsigned stage, long long off)
{
    constexpr int CH = HD * sizeof(T) / 16;      // 16-byte chunks per row
    constexpr int RPI = CH >= 32 ? 1 : 32 / CH;  // rows per instruction
    constexpr int ROWS = PA_ROWS<T, HD>;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < ROWS / RPI; ++j) {
        const int row = j * RPI + lane / CH, ch = lane % CH;
        const long long o = __shfl_sync(0xffffffffu, off, row);
        const long long byte = (o < 0 ? 0 : o) * (long long)sizeof(T) + ch * 16;
        const unsigned dst = stage + row * (HD * (int)sizeof(T)) + ((ch ^ (row & 7)) << 4);
        copy16(dst, A.C.k + byte, o >= 0);
        copy16(dst + ROWS * HD * (int)sizeof(T), A.C.v + byte, o >= 0);
    }
}

// One warp's state for an item: scores by mma for bf16 (16 query heads per tile, the rest zero).
template <int HD>
struct PaBf16 {
    static constexpr int GM = 16, ROWS = PA_ROWS<bf16, HD>, NK = ROWS / 8;  // key octets
    unsigned qf[HD / 16][4];
    float o[HD / 8][4], m[2], l[2];

    __device__ __forceinline__ void begin(const PaArgs& A, const PaWalk& w, float*)
    {
        const int lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
        const int h0 = (w.hb / A.nhb) * A.g + (w.hb % A.nhb) * GM, nh = min(GM, A.g - (w.hb % A.nhb) * GM);
        const char* q = A.q + ((long long)w.s * A.q_stride + (long long)h0 * HD) * 2;
#pragma unroll
        for (int k = 0; k < HD / 16; ++k)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int row = r + (x & 1) * 8, e = 16 * k + 2 * t + (x >> 1) * 8;
                qf[k][x] = row < nh ? __ldg(reinterpret_cast<const unsigned*>(q + (row * HD + e) * 2)) : 0u;
            }
#pragma unroll
        for (int j = 0; j < HD / 8; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[j][x] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }

    __device__ __forceinline__ void tile(unsigned stage, int valid, float c, float*, const float*)
    {
        const int lane = threadIdx.x & 31, t = lane & 3, mi = lane >> 3, r8 = lane & 7;
        float s[NK][4] = {};
#pragma unroll
        for (int n = 0; n < NK; n += 2) {
            const unsigned base = stage + (8 * n + r8 + (mi >> 1) * 8) * HD * 2;
#pragma unroll
            for (int k = 0; k < HD / 16; ++k) {
                unsigned b[4];
                ldm4(base + (((2 * k + (mi & 1)) ^ r8) << 4), b);
                mma_bf16(s[n], qf[k], b[0], b[1]);
                mma_bf16(s[n + 1], qf[k], b[2], b[3]);
            }
        }
        if (valid < ROWS) {
#pragma unroll
            for (int n = 0; n < NK; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (8 * n + 2 * t + (x & 1) >= valid) s[n][x] = -INFINITY;
        }
        float mn[2], scale[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v = fmaxf(s[0][2 * h], s[0][2 * h + 1]);
#pragma unroll
            for (int n = 1; n < NK; ++n) v = fmaxf(v, fmaxf(s[n][2 * h], s[n][2 * h + 1]));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
            mn[h] = fmaxf(m[h], v);
            scale[h] = m[h] == mn[h] ? 1.f : exp2f((m[h] - mn[h]) * c);
        }
        if (__any_sync(0xffffffffu, scale[0] != 1.f || scale[1] != 1.f)) {
#pragma unroll
            for (int j = 0; j < HD / 8; ++j)
#pragma unroll
                for (int x = 0; x < 4; ++x) o[j][x] *= scale[x >> 1];
        }
        // The weights, rounded to bf16 (2^-8 of each at most), since the matrix instruction takes both operands in one type and
        // the values are bf16; the sums take them unrounded.  Outputs are off by 2.1 - 2.3e-3 of their size against 64 bits
        // (1.7e-3 with fp32 weights: the outputs' own rounding).
        unsigned p[NK / 2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            m[h] = mn[h];
            const float sub = mn[h] == -INFINITY ? 0.f : mn[h];  // scores of -infinity alone so far: weights 0, not NaN
            float sum = 0.f;
#pragma unroll
            for (int n = 0; n < NK; ++n) {
                const float a = exp2f((s[n][2 * h] - sub) * c), b = exp2f((s[n][2 * h + 1] - sub) * c);
                sum += a + b;
                p[n / 2][2 * (n & 1) + h] = pack_bf16(a, b);
            }
            l[h] = l[h] * scale[h] + sum;
        }
#pragma unroll
        for (int n = 0; n < NK / 2; ++n) {
            const unsigned base = stage + (ROWS + 16 * n + r8 + (mi & 1) * 8) * HD * 2;
#pragma unroll
            for (int j = 0; j < HD / 8; j += 2) {
                unsigned b[4];
                ldm4t(base + (((j + (mi >> 1)) ^ r8) << 4), b);
                mma_bf16(o[j], p[n], b[0], b[1]);
                mma_bf16(o[j + 1], p[n], b[2], b[3]);
            }
        }
    }

    // whole sums over the quad's keys
    __device__ __forceinline__ void finish()
    {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        }
    }

    __device__ __forceinline__ void write(float* piece)
    {
        const int lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
#pragma unroll
        for (int j = 0; j < HD / 8; ++j)
#pragma unroll
            for (int x = 0; x < 4; x += 2)
                *reinterpret_cast<float2*>(piece + pa_at<HD>((r + 4 * x) * HD + 8 * j + 2 * t)) = make_float2(o[j][x], o[j][x + 1]);
    }
    __device__ __forceinline__ int own_row(int h) const { return ((threadIdx.x & 31) >> 2) + 8 * h; }
    __device__ __forceinline__ bool owner() const { return (threadIdx.x & 3) == 0; }
    static constexpr int OWN = 2;  // rows a lane holds statistics of
};

// fp32: a lane scores one position over 1 / PARTS of the elements, then owns HD / 32 elements of the output.
template <int HD, int GM>
struct PaF32 {
    static constexpr int E = HD / 32, OWN = GM, ROWS = PA_ROWS<float, HD>, PARTS = 32 / ROWS;
    float o[GM][E], m[GM], l[GM];

    __device__ __forceinline__ void begin(const PaArgs& A, const PaWalk& w, float* sq)
    {
        const int lane = threadIdx.x & 31;
        const int h0 = (w.hb / A.nhb) * A.g + (w.hb % A.nhb) * GM, nh = min(GM, A.g - (w.hb % A.nhb) * GM);
        const float* q = reinterpret_cast<const float*>(A.q) + (long long)w.s * A.q_stride + (long long)h0 * HD;
        __syncwarp();
        for (int i = lane; i < GM * HD; i += 32) sq[i] = i < nh * HD ? __ldg(q + i) : 0.f;
        __syncwarp();
#pragma unroll
        for (int h = 0; h < GM; ++h) {
            m[h] = -INFINITY;
            l[h] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[h][e] = 0.f;
        }
    }

    __device__ __forceinline__ void tile(unsigned, int valid, float c, float* stage, const float* sq)
    {
        const int lane = threadIdx.x & 31, key = lane & (ROWS - 1), part = lane / ROWS;
        float s[GM];
#pragma unroll
        for (int h = 0; h < GM; ++h) s[h] = 0.f;
        const float4* kr = reinterpret_cast<const float4*>(stage + key * HD);
#pragma unroll 4
        for (int i = 0; i < HD / 4 / PARTS; ++i) {
            const int ch = part * (HD / 4 / PARTS) + i;
            const float4 k = kr[ch ^ (key & 7)];
#pragma unroll
            for (int h = 0; h < GM; ++h) {
                const float4 x = reinterpret_cast<const float4*>(sq + h * HD)[ch];
                s[h] = fmaf(x.x, k.x, fmaf(x.y, k.y, fmaf(x.z, k.z, fmaf(x.w, k.w, s[h]))));
            }
        }
        float p[GM];
#pragma unroll
        for (int h = 0; h < GM; ++h) {
            for (int x = ROWS; x < 32; x *= 2) s[h] += __shfl_xor_sync(0xffffffffu, s[h], x);
            if (key >= valid) s[h] = -INFINITY;
            float v = s[h];
            for (int x = ROWS / 2; x; x >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, x));
            const float mn = fmaxf(m[h], v), sc = m[h] == mn ? 1.f : exp2f((m[h] - mn) * c);
            m[h] = mn;
            p[h] = exp2f((s[h] - (mn == -INFINITY ? 0.f : mn)) * c);  // scores of -infinity alone so far: weights 0, not NaN
            l[h] = l[h] * sc + (part == 0 ? p[h] : 0.f);
#pragma unroll
            for (int e = 0; e < E; ++e) o[h][e] *= sc;
        }
        for (int j = 0; j < valid; ++j) {
            float v[E];
            const float* vr = stage + (ROWS + j) * HD;
            if (E == 4) {
                const float4 x = reinterpret_cast<const float4*>(vr)[lane ^ (j & 7)];
                v[0] = x.x; v[1] = x.y; v[2 % E] = x.z; v[3 % E] = x.w;
            } else {
                const float2 x = reinterpret_cast<const float2*>(vr)[((lane >> 1) ^ (j & 7)) * 2 + (lane & 1)];
                v[0] = x.x; v[1] = x.y;
            }
#pragma unroll
            for (int h = 0; h < GM; ++h) {
                const float pj = __shfl_sync(0xffffffffu, p[h], j);
#pragma unroll
                for (int e = 0; e < E; ++e) o[h][e] = fmaf(pj, v[e], o[h][e]);
            }
        }
    }

    __device__ __forceinline__ void finish()
    {
#pragma unroll
        for (int h = 0; h < GM; ++h)
            for (int x = 16; x; x >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], x);
    }

    __device__ __forceinline__ void write(float* piece)
    {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int h = 0; h < GM; ++h)
#pragma unroll
            for (int e = 0; e < E; e += 2)
                *reinterpret_cast<float2*>(piece + pa_at<HD>(h * HD + lane * E + e)) = make_float2(o[h][e], o[h][e + 1]);
    }
    __device__ __forceinline__ int own_row(int h) const { return h; }
    __device__ __forceinline__ bool owner() const { return (threadIdx.x & 31) == 0; }
};

// x y / z for x <= PA_WARPS * PA_MAX_CTAS or so; 32 bits where they suffice (a 64-bit division takes about 100 instructions)
__device__ __forceinline__ long long muldiv(long long x, long long y, long long z)
{
    if (y < (1ll << 20) && x < 4096) return (unsigned)x * (unsigned)y / (unsigned)z;
    return x * y / z;
}

template <typename T, int HD, int GM>
struct PaLayout {
    static constexpr int STAGE = PA_ROWS<T, HD> * HD * (int)sizeof(T) * 2;  // keys and values of a tile
    static constexpr int RING = PA_WARPS * PA_STAGES * STAGE;
    static constexpr int Q = sizeof(T) == 4 ? PA_WARPS * GM * HD * 4 : 0;
    static constexpr int FRONTS = PA_WARPS * GM * HD * 4;  // an item's end per warp, kept until the CTA's warps are done
    static constexpr int BYTES = RING + FRONTS + Q;
    static_assert(GM * HD * 4 <= STAGE, "a warp's piece takes a stage's place");
};

// A piece of an item that a warp could not finish: whether the item's first and last tile were in it, and the
// CTA that holds the last one.  s = -1: none.
struct PaPiece {
    int s, hb, first, last, last_cta, stage;  // stage: of the warp's ring, where the piece lies
};

template <typename T, int HD, int GM>
__global__ void __launch_bounds__(PA_WARPS * 32, 2) paged_attention_kernel(const __grid_constant__ PaArgs A)
{
    using L = PaLayout<T, HD, GM>;
    using State = typename std::conditional<sizeof(T) == 2, PaBf16<HD>, PaF32<HD, GM>>::type;
    constexpr int S = PA_STAGES, ROWS = PA_ROWS<T, HD>;
    extern __shared__ __align__(128) char pa_raw[];
    __shared__ long long sh_tiles[PA_WARPS];
    __shared__ PaPiece sh_piece[2 * PA_WARPS];
    __shared__ float2 sh_ml[2 * PA_WARPS][GM];
    __shared__ float sh_w[2 * PA_WARPS][GM];
    __shared__ float2 sh_sum[2 * PA_WARPS][GM];  // maximum and sum of the pieces of an item, at its first
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int Hx = A.C.n_kv_heads * A.nhb, G = gridDim.x, cta = blockIdx.x;
    float* fronts = reinterpret_cast<float*>(pa_raw + L::RING);
    float* sq = fronts + (PA_WARPS + warp) * GM * HD;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // sequences of no length: zeros
    for (int s = cta; s < A.n_seqs; s += G)
        if (__ldg(A.kv_len + s) <= 0)
            for (int i = tid; i < A.hq * HD; i += PA_WARPS * 32)
                reinterpret_cast<T*>(A.out)[(long long)s * A.out_stride + i] = from_f<T>(0.f);

    // the tiles of the call, PA_ITEM more for each item
    auto tiles_of = [&](int s) {
        PaWalk w;
        w.s = s;
        pa_sequence<ROWS>(A, w);
        return w.ntiles ? w.ntiles + PA_ITEM : 0;
    };
    long long mine = 0;
    for (int s = tid; s < A.n_seqs; s += PA_WARPS * 32) mine += tiles_of(s);
    for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) sh_tiles[warp] = mine;
    if (tid < 2 * PA_WARPS) sh_piece[tid].s = -1;
    __syncthreads();
    const long long total = ((sh_tiles[0] + sh_tiles[1]) + (sh_tiles[2] + sh_tiles[3])) * Hx;
    const long long shares = min(total, (long long)G * PA_WARPS);
    const int share = cta * PA_WARPS + warp;
    if (cta * PA_WARPS >= shares) {
        if (tid == 0) A.rec[cta] = make_int4(-1, 0, 0, 0);
        return;
    }
    if (share < shares) {
        const long long t0 = muldiv(share, total, shares), t1 = muldiv(share + 1, total, shares);
        // where the share starts
        PaWalk use;
        long long item_first = 0;  // where the item begins: PA_ITEM empty places, then its tiles
        for (int b = 0; b < A.n_seqs; b += 32) {
            const int s = b + lane;
            const long long v = s < A.n_seqs ? (long long)tiles_of(s) * Hx : 0;
            long long inc = v;
            for (int o = 1; o < 32; o <<= 1) {
                const long long x = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += x;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, item_first + inc > t0);
            if (hit) {
                const int l = __ffs(hit) - 1;
                use.s = b + l;
                item_first += __shfl_sync(0xffffffffu, inc - v, l);
                break;
            }
            item_first += __shfl_sync(0xffffffffu, inc, 31);
        }
        pa_sequence<ROWS>(A, use);
        const long long in = t0 - item_first;
        use.hb = (int)(in >> 32 ? in / (use.ntiles + PA_ITEM) : (unsigned)in / (unsigned)(use.ntiles + PA_ITEM));
        item_first += (long long)use.hb * (use.ntiles + PA_ITEM);
        use.tile = max(0, (int)(t0 - item_first) - PA_ITEM);
        long long at = item_first + PA_ITEM + use.tile;  // where the tile of `use` lies
        PaWalk load = use;
        char* ring_p = pa_raw + warp * (S * L::STAGE);
        const unsigned ring = su32(ring_p);

        // the CTA whose share ends with or holds the tile before `end`: the last share with muldiv(share, total, shares) < end
        auto owner = [&](long long end) {
            const long long x = end * shares - 1;
            return (int)((x >> 32 ? x / total : (unsigned)x / (unsigned)total) / PA_WARPS);
        };
        long long at_load = at;  // the same of `load`: the loads run ahead of the products, across items
        unsigned bad_ring = 0;   // bit i: the tile in stage i has a row without a valid page
        bool next_bad = false;
        long long off = at < t1 ? pa_offset<ROWS>(A, load, next_bad) : -1;
        auto issue = [&](int stage) {
            if (at_load < t1) {
                pa_issue<T, HD>(A, ring + stage * L::STAGE, off);
                bad_ring = (bad_ring & ~(1u << stage)) | (__any_sync(0xffffffffu, next_bad) ? 1u << stage : 0u);
                next_bad = false;
                at_load += load.tile + 1 < load.ntiles ? 1 : 1 + PA_ITEM;
                if (at_load < t1) {
                    pa_next<ROWS>(A, load);
                    off = pa_offset<ROWS>(A, load, next_bad);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int i = 0; i < S; ++i) issue(i);

        State st;
        bool fresh = true, bad = false, front = false;
        int stage = 0;
        while (at < t1) {
            if (fresh) {
                st.begin(A, use, sq);
                fresh = false;
                bad = false;
                front = use.tile == 0;  // the item begins in this share
            }
            asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
            __syncwarp();
            const int nh = min(GM, A.g - (use.hb % A.nhb) * GM);
            st.tile(ring + stage * L::STAGE, min(ROWS, use.len - (use.lo + use.tile * ROWS)), A.c,
                    reinterpret_cast<float*>(ring_p + stage * L::STAGE), sq);
            bad = bad || ((bad_ring >> stage) & 1u);
            __syncwarp();
            const bool ends = use.tile + 1 == use.ntiles;
            at += ends ? 1 + PA_ITEM : 1;
            const bool end = at >= t1;
            if (ends || end) {
                // the item's output, through the stage just read: one place in the code writes the accumulators, which
                // matters where a call is mostly fetching instructions
                st.finish();
                if (bad) {
#pragma unroll
                    for (int h = 0; h < State::OWN; ++h) st.l[h] = NAN;
                }
                float* piece = reinterpret_cast<float*>(ring_p + stage * L::STAGE);
                const int slot = 2 * warp + (end || (ends && front));
                st.write(piece);
                if (st.owner()) {
#pragma unroll
                    for (int h = 0; h < State::OWN; ++h) sh_ml[slot][st.own_row(h)] = make_float2(st.m[h], st.l[h]);
                }
                __syncwarp();
                if (ends && front) {
                    const int h0 = (use.hb / A.nhb) * A.g + (use.hb % A.nhb) * GM;
                    T* o = reinterpret_cast<T*>(A.out) + (long long)use.s * A.out_stride + (long long)h0 * HD;
                    for (int x = 4 * lane; x < nh * HD; x += 128) {
                        const float4 v = *reinterpret_cast<const float4*>(piece + pa_at<HD>(x));
                        put4(o + x, v, 1.f / sh_ml[slot][x / HD].y);
                    }
                    __syncwarp();
                } else {
                    // stays in the ring if that has nothing more to come; else (the end of an item begun before the share:
                    // once per warp at most) into a place of its own
                    if (!end) {
                        float* o = fronts + warp * GM * HD;
                        for (int x = 4 * lane; x < nh * HD; x += 128)
                            *reinterpret_cast<float4*>(o + pa_at<HD>(x)) = *reinterpret_cast<const float4*>(piece + pa_at<HD>(x));
                        __syncwarp();
                    }
                    if (lane == 0)
                        sh_piece[slot] = {use.s, use.hb, front, ends, owner(item_first + PA_ITEM + use.ntiles), stage};
                }
                fresh = true;
            }
            issue(stage);
            stage = stage + 1 == S ? 0 : stage + 1;
            if (!end) {
                if (ends) item_first += use.ntiles + PA_ITEM;
                pa_next<ROWS>(A, use);
            }
        }
    }
    __syncthreads();
    // the pieces of each item, in order; `held`, `ended`: bit i: there is a piece i, and it is its item's last
    const bool is = lane < 2 * PA_WARPS && sh_piece[lane].s >= 0;
    const unsigned held = __ballot_sync(0xffffffffu, is), ended = __ballot_sync(0xffffffffu, is && sh_piece[lane].last);
    auto last_of = [&](int i) { return ended >> i ? i + __ffs(ended >> i) - 1 : 31 - __clz(held); };
    // weights first, a thread per row and piece that is its item's first here
    if (tid / GM < 2 * PA_WARPS) {
        const int i = tid / GM, row = tid % GM;
        const unsigned below = held & ((1u << i) - 1);
        if ((held >> i & 1) && (!below || (ended >> (31 - __clz(below)) & 1)) && row < A.g - (sh_piece[i].hb % A.nhb) * GM) {
            const unsigned item = held & ((2u << last_of(i)) - (1u << i));
            float mx = -INFINITY, l = 0.f;
            for (unsigned r = item; r; r &= r - 1) mx = fmaxf(mx, sh_ml[__ffs(r) - 1][row].x);
            for (unsigned r = item; r; r &= r - 1) {
                const int k = __ffs(r) - 1;
                const float2 ml = sh_ml[k][row];
                const float w = ml.x == mx ? 1.f : exp2f((ml.x - mx) * A.c);
                sh_w[k][row] = w;
                l = fmaf(ml.y, w, l);
            }
            sh_sum[i][row] = make_float2(mx, l);
        }
    }
    __syncthreads();
    if (tid == 0) A.rec[cta] = make_int4(-1, 0, 0, 0);
    for (int i = 0, j; held >> i; i = j + 1) {
        i += __ffs(held >> i) - 1;
        j = last_of(i);
        const unsigned item = held & ((2u << j) - (1u << i));
        const PaPiece p0 = sh_piece[i], p1 = sh_piece[j];
        const int nh = min(GM, A.g - (p0.hb % A.nhb) * GM);
        const bool whole = p0.first && p1.last;
        const int h0 = (p0.hb / A.nhb) * A.g + (p0.hb % A.nhb) * GM;
        T* out = reinterpret_cast<T*>(A.out) + (long long)p0.s * A.out_stride + (long long)h0 * HD;
        const long long slot = (long long)cta * 2 + (p0.first ? 1 : 0);
        for (int x = 4 * tid; x < nh * HD; x += PA_WARPS * 128) {
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            const int row = x / HD;
            for (unsigned r = item; r; r &= r - 1) {
                const int k = __ffs(r) - 1;
                const float* o = k & 1 ? reinterpret_cast<const float*>(pa_raw + ((k >> 1) * S + sh_piece[k].stage) * L::STAGE)
                                       : fronts + (k >> 1) * GM * HD;
                const float4 v = *reinterpret_cast<const float4*>(o + pa_at<HD>(x));
                const float w = sh_w[k][row];
                acc = make_float4(fmaf(v.x, w, acc.x), fmaf(v.y, w, acc.y), fmaf(v.z, w, acc.z), fmaf(v.w, w, acc.w));
            }
            if (whole) put4(out + x, acc, 1.f / sh_sum[i][row].y);
            else *reinterpret_cast<float4*>(A.part_o + slot * GM * HD + x) = acc;
        }
        if (!whole) {
            if (tid < nh) A.part_ml[slot * GM + tid] = sh_sum[i][tid];
            if (tid == 0 && p0.first) A.rec[cta] = make_int4(p0.s, p0.hb, p1.last_cta, 0);
        }
    }
}

// Joins the pieces of the items that cross CTAs: a block per CTA that began one and one or two query heads, HD / 2
// threads for each head and group of pieces, of which a group takes eight at a time, all on their way together.  Small
// blocks, as they start while the last CTAs of the first kernel still hold their registers: 4 ragged contexts of up to
// 1000, 32 + 8 heads of 128: 10.9 us (11.6 us by blocks of 512).
constexpr int PJ_THREADS = 256;

template <typename T, int HD, int GM>
__global__ void __launch_bounds__(PJ_THREADS) paged_attention_join(const __grid_constant__ PaArgs A)
{
    constexpr int LANES = HD / 2, SLOTS = PJ_THREADS / LANES;
    const int groups = SLOTS >> A.join_rows;
    __shared__ float2 s_acc[SLOTS][LANES], s_ml[SLOTS];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int cta = blockIdx.x, e = threadIdx.x % LANES, slot = threadIdx.x / LANES, group = slot >> A.join_rows;
    const int4 r = A.rec[cta];
    if (r.x < 0) return;
    const int row = (blockIdx.y << A.join_rows) + (slot & ((1 << A.join_rows) - 1)), nh = min(GM, A.g - (r.y % A.nhb) * GM);
    const int np = row < nh ? r.z - cta + 1 : 0;  // pieces: (cta, 1), then (cta + i, 0)
    float mx = -INFINITY, l = 0.f;
    float2 acc = make_float2(0.f, 0.f);
    for (int i0 = 8 * group; i0 < np; i0 += 8 * groups) {
        float2 ml[8], o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const long long at = ((long long)(cta + i0 + i) * 2 + (i0 + i == 0)) * GM + row;
            ml[i] = i0 + i < np ? A.part_ml[at] : make_float2(-INFINITY, 0.f);
            o[i] = i0 + i < np ? reinterpret_cast<const float2*>(A.part_o + at * HD)[e] : make_float2(0.f, 0.f);
        }
        float mn = mx;
#pragma unroll
        for (int i = 0; i < 8; ++i) mn = fmaxf(mn, ml[i].x);
        const float a = mx == mn ? 1.f : exp2f((mx - mn) * A.c);
        mx = mn;
        acc = make_float2(acc.x * a, acc.y * a);
        l *= a;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float w = ml[i].x == mx ? 1.f : exp2f((ml[i].x - mx) * A.c);
            l = fmaf(ml[i].y, w, l);
            acc = make_float2(fmaf(o[i].x, w, acc.x), fmaf(o[i].y, w, acc.y));
        }
    }
    if (r.z - cta >= 8) {  // the groups, in order
        s_acc[slot][e] = acc;
        if (e == 0) s_ml[slot] = make_float2(mx, l);
        __syncthreads();
        if (group == 0) {
            const int ng = min(groups, (np + 7) / 8);
            for (int k = 1; k < ng; ++k) mx = fmaxf(mx, s_ml[slot + (k << A.join_rows)].x);
            l = 0.f;
            acc = make_float2(0.f, 0.f);
            for (int k = 0; k < ng; ++k) {
                const float2 ml = s_ml[slot + (k << A.join_rows)], o = s_acc[slot + (k << A.join_rows)][e];
                const float w = ml.x == mx ? 1.f : exp2f((ml.x - mx) * A.c);
                l = fmaf(ml.y, w, l);
                acc = make_float2(fmaf(o.x, w, acc.x), fmaf(o.y, w, acc.y));
            }
        }
    }
    if (group || !np) return;
    const int h = (r.y / A.nhb) * A.g + (r.y % A.nhb) * GM + row;
    T* out = reinterpret_cast<T*>(A.out) + (long long)r.x * A.out_stride + (long long)h * HD + 2 * e;
    out[0] = from_f<T>(acc.x / l);
    out[1] = from_f<T>(acc.y / l);
}

size_t attention_workspace(int dtype, int hd)
{
    const size_t gm = dtype == MFS_DTYPE_BF16 ? PA_GM_MAX<bf16> : PA_GM_MAX<float>;
    return (size_t)PA_MAX_CTAS * (2 * gm * hd * sizeof(float) + 2 * gm * sizeof(float2) + sizeof(int4));
}

template <typename T, int HD, int GM>
int attention(PaArgs A, char* workspace, cudaStream_t st)
{
    using L = PaLayout<T, HD, GM>;
    A.nhb = (A.g + GM - 1) / GM;
    A.part_o = reinterpret_cast<float*>(workspace);
    A.part_ml = reinterpret_cast<float2*>(A.part_o + (size_t)PA_MAX_CTAS * 2 * GM * HD);
    A.rec = reinterpret_cast<int4*>(A.part_ml + (size_t)PA_MAX_CTAS * 2 * GM);
    const int rows = A.g < GM ? A.g : GM;
    // two heads per block of the join, or one where the items are so few that each has over a dozen pieces: one context of
    // 100000, 8 heads on one kv head: 28 us (34 us by two), one of 20000, 32 + 8 heads: 24.3 us (25.4 us); but 4 of up to
    // 1000, 32 + 8 heads: 11.2 us (10.8 us by two)
    A.join_rows = rows > 1 && (long long)A.n_seqs * A.C.n_kv_heads * A.nhb > 16 ? 1 : 0;
    int sms = 0;
    static mfs::PerDevice ready;
    cudaError_t e = mfs::op_device(ready, (const void*)paged_attention_kernel<T, HD, GM>, L::BYTES, &sms);
    if (e != cudaSuccess) return mfs::op_launched("paged_attention", e);
    const int G = 2 * sms < PA_MAX_CTAS ? 2 * sms : PA_MAX_CTAS;
    paged_attention_kernel<T, HD, GM><<<G, PA_WARPS * 32, L::BYTES, st>>>(A);
    e = cudaGetLastError();
    if (e != cudaSuccess) return mfs::op_launched("paged_attention", e);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)G, (unsigned)((rows - 1) >> A.join_rows) + 1);
    cfg.blockDim = dim3(PJ_THREADS);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return mfs::op_launched("paged_attention", cudaLaunchKernelEx(&cfg, paged_attention_join<T, HD, GM>, A));
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
    if (q && (n_q_heads < 1 || n_q_heads > MFS_MAX_HEADS)) return mfs::op_fail(MFS_E_ARG, op, "n_q_heads outside [1, 65535]");
    if (!mfs::rows_ok(k, k_stride, cache->n_kv_heads, hd, elem) || !mfs::rows_ok(v, v_stride, cache->n_kv_heads, hd, elem) ||
        (k_out && !mfs::rows_ok(k_out, k_out_stride, cache->n_kv_heads, hd, elem)) ||
        (q && (!mfs::rows_ok(q, q_stride, n_q_heads, hd, elem) || !mfs::rows_ok(q_out, q_out_stride, n_q_heads, hd, elem))))
        return mfs::op_fail(MFS_E_ARG, op, "pointers and token strides must be multiples of 16 bytes, a stride at least heads x head_dim");
    Turns turns = {};
    if (rope) {
        // powers of the first ratio, each the product of two before it: at most 7 roundings of 2^-53, where 64 calls of
        // pow cost the caller 2 us
        turns.f[0] = 1.0;
        for (int b = 1; b < hd / 2; b *= 2) {
            turns.f[b] = pow(theta, -2.0 * b / hd);
            for (int i = 1; i < b; ++i) turns.f[b + i] = turns.f[b] * turns.f[i];
        }
        for (int i = 0; i < hd / 2; ++i) turns.f[i] /= 6.283185307179586476925;
    }
    const Cache C = cache_of(cache);
    const int hq = q ? n_q_heads : 0;
    cudaStream_t st = (cudaStream_t)cuda_stream;
    return cache->dtype == MFS_DTYPE_BF16
               ? append_typed<bf16>(C, n_tokens, n_seqs, cu, kv_len, q, q_stride, hq, q_out, q_out_stride, k, k_stride, k_out,
                              k_out_stride, v, v_stride, hd, rope, turns, st)
               : append_typed<float>(C, n_tokens, n_seqs, cu, kv_len, q, q_stride, hq, q_out, q_out_stride, k, k_stride, k_out,
                               k_out_stride, v, v_stride, hd, rope, turns, st);
}

extern "C" size_t mfs_paged_attention_workspace(const mfs_paged_kv* cache, int n_q_heads)
{
    (void)n_q_heads;  // the pieces in flight are bounded by the grid, whatever the heads and lengths
    if (mfs::paged_kv_problem(cache)) return 0;
    return attention_workspace(cache->dtype, cache->head_dim);
}

extern "C" int mfs_paged_attention(const mfs_paged_kv* cache, int n_seqs, const int32_t* kv_len, const void* q,
                                   long long q_stride, int n_q_heads, void* out, long long out_stride, float scale, int window,
                                   void* workspace, size_t workspace_bytes, void* cuda_stream)
{
    const char* op = "paged_attention";
    if (const char* why = mfs::paged_kv_problem(cache)) return mfs::op_fail(MFS_E_ARG, op, why);
    if (n_seqs < 0 || window < 0) return mfs::op_fail(MFS_E_ARG, op, "need n_seqs >= 0 and window >= 0");
    if (n_q_heads < 1 || n_q_heads % cache->n_kv_heads || n_q_heads > MFS_MAX_HEADS)
        return mfs::op_fail(MFS_E_ARG, op, "n_q_heads must be a multiple of n_kv_heads, at most 65535");
    if (!(scale > 0.f && scale <= 1e30f)) return mfs::op_fail(MFS_E_ARG, op, "scale must be positive and finite");
    if (n_seqs == 0) return MFS_OK;
    if (!kv_len || !q || !out || !workspace) return mfs::op_fail(MFS_E_ARG, op, "null kv_len, q, out or workspace");
    const int hd = cache->head_dim, elem = cache->dtype == MFS_DTYPE_BF16 ? 2 : 4;
    if (!mfs::rows_ok(q, q_stride, n_q_heads, hd, elem) || !mfs::rows_ok(out, out_stride, n_q_heads, hd, elem))
        return mfs::op_fail(MFS_E_ARG, op, "pointers and token strides must be multiples of 16 bytes, a stride at least heads x head_dim");
    if (((uintptr_t)workspace & 15u) || workspace_bytes < mfs_paged_attention_workspace(cache, n_q_heads))
        return mfs::op_fail(MFS_E_ARG, op, "workspace too small or not 16-byte aligned");
    PaArgs A = {};
    A.C = cache_of(cache);
    A.kv_len = kv_len;
    A.q = (const char*)q;
    A.out = (char*)out;
    A.q_stride = q_stride;
    A.out_stride = out_stride;
    A.n_seqs = n_seqs;
    A.hq = n_q_heads;
    A.g = n_q_heads / cache->n_kv_heads;
    A.window = window;
    A.c = scale * 1.44269504088896340736f;
    cudaStream_t st = (cudaStream_t)cuda_stream;
    char* ws = (char*)workspace;
    if (cache->dtype == MFS_DTYPE_BF16) return hd == 128 ? attention<bf16, 128, 16>(A, ws, st) : attention<bf16, 64, 16>(A, ws, st);
    auto fn = hd == 128 ? (A.g == 1 ? attention<float, 128, 1> : A.g <= 4 ? attention<float, 128, 4> : attention<float, 128, 8>)
                        : (A.g == 1 ? attention<float, 64, 1> : A.g <= 4 ? attention<float, 64, 4> : attention<float, 64, 8>);
    return fn(A, ws, st);
}
