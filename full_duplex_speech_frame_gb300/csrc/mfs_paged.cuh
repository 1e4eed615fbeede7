// The paged key/value cache as the operators see it, and the kernels of one-token attention over it, whatever type
// the cache holds (mfs_paged.cu: fp32 and bf16; mfs_quant.cu: 8 bits; mfs_shared.cu: behind a shared prefix).
#pragma once
#include <string.h>
#include <type_traits>

#include "mfs_mma.cuh"
#include "mfs_ops.cuh"

namespace {

using bf16 = __nv_bfloat16;

struct Cache {
    char* k;
    char* v;
    const int32_t* table;
    int table_width, n_pages, page_size, n_kv_heads;
    long long table_stride, page_stride, head_stride, row_stride;  // elements
    unsigned by, shift;  // p / page_size = (p by) >> (32 + shift) for 0 <= p < 2^31
};

Cache cache_of(const mfs_paged_kv* c)
{
    // by = 2^(32 + shift) / page_size rounded up with shift the least that 2^(shift + 1) >= page_size: by < 2^32, and its excess
    // of less than 1 makes (p by) / 2^(32 + shift) too large by less than 2^31 / 2^(32 + shift) <= 1 / page_size
    unsigned shift = 0;
    while ((2 << shift) < c->page_size) ++shift;
    const unsigned by = c->page_size == 1 ? 0xffffffffu : (unsigned)(((1ull << (32 + shift)) + c->page_size - 1) / c->page_size);
    return {(char*)c->k, (char*)c->v, c->table, c->table_width, c->n_pages, c->page_size, c->n_kv_heads,
            c->table_stride, c->page_stride, c->head_stride, c->row_stride, by, shift};
}

// p / page_size for p >= 0
__device__ __forceinline__ int page_of(const Cache& C, int p)
{
    return C.page_size == 1 ? p : (int)(__umulhi((unsigned)p, C.by) >> C.shift);
}

// Page and row of position p of sequence s; false where the table has no valid page for it.
__device__ __forceinline__ bool row_place(const Cache& C, int s, int p, int& page, int& row)
{
    const int j = page_of(C, p);
    if (p < 0 || j >= C.table_width) return false;
    page = __ldg(C.table + s * C.table_stride + j);
    row = p - j * C.page_size;
    return page >= 0 && page < C.n_pages;
}

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
constexpr int PA_SMS = 152;
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

// Where 16-byte chunk ch of a tile's row lies in it, for rows of CH chunks: eight rows' chunks of one number, which a matrix
// load takes together, meet different banks.
template <int CH>
__device__ __forceinline__ int pa_chunk(int row, int ch) { return CH >= 8 ? ch ^ (row & 7) : ch ^ ((row >> 1) & 3); }

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
    // 8-bit caches: an exponent per row
    const uint8_t *kx, *vx;
    long long x_page, x_head, x_row;
    float* fronts;    // [CTA][PA_WARPS][GM][HD]
    // behind a shared prefix: what follows it is attended to, and what comes of it goes to own_o [n_seqs][hq][HD] and own_ml
    // [n_seqs][hq] (maximum, sum)
    const int32_t *groups, *prefix_len;
    int n_groups;
    float* own_o;
    float2* own_ml;
    int2* own_at;     // [n_seqs][head blocks] of what follows: {first CTA or -1: it is in own_o, last CTA} of its pieces
};

// The last group that begins at or before sequence s.
__device__ __forceinline__ int group_of(const int32_t* groups, int n_groups, int s)
{
    int lo = 0, hi = n_groups - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(groups + mid) <= s) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Group g's first sequence and how many it has.
__device__ __forceinline__ void group_span(const int32_t* groups, int g, int n_seqs, int& first, int& ns)
{
    first = min(max(__ldg(groups + g), 0), n_seqs);
    ns = max(min(__ldg(groups + g + 1), n_seqs) - first, 0);
}

// Positions that sequence s, which sees [lo, len), has from its group's prefix: the prefix, or none where it does not see it
// whole or is alone in its group.
__device__ __forceinline__ int shared_part(const int32_t* groups, int n_groups, const int32_t* prefix_len, int n_seqs, int s, int lo, int len)
{
    if (lo > 0 || n_groups == 0) return 0;
    const int g = group_of(groups, n_groups, s);
    int first, ns;
    group_span(groups, g, n_seqs, first, ns);
    if (s < first || s >= first + ns || ns < 2) return 0;
    const int p = max(__ldg(prefix_len + g), 0);
    return p <= len ? p : 0;
}

// Where a walk through the tiles stands.
struct PaWalk {
    int s, hb, tile, ntiles, lo, len;
};

template <typename K>
__device__ __forceinline__ void pa_sequence(const PaArgs& A, PaWalk& w)
{
    constexpr int ROWS = K::ROWS;
    w.len = __ldg(A.kv_len + w.s);
    w.lo = A.window > 0 && w.len > A.window ? w.len - A.window : 0;
    if (K::SHARED) w.lo += shared_part(A.groups, A.n_groups, A.prefix_len, A.n_seqs, w.s, w.lo, w.len);
    w.ntiles = w.len > w.lo ? (int)(((long long)w.len - w.lo + ROWS - 1) / ROWS) : 0;
}

template <typename K>
__device__ __forceinline__ void pa_next(const PaArgs& A, PaWalk& w)
{
    if (++w.tile < w.ntiles) return;
    w.tile = 0;
    if (++w.hb < A.C.n_kv_heads * A.nhb) return;
    w.hb = 0;
    do {
        ++w.s;
        if (w.s >= A.n_seqs) return;
        pa_sequence<K>(A, w);
    } while (w.ntiles == 0);
}

// Element offset of this lane's row (lane mod ROWS) of the tile, or -1; 8-bit caches: where its exponents lie.
template <typename K>
__device__ __forceinline__ long long pa_offset(const PaArgs& A, const PaWalk& w, bool& bad, long long& at)
{
    constexpr int ROWS = K::ROWS;
    const int p = w.lo + w.tile * ROWS + (threadIdx.x & (ROWS - 1));
    if ((unsigned)p >= (unsigned)w.len) return -1;  // a last tile may reach past 2^31 - 1
    int page, row;
    if (!row_place(A.C, w.s, p, page, row)) { bad = true; return -1; }
    const int h = w.hb / A.nhb;
    if (K::QUANT) at = (long long)page * A.x_page + (long long)row * A.x_row + (long long)h * A.x_head;
    return (long long)page * A.C.page_stride + (long long)row * A.C.row_stride + (long long)h * A.C.head_stride;
}

template <typename K>
__device__ __forceinline__ void pa_issue(const PaArgs& A, unsigned stage, long long off)
{
    constexpr int CE = K::CE, HD = K::HD;        // bytes of an element of the cache
    constexpr int CH = HD * CE / 16;             // 16-byte chunks per row
    constexpr int RPI = CH >= 32 ? 1 : 32 / CH;  // rows per instruction
    constexpr int ROWS = K::ROWS;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < ROWS / RPI; ++j) {
        const int row = j * RPI + lane / CH, ch = lane % CH;
        const long long o = __shfl_sync(0xffffffffu, off, row);
        const long long byte = (o < 0 ? 0 : o) * (long long)CE + ch * 16;
        const unsigned dst = stage + row * (HD * CE) + (pa_chunk<CH>(row, ch) << 4);
        copy16(dst, A.C.k + byte, o >= 0);
        copy16(dst + ROWS * HD * CE, A.C.v + byte, o >= 0);
    }
}

// The same for codes, in fewer instructions: a tile takes half the copies' time.  left: positions from the tile's first on.
template <typename K>
__device__ __forceinline__ void pa_issue_codes(const PaArgs& A, unsigned stage, long long off, int left)
{
    constexpr int HD = K::HD, CH = HD / 16, RPI = 32 / CH, ROWS = K::ROWS, SAME = 8 / RPI;  // instructions until the banks repeat
    const int lane = threadIdx.x & 31, ch = lane % CH, sub = lane / CH;
    const unsigned long long first = (unsigned long long)A.C.k, row = first + (off < 0 ? 0 : off);  // without a page: the cache's first, whatever it is
    const unsigned long long to_v = (unsigned long long)A.C.v - first;
    unsigned at[SAME];
#pragma unroll
    for (int j = 0; j < SAME; ++j) at[j] = stage + (j * RPI + sub) * HD + (pa_chunk<CH>(j * RPI + sub, ch) << 4);
    auto copy = [&](auto whole) {
#pragma unroll
        for (int j = 0; j < ROWS / RPI; ++j) {
            const unsigned long long src = __shfl_sync(0xffffffffu, row, j * RPI + sub) + 16 * ch;
            const unsigned dst = at[j % SAME] + j / SAME * (8 * HD);
            const bool in = decltype(whole)::value || j * RPI + sub < left;
            copy16(dst, (const void*)src, in);
            copy16(dst + ROWS * HD, (const void*)(src + to_v), in);
        }
    };
    if (left >= ROWS) copy(std::true_type());
    else copy(std::false_type());
}

// One warp's state for an item: scores by mma for bf16 (16 query heads per tile, the rest zero).
template <int HD>
struct PaBf16 {
    static constexpr int GM = 16, ROWS = 2048 / HD, NK = ROWS / 8;  // key octets
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

    __device__ __forceinline__ void tile(unsigned stage, int valid, float c, float*, const float*, const uint8_t*)
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
    static constexpr int E = HD / 32, OWN = GM, ROWS = 1024 / HD, PARTS = 32 / ROWS;
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

    __device__ __forceinline__ void tile(unsigned, int valid, float c, float* stage, const float* sq, const uint8_t*)
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

// x y / z for x <= 4096 or so; 32 bits where they suffice (a 64-bit division takes about 100 instructions)
__device__ __forceinline__ long long muldiv(long long x, long long y, long long z)
{
    if (y < (1ll << 20) && x < 4096) return (unsigned)x * (unsigned)y / (unsigned)z;
    return x * y / z;
}

// What a cache holds and how its tiles are taken: T the type of queries and outputs, CE bytes of an element of the cache, GM
// query heads per block, ROWS positions per tile (4 KB of keys and 4 KB of values, except heads of 64 in 8 bits), STAGES of a
// warp's ring (16 KB).
template <int HD_, bool SHARED_ = false>
struct PaKindBf16 {
    using T = bf16;
    using State = PaBf16<HD_>;
    static constexpr int HD = HD_, GM = 16, CE = 2, ROWS = 2048 / HD, STAGES = PA_STAGES, Q = 0;
    static constexpr int BLOCKS = 2, ITEM = PA_ITEM;  // per SM
    static constexpr bool QUANT = false, SHARED = SHARED_;
};
template <int HD_, int GM_, bool SHARED_ = false>
struct PaKindF32 {
    using T = float;
    using State = PaF32<HD_, GM_>;
    static constexpr int HD = HD_, GM = GM_, CE = 4, ROWS = 1024 / HD, STAGES = PA_STAGES, Q = PA_WARPS * GM * HD * 4;
    static constexpr int BLOCKS = 2, ITEM = PA_ITEM;  // per SM
    static constexpr bool QUANT = false, SHARED = SHARED_;
};

template <typename K>
struct PaLayout {
    static constexpr int HD = K::HD, GM = K::GM, Q = K::Q;
    static constexpr int STAGE = K::ROWS * HD * K::CE * 2;  // keys and values of a tile
    static constexpr int RING = PA_WARPS * K::STAGES * STAGE;
    // an item's end per warp, kept until the CTA's warps are done; 8-bit caches: in the workspace, so that a third block fits
    static constexpr int FRONTS = K::QUANT ? 0 : PA_WARPS * GM * HD * 4;
    static constexpr int BYTES = RING + FRONTS + Q;
    static_assert(GM * HD * 4 <= STAGE, "a warp's piece takes a stage's place");
};

// A piece of an item that a warp could not finish: whether the item's first and last tile were in it, and the
// CTA that holds the last one.  s = -1: none.
struct PaPiece {
    int s, hb, first, last, last_cta, stage;  // stage: of the warp's ring, where the piece lies
};

template <typename K>
__global__ void __launch_bounds__(PA_WARPS * 32, K::BLOCKS) paged_attention_kernel(const __grid_constant__ PaArgs A)
{
    using L = PaLayout<K>;
    using T = typename K::T;
    using State = typename K::State;
    constexpr int S = K::STAGES, ROWS = K::ROWS, HD = K::HD, GM = K::GM;
    // 8-bit caches: the exponents of the ring's tiles, keys' and values'
    __shared__ __align__(16) uint8_t sh_x[K::QUANT ? PA_WARPS : 1][K::QUANT ? S : 1][2][32];
    extern __shared__ __align__(128) char pa_raw[];
    __shared__ long long sh_tiles[PA_WARPS];
    __shared__ PaPiece sh_piece[2 * PA_WARPS];
    __shared__ float2 sh_ml[2 * PA_WARPS][GM];
    __shared__ float sh_w[2 * PA_WARPS][GM];
    __shared__ float2 sh_sum[2 * PA_WARPS][GM];  // maximum and sum of the pieces of an item, at its first
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int Hx = A.C.n_kv_heads * A.nhb, G = gridDim.x, cta = blockIdx.x;
    float* fronts = K::QUANT ? A.fronts + (long long)cta * PA_WARPS * GM * HD : reinterpret_cast<float*>(pa_raw + L::RING);
    float* sq = reinterpret_cast<float*>(pa_raw + L::RING) + (PA_WARPS + warp) * GM * HD;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // sequences of no length: zeros
    for (int s = cta; s < A.n_seqs && !K::SHARED; s += G)
        if (__ldg(A.kv_len + s) <= 0)
            for (int i = tid; i < A.hq * HD; i += PA_WARPS * 32)
                reinterpret_cast<T*>(A.out)[(long long)s * A.out_stride + i] = from_f<T>(0.f);

    // the tiles of the call, K::ITEM more for each item
    auto tiles_of = [&](int s) {
        PaWalk w;
        w.s = s;
        pa_sequence<K>(A, w);
        return w.ntiles ? w.ntiles + K::ITEM : 0;
    };
    // behind a shared prefix a sequence's tiles take several dependent reads to find: once, and kept
    constexpr int KEPT = K::SHARED ? 1024 : 1;
    __shared__ int sh_kept[KEPT];
    long long mine = 0;
    for (int s = tid; s < A.n_seqs; s += PA_WARPS * 32) {
        const int v = tiles_of(s);
        if (K::SHARED && s < KEPT) sh_kept[s] = v;
        mine += v;
    }
    for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) sh_tiles[warp] = mine;
    if (tid < 2 * PA_WARPS) sh_piece[tid].s = -1;
    __syncthreads();
    const long long total = ((sh_tiles[0] + sh_tiles[1]) + (sh_tiles[2] + sh_tiles[3])) * Hx;
    const long long shares = min(total, (long long)G * PA_WARPS);
    const int share = cta * PA_WARPS + warp;
    if (cta * PA_WARPS >= shares) {
        if (!K::SHARED && tid == 0) A.rec[cta] = make_int4(-1, 0, 0, 0);
        if (K::SHARED) asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    if (share < shares) {
        const long long t0 = muldiv(share, total, shares), t1 = muldiv(share + 1, total, shares);
        // where the share starts
        PaWalk use;
        long long item_first = 0;  // where the item begins: K::ITEM empty places, then its tiles
        for (int b = 0; b < A.n_seqs; b += 32) {
            const int s = b + lane;
            const long long v = s < A.n_seqs ? (long long)(K::SHARED && s < KEPT ? sh_kept[s] : tiles_of(s)) * Hx : 0;
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
        pa_sequence<K>(A, use);
        const long long in = t0 - item_first;
        use.hb = (int)(in >> 32 ? in / (use.ntiles + K::ITEM) : (unsigned)in / (unsigned)(use.ntiles + K::ITEM));
        item_first += (long long)use.hb * (use.ntiles + K::ITEM);
        use.tile = max(0, (int)(t0 - item_first) - K::ITEM);
        long long at = item_first + K::ITEM + use.tile;  // where the tile of `use` lies
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
        long long x_at = 0;      // where the row's exponents lie
        unsigned x_next = 0;     // they, on their way: put into shared memory by the next call
        int x_stage = -1;
        long long off = at < t1 ? pa_offset<K>(A, load, next_bad, x_at) : -1;
        auto issue = [&](int stage) {
            if constexpr (K::QUANT) {
                static_assert(ROWS <= 32 && S >= 2, "a lane has a row's exponents, and they are there a tile later");
                if (x_stage >= 0 && lane < ROWS) {
                    sh_x[warp][x_stage][0][lane] = (uint8_t)x_next;
                    sh_x[warp][x_stage][1][lane] = (uint8_t)(x_next >> 8);
                }
                x_stage = -1;
                if (at_load < t1) {
                    x_next = off < 0 ? 0u : (unsigned)__ldg(A.kx + x_at) | (unsigned)__ldg(A.vx + x_at) << 8;
                    x_stage = stage;
                }
            }
            if (at_load < t1) {
                if constexpr (K::QUANT) pa_issue_codes<K>(A, ring + stage * L::STAGE, off, load.len - (load.lo + load.tile * ROWS));
                else pa_issue<K>(A, ring + stage * L::STAGE, off);
                bad_ring = (bad_ring & ~(1u << stage)) | (__any_sync(0xffffffffu, next_bad) ? 1u << stage : 0u);
                next_bad = false;
                at_load += load.tile + 1 < load.ntiles ? 1 : 1 + K::ITEM;
                if (at_load < t1) {
                    pa_next<K>(A, load);
                    off = pa_offset<K>(A, load, next_bad, x_at);
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
                    reinterpret_cast<float*>(ring_p + stage * L::STAGE), sq, sh_x[K::QUANT ? warp : 0][K::QUANT ? stage : 0][0]);
            bad = bad || ((bad_ring >> stage) & 1u);
            __syncwarp();
            const bool ends = use.tile + 1 == use.ntiles;
            at += ends ? 1 + K::ITEM : 1;
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
                    if constexpr (K::SHARED) {
                        const long long row0 = (long long)use.s * A.hq + h0;
                        for (int x = 4 * lane; x < nh * HD; x += 128)
                            *reinterpret_cast<float4*>(A.own_o + row0 * HD + x) = *reinterpret_cast<const float4*>(piece + pa_at<HD>(x));
                        if (lane < nh) A.own_ml[row0 + lane] = sh_ml[slot][lane];
                        if (lane == 0) A.own_at[(long long)use.s * Hx + use.hb] = make_int2(-1, 0);
                    } else {
                        T* o = reinterpret_cast<T*>(A.out) + (long long)use.s * A.out_stride + (long long)h0 * HD;
                        for (int x = 4 * lane; x < nh * HD; x += 128) {
                            const float4 v = *reinterpret_cast<const float4*>(piece + pa_at<HD>(x));
                            put4(o + x, v, 1.f / sh_ml[slot][x / HD].y);
                        }
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
                        sh_piece[slot] = {use.s, use.hb, front, ends, owner(item_first + K::ITEM + use.ntiles), stage};
                }
                fresh = true;
            }
            issue(stage);
            stage = stage + 1 == S ? 0 : stage + 1;
            if (!end) {
                if (ends) item_first += use.ntiles + K::ITEM;
                pa_next<K>(A, use);
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
    if (!K::SHARED && tid == 0) A.rec[cta] = make_int4(-1, 0, 0, 0);
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
            if (whole && K::SHARED) *reinterpret_cast<float4*>(A.own_o + ((long long)p0.s * A.hq + h0) * HD + x) = acc;
            else if (whole) put4(out + x, acc, 1.f / sh_sum[i][row].y);
            else *reinterpret_cast<float4*>(A.part_o + slot * GM * HD + x) = acc;
        }
        if (!whole) {
            if (tid < nh) A.part_ml[slot * GM + tid] = sh_sum[i][tid];
            if (tid == 0 && p0.first) {
                if (K::SHARED) A.own_at[(long long)p0.s * Hx + p0.hb] = make_int2(cta, p1.last_cta);
                else A.rec[cta] = make_int4(p0.s, p0.hb, p1.last_cta, 0);
            }
        } else if (K::SHARED && tid < nh) {
            A.own_ml[(long long)p0.s * A.hq + h0 + tid] = sh_sum[i][tid];
            if (tid == 0) A.own_at[(long long)p0.s * Hx + p0.hb] = make_int2(-1, 0);
        }
    }
    // behind a shared prefix this kernel runs beside the prefix's, and ends after it: what waits for this one has both
    if (K::SHARED) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Joins the pieces of the items that cross CTAs: a block per CTA that began one and one or two query heads, HD / 2
// threads for each head and group of pieces, of which a group takes eight at a time, all on their way together.  Small
// blocks, as they start while the last CTAs of the first kernel still hold their registers: 4 ragged contexts of up to
// 1000, 32 + 8 heads of 128: 10.9 us (11.6 us by blocks of 512).
constexpr int PJ_THREADS = 256;

template <typename K>
__global__ void __launch_bounds__(PJ_THREADS) paged_attention_join(const __grid_constant__ PaArgs A)
{
    using T = typename K::T;
    constexpr int HD = K::HD, GM = K::GM;
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

// Bytes of the pieces in flight, which the grid bounds, whatever the heads and lengths.
inline size_t pa_fronts(int gm, int hd, int blocks) { return (size_t)PA_SMS * blocks * PA_WARPS * gm * hd * sizeof(float); }
inline size_t pa_workspace(int gm, int hd, int blocks = 2)
{
    return (size_t)PA_SMS * blocks * (2 * gm * hd * sizeof(float) + 2 * gm * sizeof(float2) + sizeof(int4));
}

template <typename K>
float2* pa_part_ml(char* workspace) { return reinterpret_cast<float2*>(reinterpret_cast<float*>(workspace) + (size_t)PA_SMS * K::BLOCKS * 2 * K::GM * K::HD); }

template <typename K>
int attention(PaArgs A, char* workspace, cudaStream_t st, const char* op = "paged_attention")
{
    using L = PaLayout<K>;
    constexpr int HD = K::HD, GM = K::GM;
    A.nhb = (A.g + GM - 1) / GM;
    A.part_o = reinterpret_cast<float*>(workspace);
    A.part_ml = pa_part_ml<K>(workspace);
    A.rec = reinterpret_cast<int4*>(A.part_ml + (size_t)PA_SMS * K::BLOCKS * 2 * GM);
    if (K::QUANT) A.fronts = reinterpret_cast<float*>(workspace + ((pa_workspace(GM, HD, K::BLOCKS) + 15) & ~(size_t)15));
    const int rows = A.g < GM ? A.g : GM;
    // two heads per block of the join, or one where the items are so few that each has over a dozen pieces: one context of
    // 100000, 8 heads on one kv head: 28 us (34 us by two), one of 20000, 32 + 8 heads: 24.3 us (25.4 us); but 4 of up to
    // 1000, 32 + 8 heads: 11.2 us (10.8 us by two)
    A.join_rows = rows > 1 && (long long)A.n_seqs * A.C.n_kv_heads * A.nhb > 16 ? 1 : 0;
    int sms = 0;
    static mfs::PerDevice ready;
    cudaError_t e = mfs::op_device(ready, (const void*)paged_attention_kernel<K>, L::BYTES, &sms);
    if (e != cudaSuccess) return mfs::op_launched(op, e);
    const int G = K::BLOCKS * (sms < PA_SMS ? sms : PA_SMS);
    cudaLaunchConfig_t cfg = {};
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (K::SHARED) {
        cfg.gridDim = dim3((unsigned)G);
        cfg.blockDim = dim3(PA_WARPS * 32);
        cfg.dynamicSmemBytes = L::BYTES;
        e = cudaLaunchKernelEx(&cfg, paged_attention_kernel<K>, A);
        cfg.dynamicSmemBytes = 0;
    } else {
        paged_attention_kernel<K><<<G, PA_WARPS * 32, L::BYTES, st>>>(A);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess || K::SHARED) return mfs::op_launched(op, e);  // behind a shared prefix one kernel joins all parts
    cfg.gridDim = dim3((unsigned)G, (unsigned)((rows - 1) >> A.join_rows) + 1);
    cfg.blockDim = dim3(PJ_THREADS);
    if constexpr (!K::SHARED) e = cudaLaunchKernelEx(&cfg, paged_attention_join<K>, A);
    return mfs::op_launched(op, e);
}

// The checks that the attention calls share, and what they fill in; 0: go on, 1: nothing to do, else an error's code.
inline int pa_checked(const char* op, PaArgs& A, int dtype, int hd, int n_seqs, const int32_t* kv_len, const void* q, long long q_stride,
                      int n_q_heads, void* out, long long out_stride, float scale, int window, const void* workspace, size_t workspace_bytes,
                      size_t workspace_needed)
{
    if (dtype != MFS_DTYPE_F32 && dtype != MFS_DTYPE_BF16) return mfs::op_fail(MFS_E_ARG, op, "dtype must be fp32 or bf16");
    if (n_seqs < 0 || window < 0) return mfs::op_fail(MFS_E_ARG, op, "need n_seqs >= 0 and window >= 0");
    if (n_q_heads < 1 || n_q_heads % A.C.n_kv_heads || n_q_heads > MFS_MAX_HEADS)
        return mfs::op_fail(MFS_E_ARG, op, "n_q_heads must be a multiple of n_kv_heads, at most 65535");
    if (!(scale > 0.f && scale <= 1e30f)) return mfs::op_fail(MFS_E_ARG, op, "scale must be positive and finite");
    if (n_seqs == 0) return 1;
    if (!kv_len || !q || !out || !workspace) return mfs::op_fail(MFS_E_ARG, op, "null kv_len, q, out or workspace");
    const int elem = dtype == MFS_DTYPE_BF16 ? 2 : 4;
    if (!mfs::rows_ok(q, q_stride, n_q_heads, hd, elem) || !mfs::rows_ok(out, out_stride, n_q_heads, hd, elem))
        return mfs::op_fail(MFS_E_ARG, op, "pointers and token strides must be multiples of 16 bytes, a stride at least heads x head_dim");
    if (((uintptr_t)workspace & 15u) || workspace_bytes < workspace_needed)
        return mfs::op_fail(MFS_E_ARG, op, "workspace too small or not 16-byte aligned");
    A.kv_len = kv_len;
    A.q = (const char*)q;
    A.out = (char*)out;
    A.q_stride = q_stride;
    A.out_stride = out_stride;
    A.n_seqs = n_seqs;
    A.hq = n_q_heads;
    A.g = n_q_heads / A.C.n_kv_heads;
    A.window = window;
    A.c = scale * 1.44269504088896340736f;
    return 0;
}

}  // namespace
