// mfs_sample_rows: one token per row of logits, drawn with the caller's uniform
// after temperature, min-p, top-k and top-p.
//
// All three filters keep a prefix of the columns ordered by (logit descending,
// column ascending), so the candidates are {logit > tau} and the columns up to
// `tie` among {logit == tau}, and the row is never sorted.  Where few columns can
// be candidates they are listed: those above the k-th largest of the threads' own
// maxima (at least k columns reach it, and rarely many more), or above min-p's
// bound, in column order.  One CTA then finds each one's rank by comparing all with
// all, cuts the list and finds the token.  Otherwise a histogram, linear in the
// distance to the maximum in octaves of the weight, finds the bin that holds a
// filter's border, only that bin's columns are listed, and the token is found by
// sums in column order, per CTA, per thread, and within that thread's columns.
// Where a filter leaves few columns, each thread notes the places of its own first,
// so that a warp's lanes weigh columns together and not one by one.
//
// A row is taken by a cluster of 1 to 8 CTAs, as many as it takes to keep its
// part of the row in shared memory beside another CTA's, and to use the SMs when
// there are few rows; the CTAs exchange maxima, histograms, lists and sums through
// distributed shared memory.  The logits are read from memory once; what bounds
// the call is the passes over shared memory, the weighing (about 80 instructions a
// column with the loop around it) and the latency of the exchanges; with many long
// rows also the second wave, as a row takes most of an SM's shared memory.  Top-k of
// 16 rows of 2048 fp32: 8 us, of 32 rows of 32000: 10 us; top-p with min-p of 256 rows
// of 32000: 46 us; 128 rows of 131072 bf16: top-k 35 us, no filter 61 to 72 us (by how many
// rows are done again), top-p alone, which weighs all columns, 130 us.  Rows left in memory
// instead, read again from L2 by every pass, need no second wave but took 1.3 to 1.6 times as
// long in the last two.  The bf16 forms spill about 44 bytes a thread at 64 registers.
//
// Weights are unsigned fixed point (2^scale for the maximum's), so sums are exact
// whatever order the atomics take, and the row's token is the same on every run.
// A weight is 2^-y = 2^-n 2^-(i/64) 2^-r with y a pair of fp32, a table for i and
// three terms for |r| < 1/128: off by less than 2^-28 of itself (2^-30.2 from the
// terms' own rounding, 2^-31 each from the table's and the result's, 2^-31.5 each
// from r's, the table's in fp32 and the product's, 2^-34.7 from the terms left out).
// Each comparison of sums is made with a bound on that error, and a row in which one
// falls inside the bound is done again with exponentials of about 2^-40 relative
// error (pairs of fp32), in units fitted to the row's sum, 2^-61 of it or less (a
// list's: fitted to its length), which decides it.  64-bit floating point, two products a
// cycle and SM here, is kept to one thread per CTA; fractions of sums are taken in
// 128-bit integers.
#include <cooperative_groups.h>

#include "mfs_ops.cuh"

namespace cg = cooperative_groups;

namespace {

using u64 = unsigned long long;
using bf16 = __nv_bfloat16;

constexpr int SR_NB = 1024;           // histogram bins, of 1 / 16 octave
constexpr float SR_REACH = 64.f;      // columns below 2^-64 of the maximum's weight can hold no border and no draw
constexpr float SR_LEAST_T = 1.5e-30f;  // lower temperatures count as this: weights stay pairs of normal fp32 numbers
// Columns that a thread notes at most.  With 6, 12 and 16: top-p and min-p of 256 rows of 32000 36.9, 34.6 and 34.7 us
// (temperature 0.8), top-k 400 of 16 rows of 8192 18.0, 15.1 and 15.2 us; top-k 50 of 128 rows of 131072 bf16 33.4, 33.4
// and 46.6 us, as 16 take the shared memory of a second block.
constexpr int SR_SLOTS = 12;
constexpr int SR_MAX_C = 8;           // CTAs per row
constexpr int SR_STAGE_BYTES = 168 * 1024;  // a CTA's part of the row in shared memory at most
constexpr int SR_WIDE_BYTES = 140 * 1024;   // the same for CTAs of 1024 threads

// A pair of fp32 whose sum is the value (error-free sums and products by Dekker and Knuth).
struct F2 {
    float h, l;
};

// Of a CTA of NT threads; at most NT columns are listed.
template <int NT>
struct __align__(16) SrShared {
    unsigned count[SR_NB], lo[SR_NB], hi[SR_NB];  // this CTA's histogram: columns, sums of weights in two words
    u64 sum[SR_NB];                               // the row's sums of weights
    unsigned num[SR_NB];                          // and columns
    u64 list[NT];                                 // listed columns, ascending: key << 32 | ~column
    u64 ranked[NT];                               // their weights or keys by rank
    unsigned keys[NT];                            // the list's keys
    unsigned short rank[NT];
    unsigned short idx[NT][SR_SLOTS];             // noted columns, ascending, as places in the part
    uint2 table[64];                              // 2^(31 - i / 64), as an integer and as fp32
    u64 ws[(NT / 32)];
    float wf[(NT / 32)];
    int wi[(NT / 32)];
    // one entry per CTA of the row, written by that CTA in every CTA's copy
    float r_max[SR_MAX_C], r_edge[SR_MAX_C];
    int r_idx[SR_MAX_C];
    unsigned r_klo[SR_MAX_C], r_khi[SR_MAX_C], r_n[SR_MAX_C];
    u64 r_sum[SR_MAX_C];
    // results of a search
    int where, token, unsure;
    u64 before, inside;
    // the row's constants
    float lmin;
    F2 c;
    double reach;
};

struct Table {
    uint2 at[64];
};
constexpr Table make_table()
{
    Table t = {};
    double x = 2147483648.0;
    for (int i = 0; i < 64; ++i) {
        t.at[i].x = (unsigned)(x + 0.5);
        t.at[i].y = 0;
        x *= 0.989228013193975484129124959065583667774674335384985;  // 2^(-1/64)
    }
    return t;
}
__constant__ Table sr_table = make_table();

// larger logit = larger key (NaN columns are never asked for theirs); -0 and +0 are the same logit
__device__ __forceinline__ unsigned order_key(float x)
{
    const unsigned b = __float_as_uint(x + 0.f);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float key_value(unsigned k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu)); }

__device__ __forceinline__ F2 two_sum(float a, float b)
{
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ F2 quick_sum(float a, float b)
{
    const float s = __fadd_rn(a, b);
    return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    const float p = __fmul_rn(a.h, b.h);
    const float e = __fmaf_rn(a.h, b.h, -p);
    return quick_sum(p, __fadd_rn(e, __fmaf_rn(a.h, b.l, __fmul_rn(a.l, b.h))));
}
__device__ __forceinline__ F2 add2(F2 a, F2 b)
{
    F2 s = two_sum(a.h, b.h);
    return quick_sum(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ constexpr F2 split2(double x) { return {(float)x, (float)(x - (double)(float)x)}; }

// 2^(scale - y), y = (mx - x) c, to about 2^-40 of it; 0 where the difference is past the largest fp32 number, as the fast
// weight has it.
__device__ __noinline__ u64 precise_weight(float x, float mx, F2 c, int scale)
{
    const F2 y = mul2(two_sum(mx, -x), c);
    if (!(y.h < 128.f)) return 0;
    const float n = rintf(y.h);
    F2 z = mul2(quick_sum(__fsub_rn(y.h, n), y.l), split2(0.69314718055994530942));  // |z| <= 0.35
    z.h = -z.h;
    z.l = -z.l;
    // the series of exp: terms 7 .. 12 need 24 bits only (the 7th is below 2^-22), the lower ones pairs
    float t = 1.f / 479001600.f;
    t = fmaf(t, z.h, 1.f / 39916800.f);
    t = fmaf(t, z.h, 1.f / 3628800.f);
    t = fmaf(t, z.h, 1.f / 362880.f);
    t = fmaf(t, z.h, 1.f / 40320.f);
    t = fmaf(t, z.h, 1.f / 5040.f);
    F2 s = {t, 0.f};
    s = add2(mul2(s, z), split2(1.0 / 720.0));
    s = add2(mul2(s, z), split2(1.0 / 120.0));
    s = add2(mul2(s, z), split2(1.0 / 24.0));
    s = add2(mul2(s, z), split2(1.0 / 6.0));
    s = add2(mul2(s, z), split2(0.5));
    s = add2(mul2(s, z), split2(1.0));
    s = add2(mul2(s, z), split2(1.0));
    const float up = exp2f((float)scale - n);  // an exact power of two
    return (u64)((long long)__float2ull_rn(s.h * up) + __float2ll_rn(s.l * up));
}

struct Weigher {
    float mx;      // the row's maximum
    F2 c;          // log2(e) / T
    int scale;     // the maximum's weight is 2^scale: sums over a row stay below 2^62
    bool precise;
    const uint2* table;

    // The 64ths of an octave, to the nearest, that x's weight lies below the maximum's (one answer for one x, and
    // never less for a smaller x); q: the same as a float, plus 1.5 2^23.
    __device__ __forceinline__ int steps(float x, float& q) const
    {
        q = fmaf(x == mx ? 0.f : __fmul_rn(mx - x, c.h), 64.f, 12582912.f);  // the integer is in the low bits
        return __float_as_int(q) - 0x4b400000;
    }
    __device__ __forceinline__ u64 operator()(float x) const
    {
        float q;
        return weight(x, steps(x, q), q);
    }
    __device__ __forceinline__ u64 weight(float x, int k, float q) const
    {
        if (x == mx) return 1ull << scale;
        if (precise) return precise_weight(x, mx, c, scale);
        const F2 d = two_sum(mx, -x);
        const float h = __fmul_rn(d.h, c.h);
        const float l = fmaf(d.l, c.h, fmaf(d.h, c.l, fmaf(d.h, c.h, -h)));
        const float r = fmaf(q - 12582912.f, -1.f / 64.f, h) + l;
        const uint2 t = table[k & 63];
        const float f = r * fmaf(r, fmaf(r, -0.0555041087f, 0.240226507f), -0.693147181f);  // 2^-r - 1
        const unsigned v = t.x + (unsigned)__float2int_rn(f * __uint_as_float(t.y));
        return ((u64)v << (scale - 31)) >> min(k >> 6, 63);
    }
};

// f x s for f in [0, 1), rounded down or up, exactly
__device__ __forceinline__ u64 fraction(float f, u64 s, bool up)
{
    if (!(f > 0.f)) return 0;
    const unsigned b = __float_as_uint(f), ex = max(b >> 23, 1u);
    const u64 m = b >> 23 ? (b & 0x7fffffu) | 0x800000u : b;
    const unsigned sh = 150 - ex;  // f = m 2^-sh, sh >= 24
    const u64 lo = m * s, hi = __umul64hi(m, s);
    u64 r, rest;
    if (sh < 64) {
        r = (hi << (64 - sh)) | (lo >> sh);
        rest = lo << (64 - sh);
    } else {
        r = sh < 128 ? hi >> (sh - 64) : 0;
        rest = lo | (sh < 128 ? hi & ((1ull << (sh - 64)) - 1) : hi);
    }
    return r + (up && rest);
}

__device__ __forceinline__ u64 warp_sum(u64 v)
{
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ u64 warp_inclusive(u64 v)
{
    const int lane = threadIdx.x & 31;
    for (int o = 1; o < 32; o <<= 1) {
        const u64 t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
    }
    return v;
}

// A CTA's part of a row, in 16-byte vectors of VE elements.  Vector v holds columns c0 + v * VE ..; those outside
// the part (at the ends, where the row is not 16-byte aligned) read as NaN.  Thread t has vectors t * per .. (t + 1) * per - 1.
template <typename T>
struct Part {
    static constexpr int VE = 16 / sizeof(T);
    const T* g;      // column 0 of the row
    unsigned kept;   // the vectors' address in shared memory, 0: they are read from memory
    int lo, hi, c0;  // columns [lo, hi)
    int nvec, per;   // vectors, and vectors per thread (odd: threads' vectors lie in different banks)

    __device__ __noinline__ static uint4 ragged(const T* g, int c, int lo, int hi)
    {
        uint4 r;
        T e[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            if constexpr (sizeof(T) == 4) e[i] = c + i >= lo && c + i < hi ? __ldg(g + c + i) : __uint_as_float(0x7fc00000u);
            else e[i] = c + i >= lo && c + i < hi ? g[c + i] : __ushort_as_bfloat16(0x7fc0);
        }
        memcpy(&r, e, 16);
        return r;
    }
    __device__ __forceinline__ uint4 fetch(int v) const
    {
        const int c = c0 + v * VE;
        if (c >= lo && c + VE <= hi) return __ldg(reinterpret_cast<const uint4*>(g + c));
        return ragged(g, c, lo, hi);
    }
    __device__ __forceinline__ uint4 vec(int v) const
    {
        if (!kept) return fetch(v);
        uint4 r;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(kept + 16 * v));
        return r;
    }
    static __device__ __forceinline__ float elem(const uint4& r, int i)
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w);
        const unsigned w = (i >> 1) == 0 ? r.x : (i >> 1) == 1 ? r.y : (i >> 1) == 2 ? r.z : r.w;
        return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
    }
    // the largest element (NaN: only if all are)
    static __device__ __forceinline__ float largest(const uint4& r)
    {
        if constexpr (sizeof(T) == 4) {
            return fmaxf(fmaxf(elem(r, 0), elem(r, 1)), fmaxf(elem(r, 2), elem(r, 3)));
        } else {
            __nv_bfloat162 b[4];
            memcpy(b, &r, 16);
            const __nv_bfloat162 m = __hmax2(__hmax2(b[0], b[1]), __hmax2(b[2], b[3]));
            return fmaxf(__low2float(m), __high2float(m));
        }
    }
    __device__ __forceinline__ float value(int i) const  // column c0 + i
    {
        if constexpr (sizeof(T) == 4) {
            if (!kept) return __ldg(g + c0 + i);
            float x;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(kept + 4 * i));
            return x;
        } else {
            unsigned short x;
            if (!kept) x = __ldg(reinterpret_cast<const unsigned short*>(g) + c0 + i);
            else asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(kept + 2 * i));
            return __uint_as_float((unsigned)x << 16);
        }
    }
    // f(column, logit) for this thread's columns of at least `least`, in ascending order
    template <typename F>
    __device__ __forceinline__ void each(float least, F f) const
    {
        const int v1 = min(nvec, (int)(threadIdx.x + 1) * per);
        for (int v = threadIdx.x * per; v < v1; ++v) {
            const uint4 r = vec(v);
            if (!(largest(r) >= least)) continue;
#pragma unroll
            for (int i = 0; i < VE; ++i)
                if (elem(r, i) >= least) f(c0 + v * VE + i, elem(r, i));
        }
    }
};

// What the functions below share.
template <typename T, int NT>
struct Row {
    Part<T> p;
    Weigher W;
    float lmin;  // columns below it are no candidates
    float mine;  // the largest logit among this thread's columns
    int C, rank, cols;
    int noted;  // columns of this thread in S->idx, or -1: its part of the row is gone through
    SrShared<NT>* S;

    __device__ __forceinline__ void sync() const
    {
        if (C > 1) cg::this_cluster().sync();
        else __syncthreads();
    }
    __device__ __forceinline__ SrShared<NT>* of(int r) const { return C > 1 ? cg::this_cluster().map_shared_rank(S, r) : S; }
    static __device__ __forceinline__ int bin_of(int steps) { return min(steps >> 2, SR_NB - 1); }
    __device__ __forceinline__ int bin(float x) const
    {
        float q;
        return bin_of(W.steps(x, q));
    }
    // f(column, logit) for this thread's columns of at least `least`, in ascending order
    template <typename F>
    __device__ __forceinline__ void each(float least, F f) const
    {
        if (noted < 0) return p.each(least, f);
        for (int i = 0; i < noted; ++i) {
            const int c = S->idx[threadIdx.x][i];
            const float x = p.value(c);
            if (x >= least) f(p.c0 + c, x);
        }
    }
    // how far a comparison of two sums of fast weights may be off: less than 2^-28 of each, a unit per column
    __device__ __forceinline__ u64 band(u64 total) const { return W.precise ? 0 : (total >> 27) + 2ull * cols + 2; }
};

// Inclusive sums of v over the CTA's threads, and their total.
template <int NT>
__device__ __forceinline__ u64 scan_weights(SrShared<NT>* S, u64 v, u64& total)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const u64 inc = warp_inclusive(v);
    __syncthreads();
    if (lane == 31) S->ws[warp] = inc;
    __syncthreads();
    const u64 all = warp_inclusive(lane < NT / 32 ? S->ws[lane] : 0);  // every warp scans the warps' sums
    total = __shfl_sync(0xffffffffu, all, 31);
    const u64 before = __shfl_sync(0xffffffffu, all, max(warp - 1, 0));
    return inc + (warp ? before : 0);
}

// The sum of v over the CTA's threads, for all of them.
template <int NT>
__device__ __forceinline__ u64 all_sum(SrShared<NT>* S, u64 v)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    v = warp_sum(v);
    __syncthreads();
    if (lane == 0) S->ws[warp] = v;
    __syncthreads();
    return warp_sum(lane < NT / 32 ? S->ws[lane] : 0);
}

// The first of 1024 values a (in shared memory) at which the running sum, starting at `start`, exceeds target;
// S->where = its place (or -1), S->before = the sum before it.
template <int NT, typename U>
__device__ void block_find(SrShared<NT>* S, const U* a, u64 start, u64 target)
{
    const int tid = threadIdx.x;
    u64 v[(SR_NB / NT)], mine = 0;
#pragma unroll
    for (int i = 0; i < (SR_NB / NT); ++i) {
        v[i] = (u64)a[tid * (SR_NB / NT) + i];
        mine += v[i];
    }
    if (tid == 0) S->where = -1;
    u64 total;
    u64 run = start + scan_weights(S, mine, total) - mine;
    if (run <= target && run + mine > target) {
#pragma unroll
        for (int i = 0; i < (SR_NB / NT); ++i) {
            if (run <= target && run + v[i] > target) { S->where = tid * (SR_NB / NT) + i; S->before = run; }
            run += v[i];
        }
    }
    __syncthreads();
}

// Sums of the first `n` of 1024 values, for all threads.
template <int NT, typename U>
__device__ u64 block_sum(SrShared<NT>* S, const U* a, int n)
{
    const int tid = threadIdx.x;
    u64 mine = 0;
#pragma unroll
    for (int i = 0; i < (SR_NB / NT); ++i)
        if (tid * (SR_NB / NT) + i < n) mine += (u64)a[tid * (SR_NB / NT) + i];
    return all_sum(S, mine);
}

// Adds this CTA's histogram to the others' into S->num and S->sum.
template <int NT, typename T>
__device__ void gather_histogram(const Row<T, NT>& R, bool counts, bool sums)
{
    SrShared<NT>* S = R.S;
    R.sync();
    for (int i = threadIdx.x; i < SR_NB; i += NT) {
        u64 m = 0;
        unsigned n = 0;
        for (int r = 0; r < R.C; ++r) {
            const SrShared<NT>* o = R.of(r);
            if (counts) n += o->count[i];
            if (sums) m += ((u64)o->hi[i] << 32) + o->lo[i];
        }
        S->num[i] = n;
        S->sum[i] = m;
    }
    R.sync();  // the others' histograms have been read
}

template <int NT>
__device__ __forceinline__ void clear_histogram(SrShared<NT>* S)
{
    for (int i = threadIdx.x; i < SR_NB; i += NT) S->count[i] = S->lo[i] = S->hi[i] = 0;
    __syncthreads();
}

template <int NT>
__device__ __forceinline__ void add_weight(SrShared<NT>* S, int b, u64 w)
{
    if (!w) return;
    const unsigned wl = (unsigned)w, old = atomicAdd(&S->lo[b], wl);
    const unsigned wh = (unsigned)(w >> 32) + (old + wl < old);
    if (wh) atomicAdd(&S->hi[b], wh);
}

// Histogram of the columns of at least `least` by put(column, x) (-1: in none), over all CTAs of the row.
template <int NT, typename T, typename F>
__device__ void histogram(const Row<T, NT>& R, float least, bool counts, bool sums, F put)
{
    SrShared<NT>* S = R.S;
    clear_histogram(S);
    R.each(least, [&](int col, float x) {
        const int b = put(col, x);
        if (b < 0) return;
        if (counts) atomicAdd(&S->count[b], 1u);
        if (sums) add_weight(S, b, R.W(x));
    });
    gather_histogram(R, counts, sums);
}

// Exclusive sums of n over the CTA's threads, and their total.
template <int NT>
__device__ __forceinline__ unsigned scan_counts(SrShared<NT>* S, unsigned n, unsigned& total)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned inc = n;
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += t;
    }
    __syncthreads();
    if (lane == 31) S->wi[warp] = inc;
    __syncthreads();
    // every warp scans the warps' sums
    unsigned all = lane < NT / 32 ? S->wi[lane] : 0;
    for (int o = 1; o < NT / 32; o <<= 1) {
        const unsigned t = __shfl_up_sync(0xffffffffu, all, o);
        if (lane >= o) all += t;
    }
    total = __shfl_sync(0xffffffffu, all, NT / 32 - 1);
    const unsigned before = __shfl_sync(0xffffffffu, all, max(warp - 1, 0));
    return inc - n + (warp ? before : 0);
}

// Each thread notes its columns of at least `least`, if no thread of the CTA has too many.
template <int NT, typename T>
__device__ __forceinline__ void note_columns(Row<T, NT>& R, float least)
{
    SrShared<NT>* S = R.S;
    if (R.noted >= 0 || R.p.nvec * R.p.VE > 65536) return;
    int n = 0;
    R.p.each(least, [&](int col, float) {
        if (n < SR_SLOTS) S->idx[threadIdx.x][n] = (unsigned short)(col - R.p.c0);
        ++n;
    });
    if (!__syncthreads_or(n > SR_SLOTS)) R.noted = n;
}

// The columns of at least `least` that take(x) names, of all CTAs and in ascending order, into the S->list of the row's
// first CTA, or of all; their number (more than NT: the list is not complete).
template <int NT, typename T, typename F>
__device__ unsigned list_columns(const Row<T, NT>& R, float least, bool all, F take)
{
    SrShared<NT>* S = R.S;
    unsigned n = 0, here;
    R.each(least, [&](int, float x) { n += take(x); });
    unsigned at = scan_counts(S, n, here), total = here;
    if (R.C > 1) {
        if (threadIdx.x < R.C) R.of(threadIdx.x)->r_n[R.rank] = here;
        R.sync();
        total = 0;
        for (int r = 0; r < R.C; ++r) {
            if (r < R.rank) at += S->r_n[r];
            total += S->r_n[r];
        }
    }
    if (n && total <= NT)
        R.each(least, [&](int col, float x) {
            if (!take(x)) return;
            const u64 e = ((u64)order_key(x) << 32) | (unsigned)~col;
            if (all)
                for (int r = 0; r < R.C; ++r) R.of(r)->list[at] = e;
            else
                R.of(0)->list[at] = e;
            ++at;
        });
    R.sync();
    return total;
}

// The ranks of the n listed columns among the candidates, into S->rank: each entry's keys are compared with all, by as
// many threads as there are for it.  A lower entry of the same key comes first.
template <int NT>
__device__ __forceinline__ void rank_list(SrShared<NT>* S, unsigned n)
{
    const unsigned tid = threadIdx.x;
    S->keys[tid] = tid < n ? (unsigned)(S->list[tid] >> 32) : 0;
    __syncthreads();
    int g = 1;
    while (g < 32 && n * (2 * g) <= NT) g *= 2;
    const unsigned me = tid / g;
    if (me < n || g > 1) {
        const unsigned k = S->keys[me < n ? me : 0];
        unsigned rank = 0;
        const uint4* keys = reinterpret_cast<const uint4*>(S->keys);
        for (unsigned c = tid & (g - 1); c < (n + 3) / 4; c += g) {
            const uint4 x = keys[c];
            const unsigned t = c < me / 4 ? k - 1 : k;  // keys are above 0
            rank += (x.x > t) + (x.y > t) + (x.z > t) + (x.w > t);
        }
        if ((tid & (g - 1)) == 0)
            for (unsigned i = me & ~3u; i < me && i < n; ++i) rank += S->keys[i] == k;
        for (int o = g / 2; o; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
        if (me < n && (tid & (g - 1)) == 0) S->rank[me] = (unsigned short)rank;
    }
    __syncthreads();
}

// The first column, in ascending order over the whole row, at which the running sum of wt(column, x) over the columns of
// at least `least` exceeds goal(total): only the CTA that holds it returns true, with S->where = the column,
// S->before = the sum before it and S->inside = its weight.
template <int NT, typename T, typename F, typename G>
__device__ bool find_in_order(const Row<T, NT>& R, float least, F wt, G goal)
{
    SrShared<NT>* S = R.S;
    const Part<T>& P = R.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    u64 mine = 0;
    R.each(least, [&](int col, float x) { mine += wt(col, x); });
    u64 here;
    u64 run = scan_weights(S, mine, here) - mine;
    u64 before = 0, total = here;
    if (R.C > 1) {
        if (tid < R.C) R.of(tid)->r_sum[R.rank] = here;
        R.sync();
        total = 0;
        for (int r = 0; r < R.C; ++r) {
            if (r < R.rank) before += S->r_sum[r];
            total += S->r_sum[r];
        }
    }
    const u64 target = goal(total);
    run += before;
    // the thread whose columns hold it, and its warp: that thread's columns, one per lane
    const unsigned hit = __ballot_sync(0xffffffffu, run <= target && run + mine > target);
    if (hit) {
        const int l = __ffs(hit) - 1, t = warp * 32 + l, first = t * P.per * P.VE;
        const int n = R.noted < 0 ? min(P.nvec, (t + 1) * P.per) * P.VE - first : __shfl_sync(0xffffffffu, R.noted, l);
        run = __shfl_sync(0xffffffffu, run, l);
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int i = i0 + lane;
            u64 w = 0;
            int col = 0;
            if (i < n) {
                const int c = R.noted < 0 ? first + i : S->idx[t][i];
                col = P.c0 + c;
                if (col >= P.lo && col < P.hi) {
                    const float x = P.value(c);
                    if (x >= least) w = wt(col, x);
                }
            }
            const u64 sum = warp_inclusive(w);
            const unsigned found = __ballot_sync(0xffffffffu, run + sum > target);
            if (found) {
                if (lane == __ffs(found) - 1) {
                    S->where = col;
                    S->before = run + sum - w;
                    S->inside = w;
                }
                break;
            }
            run += __shfl_sync(0xffffffffu, sum, 31);
        }
    }
    __syncthreads();
    return before <= target && before + here > target;
}

// The candidates: logits above tau, and those equal to it up to column tie.
struct Border {
    float tau;
    int tie;
};

// The last of the shortest prefix, in the candidates' order, of the n listed columns that, after sums of `mass` and
// `count` before the list, reaches `target` (weights if BY_MASS, less than `band` off; columns if not).
template <bool BY_MASS, int NT, typename T>
__device__ Border border_in_list(const Row<T, NT>& R, unsigned n, u64 mass, u64 count, u64 target, u64 band)
{
    SrShared<NT>* S = R.S;
    const int tid = threadIdx.x;
    rank_list(S, n);
    if (tid < n) {
        const unsigned rank = S->rank[tid];
        if (BY_MASS) S->ranked[rank] = S->list[tid];
        else if (rank == target - 1 - count) S->inside = S->list[tid];
    }
    __syncthreads();
    if (BY_MASS) {
        const u64 f = tid < n ? S->ranked[tid] : 0, w = tid < n ? R.W(key_value((unsigned)(f >> 32))) : 0;
        u64 total;
        const u64 upto = mass + scan_weights(S, w, total);
        if (tid < n && upto - w < target && (upto >= target || tid + 1 == n)) {
            S->inside = f;
            // the border is certain if no error of the sums can move it
            if (upto < target + band || (upto > w && upto - w + band >= target)) S->unsure = 1;
        }
        __syncthreads();
    }
    const u64 b = S->inside;
    __syncthreads();
    return {key_value((unsigned)(b >> 32)), (int)~(unsigned)b};
}

// The same among the CTA's threads, one entry e of weight w each where `in` is set: the entry that is the last of the
// shortest prefix, in descending order of the entries, that reaches `target` (weights if BY_MASS, entries if not), by a
// histogram and a comparison of all with all in the border's bin.
template <bool BY_MASS, int NT, typename T>
__device__ u64 border_among(const Row<T, NT>& R, u64 e, u64 w, bool in, u64 target, u64 band)
{
    SrShared<NT>* S = R.S;
    const int tid = threadIdx.x, b = in ? R.bin(key_value((unsigned)(e >> 32))) : -1;
    clear_histogram(S);
    if (in) {
        if (BY_MASS) add_weight(S, b, w);
        else atomicAdd(&S->count[b], 1u);
    }
    __syncthreads();
    if (BY_MASS) {
        for (int i = tid; i < SR_NB; i += NT) S->sum[i] = ((u64)S->hi[i] << 32) + S->lo[i];
        __syncthreads();
        block_find(S, S->sum, 0, target - 1);
    } else {
        block_find(S, S->count, 0, target - 1);
    }
    const bool here = in && b == S->where;
    u64 above = S->before;
    unsigned m;
    const unsigned at = scan_counts(S, here, m);
    u64* weight = S->sum;
    if (here) {
        S->ranked[at] = e;
        weight[at] = w;
    }
    __syncthreads();
    if (here) {
        for (unsigned i = 0; i < m; ++i)
            if (S->ranked[i] > e) above += BY_MASS ? weight[i] : 1;
        const u64 upto = above + (BY_MASS ? w : 1);
        if (above < target && upto >= target) {
            S->inside = e;
            if (BY_MASS && (upto < target + band || (above > 0 && above + band >= target))) S->unsure = 1;
        }
    }
    __syncthreads();
    const u64 border = S->inside;
    __syncthreads();
    return border;
}

// The token of a row whose candidates are all among the n listed columns.  False if an error bound left a choice open.
template <int NT, typename T>
__device__ __forceinline__ bool sample_list(const Row<T, NT>& R, unsigned n, int top_k, float top_p, float u, int32_t* token)
{
    SrShared<NT>* S = R.S;
    const int tid = threadIdx.x;
    const u64 e = tid < n ? S->list[tid] : 0;
    const u64 w = tid < n ? R.W(key_value((unsigned)(e >> 32))) : 0;
    u64 total;
    if (tid == 0) S->unsure = 0;
    __syncthreads();
    unsigned keep = top_k > 0 ? min(n, (unsigned)top_k) : n;  // columns kept, of the largest
    bool in = tid < n;
    // Up to 256 columns all are ranked against all, longer lists go through a histogram.  Lists of about 130 (16 rows of 2048,
    // top-k 100 and top-p): ranked 7.7 us, by histogram 8.8; of about 316 (top-k 250): 10.8 and 7.6; 256 rows of 32000, top-k
    // 100 and top-p: 23.5 and 26.4, top-k 400: 39.0 and 25.0.
    if (n > 256) {
        if (keep < n) {  // all threads take part
            const u64 border = border_among<false>(R, e, w, in, keep, 0);
            in = in && e >= border;
        }
        if (top_p < 1.f) {
            total = all_sum(S, in ? w : 0);
            const u64 border = border_among<true>(R, e, w, in, max((u64)1, fraction(top_p, total, true)), R.band(total));
            in = in && e >= border;
        }
    } else if (keep < n || top_p < 1.f) {
        rank_list(S, n);
        const unsigned rank = tid < n ? S->rank[tid] : n;
        if (top_p < 1.f) {
            if (tid < n) S->ranked[rank] = w;
            __syncthreads();
            const u64 v = tid < keep ? S->ranked[tid] : 0;
            const u64 upto = scan_weights(S, v, total), target = max((u64)1, fraction(top_p, total, true)), band = R.band(total);
            if (tid < keep && upto - v < target && upto >= target) {
                S->where = tid + 1;
                if (upto < target + band || (upto > v && upto - v + band >= target)) S->unsure = 1;
            }
            __syncthreads();
            keep = S->where;
        }
        in = rank < keep;
    }
    // the draw, in column order
    const u64 mine = in ? w : 0;
    const u64 upto = scan_weights(S, mine, total);
    const u64 target = u < 1.f || !(u == u) ? fraction(u, total, false) : total - 1, band = R.band(total);
    if (mine && upto > target && upto - mine <= target) {
        *token = (int)~(unsigned)e;
        if (upto <= target + band || (upto > mine && upto - mine + band > target)) S->unsure = 1;
    }
    __syncthreads();
    const bool open = S->unsure != 0;
    __syncthreads();
    return R.W.precise || !open;
}

// The border of the shortest prefix that holds `target` columns (BY_MASS = false) or weights summing to at least `target`
// (less than `band` off), from the linear histogram in S->num / S->sum.
template <bool BY_MASS, int NT, typename T>
__device__ Border find_border(Row<T, NT>& R, float least, u64 target, u64 band)
{
    SrShared<NT>* S = R.S;
    const int tid = threadIdx.x;
    if (BY_MASS) block_find(S, S->sum, 0, target - 1);
    else block_find(S, S->num, 0, target - 1);
    const int b = S->where;
    u64 mass = BY_MASS ? S->before : 0, count = BY_MASS ? 0 : S->before;  // before the bin
    unsigned klo = 0, khi = 0xffffffffu;
    bool keyed = false;
    // the bin's edges, widened by more than its arithmetic may be off, spare most columns the arithmetic
    float upper = INFINITY, from = least;
    if (R.W.c.h > 0.f) {
        const float step = SR_REACH / SR_NB / R.W.c.h;
        upper = R.W.mx - ((float)b - 0.2f) * step * 0.99999f;
        if (upper == -INFINITY) upper = INFINITY;  // past the largest fp32 number
        if (b < SR_NB - 1) from = fmaxf(least, R.W.mx - (float)(b + 1) * step * 1.00001f);
    }
    note_columns(R, from);
    unsigned n = list_columns(R, from, true, [&](float x) { return x <= upper && R.bin(x) == b; });
    while (n > NT) {
        // too many: split the bin's range of keys, down to one key
        if (!keyed) {
            unsigned lo = 0xffffffffu, hi = 0;
            R.each(least, [&](int, float x) {
                if (R.bin(x) == b) {
                    const unsigned k = order_key(x);
                    lo = min(lo, k);
                    hi = max(hi, k);
                }
            });
            lo = __reduce_min_sync(0xffffffffu, lo);
            hi = __reduce_max_sync(0xffffffffu, hi);
            if (tid == 0) { S->r_klo[R.rank] = 0xffffffffu; S->r_khi[R.rank] = 0; }
            __syncthreads();
            if ((tid & 31) == 0) { atomicMin(&S->r_klo[R.rank], lo); atomicMax(&S->r_khi[R.rank], hi); }
            __syncthreads();
            if (tid < R.C) {
                R.of(tid)->r_klo[R.rank] = S->r_klo[R.rank];
                R.of(tid)->r_khi[R.rank] = S->r_khi[R.rank];
            }
            R.sync();
            klo = 0xffffffffu;
            khi = 0;
            for (int r = 0; r < R.C; ++r) {
                klo = min(klo, S->r_klo[r]);
                khi = max(khi, S->r_khi[r]);
            }
            keyed = true;
        }
        if (klo == khi) break;
        const int bits = 32 - __clz(khi - klo), sh = bits > 10 ? bits - 10 : 0;
        histogram(R, least, true, BY_MASS, [&](int, float x) {
            const unsigned k = order_key(x);
            return k >= klo && k <= khi ? (int)((khi - k) >> sh) : -1;
        });
        if (BY_MASS) block_find(S, S->sum, mass, target - 1);
        else block_find(S, S->num, count, target - 1);
        const int sub = S->where;
        n = S->num[sub];
        if (BY_MASS) mass = S->before;
        else count = S->before;
        const unsigned top = khi - ((unsigned)sub << sh);
        klo = max(klo, sh ? top - ((1u << sh) - 1u) : top);
        khi = top;
        if (n <= NT) n = list_columns(R, least, true, [&](float x) { const unsigned k = order_key(x); return k >= klo && k <= khi; });
    }
    if (n <= NT) return border_in_list<BY_MASS>(R, n, mass, count, target, band);
    // one key, many columns: the last of them taken, in column order
    const u64 w = R.W(key_value(klo));
    u64 take = target - count;
    if (BY_MASS) {
        take = w ? max((u64)1, (target - mass + w - 1) / w) : 1;
        const u64 upto = mass + take * w;
        if ((upto < target + band || (upto > w && upto - w + band >= target)) && tid == 0) S->unsure = 1;
    }
    const bool mine = find_in_order(R, least, [&](int, float x) { return (u64)(order_key(x) == klo); }, [&](u64) { return take - 1; });
    const int at = mine ? S->where : -1;
    R.sync();
    if (mine && tid < R.C) R.of(tid)->token = at;
    R.sync();
    const Border B = {key_value(klo), S->token};
    __syncthreads();
    return B;
}

// The token of the row into `token` by the CTA that finds it, for rows whose candidates are not listed; all: the sum of
// their weights before top-p.  False if an error bound left a choice open (never with precise weights).
template <int NT, typename T>
__device__ __forceinline__ bool sample_row(Row<T, NT>& R, int top_k, float top_p, float u, int32_t* token, u64& all)
{
    SrShared<NT>* S = R.S;
    const int tid = threadIdx.x;
    Border B = {R.lmin, 0x7fffffff};
    if (tid == 0) S->unsure = 0;
    if (top_k > 0 && top_k < R.cols) {
        histogram(R, R.lmin, true, false, [&](int, float x) { return R.bin(x); });
        if (block_sum(S, S->num, SR_NB) > (u64)top_k) B = find_border<false>(R, R.lmin, (u64)top_k, 0);
    }
    if (top_p < 1.f) {
        // Columns of less than (1 - p) / cols of the maximum's weight hold at most 1 - p of the total: the border
        // lies above them, and only their sum is needed.
        const float deep = log2f((float)R.cols / (1.f - fmaxf(top_p, 0.f))) + 1.f;
        const float shallow = fmaxf(B.tau, R.W.mx - deep / R.W.c.h);
        clear_histogram(S);
        u64 rest = 0;
        R.each(B.tau, [&](int col, float x) {
            if (x == B.tau && col > B.tie) return;
            float q;
            const int steps = R.W.steps(x, q);
            const u64 w = R.W.weight(x, steps, q);
            if (x >= shallow) add_weight(S, R.bin_of(steps), w);
            else rest += w;
        });
        rest = all_sum(S, rest);
        if (R.C > 1 && tid < R.C) R.of(tid)->r_sum[R.rank] = rest;
        gather_histogram(R, false, true);
        if (R.C > 1) {
            rest = 0;
            for (int r = 0; r < R.C; ++r) rest += S->r_sum[r];
        }
        const u64 total = block_sum(S, S->sum, SR_NB) + rest;
        all = total;
        const Border Q = find_border<true>(R, shallow, max((u64)1, fraction(top_p, total, true)), R.band(total));
        if (!(Q.tau == B.tau && Q.tie > B.tie)) B = Q;
    }
    // the draw, in column order
    if (top_k > 0 || top_p < 1.f) note_columns(R, B.tau);
    u64 target = 0, total = 0;
    const bool mine = find_in_order(
        R, B.tau, [&](int col, float x) { return x == B.tau && col > B.tie ? (u64)0 : R.W(x); },
        [&](u64 sum) {
            total = sum;
            target = u < 1.f || !(u == u) ? fraction(u, sum, false) : sum - 1;
            return target;
        });
    if (mine && tid == 0) {
        const u64 band = R.band(total);
        // the chosen column's weight spans [before, before + inside)
        if (!R.W.precise && (S->before + S->inside <= target + band || (S->before > 0 && S->before + band > target)))
            for (int r = 0; r < R.C; ++r) R.of(r)->unsure = 1;
        *token = S->where;
    }
    if (!(top_p < 1.f)) all = total;
    R.sync();
    const bool open = S->unsure != 0;
    __syncthreads();  // read by all before another pass clears it
    return R.W.precise || !open;
}

template <int NT, typename T>
__global__ void __launch_bounds__(NT, 1024 / NT) sample_rows_kernel(const T* __restrict__ logits, int cols, long long ld,
                                                               const float* __restrict__ temperature,
                                                               const int32_t* __restrict__ top_k,
                                                               const float* __restrict__ top_p,
                                                               const float* __restrict__ min_p,
                                                               const float* __restrict__ uniforms, int32_t* __restrict__ tokens,
                                                               int C, int stage)
{
    extern __shared__ __align__(16) char sr_raw[];
    SrShared<NT>* S = reinterpret_cast<SrShared<NT>*>(sr_raw);
    const int r = blockIdx.x / C, rank = blockIdx.x % C, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float T_ = temperature ? __ldg(temperature + r) : 1.f;
    if (T_ > 0.f) T_ = fmaxf(T_, SR_LEAST_T);
    const int k = top_k ? __ldg(top_k + r) : 0;
    const float p = top_p ? __ldg(top_p + r) : 1.f, mp = min_p ? __ldg(min_p + r) : 0.f, u = __ldg(uniforms + r);
    if (tid < 64) {
        const unsigned t = sr_table.at[tid].x;
        S->table[tid] = make_uint2(t, __float_as_uint((float)t));
    }
    Row<T, NT> R;
    constexpr int VE = Part<T>::VE;
    R.C = C;
    R.rank = rank;
    R.cols = cols;
    R.S = S;
    R.p.g = logits + (long long)r * ld;
    const int each = (cols + C - 1) / C;
    R.p.lo = min(cols, rank * each);
    R.p.hi = min(cols, R.p.lo + each);
    R.p.c0 = R.p.lo - (int)((reinterpret_cast<uintptr_t>(R.p.g + R.p.lo) & 15u) / sizeof(T));
    R.p.nvec = R.p.hi > R.p.lo ? (R.p.hi - R.p.c0 + VE - 1) / VE : 0;
    R.p.per = ((R.p.nvec + NT - 1) / NT) | 1;
    R.p.kept = 0;
    R.noted = -1;
    const unsigned kept = (unsigned)__cvta_generic_to_shared(sr_raw + sizeof(SrShared<NT>));
    if (C > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (tid == NT - 1) {  // the row's 64-bit arithmetic, while the logits are on their way
        S->c = split2(1.4426950408889634 / (double)T_);
        S->reach = mp >= 1.f ? 0.0 : mp > 0.f ? -(double)T_ * log((double)mp) : 0.0;
    }
    // the maximum and its lowest column, and the row's part into shared memory
    float v = -INFINITY;
    int idx = 0x7fffffff;
    constexpr int DEEP = 8;
    for (int b = tid; b < R.p.nvec; b += NT * DEEP) {
        uint4 x[DEEP];
#pragma unroll
        for (int i = 0; i < DEEP; ++i)
            if (b + NT * i < R.p.nvec) x[i] = R.p.fetch(b + NT * i);
#pragma unroll
        for (int i = 0; i < DEEP; ++i)
            if (b + NT * i < R.p.nvec) {
                if (stage)
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(kept + 16 * (b + NT * i)), "r"(x[i].x), "r"(x[i].y),
                                 "r"(x[i].z), "r"(x[i].w) : "memory");
                const float m = R.p.largest(x[i]);
                if (m > v || (m == v && idx == 0x7fffffff)) {  // columns ascend: an equal one later never wins
                    v = m;
#pragma unroll
                    for (int e = VE - 1; e >= 0; --e)
                        if (R.p.elem(x[i], e) == m) idx = R.p.c0 + (b + NT * i) * VE + e;
                }
            }
    }
    R.mine = v;
    for (int o = 16; o; o >>= 1) {
        const float ov = __shfl_xor_sync(0xffffffffu, v, o);
        const int oi = __shfl_xor_sync(0xffffffffu, idx, o);
        if (ov > v || (ov == v && oi < idx)) { v = ov; idx = oi; }
    }
    if (lane == 0) { S->wf[warp] = v; S->wi[warp] = idx; }
    __syncthreads();
    v = S->wf[lane & ((NT / 32) - 1)];
    idx = S->wi[lane & ((NT / 32) - 1)];
    for (int o = (NT / 32) / 2; o; o >>= 1) {
        const float ov = __shfl_xor_sync(0xffffffffu, v, o);
        const int oi = __shfl_xor_sync(0xffffffffu, idx, o);
        if (ov > v || (ov == v && oi < idx)) { v = ov; idx = oi; }
    }
    if (C > 1) {
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every CTA of the row has started
        if (tid < C) { R.of(tid)->r_max[rank] = v; R.of(tid)->r_idx[rank] = idx; }
        cg::this_cluster().sync();
        for (int q = 0; q < C; ++q)
            if (S->r_max[q] > v || (S->r_max[q] == v && S->r_idx[q] < idx)) { v = S->r_max[q]; idx = S->r_idx[q]; }
    }
    if (!(T_ > 0.f) || v == -INFINITY || k == 1) {
        if (tid == 0 && rank == 0) tokens[r] = idx == 0x7fffffff ? 0 : idx;
        return;
    }
    if (stage) R.p.kept = kept;
    R.W.c = S->c;
    R.W.mx = v;
    R.W.table = S->table;
    R.W.scale = 62 - (32 - __clz(cols));
    R.W.precise = false;
    R.lmin = fmaxf(v - SR_REACH / R.W.c.h, -3.402823466e38f);
    if (mp > 0.f) {
        if (tid == 0) {  // the least logit l with exp((l - max) / T) >= min_p
            const double reach = S->reach;
            float l = (float)((double)v - reach);
            for (int t = 0; t < 4 && (double)v - (double)l > reach; ++t) l = nextafterf(l, INFINITY);
            for (int t = 0; t < 4; ++t) {
                const float below = nextafterf(l, -INFINITY);
                if ((double)v - (double)below > reach) break;
                l = below;
            }
            S->lmin = l;
        }
        __syncthreads();
        R.lmin = fmaxf(R.lmin, S->lmin);
    }
    if (v == INFINITY) R.lmin = INFINITY;
    const float pp = p == p ? p : 1.f;
    // few candidates: all of them listed by one CTA
    float least = R.lmin;
    bool few = mp > 0.f;
    if (k > 0 && k <= NT) {
        // the bin that the k-th largest of the threads' maxima lies in: at least k columns reach it
        clear_histogram(S);
        if (R.mine >= R.lmin) atomicAdd(&S->count[R.bin(R.mine)], 1u);
        __syncthreads();
        block_find(S, S->count, 0, (u64)k - 1);
        float edge = -INFINITY;  // its lower edge, less what the bin's arithmetic may be off
        if (S->where >= 0) edge = v - (float)(S->where + 1) * (SR_REACH / SR_NB) * 1.00001f / R.W.c.h;
        if (C > 1) {  // the best bound of the row's CTAs
            if (tid < C) R.of(tid)->r_edge[rank] = edge;
            R.sync();
            for (int q = 0; q < C; ++q) edge = fmaxf(edge, S->r_edge[q]);
        }
        if (edge > -INFINITY) {
            least = fmaxf(least, edge);
            few = true;
        }
    }
    if (few) {
        note_columns(R, least);
        const unsigned n = list_columns(R, least, false, [](float) { return true; });
        if (n <= NT) {
            if (rank == 0) {
#pragma unroll 1
                for (int pass = 0; pass < 2; ++pass) {
                    R.W.precise = pass != 0;
                    if (pass) R.W.scale = 62 - (32 - __clz(n));
                    if (sample_list(R, n, k, pp, u, tokens + r)) break;
                }
            }
            return;
        }
        R.lmin = least;
    }
    const int noted = R.noted;
    u64 all = 0;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        R.W.precise = pass != 0;
        if (sample_row(R, k, pp, u, tokens + r, all)) break;
        R.noted = noted;  // not those of the first pass's border
        // as many bits more as the sum (and what it may be off) leaves below 2^62, so that a unit is at most 2^-61 of it
        R.W.scale += __clzll(all + (all >> 26) + 2ull * cols + 2) - 2;
    }
}

template <typename T, int NT>
int launch(int C, const void* logits, int rows, int cols, long long ld, const float* temperature, const int32_t* top_k,
           const float* top_p, const float* min_p, const float* uniforms, int32_t* tokens, cudaStream_t st)
{
    constexpr int STAGE = NT == 512 ? SR_STAGE_BYTES : SR_WIDE_BYTES + 4096;
    static_assert(sizeof(SrShared<NT>) + STAGE <= 227 * 1024, "shared memory");
    auto kernel = sample_rows_kernel<NT, T>;
    int sms = 0;
    static mfs::PerDevice ready;
    const cudaError_t e = mfs::op_device(ready, (const void*)kernel, (int)(sizeof(SrShared<NT>) + STAGE), &sms);
    if (e != cudaSuccess) return mfs::op_launched("sample_rows", e);
    const long long part = ((long long)cols + C - 1) / C * sizeof(T) + 32;
    const bool stage = part <= STAGE;
    const size_t smem = sizeof(SrShared<NT>) + (stage ? (size_t)part : 0);
    if ((long long)rows * C > 0x7fffffffLL) return mfs::op_fail(MFS_E_ARG, "sample_rows", "too many rows");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * C));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)C;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = C > 1 ? 1 : 0;
    return mfs::op_launched("sample_rows", cudaLaunchKernelEx(&cfg, kernel, (const T*)logits, cols, ld, temperature, top_k, top_p, min_p,
                                                              uniforms, tokens, C, (int)stage));
}

// CTAs of 512 threads, two on an SM: as many per row as keep its parts within 64 KB, and more where rows leave SMs
// empty.  An exchange between the CTAs of a row costs over 1 us, so a row is cut in two for that from 16384 columns on
// (16 rows of 8192: 7.8 us whole, 9.6 us in two, with top-p 17.7 and 20.3 us; of 16384: 8.5 and 9.9, 19.8 and 20.6,
// without a filter 12.0 and 9.6), further while a part keeps 8192 (16 rows of 20000 bf16, top-p: 21.6 us in two, 20.4 us
// in four).  Where many rows would each need a cluster but fit one CTA of 1024 threads, alone on an SM, they get it:
// 128 rows of 32000 fp32, top-k 10.7 us (12.9 us as pairs), top-p 25.7 (29.1), 256 rows 20.5 (23.8) and 46.5 (52.5); 16
// rows, that leave SMs empty, 12.6 us without a filter (10.0 us as clusters of four).
template <typename T>
int choose(const void* logits, int rows, int cols, long long ld, const float* temperature, const int32_t* top_k,
           const float* top_p, const float* min_p, const float* uniforms, int32_t* tokens, cudaStream_t st)
{
    int sms = 0;
    static mfs::PerDevice known;
    const cudaError_t e = mfs::op_device(known, nullptr, 0, &sms);
    if (e != cudaSuccess) return mfs::op_launched("sample_rows", e);
    const long long bytes = (long long)cols * sizeof(T);
    int C = 1;
    while (C < SR_MAX_C && (bytes / C > 64 * 1024 || ((long long)rows * C * 2 <= sms && cols / C >= (C == 1 ? 16384 : 8192)))) C *= 2;
    if (C > 1 && bytes <= SR_WIDE_BYTES && 2LL * rows > sms)
        return launch<T, 1024>(1, logits, rows, cols, ld, temperature, top_k, top_p, min_p, uniforms, tokens, st);
    return launch<T, 512>(C, logits, rows, cols, ld, temperature, top_k, top_p, min_p, uniforms, tokens, st);
}

}  // namespace

extern "C" int mfs_sample_rows(const void* logits, int dtype, int rows, int cols, long long ld, const float* temperature,
                               const int32_t* top_k, const float* top_p, const float* min_p, const float* uniforms,
                               int32_t* tokens, void* cuda_stream)
{
    const char* op = "sample_rows";
    if (rows < 0 || cols < 1 || cols > MFS_SAMPLE_MAX_COLS || ld < cols)
        return mfs::op_fail(MFS_E_ARG, op, "need rows >= 0, 1 <= cols <= 4194304, ld >= cols");
    if (dtype != MFS_DTYPE_F32 && dtype != MFS_DTYPE_BF16) return mfs::op_fail(MFS_E_ARG, op, "dtype must be fp32 or bf16");
    if (rows == 0) return MFS_OK;
    if (!logits || !uniforms || !tokens) return mfs::op_fail(MFS_E_ARG, op, "null logits, uniforms or tokens");
    if ((uintptr_t)logits % (dtype == MFS_DTYPE_BF16 ? 2 : 4)) return mfs::op_fail(MFS_E_ARG, op, "misaligned logits");
    cudaStream_t st = (cudaStream_t)cuda_stream;
    return dtype == MFS_DTYPE_BF16 ? choose<bf16>(logits, rows, cols, ld, temperature, top_k, top_p, min_p, uniforms, tokens, st)
                                   : choose<float>(logits, rows, cols, ld, temperature, top_k, top_p, min_p, uniforms, tokens, st);
}
