// mfs_sample_rows: one token per row of logits, drawn with the caller's uniform
// after temperature, min-p, top-k and top-p.
//
// All three filters keep a prefix of the columns ordered by (logit descending,
// column ascending), so the candidates are {key > tau} and the columns up to
// `tie` among {key == tau}, and nothing has to be sorted: a boundary is found by
// histograms of counts and of weights, the first one linear in the distance to
// the maximum (so that the weights spread over the bins), the next ones over the
// key range of the bin that holds the boundary.  The token is then found by
// sums over 128-column segments in column order.
//
// Weights are unsigned fixed point (2^-36 of the maximum's weight), so sums are
// exact whatever order the atomics take, and the row's token is the same on
// every run.  A weight carries the error of its fp32 exponent; each comparison of
// sums is made with a bound on that error, and a row in which one falls inside
// the bound is done again with exponentials of about 2^-40 relative error
// (pairs of fp32), which decides it.
#include "mfs_ops.cuh"

namespace {

constexpr int SR_NT = 512;            // threads per row
constexpr int SR_NW = SR_NT / 32;
constexpr int SR_NB = 1024;           // histogram bins
constexpr int SR_NSEG = 1024;         // column segments at most
constexpr float SR_REACH = 64.f;      // columns below 2^-64 of the maximum's weight can hold no boundary and no draw
constexpr int SR_STAGE_COLS = 48 * 1024;  // rows of at most this many columns are kept in shared memory
using u64 = unsigned long long;

struct SrShared {
    u64 mass[SR_NB];
    unsigned count[SR_NB];
    u64 seg[SR_NSEG];
    u64 su[SR_NW];
    float sv[SR_NW];
    int si[SR_NW];
    // results of the serial steps
    int bin, tie, token;
    unsigned cnt_before, klo, khi;
    u64 mass_before, mass_upto, total;
    double err;
    float lmin;
    int unsure;
};

// larger logit = larger key (NaN columns are never asked for theirs); -0 and +0 are the same logit
__device__ __forceinline__ unsigned order_key(float x)
{
    const unsigned b = __float_as_uint(x + 0.f);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float key_value(unsigned k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu)); }

// A pair of fp32 whose sum is the value (error-free sums and products by Dekker and Knuth).
struct F2 {
    float h, l;
};
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
__device__ __forceinline__ F2 split2(double x)
{
    const float h = (float)x;
    return {h, (float)(x - (double)h)};
}

struct Weigher {
    float mx, c;  // maximum; log2(e) / T
    F2 c2;        // the same as a pair
    F2 ln2;
    F2 inv_fact[7];  // 1 / k!

    // octaves below the maximum's weight
    __device__ __forceinline__ float octaves(float x) const { return x == mx ? 0.f : (mx - x) * c; }

    // weight in units of 2^-36 (fast) or 2^-40 (precise) of the maximum's
    template <bool PRECISE>
    __device__ __forceinline__ u64 operator()(float x) const
    {
        if (x == mx) return PRECISE ? (1ull << 40) : (1ull << 36);
        if (!PRECISE) return (u64)__float2ull_rn(exp2f(-(mx - x) * c) * 68719476736.f);
        // y = (mx - x) * c as a pair, n its nearest integer, 2^-(y - n) by the series of exp
        const F2 d = two_sum(mx, -x);
        const F2 y = mul2(d, c2);
        const float n = rintf(y.h);
        F2 z = mul2(quick_sum(__fsub_rn(y.h, n), y.l), ln2);  // |z| <= 0.35
        z.h = -z.h;
        z.l = -z.l;
        // terms 7 .. 12 of the series need 24 bits only (the 7th is below 2^-22), the lower ones pairs
        float t = 1.f / 479001600.f;
        t = fmaf(t, z.h, 1.f / 39916800.f);
        t = fmaf(t, z.h, 1.f / 3628800.f);
        t = fmaf(t, z.h, 1.f / 362880.f);
        t = fmaf(t, z.h, 1.f / 40320.f);
        t = fmaf(t, z.h, 1.f / 5040.f);
        F2 s = {t, 0.f};
#pragma unroll
        for (int k = 6; k >= 0; --k) s = add2(mul2(s, z), inv_fact[k]);
        const float up = exp2f(40.f - n);  // an exact power of two
        return (u64)((long long)__float2ull_rn(s.h * up) + __float2ll_rn(s.l * up));
    }
};

template <typename T>
struct SrRow {
    const T* g;
    const float* staged;  // or nullptr
    int n;
    __device__ __forceinline__ float at(int i) const
    {
        if (staged) return staged[i];
        if constexpr (sizeof(T) == 4) return __ldg(g + i);
        else return __uint_as_float((unsigned)__ldg(reinterpret_cast<const unsigned short*>(g) + i) << 16);
    }
};

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

// Warp 0: the first entry of a[0..m) at which the running sum exceeds `target`, and the sum
// before it (or m).
template <typename U>
__device__ __forceinline__ int warp_find(const U* a, int m, u64 target, u64& before)
{
    const int lane = threadIdx.x & 31;
    u64 run = 0;
    for (int b0 = 0; b0 < m; b0 += 32) {
        const u64 v = b0 + lane < m ? (u64)a[b0 + lane] : 0;
        const u64 inc = warp_inclusive(v);
        const unsigned hit = __ballot_sync(0xffffffffu, b0 + lane < m && run + inc > target);
        if (hit) {
            const int l = __ffs(hit) - 1;
            before = run + __shfl_sync(0xffffffffu, inc - v, l);
            return b0 + l;
        }
        run += __shfl_sync(0xffffffffu, inc, 31);
    }
    before = run;
    return m;
}

// The boundary of the shortest prefix of the candidates' order that holds `target` columns
// (BY_MASS = false) or weights summing to at least `target`.  On return S->khi is the boundary's key, S->tie the
// last column taken among those with that key, S->mass_upto the sum up to the boundary and
// S->unsure is set if the error bound `band` leaves the choice open.  The linear histogram is in
// S->count / S->mass; it is overwritten.  Every thread calls it.
template <typename T, bool PRECISE, bool BY_MASS>
__device__ void find_boundary(const SrRow<T>& row, const Weigher& W, float lmin, u64 target, u64 band, SrShared* S)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto pick_bin = [&]() {  // warp 0
        u64 before;
        if (BY_MASS) {
            const int b = min(warp_find(S->mass, SR_NB, target - 1 - S->mass_before, before), SR_NB - 1);
            u64 c = 0;
            for (int i = lane; i < b; i += 32) c += S->count[i];
            c = warp_sum(c);
            if (lane == 0) { S->bin = b; S->mass_before += before; S->cnt_before += (unsigned)c; }
        } else {
            const int b = min(warp_find(S->count, SR_NB, target - 1 - S->cnt_before, before), SR_NB - 1);
            u64 c = 0;
            for (int i = lane; i < b; i += 32) c += S->mass[i];
            c = warp_sum(c);
            if (lane == 0) { S->bin = b; S->cnt_before += (unsigned)before; S->mass_before += c; }
        }
    };
    if (tid == 0) { S->cnt_before = 0; S->mass_before = 0; S->klo = 0xffffffffu; S->khi = 0; }
    __syncthreads();
    if (warp == 0) pick_bin();
    __syncthreads();
    const int bin0 = S->bin;
    {  // the key range of the bin's columns
        unsigned lo = 0xffffffffu, hi = 0;
        for (int i = tid; i < row.n; i += SR_NT) {
            const float x = row.at(i);
            if (x >= lmin && min((int)(W.octaves(x) * (SR_NB / SR_REACH)), SR_NB - 1) == bin0) {
                const unsigned k = order_key(x);
                lo = min(lo, k);
                hi = max(hi, k);
            }
        }
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (lane == 0) { atomicMin(&S->klo, lo); atomicMax(&S->khi, hi); }
    }
    __syncthreads();
    for (;;) {
        const unsigned klo = S->klo, khi = S->khi;
        const int bits = 32 - __clz(khi - klo);
        const int sh = bits > 10 ? bits - 10 : 0;
        for (int i = tid; i < SR_NB; i += SR_NT) { S->mass[i] = 0; S->count[i] = 0; }
        __syncthreads();
        for (int i = tid; i < row.n; i += SR_NT) {
            const float x = row.at(i);
            if (!(x >= lmin)) continue;
            const unsigned k = order_key(x);
            if (k >= klo && k <= khi) {
                const unsigned b = (khi - k) >> sh;
                atomicAdd(&S->count[b], 1u);
                atomicAdd(&S->mass[b], W.template operator()<PRECISE>(x));
            }
        }
        __syncthreads();
        if (warp == 0) pick_bin();
        __syncthreads();
        if (tid == 0) {
            const unsigned top = khi - ((unsigned)S->bin << sh);
            S->khi = top;
            S->klo = sh == 0 ? top : max(klo, top - ((1u << sh) - 1u));
        }
        __syncthreads();
        if (sh == 0) break;
    }
    const unsigned tau = S->khi;
    const unsigned have = S->count[S->bin];
    const u64 w = W.template operator()<PRECISE>(key_value(tau));
    unsigned take;  // columns taken among those with the boundary's key
    if (BY_MASS) {
        const u64 r = w ? (target - S->mass_before + w - 1) / w : have;
        take = (unsigned)min((u64)have, max((u64)1, r));
    } else {
        take = min(have, max(1u, (unsigned)(target - S->cnt_before)));
    }
    const u64 upto = S->mass_before + (u64)take * w;
    __syncthreads();
    if (tid == 0) {
        S->mass_upto = upto;
        S->tie = 0x7fffffff;
        if (BY_MASS && (upto < target + band || (upto > w && upto - w + band >= target))) S->unsure = 1;
    }
    if (take < have) {  // the take-th column with that key: counts per segment, in column order
        const int per = ((row.n + 127) / 128 + SR_NSEG - 1) / SR_NSEG * 128, nseg = (row.n + per - 1) / per;
        for (int s = warp; s < nseg; s += SR_NW) {
            unsigned c = 0;
            const int end = min(row.n, (s + 1) * per);
            for (int i = s * per + lane; i < end; i += 32) {
                const float x = row.at(i);
                c += x >= lmin && order_key(x) == tau;
            }
            c = __reduce_add_sync(0xffffffffu, c);
            if (lane == 0) S->seg[s] = c;
        }
        __syncthreads();
        if (warp == 0) {
            u64 before;
            const int s = warp_find(S->seg, nseg, take - 1, before);
            unsigned left = take - (unsigned)before;
            const int end = min(row.n, (s + 1) * per);
            for (int i0 = s * per; i0 < end; i0 += 32) {
                const int i = i0 + lane;
                float x = 0.f;
                if (i < end) x = row.at(i);
                unsigned m = __ballot_sync(0xffffffffu, i < end && x >= lmin && order_key(x) == tau);
                const unsigned here = __popc(m);
                if (here >= left) {
                    while (--left) m &= m - 1;
                    if (lane == 0) S->tie = i0 + __ffs(m) - 1;
                    break;
                }
                left -= here;
            }
        }
    }
    __syncthreads();
}

// One row.  Returns false if an error bound left a choice open (never with PRECISE).
template <typename T, bool PRECISE>
__device__ bool sample_row(const SrRow<T>& row, const Weigher& W, float lmin, int top_k, float top_p, float u, SrShared* S)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = row.n;
    unsigned tau = 0;
    int tie = 0x7fffffff;
    if (tid == 0) S->unsure = 0;
    const bool cut_k = top_k > 0 && top_k < n, cut_p = top_p < 1.f;
    if (cut_k || cut_p) {
        auto histogram = [&]() {
            for (int i = tid; i < SR_NB; i += SR_NT) { S->mass[i] = 0; S->count[i] = 0; }
            __syncthreads();
            for (int i = tid; i < n; i += SR_NT) {
                const float x = row.at(i);
                if (x >= lmin) {
                    const unsigned k = order_key(x);
                    if (k > tau || (k == tau && i <= tie)) {
                        const int b = min((int)(W.octaves(x) * (SR_NB / SR_REACH)), SR_NB - 1);
                        atomicAdd(&S->count[b], 1u);
                        atomicAdd(&S->mass[b], W.template operator()<PRECISE>(x));
                    }
                }
            }
            __syncthreads();
            if (warp == 0) {  // totals, and a bound on the error of any sum of these weights
                u64 c = 0, m = 0;
                double e = 0.0;
                for (int i = lane; i < SR_NB; i += 32) {
                    c += S->count[i];
                    m += S->mass[i];
                    e += (double)S->mass[i] * (double)(i + 1);
                }
                c = warp_sum(c);
                m = warp_sum(m);
                for (int o = 16; o; o >>= 1) e += __shfl_xor_sync(0xffffffffu, e, o);
                if (lane == 0) { S->cnt_before = (unsigned)c; S->total = m; S->err = e * (SR_REACH / SR_NB); }
            }
            __syncthreads();
        };
        histogram();
        u64 total = S->total;
        if (cut_k && (unsigned)top_k < S->cnt_before) {
            find_boundary<T, PRECISE, false>(row, W, lmin, (u64)top_k, 0, S);
            tau = S->khi;
            tie = S->tie;
            total = S->mass_upto;
            __syncthreads();
            if (cut_p) histogram();
        }
        if (cut_p) {
            const double goal = fmax(0.0, (double)top_p) * (double)total;
            const u64 band = PRECISE ? 0 : (u64)(2.0 * (1.3e-7 * S->err + 2.5e-7 * (double)total + 0.5 * n)) + 2;
            const u64 target = max((u64)1, (u64)ceil(goal));
            __syncthreads();
            find_boundary<T, PRECISE, true>(row, W, lmin, target, band, S);
            // the boundary among those of top-k: a tie of its own only if it is the same key
            const int t2 = S->khi == tau ? min(tie, S->tie) : S->tie;
            tau = S->khi;
            tie = t2;
            __syncthreads();
        }
    }
    // sums of 128-column segments, in column order
    const int per = ((n + 127) / 128 + SR_NSEG - 1) / SR_NSEG * 128, nseg = (n + per - 1) / per;
    float spread = 0.f;  // sum of weight x octaves: how exact the weights are
    for (int s = warp; s < nseg; s += SR_NW) {
        u64 sum = 0;
        const int end = min(n, (s + 1) * per);
        for (int i = s * per + lane; i < end; i += 32) {
            const float x = row.at(i);
            if (x >= lmin) {
                const unsigned k = order_key(x);
                if (k > tau || (k == tau && i <= tie)) {
                    const u64 w = W.template operator()<PRECISE>(x);
                    sum += w;
                    spread += (float)w * W.octaves(x);
                }
            }
        }
        sum = warp_sum(sum);
        if (lane == 0) S->seg[s] = sum;
    }
    for (int o = 16; o; o >>= 1) spread += __shfl_xor_sync(0xffffffffu, spread, o);
    if (lane == 0) S->sv[warp] = spread;
    __syncthreads();
    if (warp == 0) {
        u64 total = 0;
        for (int s = lane; s < nseg; s += 32) total += S->seg[s];
        total = warp_sum(total);
        spread = 0.f;
        for (int w = 0; w < SR_NW; ++w) spread += S->sv[w];
        const double goal = fmax(0.0, (double)u) * (double)total;
        const u64 target = goal < (double)total ? min((u64)goal, total - 1) : total - 1;
        const u64 band = PRECISE ? 0 : (u64)(2.0 * (1.4e-7 * (double)spread + 2.5e-7 * (double)total + 0.5 * n)) + 2;
        u64 run;
        const int s = warp_find(S->seg, nseg, target, run);
        const int end = min(n, (s + 1) * per);
        for (int i0 = s * per; i0 < end; i0 += 32) {
            const int i = i0 + lane;
            u64 w = 0;
            if (i < end) {
                const float x = row.at(i);
                if (x >= lmin) {
                    const unsigned k = order_key(x);
                    if (k > tau || (k == tau && i <= tie)) w = W.template operator()<PRECISE>(x);
                }
            }
            const u64 inc = warp_inclusive(w);
            const unsigned hit = __ballot_sync(0xffffffffu, run + inc > target);
            if (hit) {
                const int l = __ffs(hit) - 1;
                if (lane == l) {
                    S->token = i;
                    // the chosen column's weight spans [run + inc - w, run + inc)
                    if (run + inc <= target + band || (run + inc - w > 0 && run + inc - w + band > target)) S->unsure = 1;
                }
                break;
            }
            run += __shfl_sync(0xffffffffu, inc, 31);
        }
    }
    __syncthreads();
    return PRECISE || S->unsure == 0;
}

template <typename T>
__global__ void __launch_bounds__(SR_NT) sample_rows_kernel(const T* __restrict__ logits, int cols, long long ld,
                                                            const float* __restrict__ temperature,
                                                            const int32_t* __restrict__ top_k,
                                                            const float* __restrict__ top_p,
                                                            const float* __restrict__ min_p,
                                                            const float* __restrict__ uniforms, int32_t* __restrict__ tokens,
                                                            int stage)
{
    extern __shared__ __align__(16) char sr_raw[];
    SrShared* S = reinterpret_cast<SrShared*>(sr_raw);
    float* st = reinterpret_cast<float*>(sr_raw + sizeof(SrShared));
    const int r = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    SrRow<T> row{logits + (long long)r * ld, nullptr, cols};
    float v = -INFINITY;
    int idx = 0x7fffffff;
    for (int i = tid; i < cols; i += SR_NT) {
        const float x = row.at(i);
        if (stage) st[i] = x;
        if (x > v || (x == v && i < idx)) { v = x; idx = i; }
    }
    for (int o = 16; o; o >>= 1) {
        const float ov = __shfl_xor_sync(0xffffffffu, v, o);
        const int oi = __shfl_xor_sync(0xffffffffu, idx, o);
        if (ov > v || (ov == v && oi < idx)) { v = ov; idx = oi; }
    }
    if (lane == 0) { S->sv[warp] = v; S->si[warp] = idx; }
    __syncthreads();
    v = S->sv[0];
    idx = S->si[0];
    for (int w = 1; w < SR_NW; ++w)
        if (S->sv[w] > v || (S->sv[w] == v && S->si[w] < idx)) { v = S->sv[w]; idx = S->si[w]; }
    __syncthreads();
    if (stage) row.staged = st;
    const float T_ = temperature ? temperature[r] : 1.f;
    const int k = top_k ? top_k[r] : 0;
    if (!(T_ > 0.f) || v == -INFINITY || k == 1) {
        if (tid == 0) tokens[r] = idx == 0x7fffffff ? 0 : idx;
        return;
    }
    const float p = top_p ? top_p[r] : 1.f, mp = min_p ? min_p[r] : 0.f;
    Weigher W;
    W.mx = v;
    const double c = fmin(1.4426950408889634 / (double)T_, 1e30);
    W.c2 = split2(c);
    W.c = W.c2.h;
    if (tid == 0) {
        float lmin = fmaxf(v - SR_REACH / W.c, -3.402823466e38f);
        if (mp > 0.f) {  // the least logit l with exp((l - max) / T) >= min_p
            const double reach = mp >= 1.f ? 0.0 : -(double)T_ * log((double)mp);
            float l = (float)((double)v - reach);
            for (int t = 0; t < 4 && (double)v - (double)l > reach; ++t) l = nextafterf(l, INFINITY);
            for (int t = 0; t < 4; ++t) {
                const float below = nextafterf(l, -INFINITY);
                if ((double)v - (double)below > reach) break;
                l = below;
            }
            lmin = fmaxf(lmin, l);
        }
        S->lmin = v == INFINITY ? INFINITY : lmin;
    }
    __syncthreads();
    const float lmin = S->lmin, u = uniforms[r];
    const float pp = p == p ? p : 1.f;
    if (!sample_row<T, false>(row, W, lmin, k, pp, u, S)) {
        __syncthreads();
        W.ln2 = split2(0.69314718055994530942);
        double f = 1.0;
        for (int i = 0; i < 7; ++i) {
            W.inv_fact[i] = split2(1.0 / f);
            f *= i + 1;
        }
        sample_row<T, true>(row, W, lmin, k, pp, u, S);
    }
    if (tid == 0) tokens[r] = S->token;
}

template <typename T>
int launch(const void* logits, int rows, int cols, long long ld, const float* temperature, const int32_t* top_k,
           const float* top_p, const float* min_p, const float* uniforms, int32_t* tokens, cudaStream_t st)
{
    const bool stage = cols <= SR_STAGE_COLS;
    const size_t smem = sizeof(SrShared) + (stage ? (size_t)cols * 4 : 0);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(sample_rows_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return mfs::op_launched("sample_rows", e);
    }
    sample_rows_kernel<T><<<rows, SR_NT, smem, st>>>((const T*)logits, cols, ld, temperature, top_k, top_p, min_p, uniforms,
                                                    tokens, stage);
    return mfs::op_launched("sample_rows", cudaGetLastError());
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
    return dtype == MFS_DTYPE_BF16
               ? launch<__nv_bfloat16>(logits, rows, cols, ld, temperature, top_k, top_p, min_p, uniforms, tokens, st)
               : launch<float>(logits, rows, cols, ld, temperature, top_k, top_p, min_p, uniforms, tokens, st);
}
