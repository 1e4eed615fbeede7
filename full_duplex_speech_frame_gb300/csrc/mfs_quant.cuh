// One-token attention over the 8-bit cache: a warp's state for an item of paged_attention_kernel.
#pragma once
#include "mfs_paged.cuh"

namespace {

__device__ __forceinline__ void mma_f16(float (&d)[4], const unsigned (&a)[4], unsigned b0, unsigned b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ unsigned pack_f16(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const unsigned*>(&v);
}

// Four e4m3 codes as two pairs of fp16, which hold them exactly.
__device__ __forceinline__ void e4m3_f16(unsigned w, unsigned& lo, unsigned& hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}" : "=r"(lo), "=r"(hi) : "r"(w));
}

__device__ __forceinline__ float pow2_of(unsigned b) { return __uint_as_float(b << 23); }  // 2^(b - 127); 0 for b = 0

__device__ __forceinline__ unsigned transposed(unsigned x)
{
    unsigned y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ float max_of_keys(float v)  // over a warp's eight groups of four lanes
{
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}

// The codes go to the matrix instruction as fp16, which holds each exactly and takes one conversion for two of them (bf16
// would take several); the rows' powers of two never meet the elements: a key's multiplies its scores, a value's goes into
// its weights.  Keys, and elements of the values, are the instruction's 16 rows, query heads its 8 columns: a group of up to
// eight heads fills it (with heads as rows half of it would be zeros).
//
// Queries: q = q' / f with a power of two f for each head that brings its largest element to [2^14, 2^15), so that fp16
// loses nothing above 2^-39 of it; a score takes f back as its key's power of two meets it, so that scores have their own size,
// whatever the query's and the key's (kept times f it would end at keys of 2^106).  bf16 queries are then exact;
// fp32 ones are the sum of two fp16 parts, 22 bits, and take two products.
//
// Weights: w_j 2^(e_j) with e_j the value's exponent, under a running maximum Y of log2 of that, times 2^BASE: so the weights'
// fp16 has its 11 bits for all that matter down to 2^-25 of the largest part of the output, and 2^-36 is lost, whatever the
// values' sizes.  fp32 queries: two parts again.  The sum of the weights is apart from this, in fp32 under the maximum of
// the scores alone.
//
// NB: blocks of eight query heads.
template <typename T, int HD, int NB>
struct PaE4m3 {
    static constexpr bool SPLIT = sizeof(T) == 4;
    static constexpr int GM = 8 * NB, ROWS = 32, MB = ROWS / 16, CH = HD / 16, OWN = 2 * NB, NP = SPLIT ? 2 : 1;
    static_assert(ROWS == 32, "a lane looks at one row's exponents");
    static constexpr float BASE = 11.f, TAKE = 4.5f;  // weights stay below 2^15.5, fp16 ends at 2^16
    unsigned qf[CH][NB][NP][2];
    float o[CH][NB][4];
    float m[OWN], l[OWN], y[OWN], inv[OWN];  // of heads 2 t and 2 t + 1 of each block; inv: 1 / f, NaN where the query is not finite

    __device__ __forceinline__ void begin(const PaArgs& A, const PaWalk& w, float*)
    {
        const int lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
        const int h0 = (w.hb / A.nhb) * A.g + (w.hb % A.nhb) * GM, nh = min(GM, A.g - (w.hb % A.nhb) * GM);
        const T* q = reinterpret_cast<const T*>(A.q) + (long long)w.s * A.q_stride + (long long)h0 * HD;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int row = r + 8 * b;
            // a lane's elements of a head: 16 k + 4 t ..., the instruction's places 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of step k, as
            // a word of codes has them
            float x[CH][4];
            unsigned top = 0, most = 0;  // largest finite element; of all, NaN above infinity
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                if constexpr (SPLIT) {
                    const float4 v = row < nh ? __ldg(reinterpret_cast<const float4*>(q + row * HD + 16 * k + 4 * t)) : make_float4(0.f, 0.f, 0.f, 0.f);
                    x[k][0] = v.x; x[k][1] = v.y; x[k][2] = v.z; x[k][3] = v.w;
                } else {
                    const uint2 v = row < nh ? __ldg(reinterpret_cast<const uint2*>(q + row * HD + 16 * k + 4 * t)) : make_uint2(0u, 0u);
                    x[k][0] = __uint_as_float(v.x << 16); x[k][1] = __uint_as_float(v.x & 0xffff0000u);
                    x[k][2] = __uint_as_float(v.y << 16); x[k][3] = __uint_as_float(v.y & 0xffff0000u);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const unsigned bits = __float_as_uint(x[k][e]) & 0x7fffffffu;
                    if (bits < 0x7f800000u) top = max(top, bits);
                    most = max(most, bits);
                }
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
            const unsigned f = min(253u, 268u - (top >> 23));  // of 2^(f - 127)
#pragma unroll
            for (int e = 0; e < 2; ++e) inv[2 * b + e] = __shfl_sync(0xffffffffu, most < 0x7f800000u ? pow2_of(254u - f) : NAN, 4 * (2 * t + e));
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                float z[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) z[e] = x[k][e] * pow2_of(f);
                qf[k][b][0][0] = pack_f16(z[0], z[1]);
                qf[k][b][0][1] = pack_f16(z[2], z[3]);
                if constexpr (SPLIT) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float rest = z[e] - __half2float(__float2half_rn(z[e]));
                        z[e] = isfinite(z[e]) ? rest : 0.f;
                    }
                    qf[k][b][NP - 1][0] = pack_f16(z[0], z[1]);
                    qf[k][b][NP - 1][1] = pack_f16(z[2], z[3]);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < OWN; ++h) {
            m[h] = y[h] = -INFINITY;
            l[h] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int x = 0; x < 4; ++x) o[k][b][x] = 0.f;
    }

    // x: exponents of the tile's 32 keys, then of its values
    __device__ __forceinline__ void tile(unsigned stage, int valid, float c, float* staged, const float*, const uint8_t* x)
    {
        const int lane = threadIdx.x & 31, r = lane >> 2, mi = lane >> 3, r8 = lane & 7;
        const bool no_key = x[lane] == 0, no_value = x[32 + lane] == 0;  // the row that this lane looks after
        float s[MB][NB][4] = {};  // keys r (0, 1) and r + 8 (2, 3) of heads 2 t (0, 2) and 2 t + 1 (1, 3)
#pragma unroll
        for (int n = 0; n < MB; ++n) {
            const int row = 16 * n + (mi & 1) * 8 + r8;
#pragma unroll
            for (int k = 0; k < CH; k += 2) {  // two steps of 16 elements of 16 keys
                unsigned w[4];
                ldm4(stage + row * HD + (pa_chunk<CH>(row, k + (mi >> 1)) << 4), w);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    unsigned a[4];
                    e4m3_f16(w[2 * i], a[0], a[2]);
                    e4m3_f16(w[2 * i + 1], a[1], a[3]);
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int p = 0; p < NP; ++p) mma_f16(s[n][b], a, qf[k + i][b][p][0], qf[k + i][b][p][1]);
                }
            }
        }
        float ve[MB][2];  // exponents of the values (0 stands for no value at all)
#pragma unroll
        for (int n = 0; n < MB; ++n)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int key = 16 * n + 8 * u + r;
                const float by = pow2_of(x[key]);
                float to[OWN];  // (finite, so that a score of 0 stays one)
#pragma unroll
                for (int h = 0; h < OWN; ++h) to[h] = fminf(by * inv[h], 0x1p127f);
                const unsigned vb = x[32 + key];
                ve[n][u] = vb ? (float)((int)vb - 127) : -INFINITY;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    s[n][b][2 * u] = key < valid ? s[n][b][2 * u] * to[2 * b] : -INFINITY;
                    s[n][b][2 * u + 1] = key < valid ? s[n][b][2 * u + 1] * to[2 * b + 1] : -INFINITY;
                }
            }
        // rows of exponent 0 are zeros, codes of NaN among theirs too (0 times NaN would not be)
        if (__any_sync(0xffffffffu, lane < valid && (no_key || no_value))) {
            uint4* row = reinterpret_cast<uint4*>(staged) + (ROWS + lane) * CH;
            for (int i = 0; i < CH && no_value; ++i) row[i] = make_uint4(0u, 0u, 0u, 0u);
            __syncwarp();
#pragma unroll
            for (int n = 0; n < MB; ++n)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (16 * n + 8 * (e >> 1) + r < valid && x[16 * n + 8 * (e >> 1) + r] == 0) s[n][b][e] = 0.f * inv[2 * b + (e & 1)];
        }
        // The maxima in use stay while no weight passes 2^8 under them, and no weight times its value's size 2^TAKE: then no lane
        // asks another.  Else (the first tile of an item, and few behind it; always where a score is NaN) they are found anew.
        float z[MB][NB][4];
        bool fits = true;
#pragma unroll
        for (int h = 0; h < OWN; ++h) {
            const int b = h / 2, e = h % 2;
#pragma unroll
            for (int n = 0; n < MB; ++n)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float a = (s[n][b][2 * u + e] - m[h]) * c;
                    z[n][b][2 * u + e] = a;
                    fits = fits && a <= 8.f && a + ve[n][u] <= y[h] + TAKE;
                }
        }
        if (!__all_sync(0xffffffffu, fits)) {
#pragma unroll
            for (int h = 0; h < OWN; ++h) {
                const int b = h / 2, e = h % 2;
                float v = -INFINITY;
#pragma unroll
                for (int n = 0; n < MB; ++n) v = fmaxf(v, fmaxf(s[n][b][e], s[n][b][e + 2]));
                const float mn = fmaxf(m[h], max_of_keys(v)), sub = mn == -INFINITY ? 0.f : mn;  // scores of -infinity alone so far: weights 0, not NaN
                const float down = m[h] == mn ? 0.f : (m[h] - mn) * c;
                float top = -INFINITY;
#pragma unroll
                for (int n = 0; n < MB; ++n)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        z[n][b][2 * u + e] = (s[n][b][2 * u + e] - sub) * c;
                        top = fmaxf(top, z[n][b][2 * u + e] + ve[n][u]);
                    }
                const float was = y[h] + down, yn = fmaxf(was, max_of_keys(top)), scale = was == yn ? 1.f : ex2(was - yn);
                l[h] *= ex2(down);
                m[h] = mn;
                y[h] = yn;
#pragma unroll
                for (int k = 0; k < CH; ++k) {
                    o[k][b][e] *= scale;
                    o[k][b][e + 2] *= scale;
                }
            }
        }
#pragma unroll
        for (int h = 0; h < OWN; ++h) {
            const int b = h / 2, e = h % 2;
            const float up = BASE - (y[h] == -INFINITY ? 0.f : y[h]);
#pragma unroll
            for (int n = 0; n < MB; ++n)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    l[h] += ex2(z[n][b][2 * u + e]);
                    s[n][b][2 * u + e] = ex2(z[n][b][2 * u + e] + (ve[n][u] + up));
                }
        }
        // the weights as the products' columns: by heads, not by keys
        unsigned p[MB][NB][NP][2];
#pragma unroll
        for (int n = 0; n < MB; ++n)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float a = s[n][b][2 * u], d = s[n][b][2 * u + 1];
                    const unsigned w = pack_f16(a, d);
                    p[n][b][0][u] = transposed(w);
                    if constexpr (SPLIT) {
                        const float2 got = __half22float2(*reinterpret_cast<const __half2*>(&w));
                        p[n][b][NP - 1][u] = transposed(pack_f16(a - got.x, d - got.y));
                    }
                }
        // a lane's word of a transposed load: positions 2 t and 2 t + 1, elements 2 r and 2 r + 1 of the chunk, the
        // instruction's rows r and r + 8
#pragma unroll
        for (int n = 0; n < MB; ++n) {
            const int row = 16 * n + (mi & 1) * 8 + r8;
#pragma unroll
            for (int k = 0; k < CH; k += 2) {
                unsigned w[4];  // chunk k: positions 0 - 7, 8 - 15; chunk k + 1
                ldm4t(stage + (ROWS + row) * HD + (pa_chunk<CH>(row, k + (mi >> 1)) << 4), w);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    unsigned a[4];
                    e4m3_f16(__byte_perm(w[2 * i], 0, 0x3120), a[0], a[1]);
                    e4m3_f16(__byte_perm(w[2 * i + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int z = 0; z < NP; ++z) mma_f16(o[k + i][b], a, p[n][b][z][0], p[n][b][z][1]);
                }
            }
        }
    }

    // whole sums over the warp's keys
    __device__ __forceinline__ void finish()
    {
#pragma unroll
        for (int h = 0; h < OWN; ++h)
            for (int d = 4; d < 32; d *= 2) l[h] += __shfl_xor_sync(0xffffffffu, l[h], d);
    }

    __device__ __forceinline__ void write(float* piece)
    {
        const int lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
#pragma unroll
        for (int h = 0; h < OWN; ++h) {
            const int b = h / 2, e = h % 2;
            // 2^(Y - BASE) in two factors: as one it would be subnormal, with few bits, where Y is next to -126
            const float by = exp2f(y[h]), base = 0x1p-11f;
            static_assert(BASE == 11.f, "the other factor");
#pragma unroll
            for (int k = 0; k < CH; ++k)
                *reinterpret_cast<float2*>(piece + pa_at<HD>((8 * b + 2 * t + e) * HD + 16 * k + 2 * r)) =
                    make_float2(o[k][b][e] * base * by, o[k][b][2 + e] * base * by);
        }
    }
    __device__ __forceinline__ int own_row(int h) const { return 8 * (h / 2) + 2 * (threadIdx.x & 3) + h % 2; }
    __device__ __forceinline__ bool owner() const { return (threadIdx.x & 31) < 4; }
};

// What bounds the loop is not one unit but the latency of its instructions (conversions, products, the softmax), so as many
// warps as their registers allow, against 32 rows a tile: 4 sequences of up to 131072, 8 kv heads of 128, 64 query heads 115 us
// (100 us at the measured copy rate), with two blocks per SM 8 us more, with four and tiles of 16 rows 16 more; 32 of up to 8192, 32
// query heads, pages of 16, 60 us, 7 more either way; in fp32 the first 122 us, 13 more with two blocks; heads of 64 40.5 us, 15
// more with two blocks.  The look at the rows of exponent 0 and the scores' own size are 1 us of the 60.
template <typename T_, int HD_, int NB, bool SHARED_ = false>
struct PaKindE4m3 {
    using T = T_;
    using State = PaE4m3<T_, HD_, NB>;
    static constexpr int HD = HD_, GM = State::GM, CE = 1, ROWS = State::ROWS, STAGES = 2, Q = 0;
    static constexpr int BLOCKS = NB == 2 ? 2 : HD == 64 && !State::SPLIT ? 4 : 3;  // per SM
    static constexpr int ITEM = 1;  // (1, 2 and 4: 64 sequences of up to 1000, 24 + 8 heads of 64 in fp32 19.8, 20.3 and 20.5 us)
    static constexpr bool QUANT = true, SHARED = SHARED_;
};

// Of any kind above, with the items' ends
inline size_t quant_workspace(int hd)
{
    const size_t a = pa_workspace(8, hd, 4) + pa_fronts(8, hd, 4), b = pa_workspace(16, hd, 2) + pa_fronts(16, hd, 2);
    return a > b ? a : b;
}

inline PaArgs quant_args(const mfs_quant_kv* c)
{
    PaArgs A = {};
    A.C = cache_of(&c->kv);
    A.kx = c->k_exp;
    A.vx = c->v_exp;
    A.x_page = c->exp_page_stride;
    A.x_head = c->exp_head_stride;
    A.x_row = c->exp_row_stride;
    return A;
}

}  // namespace
