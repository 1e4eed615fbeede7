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

// The codes go to the matrix instruction as fp16, which holds each exactly and takes one conversion for two of them (bf16
// would take several); the rows' powers of two never meet the elements: a key's multiplies its scores, a value's goes into
// its weights.
//
// Queries: q = q' / f with a power of two f for each head that brings its largest element to [2^14, 2^15), so that fp16
// loses nothing above 2^-39 of it.  bf16 queries are then exact: 16 heads, one a row of the instruction.  fp32 queries are
// two fp16 parts, 22 bits together: 8 heads, the first part in rows 0 - 7, the second in rows 8 - 15, which a lane holds
// both of.
//
// Weights: w_j 2^(e_j) with e_j the value's exponent, under a running maximum Y of log2 of that, times 2^14: so the weights'
// fp16 has its 11 bits for all that matter down to 2^-28 of the largest part of the output, and 2^-39 is lost, whatever the
// values' sizes.  fp32 queries: two parts again.  The sum of the weights is apart from this, in fp32 under the maximum of
// the scores alone.
template <typename T, int HD>
struct PaE4m3 {
    static constexpr bool SPLIT = sizeof(T) == 4;
    static constexpr int GM = SPLIT ? 8 : 16, ROWS = 32, NK = ROWS / 8, OWN = SPLIT ? 1 : 2;
    unsigned qf[HD / 16][4];
    float o[HD / 8][4], m[OWN], l[OWN], y[OWN], inv[OWN];  // m: in scores times 1 / inv until finish()

    __device__ __forceinline__ void begin(const PaArgs& A, const PaWalk& w, float*)
    {
        const int lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
        const int h0 = (w.hb / A.nhb) * A.g + (w.hb % A.nhb) * GM, nh = min(GM, A.g - (w.hb % A.nhb) * GM);
        const T* q = reinterpret_cast<const T*>(A.q) + (long long)w.s * A.q_stride + (long long)h0 * HD;
#pragma unroll
        for (int h = 0; h < OWN; ++h) {
            const int row = r + 8 * h;
            // a lane's elements of a row: 16 k + 4 t ..., the instruction's columns 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of step k
            float x[HD / 16][4];
            unsigned top = 0;
#pragma unroll
            for (int k = 0; k < HD / 16; ++k) {
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
                    const unsigned b = __float_as_uint(x[k][e]) & 0x7fffffffu;
                    if (b < 0x7f800000u) top = max(top, b);
                }
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const unsigned f = min(253u, 268u - (top >> 23));  // of 2^(f - 127)
            inv[h] = pow2_of(254u - f);
#pragma unroll
            for (int k = 0; k < HD / 16; ++k) {
                float z[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) z[e] = x[k][e] * pow2_of(f);
                qf[k][h] = pack_f16(z[0], z[1]);
                qf[k][h + 2] = pack_f16(z[2], z[3]);
                if constexpr (SPLIT) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float rest = z[e] - __half2float(__float2half_rn(z[e]));
                        z[e] = isfinite(z[e]) ? rest : 0.f;
                    }
                    qf[k][1] = pack_f16(z[0], z[1]);
                    qf[k][3] = pack_f16(z[2], z[3]);
                }
            }
            m[h] = y[h] = -INFINITY;
            l[h] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < HD / 8; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[j][x] = 0.f;
    }

    // x: exponents of the tile's 32 keys, then of its values
    __device__ __forceinline__ void tile(unsigned stage, int valid, float c, float*, const float*, const uint8_t* x)
    {
        constexpr int CH = HD / 16;
        const int lane = threadIdx.x & 31, t = lane & 3, mi = lane >> 3, r8 = lane & 7;
        float s[NK][4] = {};
#pragma unroll
        for (int n = 0; n < NK; ++n) {
            const int row = 8 * n + r8;
#pragma unroll
            for (int k = 0; k < CH; k += 4) {  // four steps of 16 elements of eight keys
                unsigned w[4];
                ldm4(stage + row * HD + (pa_chunk<CH>(row, k + mi) << 4), w);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    unsigned b0, b1;
                    e4m3_f16(w[i], b0, b1);
                    mma_f16(s[n], qf[k + i], b0, b1);
                }
            }
        }
        float ve[NK][2];  // exponents of the values (0 stands for no value at all)
#pragma unroll
        for (int n = 0; n < NK; ++n) {
            const unsigned kx = *reinterpret_cast<const unsigned short*>(x + 8 * n + 2 * t), vx = *reinterpret_cast<const unsigned short*>(x + 32 + 8 * n + 2 * t);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const unsigned kb = e ? kx >> 8 : kx & 255u, vb = e ? vx >> 8 : vx & 255u;
                const float by = pow2_of(kb);
                if constexpr (SPLIT) s[n][e] = (s[n][e] + s[n][e + 2]) * by;
                else { s[n][e] *= by; s[n][e + 2] *= by; }
                ve[n][e] = vb ? (float)((int)vb - 127) : -INFINITY;
            }
        }
        if (valid < ROWS) {
#pragma unroll
            for (int n = 0; n < NK; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (8 * n + 2 * t + e >= valid) {
                        s[n][e] = -INFINITY;
                        if (!SPLIT) s[n][e + 2] = -INFINITY;
                    }
        }
        float scale[OWN];
        unsigned p[NK / 2][4];
#pragma unroll
        for (int h = 0; h < OWN; ++h) {
            const float ch = c * inv[h];
            float v = -INFINITY;
#pragma unroll
            for (int n = 0; n < NK; ++n) v = fmaxf(v, fmaxf(s[n][2 * h], s[n][2 * h + 1]));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
            const float mn = fmaxf(m[h], v), sub = mn == -INFINITY ? 0.f : mn;  // scores of -infinity alone so far: weights 0, not NaN
            const float down = m[h] == mn ? 0.f : (m[h] - mn) * ch;
            float sum = 0.f, top = -INFINITY;
#pragma unroll
            for (int n = 0; n < NK; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float a = (s[n][2 * h + e] - sub) * ch;
                    sum += exp2f(a);
                    s[n][2 * h + e] = a + ve[n][e];
                    top = fmaxf(top, s[n][2 * h + e]);
                }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float was = y[h] + down, yn = fmaxf(was, top);
            scale[h] = was == yn ? 1.f : exp2f(was - yn);
            l[h] = l[h] * (down == 0.f ? 1.f : exp2f(down)) + sum;
            m[h] = mn;
            y[h] = yn;
            const float up = 14.f - (yn == -INFINITY ? 0.f : yn);
#pragma unroll
            for (int n = 0; n < NK; ++n) {
                const float a = exp2f(s[n][2 * h] + up), b = exp2f(s[n][2 * h + 1] + up);
                p[n / 2][2 * (n & 1) + h] = pack_f16(a, b);
                if constexpr (SPLIT) {
                    const float2 got = __half22float2(*reinterpret_cast<const __half2*>(&p[n / 2][2 * (n & 1)]));
                    p[n / 2][2 * (n & 1) + 1] = pack_f16(a - got.x, b - got.y);
                }
            }
        }
        if (__any_sync(0xffffffffu, scale[0] != 1.f || scale[OWN - 1] != 1.f)) {
#pragma unroll
            for (int j = 0; j < HD / 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[j][e] *= scale[SPLIT ? 0 : e >> 1];
        }
        // a lane's word of a transposed load: positions 2 t and 2 t + 1, elements 2 r and 2 r + 1 of the chunk; the even
        // elements make one product, the odd ones another
#pragma unroll
        for (int n = 0; n < NK / 2; ++n) {
            const int row = 16 * n + (mi & 1) * 8 + r8;
#pragma unroll
            for (int k = 0; k < CH; k += 2) {
                unsigned w[4];  // chunk k: positions 0 - 7, 8 - 15; chunk k + 1
                ldm4t(stage + (ROWS + row) * HD + (pa_chunk<CH>(row, k + (mi >> 1)) << 4), w);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    unsigned e0, o0, e1, o1;
                    e4m3_f16(__byte_perm(w[2 * i], 0, 0x3120), e0, o0);
                    e4m3_f16(__byte_perm(w[2 * i + 1], 0, 0x3120), e1, o1);
                    mma_f16(o[2 * (k + i)], p[n], e0, e1);
                    mma_f16(o[2 * (k + i) + 1], p[n], o0, o1);
                }
            }
        }
    }

    // whole sums over the quad's keys, in the scores' own scale
    __device__ __forceinline__ void finish()
    {
#pragma unroll
        for (int h = 0; h < OWN; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            m[h] *= inv[h];
        }
    }

    __device__ __forceinline__ void write(float* piece)
    {
        const int lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
#pragma unroll
        for (int h = 0; h < OWN; ++h) {
            const float by = exp2f(y[h] - 14.f);
#pragma unroll
            for (int k = 0; k < HD / 16; ++k) {
                float4 v;
                if constexpr (SPLIT)
                    v = make_float4(o[2 * k][0] + o[2 * k][2], o[2 * k + 1][0] + o[2 * k + 1][2], o[2 * k][1] + o[2 * k][3], o[2 * k + 1][1] + o[2 * k + 1][3]);
                else
                    v = make_float4(o[2 * k][2 * h], o[2 * k + 1][2 * h], o[2 * k][2 * h + 1], o[2 * k + 1][2 * h + 1]);
                *reinterpret_cast<float4*>(piece + pa_at<HD>((r + 8 * h) * HD + 16 * k + 4 * t)) = make_float4(v.x * by, v.y * by, v.z * by, v.w * by);
            }
        }
    }
    __device__ __forceinline__ int own_row(int h) const { return ((threadIdx.x & 31) >> 2) + 8 * h; }
    __device__ __forceinline__ bool owner() const { return (threadIdx.x & 3) == 0; }
};

// A warp's ring holds 16 KB as the others' does: two tiles, or four of heads of 64.
template <typename T_, int HD_, bool SHARED_ = false>
struct PaKindE4m3 {
    using T = T_;
    using State = PaE4m3<T_, HD_>;
    static constexpr int HD = HD_, GM = State::GM, CE = 1, ROWS = 32, STAGES = 256 / HD, Q = 0;
    static constexpr bool QUANT = true, SHARED = SHARED_;
};

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
