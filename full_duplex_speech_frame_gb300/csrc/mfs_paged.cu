// Paged key/value cache: mfs_kv_append (rotate and write new tokens) and
// mfs_paged_attention (one new token per sequence).
#include "mfs_paged.cuh"

namespace {

// ------------------------------------------------------------------ append

struct Turns {
    double f[64];  // turns per position of pair i: theta^(-2 i / head_dim) / (2 pi)
};

// A block takes a few tokens: one warp per token finds its sequence, position and row in the cache, and the cosines and
// sines of its angles; the block's threads then move items of two 16-byte vectors that hold whole pairs (neighbours for
// interleaved pairs, half a head apart for split ones), the next one on its way while one is rotated, the first while
// the angles are found.  What bounds it is memory: each input is read and each output written once.  8192 tokens of 32 + 8
// heads of 128 bf16: 39 us, 0.83 of the measured copy rate; blocks of 256 threads and 4 tokens 40 us, three items on
// their way per thread (fewer blocks on an SM) 45 us, 8 tokens 45 us.  The same in fp32: 77 us, 0.84.
constexpr int AP_THREADS = 128;
// 8-bit caches: 8192 tokens, half of each head rotated, 41 us for 201 MB, 0.72 of the copy rate (all of it 51 us); the row's maximum is
// three or four exchanges, and the conversion makes it issue 60 % of the time (64 registers, eight blocks per SM; 48 and ten with
// spills 25 us more).  In fp32 63 us for 386 MB, 0.91 (all of it 65 us).  A partial rotation into a plain cache: 38 us, 0.84; fp32 71 us, 0.90.
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
    // a rotation of part of the head, and its magnitude
    int dims;
    float magnitude;
    // 8-bit caches: an exponent per row
    uint8_t *kx, *vx;
    long long x_page, x_head, x_row;
};

template <typename T>
struct Vec2 {
    uint4 a, b;
};

// Sequence and position of token t, for a whole warp; false: it belongs to no sequence.
__device__ __forceinline__ bool token_place(const int32_t* cu, const int32_t* kv_len, int n_seqs, int t, int& s, long long& pos)
{
    // the last s with cu[s] <= token, 32 places at a time
    const int lane = threadIdx.x & 31;
    int lo = 0, size = n_seqs;
    while (size > 1) {
        const int step = (size + 31) / 32, at = lane * step;
        const unsigned m = __ballot_sync(0xffffffffu, at < size && __ldg(cu + lo + at) <= t);
        const int c = max(0, 31 - __clz(m));  // the last probe that is not past the token
        lo += c * step;
        size = min(step, size - c * step);
    }
    const int begin = __ldg(cu + lo), end = __ldg(cu + lo + 1);
    s = lo;
    pos = (long long)__ldg(kv_len + lo) - end + t;
    return t >= begin && t < end;
}

// Four values as e4m3, nearest, ties to even; past 448: 448.
__device__ __forceinline__ unsigned to_e4m3(float a, float b, float c, float d)
{
    unsigned short lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (unsigned)hi << 16 | lo;
}

// MODE 0: the cache has the type of k and v, whole heads are rotated.  1: the same, with a rotation of part of the head or
// a magnitude.  2: as 1, and the cache has 8 bits: the lanes that share a row find its largest value, and from it the
// exponent; the key is quantised as rotated in 32 bits, not as rounded for k_out.
template <typename T, int HD, int TT, int MODE>
__global__ void __launch_bounds__(AP_THREADS, MODE == 2 ? 8 : 10) append_kernel(const __grid_constant__ ApArgs<T> A)
{
    constexpr int VE = 16 / sizeof(T);        // elements per vector
    constexpr int IPH = HD / (2 * VE);        // items per head
    __shared__ float2 cs[TT][HD / 2];
    __shared__ long long row[TT];             // element offset of the token's row (head 0) in the cache; -1: none; -2: no token
    __shared__ long long xrow[MODE == 2 ? TT : 1];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int t0 = blockIdx.x * TT, nt = min(TT, A.n_tokens - t0);
    const int hkv = A.C.n_kv_heads, heads = A.hq + 2 * hkv, items = nt * heads * IPH;
    const bool split = A.rope == MFS_ROPE_HALF;
    const int HALF = MODE ? A.dims / 2 : HD / 2, turned = MODE ? A.dims / (2 * VE) : IPH;  // items of a head that are rotated

    // item i: token, head (queries, keys, values), place within the head
    auto where = [&](int i, int& t, int& h, int& e) {
        const int hh = i / IPH;
        e = i % IPH;
        t = TT == 1 ? 0 : hh / heads;
        h = TT == 1 ? hh : hh - t * heads;
    };
    auto vectors = [&](int e, int& first, int& second) {
        const bool apart = split && (MODE == 0 || e < turned);
        first = apart ? e * VE : 2 * e * VE;
        second = apart ? first + HALF : first + VE;
    };
    auto source = [&](int i) {
        int t, h, e, first, second;
        where(i, t, h, e);
        const long long tok = t0 + t;
        const T* p = h < A.hq ? A.q + tok * A.q_stride + h * HD : h < A.hq + hkv ? A.k + tok * A.k_stride + (h - A.hq) * HD
                                                                              : A.v + tok * A.v_stride + (h - A.hq - hkv) * HD;
        vectors(e, first, second);
        // plain loads: the queries and keys may be their own outputs
        return Vec2<T>{*reinterpret_cast<const uint4*>(p + first), *reinterpret_cast<const uint4*>(p + second)};
    };
    // MODE 1, 2: few tokens' items are dealt to several blocks each
    const int begin = MODE ? blockIdx.y * AP_THREADS + tid : tid, every = MODE ? gridDim.y * AP_THREADS : AP_THREADS;
    Vec2<T> x;
    if (begin < items) x = source(begin);

    if (warp < nt) {
        int s, page = 0, r = 0;
        long long pos;
        const bool is = token_place(A.cu, A.kv_len, A.n_seqs, t0 + warp, s, pos);
        if (lane == 0) {
            const bool has = is && pos >= 0 && pos <= 0x7fffffff && row_place(A.C, s, (int)pos, page, r);
            row[warp] = !is ? -2 : !has ? -1 : (long long)page * A.C.page_stride + (long long)r * A.C.row_stride;
            if (MODE == 2) xrow[warp] = (long long)page * A.x_page + (long long)r * A.x_row;
        }
        if (A.rope)
            for (int i = lane; i < HALF; i += 32) {
                // turns in 64 bits; what is left of one, up to half, in fp32: off by 2^-26 of a turn, 1e-7 in the cosine
                const double a = (double)pos * A.turns.f[i];
                float s, c;
                if (MODE == 2) {
                    // what fp32 leaves out of the angle and of the products with the magnitude is added: a key next to a border of
                    // its codes takes the wrong one less often
                    const double x = 2.0 * (a - rint(a));
                    const float hi = (float)x, d = 3.14159265f * (float)(x - hi) * A.magnitude;
                    sincospif(hi, &s, &c);
                    const float mc = A.magnitude * c, ms = A.magnitude * s;
                    cs[warp][i] = make_float2(mc + fmaf(-d, s, fmaf(A.magnitude, c, -mc)), ms + fmaf(d, c, fmaf(A.magnitude, s, -ms)));
                    continue;
                }
                sincospif(2.f * (float)(a - rint(a)), &s, &c);
                cs[warp][i] = MODE ? make_float2(c * A.magnitude, s * A.magnitude) : make_float2(c, s);
            }
    }
    __syncthreads();

    auto finish = [&](int i, Vec2<T> y) {
        int t, h, e, first, second;
        where(i, t, h, e);
        const long long r = row[t];
        if (r == -2) return;
        const long long tok = t0 + t;
        vectors(e, first, second);
        float f[2 * VE];  // MODE 2: the values, first vector and second
        if (MODE == 2) {
            T in[2 * VE];
            memcpy(in, &y, 32);
#pragma unroll
            for (int j = 0; j < 2 * VE; ++j) f[j] = to_f(in[j]);
        }
        if (h < A.hq + hkv && A.rope && (MODE == 0 || e < turned)) {
            T in[2 * VE], out[2 * VE];
            memcpy(in, &y, 32);
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                // pair j of the item: elements (j, j + VE) of the two vectors for split pairs, (2 j, 2 j + 1) for neighbours
                const float2 c = cs[t][e * VE + j];
                const float u = to_f(split ? in[j] : in[2 * j]), w = to_f(split ? in[j + VE] : in[2 * j + 1]);
                const float fa = u * c.x - w * c.y, fb = u * c.y + w * c.x;
                const T a = from_f<T>(fa), b = from_f<T>(fb);
                if (split) { out[j] = a; out[j + VE] = b; }
                else { out[2 * j] = a; out[2 * j + 1] = b; }
                if (MODE == 2) {
                    if (split) { f[j] = fa; f[j + VE] = fb; }
                    else { f[2 * j] = fa; f[2 * j + 1] = fb; }
                }
            }
            memcpy(&y, out, 32);
        }
        auto put = [&](T* p) {
            *reinterpret_cast<uint4*>(p + first) = y.a;
            *reinterpret_cast<uint4*>(p + second) = y.b;
        };
        if (h < A.hq) {
            put(A.q_out + tok * A.q_out_stride + h * HD);
            return;
        }
        const bool key = h < A.hq + hkv;
        const int hk = h - A.hq - (key ? 0 : hkv);
        if (key && A.k_out) put(A.k_out + tok * A.k_out_stride + hk * HD);
        if (r < 0) return;
        if constexpr (MODE == 2) {
            // the row's largest value as bits, which order a NaN above infinity above the rest
            unsigned top = 0;
#pragma unroll
            for (int j = 0; j < 2 * VE; ++j) top = max(top, __float_as_uint(f[j]) & 0x7fffffffu);
            const unsigned row_lanes = (unsigned)((1ull << IPH) - 1) << (lane & ~(IPH - 1));
#pragma unroll
            for (int d = 1; d < IPH; d *= 2) top = max(top, __shfl_xor_sync(row_lanes, top, d));
            // the least b with top <= 448 2^(b - 127), 448 = 1.75 x 2^8: 1 at least (and for subnormal rows), 0 for zeros
            int b = max(1, (int)(top >> 23) - ((top & 0x7fffffu) > 0x600000u ? 7 : 8));
            unsigned w[VE / 2];
            if (top >= 0x7f800000u) {  // not finite: the whole row is NaN
                b = 127;
#pragma unroll
                for (int j = 0; j < VE / 2; ++j) w[j] = 0x7f7f7f7fu;
            } else {
                const float by = __uint_as_float((unsigned)(254 - b) << 23);  // 2^(127 - b)
#pragma unroll
                for (int j = 0; j < VE / 2; ++j) w[j] = to_e4m3(f[4 * j] * by, f[4 * j + 1] * by, f[4 * j + 2] * by, f[4 * j + 3] * by);
                if (top == 0) b = 0;
            }
            char* c = (key ? A.C.k : A.C.v) + r + (long long)hk * A.C.head_stride;
            if constexpr (VE == 8) {
                *reinterpret_cast<uint2*>(c + first) = make_uint2(w[0], w[1]);
                *reinterpret_cast<uint2*>(c + second) = make_uint2(w[2], w[3]);
            } else {
                *reinterpret_cast<unsigned*>(c + first) = w[0];
                *reinterpret_cast<unsigned*>(c + second) = w[1];
            }
            if (e == 0) (key ? A.kx : A.vx)[xrow[t] + (long long)hk * A.x_head] = (uint8_t)b;
        } else {
            put(reinterpret_cast<T*>(key ? A.C.k : A.C.v) + r + (long long)hk * A.C.head_stride);
        }
    };
    for (int i = begin; i < items; i += every) {
        const Vec2<T> y = x;
        if (i + every < items) x = source(i + every);
        finish(i, y);
    }
}

template <typename T, int HD, int MODE>
int append(const ApArgs<T>& A, cudaStream_t st)
{
    int sms = 0;
    static mfs::PerDevice ready;
    cudaError_t e = mfs::op_device(ready, nullptr, 0, &sms);
    if (e == cudaSuccess) {
        // as many blocks for a token as its items fill, up to eight per SM in all
        const long long items = (long long)(A.hq + 2 * A.C.n_kv_heads) * (HD * (int)sizeof(T) / 32), most = (items - 1) / AP_THREADS + 1;
        const long long room = 8LL * sms / (A.n_tokens > 0 ? A.n_tokens : 1);
        const unsigned each = MODE == 0 || room < 2 ? 1u : (unsigned)(room < most ? room : most);
        // (8-bit caches: 8192 tokens of 32 + 8 heads and their reading back 54 us by ones, 57 us by twos)
        constexpr int TOKENS = MODE == 2 ? 1 : AP_TOKENS;
        if (A.n_tokens <= 8 * sms || TOKENS == 1) append_kernel<T, HD, 1, MODE><<<dim3(A.n_tokens, each), AP_THREADS, 0, st>>>(A);
        else append_kernel<T, HD, TOKENS, MODE><<<(A.n_tokens + TOKENS - 1) / TOKENS, AP_THREADS, 0, st>>>(A);
        e = cudaGetLastError();
    }
    return mfs::op_launched("kv_append", e);
}

// The arguments of an append, and all entry points' checks of them.
struct Append {
    int n_tokens, n_seqs;
    const int32_t *cu, *kv_len;
    const void* q;
    long long q_stride;
    int n_q_heads;
    void* q_out;
    long long q_out_stride;
    const void* k;
    long long k_stride;
    void* k_out;
    long long k_out_stride;
    const void* v;
    long long v_stride;
};

template <typename T>
ApArgs<T> append_args(const Append& P, const Cache& C, int rope)
{
    ApArgs<T> A = {};
    A.C = C;
    A.cu = P.cu; A.kv_len = P.kv_len;
    A.q = (const T*)P.q; A.k = (const T*)P.k; A.v = (const T*)P.v;
    A.q_out = (T*)P.q_out; A.k_out = (T*)P.k_out;
    A.q_stride = P.q_stride; A.q_out_stride = P.q_out_stride; A.k_stride = P.k_stride; A.k_out_stride = P.k_out_stride;
    A.v_stride = P.v_stride;
    A.n_tokens = P.n_tokens; A.n_seqs = P.n_seqs; A.hq = P.q ? P.n_q_heads : 0; A.rope = rope;
    A.magnitude = 1.f;
    return A;
}

// 0: go on; 1: nothing to do; else an error's code
int append_checks(const Append& P, int hkv, int hd, int elem)
{
    const char* op = "kv_append";
    if (P.n_tokens == 0 || P.n_seqs == 0) return 1;
    if (!P.cu || !P.kv_len || !P.k || !P.v) return mfs::op_fail(MFS_E_ARG, op, "null cu, kv_len, k or v");
    if ((P.q != nullptr) != (P.q_out != nullptr)) return mfs::op_fail(MFS_E_ARG, op, "q and q_out go together");
    if (P.q && (P.n_q_heads < 1 || P.n_q_heads > MFS_MAX_HEADS)) return mfs::op_fail(MFS_E_ARG, op, "n_q_heads outside [1, 65535]");
    if (!mfs::rows_ok(P.k, P.k_stride, hkv, hd, elem) || !mfs::rows_ok(P.v, P.v_stride, hkv, hd, elem) ||
        (P.k_out && !mfs::rows_ok(P.k_out, P.k_out_stride, hkv, hd, elem)) ||
        (P.q && (!mfs::rows_ok(P.q, P.q_stride, P.n_q_heads, hd, elem) || !mfs::rows_ok(P.q_out, P.q_out_stride, P.n_q_heads, hd, elem))))
        return mfs::op_fail(MFS_E_ARG, op, "pointers and token strides must be multiples of 16 bytes, a stride at least heads x head_dim");
    return 0;
}

// theta^(-2 i / dims) in turns: powers of the first ratio, each the product of two before it: at most 7 roundings of 2^-53,
// where 64 calls of pow cost the caller 2 us
void rope_turns(Turns& turns, double theta, int dims)
{
    turns.f[0] = 1.0;
    for (int b = 1; b < dims / 2; b *= 2) {
        turns.f[b] = pow(theta, -2.0 * b / dims);
        for (int i = 1; i < b && b + i < dims / 2; ++i) turns.f[b + i] = turns.f[b] * turns.f[i];
    }
    for (int i = 0; i < dims / 2; ++i) turns.f[i] /= 6.283185307179586476925;
}

// Rotation of the first `dims` elements, slower where it turns less than `high` times over the original length.
template <typename T>
void rope_of(ApArgs<T>& A, const mfs_rope* r, int hd)
{
    A.rope = r ? r->layout : MFS_ROPE_NONE;
    if (A.rope == MFS_ROPE_NONE) return;
    A.dims = r->dims ? r->dims : hd;
    A.magnitude = (float)r->magnitude;
    rope_turns(A.turns, r->theta, A.dims);
    for (int i = 0; i < A.dims / 2; ++i) {
        double kept = 0.0;
        if (r->original > 0.0) {
            kept = (A.turns.f[i] * r->original - r->low) / (r->high - r->low);
            kept = kept < 0.0 ? 0.0 : kept > 1.0 ? 1.0 : kept;
        }
        A.turns.f[i] *= kept + (1.0 - kept) / r->factor;
    }
}

template <typename T>
int append_ropes(const Append& P, const Cache& C, int hd, const mfs_rope* rope, const mfs_quant_kv* quant, cudaStream_t st)
{
    ApArgs<T> A = append_args<T>(P, C, MFS_ROPE_NONE);
    rope_of(A, rope, hd);
    if (quant) {
        A.kx = quant->k_exp; A.vx = quant->v_exp;
        A.x_page = quant->exp_page_stride; A.x_head = quant->exp_head_stride; A.x_row = quant->exp_row_stride;
        return hd == 128 ? append<T, 128, 2>(A, st) : append<T, 64, 2>(A, st);
    }
    return hd == 128 ? append<T, 128, 1>(A, st) : append<T, 64, 1>(A, st);
}

// -------------------------------------------------------------------- read

// The last rows of each sequence, packed: a block takes a few tokens (64 or 256 rows of keys and values), then others,
// until there are none.  A warp for each token finds its place, which takes several dependent reads, while the rows of the
// tokens before are on their way.
constexpr int RD_THREADS = 256, RD_TOKENS = 8, RD_BLOCKS = 8;
// Rows of a turn: 64 where the call has few, 256 else: 3000 tokens of 32 heads of 128 to bf16 18 us (20 by 256), 8 tokens with
// their append 8.9 (13.0); 131 000 of 8 heads 158 us = 5.3 TB/s, two thirds of it written, 0.78 of the measured copy rate (179 by
// 64).  What bounds it is memory; with items of 16 bytes it was the instructions that find an item's place (issue 70 %, 170 us).
constexpr int RD_FEW = 64, RD_MANY = 256;

struct RdArgs {
    Cache C;
    const int32_t *cu, *kv_len;
    char *k, *v;                    // out
    long long k_stride, v_stride;   // bytes
    int n_tokens, n_seqs;
    int tokens;        // of a block
    unsigned inverse;  // 2^32 / (2 n_kv_heads), rounded up: exact for the rows of a block, which are fewer than 2^16 where tokens > 1
    const uint8_t *kx, *vx;
    long long x_page, x_head, x_row;
};

// Four e4m3 codes under 2^(b - 127); b = 0: codes of 0
__device__ __forceinline__ float4 from_e4m3(unsigned w, unsigned b)
{
    unsigned lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}" : "=r"(lo), "=r"(hi) : "r"(w));
    const float by = __uint_as_float(b << 23);
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo)), y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return make_float4(x.x * by, x.y * by, y.x * by, y.y * by);
}

// T: of the output; the cache has the same, or 8 bits (QUANT).  An item is 32 bytes of output, and pairs of lanes exchange halves
// of theirs, so that each store writes whole sectors.
template <typename T, int HD, bool QUANT>
__global__ void __launch_bounds__(RD_THREADS, RD_BLOCKS) read_kernel(const __grid_constant__ RdArgs A)
{
    constexpr int VE = 32 / sizeof(T), IPH = HD / VE;  // elements of an item, items per row
    constexpr int CE = QUANT ? 1 : sizeof(T);
    static_assert(IPH >= 2 && IPH % 2 == 0, "a pair of lanes has two items of a row");
    __shared__ long long places[2][2][RD_TOKENS];  // of this turn's tokens and the next's: row -1: none, -2: no token; exponents
    __shared__ uint4 zeros;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, hkv = A.C.n_kv_heads;
    if (tid == 0) zeros = make_uint4(0u, 0u, 0u, 0u);
    auto look_up = [&](int t0, int turn) {
        if (warp >= A.tokens || t0 + warp >= A.n_tokens) return;
        int s, page = 0, r = 0;
        long long pos;
        const bool is = token_place(A.cu, A.kv_len, A.n_seqs, t0 + warp, s, pos);
        if (lane == 0) {
            const bool has = is && pos >= 0 && pos <= 0x7fffffff && row_place(A.C, s, (int)pos, page, r);
            places[turn][0][warp] = !is ? -2 : !has ? -1 : (long long)page * A.C.page_stride + (long long)r * A.C.row_stride;
            places[turn][1][warp] = (long long)page * A.x_page + (long long)r * A.x_row;
        }
    };
    long long t0 = (long long)blockIdx.x * A.tokens;
    const long long ahead = (long long)gridDim.x * A.tokens;
    look_up((int)t0, 0);
    __syncthreads();
    for (int turn = 0; t0 < A.n_tokens; t0 += ahead, turn ^= 1) {
        const long long *row = places[turn][0], *xrow = places[turn][1];
        const int nt = (int)min((long long)A.tokens, A.n_tokens - t0);
        bool found = t0 + ahead >= A.n_tokens;  // the next tokens' places
        // rows of a token: keys of all heads, then values; a thread has item e of every RD_THREADS / IPH-th row
        const int rows = nt * 2 * hkv, e = tid % IPH;
        const bool odd = lane & 1;
        for (int i = tid / IPH; i < rows || !found; i += RD_THREADS / IPH) {
            uint4 x[QUANT ? 1 : 2];
            unsigned b = 127;
            char* out = nullptr;  // of the pair's two items; null: nothing to write
            if (i < rows) {
                const int t = A.tokens == 1 ? 0 : (int)__umulhi((unsigned)i, A.inverse), h2 = i - t * 2 * hkv;
                const bool key = h2 < hkv;
                const int h = key ? h2 : h2 - hkv;
                const long long r = row[t];
                if (r != -2) out = (key ? A.k + (t0 + t) * A.k_stride : A.v + (t0 + t) * A.v_stride) + (long long)h * HD * sizeof(T) + (e & ~1) * 32;
                if (r == -1) {  // no page: NaN
                    const unsigned nan = QUANT ? 0x7f7f7f7fu : sizeof(T) == 2 ? 0x7fc07fc0u : 0x7fc00000u;
                    x[0] = x[QUANT ? 0 : 1] = make_uint4(nan, nan, nan, nan);
                } else if (r >= 0) {
                    const char* p = (key ? A.C.k : A.C.v) + (r + (long long)h * A.C.head_stride + e * VE) * CE;
                    if constexpr (!QUANT) {
                        x[0] = __ldg(reinterpret_cast<const uint4*>(p));
                        x[1] = __ldg(reinterpret_cast<const uint4*>(p) + 1);
                    } else {
                        if constexpr (VE == 16) {
                            x[0] = __ldg(reinterpret_cast<const uint4*>(p));
                        } else {
                            const uint2 y = __ldg(reinterpret_cast<const uint2*>(p));
                            x[0].x = y.x;
                            x[0].y = y.y;
                        }
                        b = __ldg((key ? A.kx : A.vx) + xrow[t] + (long long)h * A.x_head);
                    }
                }
            }
            if (!found) look_up((int)(t0 + ahead), turn ^ 1);
            found = true;
            if (!out) continue;  // (the same in both lanes of a pair)
            uint4 y[2];
            if constexpr (!QUANT) {
                y[0] = x[0];
                y[1] = x[1];
            } else {
                const float4 f = from_e4m3(x[0].x, b), g = from_e4m3(x[0].y, b);
                if constexpr (VE == 16) {
                    const float4 u = from_e4m3(x[0].z, b), v = from_e4m3(x[0].w, b);
                    y[0] = make_uint4(pack_bf16(f.x, f.y), pack_bf16(f.z, f.w), pack_bf16(g.x, g.y), pack_bf16(g.z, g.w));
                    y[1] = make_uint4(pack_bf16(u.x, u.y), pack_bf16(u.z, u.w), pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
                } else {
                    memcpy(&y[0], &f, 16);
                    memcpy(&y[1], &g, 16);
                }
            }
            if (QUANT && b == 0) y[0] = y[1] = zeros;  // a row of zeros, codes of NaN among its too (by loads: two instructions, not eight)
            // the even lane's second half for the odd one's first
            const unsigned both = 3u << (lane & ~1);
            const uint4 give = odd ? y[0] : y[1];
            uint4 got;
            got.x = __shfl_xor_sync(both, give.x, 1);
            got.y = __shfl_xor_sync(both, give.y, 1);
            got.z = __shfl_xor_sync(both, give.z, 1);
            got.w = __shfl_xor_sync(both, give.w, 1);
            uint4* o = reinterpret_cast<uint4*>(out) + odd;
            o[0] = odd ? got : y[0];
            o[2] = odd ? y[1] : got;
        }
        __syncthreads();
    }
}

template <typename T, bool QUANT>
int read_rows(RdArgs A, int hd, cudaStream_t st)
{
    const int rows = 2 * A.C.n_kv_heads, most = (long long)A.n_tokens * rows <= 4096 * RD_FEW ? RD_FEW : RD_MANY;
    A.tokens = rows >= most ? 1 : most / rows < RD_TOKENS ? most / rows : RD_TOKENS;
    A.inverse = (unsigned)(((1ull << 32) + rows - 1) / rows);
    int sms = 0;
    static mfs::PerDevice known;
    const cudaError_t e = mfs::op_device(known, nullptr, 0, &sms);
    if (e != cudaSuccess) return mfs::op_launched("kv_read", e);
    const int turns = (A.n_tokens - 1) / A.tokens + 1, blocks = turns < RD_BLOCKS * sms ? turns : RD_BLOCKS * sms;
    if (hd == 128) read_kernel<T, 128, QUANT><<<blocks, RD_THREADS, 0, st>>>(A);
    else read_kernel<T, 64, QUANT><<<blocks, RD_THREADS, 0, st>>>(A);
    return mfs::op_launched("kv_read", cudaGetLastError());
}

int read_checked(const mfs_paged_kv* cache, const mfs_quant_kv* quant, int dtype, int n_tokens, int n_seqs, const int32_t* cu,
                 const int32_t* kv_len, void* k_out, long long k_stride, void* v_out, long long v_stride, void* cuda_stream)
{
    const char* op = "kv_read";
    if (dtype != MFS_DTYPE_F32 && dtype != MFS_DTYPE_BF16) return mfs::op_fail(MFS_E_ARG, op, "dtype must be fp32 or bf16");
    if (n_tokens < 0 || n_seqs < 0) return mfs::op_fail(MFS_E_ARG, op, "need n_tokens >= 0 and n_seqs >= 0");
    if (n_tokens == 0 || n_seqs == 0) return MFS_OK;
    if (!cu || !kv_len || !k_out || !v_out) return mfs::op_fail(MFS_E_ARG, op, "null cu, kv_len, k_out or v_out");
    const int hd = cache->head_dim, elem = dtype == MFS_DTYPE_BF16 ? 2 : 4;
    if (!mfs::rows_ok(k_out, k_stride, cache->n_kv_heads, hd, elem) || !mfs::rows_ok(v_out, v_stride, cache->n_kv_heads, hd, elem))
        return mfs::op_fail(MFS_E_ARG, op, "pointers and token strides must be multiples of 16 bytes, a stride at least heads x head_dim");
    RdArgs A = {};
    A.C = cache_of(cache);
    A.cu = cu; A.kv_len = kv_len;
    A.k = (char*)k_out; A.v = (char*)v_out;
    A.k_stride = k_stride * elem; A.v_stride = v_stride * elem;
    A.n_tokens = n_tokens; A.n_seqs = n_seqs;
    cudaStream_t st = (cudaStream_t)cuda_stream;
    if (quant) {
        A.kx = quant->k_exp; A.vx = quant->v_exp;
        A.x_page = quant->exp_page_stride; A.x_head = quant->exp_head_stride; A.x_row = quant->exp_row_stride;
        return dtype == MFS_DTYPE_BF16 ? read_rows<bf16, true>(A, hd, st) : read_rows<float, true>(A, hd, st);
    }
    return dtype == MFS_DTYPE_BF16 ? read_rows<bf16, false>(A, hd, st) : read_rows<float, false>(A, hd, st);
}

size_t attention_workspace(int dtype, int hd)
{
    const size_t gm = dtype == MFS_DTYPE_BF16 ? PA_GM_MAX<bf16> : PA_GM_MAX<float>;
    return pa_workspace((int)gm, hd);
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
    const Append P = {n_tokens, n_seqs, cu, kv_len, q, q_stride, n_q_heads, q_out, q_out_stride, k, k_stride, k_out, k_out_stride, v, v_stride};
    const int hd = cache->head_dim;
    if (const int rc = append_checks(P, cache->n_kv_heads, hd, cache->dtype == MFS_DTYPE_BF16 ? 2 : 4)) return rc < 0 ? rc : MFS_OK;
    Turns turns = {};
    if (rope) rope_turns(turns, theta, hd);
    cudaStream_t st = (cudaStream_t)cuda_stream;
    auto typed = [&](auto zero) {
        using T = decltype(zero);
        ApArgs<T> A = append_args<T>(P, cache_of(cache), rope);
        A.turns = turns;
        return hd == 128 ? append<T, 128, 0>(A, st) : append<T, 64, 0>(A, st);
    };
    return cache->dtype == MFS_DTYPE_BF16 ? typed(bf16()) : typed(0.f);
}

extern "C" int mfs_kv_append_rope(const mfs_paged_kv* cache, int n_tokens, int n_seqs, const int32_t* cu, const int32_t* kv_len,
                                  const void* q, long long q_stride, int n_q_heads, void* q_out, long long q_out_stride,
                                  const void* k, long long k_stride, void* k_out, long long k_out_stride, const void* v,
                                  long long v_stride, const mfs_rope* rope, void* cuda_stream)
{
    const char* op = "kv_append";
    if (const char* why = mfs::paged_kv_problem(cache)) return mfs::op_fail(MFS_E_ARG, op, why);
    if (n_tokens < 0 || n_seqs < 0) return mfs::op_fail(MFS_E_ARG, op, "need n_tokens >= 0 and n_seqs >= 0");
    if (const char* why = mfs::rope_problem(rope, cache->head_dim)) return mfs::op_fail(MFS_E_ARG, op, why);
    const Append P = {n_tokens, n_seqs, cu, kv_len, q, q_stride, n_q_heads, q_out, q_out_stride, k, k_stride, k_out, k_out_stride, v, v_stride};
    if (const int rc = append_checks(P, cache->n_kv_heads, cache->head_dim, cache->dtype == MFS_DTYPE_BF16 ? 2 : 4)) return rc < 0 ? rc : MFS_OK;
    cudaStream_t st = (cudaStream_t)cuda_stream;
    return cache->dtype == MFS_DTYPE_BF16 ? append_ropes<bf16>(P, cache_of(cache), cache->head_dim, rope, nullptr, st)
                                          : append_ropes<float>(P, cache_of(cache), cache->head_dim, rope, nullptr, st);
}

extern "C" int mfs_quant_append(const mfs_quant_kv* cache, int dtype, int n_tokens, int n_seqs, const int32_t* cu, const int32_t* kv_len,
                                const void* q, long long q_stride, int n_q_heads, void* q_out, long long q_out_stride,
                                const void* k, long long k_stride, void* k_out, long long k_out_stride, const void* v,
                                long long v_stride, const mfs_rope* rope, void* cuda_stream)
{
    const char* op = "kv_append";
    if (const char* why = mfs::quant_kv_problem(cache)) return mfs::op_fail(MFS_E_ARG, op, why);
    if (dtype != MFS_DTYPE_F32 && dtype != MFS_DTYPE_BF16) return mfs::op_fail(MFS_E_ARG, op, "dtype must be fp32 or bf16");
    if (n_tokens < 0 || n_seqs < 0) return mfs::op_fail(MFS_E_ARG, op, "need n_tokens >= 0 and n_seqs >= 0");
    const int hd = cache->kv.head_dim;
    if (const char* why = mfs::rope_problem(rope, hd)) return mfs::op_fail(MFS_E_ARG, op, why);
    const Append P = {n_tokens, n_seqs, cu, kv_len, q, q_stride, n_q_heads, q_out, q_out_stride, k, k_stride, k_out, k_out_stride, v, v_stride};
    if (const int rc = append_checks(P, cache->kv.n_kv_heads, hd, dtype == MFS_DTYPE_BF16 ? 2 : 4)) return rc < 0 ? rc : MFS_OK;
    cudaStream_t st = (cudaStream_t)cuda_stream;
    return dtype == MFS_DTYPE_BF16 ? append_ropes<bf16>(P, cache_of(&cache->kv), hd, rope, cache, st)
                                   : append_ropes<float>(P, cache_of(&cache->kv), hd, rope, cache, st);
}

extern "C" int mfs_kv_read(const mfs_paged_kv* cache, int n_tokens, int n_seqs, const int32_t* cu, const int32_t* kv_len, void* k_out,
                           long long k_stride, void* v_out, long long v_stride, void* cuda_stream)
{
    if (const char* why = mfs::paged_kv_problem(cache)) return mfs::op_fail(MFS_E_ARG, "kv_read", why);
    return read_checked(cache, nullptr, cache->dtype, n_tokens, n_seqs, cu, kv_len, k_out, k_stride, v_out, v_stride, cuda_stream);
}

extern "C" int mfs_quant_read(const mfs_quant_kv* cache, int dtype, int n_tokens, int n_seqs, const int32_t* cu, const int32_t* kv_len,
                              void* k_out, long long k_stride, void* v_out, long long v_stride, void* cuda_stream)
{
    if (const char* why = mfs::quant_kv_problem(cache)) return mfs::op_fail(MFS_E_ARG, "kv_read", why);
    return read_checked(&cache->kv, cache, dtype, n_tokens, n_seqs, cu, kv_len, k_out, k_stride, v_out, v_stride, cuda_stream);
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
    PaArgs A = {};
    A.C = cache_of(cache);
    const int hd = cache->head_dim;
    if (const int rc = pa_checked(op, A, cache->dtype, hd, n_seqs, kv_len, q, q_stride, n_q_heads, out, out_stride, scale, window, workspace,
                                  workspace_bytes, mfs_paged_attention_workspace(cache, n_q_heads)))
        return rc < 0 ? rc : MFS_OK;
    cudaStream_t st = (cudaStream_t)cuda_stream;
    char* ws = (char*)workspace;
    if (cache->dtype == MFS_DTYPE_BF16) return hd == 128 ? attention<PaKindBf16<128>>(A, ws, st) : attention<PaKindBf16<64>>(A, ws, st);
    auto fn = hd == 128 ? (A.g == 1 ? attention<PaKindF32<128, 1>> : A.g <= 4 ? attention<PaKindF32<128, 4>> : attention<PaKindF32<128, 8>>)
                        : (A.g == 1 ? attention<PaKindF32<64, 1>> : A.g <= 4 ? attention<PaKindF32<64, 4>> : attention<PaKindF32<64, 8>>);
    return fn(A, ws, st, "paged_attention");
}
