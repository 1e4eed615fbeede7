// mfs_prompt_attention: causal attention over packed prompts.
//
// bf16: a CTA takes 256 query rows of one sequence and head as two 128-row tiles and walks over the
// keys they may see in tiles of 128.  Scores S = Q K^T and outputs O += P V are tcgen05 MMAs with
// accumulators in tensor memory (S 2 x 128 columns, O 2 x head_dim); K and V tiles arrive by TMA
// through a ring.  Each 128-row tile has four warps with one row per thread: they read a row of
// scores into registers, take its maximum without any exchange between threads, and write the
// weights back over the scores as bf16, where the second product reads them as its A operand.  The
// two tiles alternate: while one is in its softmax, the tensor cores work for the other.  O is
// rescaled only when a row's maximum grew by more than 2^8 (in the exponent's base 2) since the
// value in use; until then weights above 1 do no harm, the sum uses the same scale.
//
// Masked places: scores outside a row's range are replaced, not added to, so a NaN there is gone.  A
// masked weight is 0, but 0 x NaN is not, so where a tile of keys is masked for some rows (the
// diagonal, the end of a sequence, a window's edge), two warps clear the non-finite values of V in
// shared memory before the product; rows that do see one of them (it lies in their range) are
// computed again at the end by a plain pass in fp32.
#include <cuda.h>
#include <cudaTypedefs.h>

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

// ------------------------------------------------------------- tensor cores

constexpr int PT_M = 128;                    // query rows per tile, keys per tile
constexpr int PT_BLOCK = 2 * PT_M;           // query rows per CTA
constexpr int PT_THREADS = 384;              // warps 0-3, 4-7: softmax of the two tiles; 8: MMA; 9: TMA; 10, 11: V of masked tiles
constexpr unsigned long long PT_WAIT_NS = 2000000000ull;

template <int HD>
struct PtShape {
    static constexpr int BOX = PT_M * 128;        // a TMA box: 128 rows of 64 elements, 128-byte swizzle
    static constexpr int TILE = BOX * (HD / 64);  // a 128-row tile of Q, K or V
    static constexpr int STAGES = HD == 128 ? 5 : 8;
    static constexpr int BYTES = 1024 + 2 * TILE + STAGES * TILE;
};

struct PtBars {
    uint64_t q_full, kv_full[8], kv_empty[8], v_ready[8], s_full[2], p_full[2], o_full[2], drained;
    uint32_t tmem;
    int abort, cleared;        // a wait gave up; a non-finite value of V was cleared
    int seq, blk, b, len;      // the CTA's work
    int scan[PT_THREADS / 32];
};

__device__ __forceinline__ unsigned su32(const void* p) { return (unsigned)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void bar_init(uint64_t* b, unsigned n)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(su32(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* b, unsigned bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(su32(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* b)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(su32(b)) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t* b, unsigned par)
{
    unsigned ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(su32(b)), "r"(par) : "memory");
    return ok != 0;
}
__device__ __forceinline__ unsigned long long gtime()
{
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// Waits for the phase of parity `par`; false if it took too long or another wait of the CTA gave up.
__device__ __forceinline__ bool bar_wait(uint64_t* b, unsigned par, int* abort)
{
    unsigned long long t0 = 0;
    for (unsigned n = 1;; ++n) {
        if (bar_try(b, par)) return true;
        if (n & 63u) continue;
        if (*(volatile int*)abort) return false;
        const unsigned long long t = gtime();
        if (t0 == 0) {
            t0 = t;
        } else if (t - t0 > PT_WAIT_NS) {
            *(volatile int*)abort = 1;
            return false;
        }
    }
}
__device__ __forceinline__ void bar_drain(uint64_t* b, unsigned par)
{
    const unsigned long long t0 = gtime();
    while (!bar_try(b, par) && gtime() - t0 <= PT_WAIT_NS) {
    }
}

// Shared-memory operand, 128-byte swizzle, groups of 8 rows 1024 bytes apart; `lead`: bytes between
// 64-element blocks of the contiguous dimension where that is the MMA's M or N (V), else unused.
__device__ __forceinline__ uint64_t desc(unsigned saddr, unsigned lead)
{
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
           ((uint64_t)2 << 61);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void commit(uint64_t* b)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(su32(b)) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

#define PT_R4(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3])
#define PT_R16(r, i) PT_R4(r, i), PT_R4(r, i + 4), PT_R4(r, i + 8), PT_R4(r, i + 12)
#define PT_I4(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3])
#define PT_I16(r, i) PT_I4(r, i), PT_I4(r, i + 4), PT_I4(r, i + 8), PT_I4(r, i + 12)

// 32 columns of this thread's row (no wait)
__device__ __forceinline__ void tld32(uint32_t t, uint32_t* r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
                 "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];" : PT_R16(r, 0), PT_R16(r, 16) : "r"(t));
}
__device__ __forceinline__ void tst32(uint32_t t, const uint32_t* r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
                 "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(t), PT_I16(r, 0), PT_I16(r, 16) : "memory");
}
__device__ __forceinline__ void tld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tst_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t r, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

struct PtArgs {
    const int32_t* cu;
    const bf16 *q, *k, *v;
    bf16* out;
    long long q_stride, k_stride, v_stride, out_stride;
    int n_tokens, n_seqs, hq, g, window;
    float c;  // scale * log2(e)
};

// Row t (token) of head h again, by the warp: the running maximum and sum over keys lo .. t.
template <int HD>
__device__ __noinline__ void plain_row(const PtArgs& A, int t, int h, int lo)
{
    constexpr int E = HD / 32;
    const int lane = threadIdx.x & 31;
    float qf[E], o[E], m = -INFINITY, l = 0.f;
    for (int e = 0; e < E; ++e) {
        qf[e] = to_f(A.q[(long long)t * A.q_stride + h * HD + lane * E + e]);
        o[e] = 0.f;
    }
    for (int j = lo; j <= t; ++j) {
        const bf16* kr = A.k + (long long)j * A.k_stride + (h / A.g) * HD + lane * E;
        const bf16* vr = A.v + (long long)j * A.v_stride + (h / A.g) * HD + lane * E;
        float a = 0.f;
        for (int e = 0; e < E; ++e) a = fmaf(qf[e], to_f(kr[e]), a);
        for (int x = 16; x; x >>= 1) a += __shfl_xor_sync(0xffffffffu, a, x);
        const float mn = fmaxf(m, a), cc = m == mn ? 1.f : exp2f((m - mn) * A.c), p = a == mn ? 1.f : exp2f((a - mn) * A.c);
        l = l * cc + p;
        for (int e = 0; e < E; ++e) o[e] = o[e] * cc + p * to_f(vr[e]);
        m = mn;
    }
    for (int e = 0; e < E; ++e) put(A.out + (long long)t * A.out_stride + h * HD + lane * E + e, o[e] / l);
}

__device__ __forceinline__ bool not_finite2(uint32_t x) { return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u; }

template <int HD>
__global__ void __launch_bounds__(PT_THREADS, 1) prompt_mma_kernel(const __grid_constant__ CUtensorMap mq,
                                                                   const __grid_constant__ CUtensorMap mk,
                                                                   const __grid_constant__ CUtensorMap mv,
                                                                   const __grid_constant__ PtArgs A)
{
    using S = PtShape<HD>;
    extern __shared__ char pt_raw[];
    __shared__ PtBars B;
    char* base = (char*)(((uintptr_t)pt_raw + 1023) & ~(uintptr_t)1023);
    char* sq = base;
    char* ring = base + 2 * S::TILE;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x % A.hq, y = blockIdx.x / A.hq;

    // this CTA's sequence and block of rows, the last block of a sequence first
    {
        const int per = (A.n_seqs + PT_THREADS - 1) / PT_THREADS;
        auto length = [&](int s, int& b) {
            b = min(max(__ldg(A.cu + s), 0), A.n_tokens);
            return max(min(__ldg(A.cu + s + 1), A.n_tokens) - b, 0);
        };
        int mine = 0, b;
        for (int s = tid * per; s < min(A.n_seqs, (tid + 1) * per); ++s) mine += (length(s, b) + PT_BLOCK - 1) / PT_BLOCK;
        int inc = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += x;
        }
        if (lane == 31) B.scan[warp] = inc;
        if (tid == 0) {
            B.seq = -1;
            B.abort = B.cleared = 0;
            bar_init(&B.q_full, 1);
            for (int i = 0; i < S::STAGES; ++i) {
                bar_init(&B.kv_full[i], 1);
                bar_init(&B.kv_empty[i], 1);
            }
            for (int i = 0; i < 8; ++i) bar_init(&B.v_ready[i], 64);
            for (int i = 0; i < 2; ++i) {
                bar_init(&B.s_full[i], 1);
                bar_init(&B.p_full[i], PT_M);
                bar_init(&B.o_full[i], 1);
            }
            bar_init(&B.drained, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncthreads();
        int run = inc - mine;
        for (int w = 0; w < warp; ++w) run += B.scan[w];
        if (y >= run && y < run + mine)
            for (int s = tid * per; s < A.n_seqs; ++s) {
                const int len = length(s, b), nb = (len + PT_BLOCK - 1) / PT_BLOCK;
                if (y < run + nb) {
                    B.seq = s;
                    B.blk = nb - 1 - (y - run);
                    B.b = b;
                    B.len = len;
                    break;
                }
                run += nb;
            }
        __syncthreads();
        if (B.seq < 0) return;
    }
    const int b = B.b, len = B.len, r0 = B.blk * PT_BLOCK, W = A.window;
    // tiles of keys: [a0, a1) for the first row tile, [b0, b1) for the second
    const int a0 = W > 0 ? max(0, r0 - W + 1) / PT_M : 0, a1 = r0 / PT_M + 1;
    const bool two = len > r0 + PT_M;
    const int b0 = W > 0 ? max(0, r0 + PT_M - W + 1) / PT_M : 0, b1 = two ? a1 + 1 : 0;
    const int t_end = two ? b1 : a1;
    // does some row of tile x (0, 1) not see some key of tile t?
    auto masked = [&](int x, int t) { return t == (x ? b1 : a1) - 1 || (W > 0 && PT_M * t < r0 + PT_M * (x + 1) - W); };
    auto active = [&](int x, int t) { return x ? t >= b0 && t < b1 : t < a1; };
    auto edge = [&](int t) { return (active(0, t) && masked(0, t)) || (active(1, t) && masked(1, t)); };

    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&B.tmem)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, B.tmem, 0);  // columns: S of tile 0, S of tile 1, O of tile 0, O of tile 1
    const int ntile = t_end - a0;

    // registers: 384 threads x 168 at launch; the softmax warps take more, the others less
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 9) {
        if (lane == 0) {
            auto load = [&](const CUtensorMap* m, char* dst, int head, int row, uint64_t* bar) {
#pragma unroll
                for (int x = 0; x < HD / 64; ++x)
                    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                                 ::"r"(su32(dst + x * S::BOX)), "l"(m), "r"(64 * x), "r"(head), "r"(row), "r"(su32(bar)) : "memory");
            };
            bar_expect(&B.q_full, (two ? 2 : 1) * S::TILE);
            load(&mq, sq, h, b + r0, &B.q_full);
            if (two) load(&mq, sq + S::TILE, h, b + r0 + PT_M, &B.q_full);
            int i = 0, slot = 0;
            unsigned par = 1;
            bool ok = true;
            for (int t = a0; t < t_end && ok; ++t)
                for (int kv = 0; kv < 2; ++kv, ++i) {
                    if (!bar_wait(&B.kv_empty[slot], par, &B.abort)) { ok = false; break; }
                    bar_expect(&B.kv_full[slot], S::TILE);
                    load(kv ? &mv : &mk, ring + slot * S::TILE, h / A.g, b + t * PT_M, &B.kv_full[slot]);
                    if (++slot == S::STAGES) { slot = 0; par ^= 1; }
                }
            if (!ok) {  // the copies in flight
                bar_drain(&B.q_full, 0);
                for (int k = max(0, i - S::STAGES); k < i; ++k) bar_drain(&B.kv_full[k % S::STAGES], (k / S::STAGES) & 1);
            }
        }
    } else if (warp == 8) {
        {
            unsigned leader;
            asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(leader));
            constexpr uint32_t id_s = (1u << 4) | (1u << 7) | (1u << 10) | ((PT_M >> 3) << 17) | ((PT_M >> 4) << 24);
            constexpr uint32_t id_o = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((HD >> 3) << 17) | ((PT_M >> 4) << 24);
            // one thread issues everything: descriptors are built once and stepped, ring positions counted
            const uint64_t dq = desc(su32(sq), 16), dk = desc(su32(ring), 16), dv = desc(su32(ring), S::BOX);
            auto scores = [&](int x, int slot) {
                const uint64_t qa = dq + (uint64_t)(x * (S::TILE >> 4)), ka = dk + (uint64_t)(slot * (S::TILE >> 4));
                const uint32_t d = tm + x * PT_M;
#pragma unroll
                for (int k = 0; k < HD / 16; ++k) {
                    const uint64_t at = (k / 4) * (S::BOX >> 4) + (k % 4) * 2;
                    if (leader) mma_ss(d, qa + at, ka + at, id_s, k > 0);
                }
            };
            auto outputs = [&](int x, int slot, bool first) {
                const uint64_t va = dv + (uint64_t)(slot * (S::TILE >> 4));
                const uint32_t d = tm + 2 * PT_M + x * HD, pa = tm + x * PT_M;
                if (leader) mma_ts(d, pa, va, id_o, !first);
#pragma unroll
                for (int k = 1; k < PT_M / 16; ++k) if (leader) mma_ts(d, pa + 8 * k, va + (uint64_t)(k * 128), id_o, 1);
            };
            int slot = 0;  // of the next tile of the ring
            unsigned par = 0, v_par = 0, p_par[2] = {0, 0};
            auto step = [&]() {
                if (++slot == S::STAGES) { slot = 0; par ^= 1; }
            };
            bool ok = bar_wait(&B.q_full, 0, &B.abort) && bar_wait(&B.kv_full[0], 0, &B.abort);
            if (ok) {
                fence_after();
                scores(0, 0);
                if (leader) commit(&B.s_full[0]);
                if (active(1, a0)) {
                    scores(1, 0);
                    if (leader) commit(&B.s_full[1]);
                }
                if (leader) commit(&B.kv_empty[0]);
                step();
            }
            for (int n = 0; n < ntile && ok; ++n) {
                const int t = a0 + n;
                const bool next = n + 1 < ntile;
                const int vs = slot;
                ok = bar_wait(&B.kv_full[vs], par, &B.abort) && bar_wait(&B.v_ready[n & 7], v_par, &B.abort);
                if ((n & 7) == 7) v_par ^= 1;
                step();
                const int ks = slot;
                if (ok && next) ok = bar_wait(&B.kv_full[ks], par, &B.abort);
                if (next) step();
                if (!ok) break;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const bool now = active(x, t), then = next && active(x, t + 1);
                    if (now) {
                        ok = bar_wait(&B.p_full[x], p_par[x], &B.abort);
                        if (!ok) break;
                        p_par[x] ^= 1;
                        fence_after();
                        outputs(x, vs, t == (x ? b0 : a0));
                    }
                    if (then) {
                        scores(x, ks);
                        if (leader) commit(&B.s_full[x]);
                    } else if (now) {
                        if (leader) commit(&B.o_full[x]);
                    }
                }
                if (!ok) break;
                if (leader) commit(&B.kv_empty[vs]);
                if (next) if (leader) commit(&B.kv_empty[ks]);
            }
            if (leader) commit(&B.drained);
            if (leader) bar_drain(&B.drained, 0);
        }
    } else {
        // V of the tiles that some row does not see whole: non-finite values become 0
        const int th = tid - 10 * 32;
        bool ok = true;
        for (int n = 0; n < ntile && ok; ++n) {
            const int t = a0 + n, i = 2 * n + 1, slot = i % S::STAGES;
            // every tile is waited for and passed on, so that these warps stay in step with the ring
            ok = bar_wait(&B.kv_full[slot], (i / S::STAGES) & 1, &B.abort);
            if (!ok) break;
            bool wrote = false;
            for (int c = edge(t) ? th : S::TILE; c < S::TILE / 16; c += 64) {
                uint4* p = reinterpret_cast<uint4*>(ring + slot * S::TILE) + c;
                const uint4 x = *p;
                if (not_finite2(x.x) || not_finite2(x.y) || not_finite2(x.z) || not_finite2(x.w)) {
                    uint32_t w[4] = {x.x, x.y, x.z, x.w};
                    for (int e = 0; e < 4; ++e) {
                        if ((w[e] & 0x7f80u) == 0x7f80u) w[e] &= 0xffff0000u;
                        if ((w[e] & 0x7f800000u) == 0x7f800000u) w[e] &= 0xffffu;
                    }
                    *p = make_uint4(w[0], w[1], w[2], w[3]);
                    wrote = true;
                    if (t * PT_M + (c * 16 % S::BOX) / 128 < len) *(volatile int*)&B.cleared = 1;
                }
            }
            if (wrote) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            bar_arrive(&B.v_ready[n % 8]);
        }
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int x = warp >> 2, row = tid & (PT_M - 1);
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tm + lanes + x * PT_M, to = tm + lanes + 2 * PT_M + x * HD;
        const int first = x ? b0 : a0, last = x ? b1 : a1;
        const float c = A.c;
        float m = -INFINITY;     // the maximum in use (raw scores), exact up to 2^8 in the weights
        uint64_t l2[2] = {0, 0};  // the sum, in four parts
        bool ok = true;
        const int rr = r0 + x * PT_M + row;  // the row in its sequence
        for (int t = first; t < last; ++t) {
            if (!bar_wait(&B.s_full[x], (t - first) & 1, &B.abort)) { ok = false; break; }
            fence_after();
            uint32_t s[PT_M];
            tld32(ts, s);
            tld32(ts + 32, s + 32);
            tld_wait();
            tld32(ts + 64, s + 64);  // on its way while the first half's maximum is taken
            tld32(ts + 96, s + 96);
            const bool some = masked(x, t);
            const int hi = rr - PT_M * t, lo = W > 0 ? hi - W + 1 : 0;
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (half) tld_wait();
                if (some) {
#pragma unroll
                    for (int i = 64 * half; i < 64 * half + 64; ++i)
                        if (i > hi || i < lo) s[i] = 0xff800000u;
                }
#pragma unroll
                for (int i = 64 * half; i < 64 * half + 64; i += 8)
#pragma unroll
                    for (int y2 = 0; y2 < 4; ++y2) mx[y2] = max3(mx[y2], __uint_as_float(s[i + y2]), __uint_as_float(s[i + 4 + y2]));
            }
            const float mt = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
            if (t == first) {
                m = mt;
            } else {
                const bool up = mt > m && !((mt - m) * c <= 8.f);
                if (__any_sync(0xffffffffu, up)) {
                    const float a = !up ? 1.f : m == -INFINITY ? 0.f : ex2((m - mt) * c);
                    if (up) m = mt;
                    l2[0] = mul2(l2[0], pair(a, a));
                    l2[1] = mul2(l2[1], pair(a, a));
#pragma unroll
                    for (int i = 0; i < HD; i += 32) {
                        uint32_t o[32];
                        tld32(to + i, o);
                        tld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                        tst32(to + i, o);
                    }
                }
            }
            const float base_ = m == -INFINITY ? 0.f : -m * c;
            const uint64_t cc = pair(c, c), bb = pair(base_, base_);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t p[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int e = 64 * half + 2 * i;
                    float u, w;
                    unpair(fma2(pair(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), cc, bb), u, w);
                    u = ex2(u);
                    w = ex2(w);
                    l2[i & 1] = add2(l2[i & 1], pair(u, w));
                    p[i] = pack_bf16(u, w);
                }
                tst32(ts + 32 * half, p);
            }
            tst_wait();
            fence_before();
            bar_arrive(&B.p_full[x]);
        }
        if (last > first) {
            if (ok) ok = bar_wait(&B.o_full[x], 0, &B.abort);
            __syncwarp();
            fence_after();
            float l0, l1;
            unpair(add2(l2[0], l2[1]), l0, l1);
            const float inv = ok ? 1.f / (l0 + l1) : NAN;
            bf16* o = A.out + (long long)(b + rr) * A.out_stride + h * HD;
#pragma unroll
            for (int i = 0; i < HD; i += 32) {
                uint32_t r[32];
                tld32(to + i, r);
                tld_wait();
                if (rr < len) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint4 w;
                        w.x = pack_bf16(__uint_as_float(r[e]) * inv, __uint_as_float(r[e + 1]) * inv);
                        w.y = pack_bf16(__uint_as_float(r[e + 2]) * inv, __uint_as_float(r[e + 3]) * inv);
                        w.z = pack_bf16(__uint_as_float(r[e + 4]) * inv, __uint_as_float(r[e + 5]) * inv);
                        w.w = pack_bf16(__uint_as_float(r[e + 6]) * inv, __uint_as_float(r[e + 7]) * inv);
                        *reinterpret_cast<uint4*>(o + i + e) = w;
                    }
                }
            }
        }
    }
    fence_before();
    __syncthreads();
    if (warp == 8) {
        __syncwarp();
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512u));
    }
    if (B.cleared) {
        // rows that see a value that was cleared are computed again
        const int kv = h / A.g;
        for (int rr = r0 + warp; rr < min(len, r0 + PT_BLOCK); rr += PT_THREADS / 32) {
            const int lo = W > 0 ? max(0, rr - W + 1) : 0;
            bool sees = false;
            for (int t = max(a0, lo / PT_M); t <= rr / PT_M && !sees; ++t) {
                if (!edge(t)) continue;
                for (int j = max(lo, t * PT_M); j <= min(rr, t * PT_M + PT_M - 1); ++j) {
                    const uint32_t* p = reinterpret_cast<const uint32_t*>(A.v + (long long)(b + j) * A.v_stride + kv * HD);
                    for (int e = lane; e < HD / 2; e += 32) sees = sees || not_finite2(__ldg(p + e));
                }
                sees = __any_sync(0xffffffffu, sees);
            }
            if (sees) plain_row<HD>(A, b + rr, h, b + lo);
        }
    }
}

template <int HD>
int run_mma(int n_tokens, int n_seqs, const int32_t* cu, const void* q, long long q_stride, int hq, const void* k, long long k_stride,
            const void* v, long long v_stride, int hkv, void* out, long long out_stride, float scale, int window, cudaStream_t st)
{
    using S = PtShape<HD>;
    const char* op = "prompt_attention";
    static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    if (!encode) {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &r) != cudaSuccess || !fn)
            return mfs::op_fail(MFS_E_CUDA, op, "cuTensorMapEncodeTiled is not available");
        encode = (PFN_cuTensorMapEncodeTiled_v12000)fn;
    }
    CUtensorMap maps[3];
    const void* p[3] = {q, k, v};
    const long long stride[3] = {q_stride, k_stride, v_stride};
    const int heads[3] = {hq, hkv, hkv};
    for (int i = 0; i < 3; ++i) {
        const cuuint64_t dim[3] = {(cuuint64_t)HD, (cuuint64_t)heads[i], (cuuint64_t)n_tokens};
        const cuuint64_t str[2] = {(cuuint64_t)HD * 2, (cuuint64_t)stride[i] * 2};
        const cuuint32_t box[3] = {64, 1, PT_M}, es[3] = {1, 1, 1};
        if (encode(&maps[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p[i]), dim, str, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return mfs::op_fail(MFS_E_ARG, op, "the tensor is too large for a tensor map");
    }
    PtArgs A = {cu, (const bf16*)q, (const bf16*)k, (const bf16*)v, (bf16*)out, q_stride, k_stride, v_stride, out_stride,
                n_tokens, n_seqs, hq, hq / hkv, window, scale * 1.44269504088896340736f};
    const long long blocks = ((long long)n_tokens / PT_BLOCK + n_seqs) * hq;  // at least as many as there are
    if (blocks > 0x7fffffffLL) return mfs::op_fail(MFS_E_ARG, op, "too many tokens and sequences");
    cudaError_t e = cudaFuncSetAttribute(prompt_mma_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::BYTES);
    if (e == cudaSuccess) {
        prompt_mma_kernel<HD><<<(unsigned)blocks, PT_THREADS, S::BYTES, st>>>(maps[0], maps[1], maps[2], A);
        e = cudaGetLastError();
    }
    return mfs::op_launched(op, e);
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
    auto fn = dtype == MFS_DTYPE_BF16 ? (head_dim == 128 ? run_mma<128> : run_mma<64>)
                                      : (head_dim == 128 ? run<float, 128> : run<float, 64>);
    return fn(n_tokens, n_seqs, cu, q, q_stride, n_q_heads, k, k_stride, v, v_stride, n_kv_heads, out, out_stride, scale, window, st);
}
