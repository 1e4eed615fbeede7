// mfs_prompt_attention: causal attention over packed prompts.
//
// bf16: one CTA per SM takes blocks of two 128-row tiles of queries and walks over the keys they may
// see in tiles of 128.  The two tiles are the same rows of two heads that share keys, or, where the heads
// of a group are odd in number, 256 rows of one head (whose second tile sees one tile of keys more, so
// that the first one's warps wait at the end).  Scores S = Q K^T and outputs O += P V are
// tcgen05 MMAs with accumulators in tensor memory (S 2 x 128 columns, O 2 x head_dim); Q, K and V
// tiles arrive by TMA, K and V through a ring.  Each 128-row tile has four warps with one row per
// thread: they read a row of scores into registers, take its maximum without any exchange between
// threads, and write the weights back over the scores as bf16, where the second product reads them as
// its A operand.  The two tiles alternate: while one is in its softmax, the tensor cores work for the
// other.  The weights of a tile are taken against the maximum in use so far, while the tile's own is
// found; only where that is more than 2^8 larger (in the exponent's base 2) is O rescaled and the tile
// weighted again.  Until then weights above 1 do no harm: the sum uses the same scale.
//
// The blocks of a call, those with the most keys first, are dealt out to the CTAs back and forth, so
// that each gets about the same work; a CTA loads and multiplies for its next block while the last
// rows of the one before are written.
//
// What bounds it is the softmax's instructions on each score (maximum, exponential, sum, conversion)
// beside the tensor pipe, which is 70 % busy.  8192 tokens, 32 + 8 heads of 128: 341 us = 1610 TFLOP/s in
// replays of a graph, 0.84 of the measured matrix rate, 364 us by calls one behind the other, where the
// power limit holds the clock lower (with two row tiles of one head 353 us in replays; 32 + 32 heads, which
// have no other form, 380 us); 12 packed prompts of the same total 74 us (95 us): short ones are bounded by
// the blocks' starts and ends, where both row tiles end together and the softmax warps write.
// Heads of 64 halve the products but not the softmax: 8192 tokens 269 us = 1023 TFLOP/s, tensor pipe 44 %
// busy, exponentials 44 %, issue 47 %: the chain of one row per thread, with three warps per scheduler.  Their
// O leaves columns to keep the weights apart from the scores, so that the next scores are made while the softmax
// of these runs (294 us with the weights over the scores; 12 packed prompts 61 us against 60 us).
//
// The weights are rounded to bf16, since the tensor cores take both operands of a product in one type and the
// values are bf16; a weight is then off by at most half a step, 2^-8 of itself, as the output is when it is
// rounded.  Against 64 bits the outputs are off by 1.9 - 2.1e-3 of their size (1.6e-3 with the weights in fp32:
// the outputs' own rounding).  The sums take the weights unrounded; the exponential is the hardware's, 2^-22.
//
// Masked places: scores outside a row's range are replaced, not added to, so a NaN there is gone.  A
// masked weight is 0, but 0 x NaN is not, so where a tile of keys is masked for some rows (the
// diagonal, the end of a sequence, a window's edge), a warp clears the non-finite values of V in
// shared memory before the product; the rows that do see one of them (it lies in their range) get it
// added to their outputs at the end.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <type_traits>

#include "mfs_mma.cuh"
#include "mfs_ops.cuh"

namespace {

using bf16 = __nv_bfloat16;
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(bf16* p, float x) { *p = __float2bfloat16_rn(x); }

// ------------------------------------------------------------- tensor cores

constexpr int PT_M = 128;                    // query rows per tile, keys per tile
// warps 0-3, 4-7: softmax of the two tiles; 8: MMA; 9: TMA; 10, 11: V of masked tiles (11 also the next block)
constexpr int PT_THREADS = 384;
// A test build may shorten the waits' limit, and have every CTA lose one tile of its ring (never ask for it), so that they
// run out.
#ifndef MFS_PROMPT_LOST_TILE
#define MFS_PROMPT_LOST_TILE -1
#endif

template <int HD>
struct PtShape {
    static constexpr int BOX = PT_M * 128;        // a TMA box: 128 rows of 64 elements, 128-byte swizzle
    static constexpr int TILE = BOX * (HD / 64);  // a 128-row tile of Q, K or V
    static constexpr int STAGES = HD == 128 ? 5 : 8;
    static constexpr int BYTES = 1024 + 2 * TILE + STAGES * TILE;
};

// A block: rows r0 .. of the sequence of len tokens from token b, of head h; h < 0: no more.
struct __align__(16) PtWork {
    int b, len, r0, h;
};

struct PtBars {
    uint64_t q_full[2], q_empty[2], kv_full[8], kv_empty[8], v_ready[8], s_full[2], s_read[2], p_full[2], o_full[2], work_full[4], work_empty[4], drained;
    uint32_t tmem;
    int abort;          // a wait gave up
    int cleared[4];     // a non-finite value of V was cleared
    PtWork work[4];     // block i in place i mod 4
};
constexpr int PT_READERS = PT_THREADS / 32;  // warps that read the work

// Has a wait of the CTA given up?  For a whole warp.
__device__ __forceinline__ bool gave_up(PtBars& B) { return __any_sync(0xffffffffu, *(volatile int*)&B.abort); }
struct PtArgs {
    const int32_t* cu;
    const bf16 *q, *k, *v;
    bf16* out;
    long long q_stride, k_stride, v_stride, out_stride;
    int n_tokens, n_seqs, hq, g, window;
    int down, across;  // rows and heads from a block's first tile to its second: 0 and 1, or 128 and 0
    float c;           // scale * log2(e)
};

// s plus the products of two pairs of bf16
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float s)
{
    return fmaf(__uint_as_float(a << 16), __uint_as_float(b << 16), fmaf(__uint_as_float(a & 0xffff0000u), __uint_as_float(b & 0xffff0000u), s));
}

__device__ __forceinline__ bool not_finite2(uint32_t x) { return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u; }

// The tiles of keys of a block.
struct PtItem {
    int b, len, r0, h, W, down;
    int first[2], last[2];  // of each row tile
    int t0, t1;             // of both

    __device__ __forceinline__ bool two() const { return last[1] > first[1]; }
    // does some row of tile x not see some key of tile t?
    __device__ __forceinline__ bool masked(int x, int t) const { return t == last[x] - 1 || (W > 0 && PT_M * t < r0 + down * x + PT_M - W); }
    __device__ __forceinline__ bool active(int x, int t) const { return t >= first[x] && t < last[x]; }
    __device__ __forceinline__ bool edge(int t) const { return (active(0, t) && masked(0, t)) || (active(1, t) && masked(1, t)); }
};

// Block i of this CTA, for a whole warp; false: no more (or the wait gave up).
__device__ __forceinline__ bool next_item(PtBars& B, int i, const PtArgs& A, PtItem& I)
{
    if (!bar_wait(&B.work_full[i & 3], (i >> 2) & 1, &B.abort)) return false;
    const PtWork w = B.work[i & 3];
    if (w.h < 0) return false;
    I.b = w.b;
    I.len = w.len;
    I.r0 = w.r0;
    I.h = w.h;
    const int W = A.window;
    I.W = W;
    I.down = A.down;
    for (int x = 0; x < 2; ++x) {
        const int r = w.r0 + A.down * x;
        I.first[x] = W > 0 ? max(0, r - W + 1) / PT_M : 0;
        I.last[x] = r < w.len ? r / PT_M + 1 : I.first[x];
    }
    I.t0 = I.first[0];
    I.t1 = max(I.last[0], I.last[1]);
    if (!I.two()) I.t1 = I.last[0];
    return true;
}

__device__ __forceinline__ void done_with_item(PtBars& B, int i)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0) bar_arrive(&B.work_empty[i & 3]);
}

// Deals out the call's blocks, of `rows` rows and one of `hq` heads or pairs of heads.  Pairs (row block, sequence) are
// ordered by block number, largest first (about the number of their keys), then by sequence; an item is a pair and a
// head, heads innermost, so that neighbouring CTAs share keys; round r of G items goes to the CTAs in ascending order for
// even r, descending for odd r.
struct PtDealer {
    const int32_t* cu;
    int n_tokens, n_seqs, hq, rows;
    int level, above, upto;  // the current block number; pairs of larger numbers; those and its own

    __device__ __forceinline__ int blocks(int s, int& b, int& len) const
    {
        b = min(max(__ldg(cu + s), 0), n_tokens);
        len = max(min(__ldg(cu + s + 1), n_tokens) - b, 0);
        return (len + rows - 1) / rows;
    }
    __device__ int pairs_from(int lv) const
    {
        int n = 0, b, len;
        for (int s = threadIdx.x & 31; s < n_seqs; s += 32) n += max(0, blocks(s, b, len) - lv);
        return __reduce_add_sync(0xffffffffu, n);
    }
    __device__ __forceinline__ PtDealer(const int32_t* cu_, int n_tokens_, int n_seqs_, int hq_, int rows_)
        : cu(cu_), n_tokens(n_tokens_), n_seqs(n_seqs_), hq(hq_), rows(rows_), level(0), above(0), upto(0)
    {
    }
    __device__ void start()
    {
        int n = 0, b, len;
        for (int s = threadIdx.x & 31; s < n_seqs; s += 32) n = max(n, blocks(s, b, len));
        level = __reduce_max_sync(0xffffffffu, n);
    }
    // item r of this CTA, false: there is none
    __device__ bool get(int r, PtWork& w)
    {
        const long long G = gridDim.x, it = r * G + (r & 1 ? G - 1 - blockIdx.x : blockIdx.x);
        const long long pair = it / hq;
        while (pair >= upto) {
            if (level == 0) return false;
            --level;
            above = upto;
            upto = pairs_from(level);
        }
        int k = (int)(pair - above);  // the k-th sequence with such a block
        const int lane = threadIdx.x & 31;
        for (int s0 = 0; s0 < n_seqs; s0 += 32) {
            int b = 0, len = 0;
            const bool has = s0 + lane < n_seqs && blocks(s0 + lane, b, len) > level;
            unsigned m = __ballot_sync(0xffffffffu, has);
            if (k >= __popc(m)) { k -= __popc(m); continue; }
            while (k--) m &= m - 1;
            const int l = __ffs(m) - 1;
            w.b = __shfl_sync(0xffffffffu, b, l);
            w.len = __shfl_sync(0xffffffffu, len, l);
            w.r0 = level * rows;
            w.h = (int)(it % hq);
            return true;
        }
        return false;
    }
};

// A warp's 32 rows of block i, tile x, one per lane, whose outputs are written: adds the non-finite values that were cleared
// to the rows that see them, each in its own column, or NaN where the key's weight is 0.  m: the row's maximum in use.  Only
// tiles of keys that some row does not see whole were cleared (the last ones, and the window's first), so this takes the same
// time however long the prompt is: to 0.35 ms of 8192 tokens, 32 + 8 heads of 128, one such value adds 0.07 ms,
// one in every 64th token and head 0.5 ms, NaN in all values 0.9 ms.
template <int HD>
__device__ __noinline__ void put_cleared(const PtArgs& A, PtBars& B, int i, int x, int quarter, float m)
{
    PtItem I;
    const int W = A.window, lane = threadIdx.x & 31;
    if (!next_item(B, i, A, I)) return;  // published long ago
    const int r1 = I.r0 + x * A.down + 32 * quarter, r = r1 + lane, h = I.h + x * A.across;
    if (r1 >= I.len) return;
    const bool row = r < I.len;
    const int lo = W > 0 ? max(0, r - W + 1) : 0;
    const int from = W > 0 ? max(0, r1 - W + 1) : 0, upto = min(I.len, r1 + 32) - 1;  // the keys that the warp's rows see
    const float base_ = m == -INFINITY ? 0.f : -m * A.c;
    const uint4* q = reinterpret_cast<const uint4*>(A.q + (long long)(I.b + (row ? r : r1)) * A.q_stride + h * HD);
    bf16* o = A.out + (long long)(I.b + (row ? r : r1)) * A.out_stride + h * HD;
    uint32_t done[HD / 64] = {};  // words that are NaN in all of the warp's rows: a prompt of NaN values takes each once
    for (int t = from / PT_M; t <= upto / PT_M; ++t) {
        if (!I.edge(t)) continue;
        for (int j = max(from, t * PT_M); j <= min(upto, t * PT_M + PT_M - 1); ++j) {
            const uint32_t* v = reinterpret_cast<const uint32_t*>(A.v + (long long)(I.b + j) * A.v_stride + h / A.g * HD);
            uint32_t y[HD / 64], bad[HD / 64], any = 0;
#pragma unroll
            for (int e = 0; e < HD / 64; ++e) {
                y[e] = __ldg(v + 32 * e + lane);
                bad[e] = __ballot_sync(0xffffffffu, not_finite2(y[e])) & ~done[e];
                any |= bad[e];
            }
            if (!any) continue;
            const uint4* k = reinterpret_cast<const uint4*>(A.k + (long long)(I.b + j) * A.k_stride + h / A.g * HD);
            float s = 0.f;
            for (int e = 0; e < HD / 8; ++e) {
                const uint4 a = __ldg(q + e), b = __ldg(k + e);
                s = dot2(a.x, b.x, dot2(a.y, b.y, dot2(a.z, b.z, dot2(a.w, b.w, s))));
            }
            const bool sees = row && j >= lo && j <= r, weighs = ex2(fmaf(s, A.c, base_)) > 0.f;
            const bool all = __all_sync(0xffffffffu, sees || !row);
#pragma unroll
            for (int e = 0; e < HD / 64; ++e) {
                for (unsigned u = bad[e]; u; u &= u - 1) {
                    const int at = __ffs(u) - 1;
                    const uint32_t z = __shfl_sync(0xffffffffu, y[e], at);
                    bf16* p = o + 2 * (32 * e + at);
                    if (sees && (z & 0x7f80u) == 0x7f80u) put(p, to_f(*p) + (weighs ? __uint_as_float(z << 16) : NAN));
                    if (sees && (z & 0x7f800000u) == 0x7f800000u) put(p + 1, to_f(p[1]) + (weighs ? __uint_as_float(z & 0xffff0000u) : NAN));
                }
                const uint32_t nan = __ballot_sync(0xffffffffu, (y[e] & 0x7fffu) > 0x7f80u && (y[e] & 0x7fffffffu) > 0x7f80ffffu);
                if (all) done[e] |= nan;
            }
        }
    }
}

// The top bit of each half is set if that half's exponent is all ones (a bf16 infinity or NaN).
__device__ __forceinline__ uint32_t ones_exponent(uint32_t x) { return (x & 0x7f807f80u) + 0x00800080u; }

template <int HD, bool PAIRED>
__global__ void __launch_bounds__(PT_THREADS, 1) prompt_mma_kernel(const __grid_constant__ CUtensorMap mq,
                                                                   const __grid_constant__ CUtensorMap mk,
                                                                   const __grid_constant__ CUtensorMap mv,
                                                                   const __grid_constant__ PtArgs A)
{
    using S = PtShape<HD>;
    // heads of 64 leave columns for the weights beside the scores, which are then replaced while their softmax runs
    constexpr bool APART = HD == 64 && PAIRED;
    extern __shared__ char pt_raw[];
    __shared__ PtBars B;
    char* base = (char*)(((uintptr_t)pt_raw + 1023) & ~(uintptr_t)1023);
    char* sq = base;
    char* ring = base + 2 * S::TILE;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        B.abort = 0;
        for (int i = 0; i < S::STAGES; ++i) {
            bar_init(&B.kv_full[i], 1);
            bar_init(&B.kv_empty[i], 1);
        }
        for (int i = 0; i < 8; ++i) bar_init(&B.v_ready[i], 2);
        for (int i = 0; i < 2; ++i) {
            bar_init(&B.q_full[i], 1);
            bar_init(&B.q_empty[i], 1);
            bar_init(&B.s_full[i], 1);
            bar_init(&B.s_read[i], PT_M);
            bar_init(&B.p_full[i], PT_M);
            bar_init(&B.o_full[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            bar_init(&B.work_full[i], 1);
            bar_init(&B.work_empty[i], PT_READERS);
        }
        bar_init(&B.drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&B.tmem)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    PtDealer deal(A.cu, A.n_tokens, A.n_seqs, A.hq >> A.across, PT_M + A.down);
    if (warp == 11) deal.start();
    if (tid == 9 * 32) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&mq) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&mk) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&mv) : "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, B.tmem, 0);  // columns: S of tile 0, S of tile 1, O of tile 0, O of tile 1, APART: P of each
    const int W = A.window;

    // registers: 384 threads x 168 at launch; the softmax warps take more, the others less
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 9) {
            auto load = [&](const CUtensorMap* m, char* dst, int head, int row, uint64_t* bar) {
                bar_expect(bar, S::TILE);
#pragma unroll
                for (int x = 0; x < HD / 64; ++x)
                    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                                 ::"r"(su32(dst + x * S::BOX)), "l"(m), "r"(64 * x), "r"(head), "r"(row), "r"(su32(bar)) : "memory");
            };
            PtItem I;
            int n = 0, slot = 0;               // tiles asked for
            unsigned par = 1, q_par[2] = {1, 1};
            bool ok = true, q_used[2] = {false, false};
            // After a wait that gave up nothing more is asked for: the issuing warp may then free a place of the ring whose tile
            // is still on its way (a test for that there, where it would be made first, takes 5 % of a long prompt's time).
            for (int i = 0; ok && next_item(B, i, A, I); ++i) {
                auto query = [&](int x) {
                    if (!bar_wait(&B.q_empty[x], q_par[x], &B.abort) || gave_up(B)) return false;
                    if (lane == 0) load(&mq, sq + x * S::TILE, I.h + A.across * x, I.b + I.r0 + A.down * x, &B.q_full[x]);
                    q_par[x] ^= 1;
                    q_used[x] = true;
                    return true;
                };
                ok = query(0);
                for (int t = I.t0; t < I.t1 && ok; ++t)
                    for (int kv = 0; kv < 2 && ok; ++kv) {
                        ok = bar_wait(&B.kv_empty[slot], par, &B.abort) && !gave_up(B);
                        if (!ok) break;
                        if (lane == 0 && n != MFS_PROMPT_LOST_TILE) load(kv ? &mv : &mk, ring + slot * S::TILE, I.h / A.g, I.b + t * PT_M, &B.kv_full[slot]);
                        __syncwarp();
                        ++n;
                        if (++slot == S::STAGES) { slot = 0; par ^= 1; }
                        if (t == I.t0 && kv == 0 && I.two()) ok = query(1);
                    }
                done_with_item(B, i);
            }
            if (lane == 0) {  // no copy is in flight when the CTA ends, whichever warp gave up
                for (int x = 0; x < 2; ++x)
                    if (q_used[x]) bar_drain(&B.q_full[x], q_par[x]);
                for (int k = max(0, n - S::STAGES); k < n; ++k) bar_drain(&B.kv_full[k % S::STAGES], (k / S::STAGES) & 1);
            }
        } else if (warp == 8) {
            // the whole warp runs the loop and an elected lane issues: the operands' descriptors stay in uniform
            // registers (a single thread's loop took 70-80 cycles an MMA to move them there, an MMA takes 64)
            constexpr uint32_t id_s = (1u << 4) | (1u << 7) | (1u << 10) | ((PT_M >> 3) << 17) | ((PT_M >> 4) << 24);
            constexpr uint32_t id_o = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((HD >> 3) << 17) | ((PT_M >> 4) << 24);
            unsigned leader;
            asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(leader));
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
                const uint32_t d = tm + 2 * PT_M + x * HD, pa = tm + (APART ? 2 * (PT_M + HD) + x * (PT_M / 2) : x * PT_M);
                if (leader) mma_ts(d, pa, va, id_o, !first);
#pragma unroll
                for (int k = 1; k < PT_M / 16; ++k)
                    if (leader) mma_ts(d, pa + 8 * k, va + (uint64_t)(k * 128), id_o, 1);
            };
            auto signal = [&](uint64_t* bar) {
                if (leader) commit(bar);
            };
            int slot = 0;  // of the next tile of the ring
            unsigned par = 0, v_at = 0, p_par[2] = {0, 0}, q_par[2] = {0, 0}, r_par = 0;
            auto step = [&]() {
                if (++slot == S::STAGES) { slot = 0; par ^= 1; }
            };
            bool ok = true;
            PtItem I;
            if constexpr (PAIRED) {
                // Both row tiles see the same tiles of keys.  The steps of all blocks follow each other: the scores of the
                // next step, of the next block after the last tile, go behind each outputs.
                bool have = next_item(B, 0, A, I), fresh = true;  // fresh: the step is its block's first
                int i = 0, t = I.t0, t1 = I.t1;
                auto score_tile = [&](int x, int ks, bool first, bool last) {
                    if (first) {
                        if (!bar_wait(&B.q_full[x], q_par[x], &B.abort)) return false;
                        q_par[x] ^= 1;
                        fence_after();
                    }
                    scores(x, ks);
                    signal(&B.s_full[x]);
                    if (last) signal(&B.q_empty[x]);
                    return true;
                };
                if (have) {
                    ok = bar_wait(&B.kv_full[slot], par, &B.abort);
                    fence_after();
#pragma unroll
                    for (int x = 0; x < 2; ++x) ok = ok && score_tile(x, slot, true, t + 1 == t1);
                    signal(&B.kv_empty[slot]);
                    step();
                }
                while (ok && have) {
                    const bool ends = t + 1 == t1, was_fresh = fresh;
                    if (ends) {
                        have = next_item(B, i + 1, A, I);
                        t = I.t0;
                        t1 = I.t1;
                    } else {
                        ++t;
                    }
                    fresh = ends;
                    const int vs = slot;
                    step();
                    const int ks = slot;
                    if (have) {
                        ok = bar_wait(&B.kv_full[ks], par, &B.abort);
                        step();
                    }
                    if constexpr (APART)
                        if (have) {
                            // the next scores as soon as these are in registers
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                ok = ok && bar_wait(&B.s_read[x], r_par, &B.abort);
                                if (!ok) break;
                                fence_after();
                                ok = score_tile(x, ks, fresh, t + 1 == t1);
                            }
                            r_par ^= 1;
                            signal(&B.kv_empty[ks]);
                        }
                    ok = ok && bar_wait(&B.v_ready[v_at & 7], (v_at >> 3) & 1, &B.abort);  // loaded, and cleared where masked
                    ++v_at;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        ok = ok && bar_wait(&B.p_full[x], p_par[x], &B.abort);
                        if (!ok) break;
                        p_par[x] ^= 1;
                        fence_after();
                        outputs(x, vs, was_fresh);
                        if (ends || APART) signal(&B.o_full[x]);
                        if (have && !APART) ok = score_tile(x, ks, fresh, t + 1 == t1);
                    }
                    signal(&B.kv_empty[vs]);
                    if (have && !APART) signal(&B.kv_empty[ks]);
                    if (ends) done_with_item(B, i++);
                }
            } else
            for (int i = 0; ok && next_item(B, i, A, I); ++i) {
                // scores of row tile x for tile t of keys, in the ring at ks; the block's Q is free after its last
                auto score_tile = [&](int x, int t, int ks) {
                    if (t == I.first[x]) {
                        if (!bar_wait(&B.q_full[x], q_par[x], &B.abort)) return false;
                        q_par[x] ^= 1;
                        fence_after();
                    }
                    scores(x, ks);
                    signal(&B.s_full[x]);
                    if (t == I.last[x] - 1) signal(&B.q_empty[x]);
                    return true;
                };
                ok = bar_wait(&B.kv_full[slot], par, &B.abort);
                if (ok) {
                    fence_after();
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        if (ok && I.active(x, I.t0)) ok = score_tile(x, I.t0, slot);
                    signal(&B.kv_empty[slot]);
                    step();
                }
                for (int t = I.t0; t < I.t1 && ok; ++t) {
                    const bool next = t + 1 < I.t1;
                    const int vs = slot;
                    ok = bar_wait(&B.v_ready[v_at & 7], (v_at >> 3) & 1, &B.abort);  // loaded, and cleared where masked
                    ++v_at;
                    step();
                    const int ks = slot;
                    if (next) {
                        ok = ok && bar_wait(&B.kv_full[ks], par, &B.abort);
                        step();
                    }
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        if (!ok) break;
                        if (I.active(x, t)) {
                            ok = bar_wait(&B.p_full[x], p_par[x], &B.abort);
                            if (!ok) break;
                            p_par[x] ^= 1;
                            fence_after();
                            outputs(x, vs, t == I.first[x]);
                            if (t == I.last[x] - 1) signal(&B.o_full[x]);
                        }
                        if (next && I.active(x, t + 1)) ok = score_tile(x, t + 1, ks);
                    }
                    signal(&B.kv_empty[vs]);
                    if (next) signal(&B.kv_empty[ks]);
                }
                done_with_item(B, i);
            }
            signal(&B.drained);
            if (leader) bar_drain(&B.drained, 0);
        } else {
            // Warp 11 deals out the blocks, one ahead; both look through V of the tiles that some row does not see whole,
            // half a tile each: non-finite values become 0.  Every tile is waited for and passed on.
            PtItem I;
            PtWork w;
            int next = 0;  // blocks published
            int slot = 1 % S::STAGES;
            unsigned par = 0, v_at = 0;
            bool ok = true, more = warp == 11;
            auto publish = [&](int i) {  // block i
                if (!more) return true;
                more = deal.get(i, w);
                w.h <<= A.across;
                if (!bar_wait(&B.work_empty[i & 3], ((i >> 2) & 1) ^ 1, &B.abort)) return false;
                if (lane == 0) {
                    if (!more) w.h = -1;
                    B.work[i & 3] = w;
                    B.cleared[i & 3] = 0;
                    bar_arrive(&B.work_full[i & 3]);
                }
                __syncwarp();
                next = i + 1;
                return true;
            };
            int i = 0;
            ok = publish(0);
            for (; ok && next_item(B, i, A, I); ++i) {
                ok = publish(i + 1);
                for (int t = I.t0; t < I.t1 && ok; ++t) {
                    ok = bar_wait(&B.kv_full[slot], par, &B.abort);
                    if (!ok) break;
                    if (I.edge(t)) {
                        bool wrote = false;
                        const int from = (warp - 10) * (S::TILE / 32);
                        uint4* tile = reinterpret_cast<uint4*>(ring + slot * S::TILE) + from + lane;
                        for (int c0 = 0; c0 < S::TILE / 32; c0 += 8 * 32) {
                            uint4 x[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] = tile[c0 + 32 * e];
                            uint32_t any = 0;
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                any |= ones_exponent(x[e].x) | ones_exponent(x[e].y) | ones_exponent(x[e].z) | ones_exponent(x[e].w);
                            if (!(any & 0x80008000u)) continue;
                            for (int e = 0; e < 8; ++e) {
                                const int c = from + c0 + 32 * e + lane;
                                const uint4 y = tile[c0 + 32 * e];
                                uint32_t v[4] = {y.x, y.y, y.z, y.w};
                                bool here = false;
                                for (int k = 0; k < 4; ++k) {
                                    here = here || not_finite2(v[k]);
                                    if ((v[k] & 0x7f80u) == 0x7f80u) v[k] &= 0xffff0000u;
                                    if ((v[k] & 0x7f800000u) == 0x7f800000u) v[k] &= 0xffffu;
                                }
                                if (!here) continue;
                                tile[c0 + 32 * e] = make_uint4(v[0], v[1], v[2], v[3]);
                                wrote = true;
                                if (t * PT_M + (c * 16 % S::BOX) / 128 < I.len) *(volatile int*)&B.cleared[i & 3] = 1;
                            }
                        }
                        if (wrote) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    }
                    __syncwarp();
                    if (lane == 0) bar_arrive(&B.v_ready[v_at & 7]);
                    ++v_at;
                    slot += 2;
                    if (slot >= S::STAGES) { slot -= S::STAGES; par ^= 1; }
                }
                done_with_item(B, i);
            }
            if (!ok && warp == 11)
                // given up: NaN for the blocks that nobody will compute; those published are the softmax warps' to write
                for (; deal.get(next, w); ++next)
                    for (int r = w.r0; r < min(w.len, w.r0 + PT_M + A.down); ++r)
                        for (int e = lane; e < HD << A.across; e += 32)
                            A.out[(long long)(w.b + r) * A.out_stride + (w.h << A.across) * HD + e] = __float2bfloat16_rn(NAN);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int x = warp >> 2, row = tid & (PT_M - 1);
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tm + lanes + x * PT_M, to = tm + lanes + 2 * PT_M + x * HD;
        const uint32_t tp = APART ? tm + lanes + 2 * (PT_M + HD) + x * (PT_M / 2) : ts;
        unsigned s_par = 0, o_par = 0;
        bool ok = true, summing = false;  // summing: APART, the last weights' product may still run
        for (int i = 0;; ++i) {
            int first, last, rr;  // rr: the row in its sequence
            {
                PtItem I;
                if (!next_item(B, i, A, I)) break;
                first = x ? I.first[1] : I.first[0];
                last = x ? I.last[1] : I.last[0];
                rr = I.r0 + x * A.down + row;
            }
            float m = -INFINITY;       // the maximum in use (raw scores), exact up to 2^8 in the weights
            uint64_t l2[2] = {0, 0};   // the sum, in four parts
            for (int t = first; t < last && ok; ++t) {
                ok = bar_wait(&B.s_full[x], s_par, &B.abort);
                if (!ok) break;
                s_par ^= 1;
                __syncwarp();
                fence_after();
                uint32_t s[PT_M];
#pragma unroll
                for (int k = 0; k < 4; ++k) tld32(ts + 32 * k, s + 32 * k);
                tld_wait();
                if constexpr (APART) {
                    fence_before();
                    bar_arrive(&B.s_read[x]);
                }
                if (t == last - 1 || (W > 0 && PT_M * t < rr - row + PT_M - W)) {  // masked for some row
                    const int hi = rr - PT_M * t, lo = W > 0 ? hi - W + 1 : 0;
#pragma unroll
                    for (int k = 0; k < PT_M; ++k)
                        if (k > hi || k < lo) s[k] = 0xff800000u;
                }
                auto summed = [&]() {  // O and the weights' place are free
                    if (APART && summing) {
                        ok = bar_wait(&B.o_full[x], o_par, &B.abort);
                        o_par ^= 1;
                        summing = false;
                        __syncwarp();
                        fence_after();
                    }
                    return ok;
                };
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < PT_M; k += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], __uint_as_float(s[k + e]), __uint_as_float(s[k + 4 + e]));
                const float mt = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
                if (t == first) {
                    m = mt;
                } else {
                    const bool up = mt > m && !((mt - m) * A.c <= 8.f);
                    if (__any_sync(0xffffffffu, up)) {
                        if (!summed()) break;
                        const float a = !up ? 1.f : m == -INFINITY ? 0.f : ex2((m - mt) * A.c);
                        if (up) m = mt;
                        l2[0] = mul2(l2[0], pair(a, a));
                        l2[1] = mul2(l2[1], pair(a, a));
#pragma unroll
                        for (int k = 0; k < HD; k += 16) {
                            uint32_t o[16];
                            tld16(to + k, o);
                            tld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                            tst16(to + k, o);
                        }
                    }
                }
                const float base_ = m == -INFINITY ? 0.f : -m * A.c;
                const uint64_t cc = pair(A.c, A.c), bb = pair(base_, base_);
#pragma unroll
                for (int quarter = 0; quarter < 4; ++quarter) {
                    uint32_t p[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const int e = 32 * quarter + 2 * k;
                        float u, w;
                        unpair(fma2(pair(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), cc, bb), u, w);
                        u = ex2(u);
                        w = ex2(w);
                        l2[k & 1] = add2(l2[k & 1], pair(u, w));
                        p[k] = pack_bf16(u, w);
                    }
                    if (quarter == 0 && !summed()) break;
                    tst16(tp + 16 * quarter, p);
                }
                if (!ok) break;
                summing = APART;
                tst_wait();
                fence_before();
                bar_arrive(&B.p_full[x]);
            }
            if (last > first) {
                if (ok) ok = bar_wait(&B.o_full[x], o_par, &B.abort);
                o_par ^= 1;
                summing = false;
                __syncwarp();
                fence_after();
                float l0, l1;
                unpair(add2(l2[0], l2[1]), l0, l1);
                const float inv = ok ? 1.f / (l0 + l1) : NAN;
                const PtWork w = B.work[i & 3];
                // 64 elements of a row at a time: the eight lanes of eight rows exchange 16-byte units so that a store
                // writes 128 bytes of each of four rows (a lane per row would touch 32 lines with each)
                const int j = lane & 7;
                bf16* o = A.out + (long long)(w.b + rr - j) * A.out_stride + (w.h + x * A.across) * HD + 8 * j;
#pragma unroll
                for (int k = 0; k < HD; k += 64) {
                    uint32_t u[8][4];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t r[32];
                        tld32(to + k + 32 * half, r);
                        tld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            u[4 * half + e / 4][e % 4] = pack_bf16(__uint_as_float(r[2 * e]) * inv, __uint_as_float(r[2 * e + 1]) * inv);
                    }
#pragma unroll
                    for (int d = 1; d < 8; d *= 2)
#pragma unroll
                        for (int y = 0; y < 8; ++y)
                            if (!(y & d)) {
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const uint32_t got = __shfl_xor_sync(0xffffffffu, j & d ? u[y][e] : u[y | d][e], d);
                                    if (j & d) u[y][e] = got;
                                    else u[y | d][e] = got;
                                }
                            }
#pragma unroll
                    for (int y = 0; y < 8; ++y)
                        if (rr - j + y < w.len)
                            *reinterpret_cast<uint4*>(o + y * A.out_stride + k) = make_uint4(u[y][0], u[y][1], u[y][2], u[y][3]);
                }
                fence_before();
                if (*(volatile int*)&B.cleared[i & 3] && ok) {
                    __syncwarp();
                    put_cleared<HD>(A, B, i, x, warp & 3, m);
                }
            }
            done_with_item(B, i);
        }
    }
    fence_before();
    __syncthreads();
    if (warp == 8) {
        __syncwarp();
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512u));
    }
}

// --------------------------------------------------------------------- fp32
//
// On the CUDA cores: a CTA of 256 threads takes 16 RT query rows of one sequence and head (RT 8, 4 or 2)
// and walks over tiles of 64 keys in shared memory.  A thread has RT rows x 4 keys of the scores and
// RT rows x HD / 16 elements of the output in registers (rows and keys 16 apart, so that a warp's 16-byte
// loads meet no bank twice), with paired fp32 products; a row's maximum and sum go over half a warp.
// Keys of the next tile are copied while the values of this one are summed, and the other way round.
// 4096 tokens, 32 + 8 heads of 128, take 3.0 ms = 46 TFLOP/s, about 0.6 of the CUDA cores' rate; the data path of
// shared memory, which feeds them, is 55 % busy, and two warps per scheduler issue 45 % of the time.  In tiles
// that some row does not see whole, unseen products are left out, not multiplied by zero.

constexpr int PF_KEYS = 64, PF_THREADS = 256;

template <int HD, int RT>
struct PfShape {
    static constexpr int ROWS = 16 * RT;                 // query rows of a CTA
    static constexpr int LD = HD + 4, LP = PF_KEYS + 4;  // row strides in shared memory
    static constexpr int BYTES = 4 * ((ROWS + 2 * PF_KEYS) * LD + ROWS * LP);
};

struct PfArgs {
    const int32_t* cu;
    const float *q, *k, *v;
    float* out;
    long long q_stride, k_stride, v_stride, out_stride;
    int n_tokens, n_seqs, hq, g, window;
    float c;  // scale * log2(e)
};

__device__ __forceinline__ void copy16(float* dst, const float* src, bool full)
{
    const int n = full ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(su32(dst)), "l"(src), "r"(n) : "memory");
}

template <int HD, int RT>
__global__ void __launch_bounds__(PF_THREADS, RT == 2 ? 2 : 1) prompt_f32_kernel(const __grid_constant__ PfArgs A)
{
    using S = PfShape<HD, RT>;
    constexpr int ROWS = S::ROWS, LD = S::LD, LP = S::LP, OC = HD / 16;
    extern __shared__ __align__(16) float pf_raw[];
    float *sq = pf_raw, *sk = sq + ROWS * LD, *sv = sk + PF_KEYS * LD, *sp = sv + PF_KEYS * LD;
    __shared__ PtWork work;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    if (tid < 32) {
        PtDealer deal(A.cu, A.n_tokens, A.n_seqs, A.hq, ROWS);
        deal.start();
        PtWork w;
        if (!deal.get(0, w)) w.h = -1;
        if (tid == 0) work = w;
    }
    __syncthreads();
    const PtWork w = work;
    if (w.h < 0) return;
    const int rows = min(ROWS, w.len - w.r0), W = A.window;
    const float* kg = A.k + (long long)w.b * A.k_stride + w.h / A.g * HD;
    const float* vg = A.v + (long long)w.b * A.v_stride + w.h / A.g * HD;
    auto copy_tile = [&](float* dst, const float* src, long long stride, int r0, int n, int limit) {
        for (int i = tid; i < n * (HD / 4); i += PF_THREADS) {
            const int r = i / (HD / 4), c = i % (HD / 4) * 4;
            const bool in = r0 + r < limit;
            copy16(dst + r * LD + c, src + (in ? (long long)(r0 + r) * stride + c : 0), in);
        }
    };
    const int t0 = (W > 0 ? max(0, w.r0 - W + 1) : 0) / PF_KEYS, t1 = (w.r0 + rows - 1) / PF_KEYS + 1;
    copy_tile(sq, A.q + (long long)(w.b + w.r0) * A.q_stride + w.h * HD, A.q_stride, 0, ROWS, rows);
    copy_tile(sk, kg, A.k_stride, t0 * PF_KEYS, PF_KEYS, w.len);
    asm volatile("cp.async.commit_group;" ::: "memory");
    copy_tile(sv, vg, A.v_stride, t0 * PF_KEYS, PF_KEYS, w.len);
    asm volatile("cp.async.commit_group;" ::: "memory");

    float o[RT][OC], m[RT], l[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int e = 0; e < OC; ++e) o[i][e] = 0.f;
    }
    for (int t = t0; t < t1; ++t) {
        const int k0 = t * PF_KEYS;
        // some row does not see some key
        const bool edge = k0 + PF_KEYS - 1 > w.r0 || (W > 0 && k0 <= w.r0 + rows - 1 - W);
        asm volatile("cp.async.wait_group 1;" ::: "memory");  // the keys
        __syncthreads();
        uint64_t acc[RT][4];
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = 0;
#pragma unroll 4
        for (int e = 0; e < HD; e += 4) {
            ulonglong2 k4[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) k4[j] = *reinterpret_cast<const ulonglong2*>(sk + (tx + 16 * j) * LD + e);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const ulonglong2 q4 = *reinterpret_cast<const ulonglong2*>(sq + (ty + 16 * i) * LD + e);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fma2(q4.y, k4[j].y, fma2(q4.x, k4[j].x, acc[i][j]));
            }
        }
        __syncthreads();  // all have read the keys
        if (t + 1 < t1) copy_tile(sk, kg, A.k_stride, k0 + PF_KEYS, PF_KEYS, w.len);
        asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int row = w.r0 + ty + 16 * i;
            float s[4], mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float a, b;
                unpair(acc[i][j], a, b);
                s[j] = a + b;
                const int key = k0 + tx + 16 * j;
                if (edge && (key > row || (W > 0 && key <= row - W))) s[j] = -INFINITY;
                mx = fmaxf(mx, s[j]);
            }
            for (int x = 8; x; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
            const float mn = fmaxf(m[i], mx), a = m[i] == mn ? 1.f : exp2f((m[i] - mn) * A.c);
            const float sub = mn == -INFINITY ? 0.f : mn;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f((s[j] - sub) * A.c);
                sum += p;
                sp[(ty + 16 * i) * LP + tx + 16 * j] = p;
            }
            m[i] = mn;
            l[i] = l[i] * a + sum;
#pragma unroll
            for (int e = 0; e < OC; ++e) o[i][e] *= a;
        }
        asm volatile("cp.async.wait_group 1;" ::: "memory");  // the values
        __syncthreads();
        auto product = [&](auto part) {  // part: some keys are left out
#pragma unroll 2
            for (int j = 0; j < PF_KEYS; j += 4) {
                float4 p4[RT];
#pragma unroll
                for (int i = 0; i < RT; ++i) p4[i] = *reinterpret_cast<const float4*>(sp + (ty + 16 * i) * LP + j);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint64_t v2[OC / 2];
#pragma unroll
                    for (int e = 0; e < OC / 4; ++e) {
                        const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(sv + (j + x) * LD + 4 * tx + 64 * e);
                        v2[2 * e] = y.x;
                        v2[2 * e + 1] = y.y;
                    }
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        const float p = x == 0 ? p4[i].x : x == 1 ? p4[i].y : x == 2 ? p4[i].z : p4[i].w;
                        if (decltype(part)::value) {
                            const int row = w.r0 + ty + 16 * i, key = k0 + j + x;
                            if (key > row || (W > 0 && key <= row - W)) continue;
                        }
                        const uint64_t pp = pair(p, p);
#pragma unroll
                        for (int e = 0; e < OC / 2; ++e) {
                            const uint64_t r = fma2(pp, v2[e], pair(o[i][2 * e], o[i][2 * e + 1]));
                            unpair(r, o[i][2 * e], o[i][2 * e + 1]);
                        }
                    }
                }
            }
        };
        if (edge) product(std::true_type());
        else product(std::false_type());
        __syncthreads();  // all have read the values
        if (t + 1 < t1) copy_tile(sv, vg, A.v_stride, k0 + PF_KEYS, PF_KEYS, w.len);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        float sum = l[i];
        for (int x = 8; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        const int r = ty + 16 * i;
        if (r >= rows) continue;
        float* p = A.out + (long long)(w.b + w.r0 + r) * A.out_stride + w.h * HD;
#pragma unroll
        for (int e = 0; e < OC / 4; ++e)
            *reinterpret_cast<float4*>(p + 4 * tx + 64 * e) =
                make_float4(o[i][4 * e] / sum, o[i][4 * e + 1] / sum, o[i][4 * e + 2] / sum, o[i][4 * e + 3] / sum);
    }
}

template <int HD, int RT>
int launch_f32(const PfArgs& A, cudaStream_t st)
{
    const char* op = "prompt_attention";
    using S = PfShape<HD, RT>;
    const long long blocks = ((long long)A.n_tokens / S::ROWS + A.n_seqs) * A.hq;  // blocks there can be
    if (blocks > 0x7fffffffLL) return mfs::op_fail(MFS_E_ARG, op, "too many tokens and sequences");
    int sms = 0;
    static mfs::PerDevice ready;
    cudaError_t e = mfs::op_device(ready, (const void*)prompt_f32_kernel<HD, RT>, S::BYTES, &sms);
    if (e == cudaSuccess) {
        prompt_f32_kernel<HD, RT><<<(unsigned)blocks, PF_THREADS, S::BYTES, st>>>(A);
        e = cudaGetLastError();
    }
    return mfs::op_launched(op, e);
}

// Row tiles of 128; of 64 or 32 where they would be fewer than one and a half per SM, or longer than the sequences on
// average.  With 128, 64 and 32 rows, heads of 128: 4096 tokens, 32 heads 3010, 3481 and 4706 us; 1000 tokens 227, 246, 322;
// 512 tokens 114, 72, 99; 8 heads 115, 67, 52; 137 tokens, 32 heads 46, 28, 26; 100 sequences of 20 408, 254, 152; 50 of
// 40 208, 134, 116; 25 of 80 168, 130, 129.
template <int HD>
int run_f32(int n_tokens, int n_seqs, const int32_t* cu, const void* q, long long q_stride, int hq, const void* k, long long k_stride,
            const void* v, long long v_stride, int hkv, void* out, long long out_stride, float scale, int window, cudaStream_t st)
{
    const PfArgs A = {cu, (const float*)q, (const float*)k, (const float*)v, (float*)out, q_stride, k_stride, v_stride, out_stride,
                      n_tokens, n_seqs, hq, hq / hkv, window, scale * 1.44269504088896340736f};
    int sms = 0;
    static mfs::PerDevice known;
    const cudaError_t e = mfs::op_device(known, nullptr, 0, &sms);
    if (e != cudaSuccess) return mfs::op_launched("prompt_attention", e);
    int rt = 8;
    while (rt > 2 && (((long long)n_tokens / (16 * rt) + n_seqs) * hq * 2 < 3 * sms || n_tokens <= 16LL * rt * n_seqs)) rt /= 2;
    return rt == 8 ? launch_f32<HD, 8>(A, st) : rt == 4 ? launch_f32<HD, 4>(A, st) : launch_f32<HD, 2>(A, st);
}

template <int HD>
int run_mma(int n_tokens, int n_seqs, const int32_t* cu, const void* q, long long q_stride, int hq, const void* k, long long k_stride,
            const void* v, long long v_stride, int hkv, void* out, long long out_stride, float scale, int window, cudaStream_t st)
{
    using S = PtShape<HD>;
    const char* op = "prompt_attention";
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> known{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 encode = known.load();
    if (!encode) {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &r) != cudaSuccess || !fn)
            return mfs::op_fail(MFS_E_CUDA, op, "cuTensorMapEncodeTiled is not available");
        known.store(encode = (PFN_cuTensorMapEncodeTiled_v12000)fn);
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
                n_tokens, n_seqs, hq, hq / hkv, window, PT_M, 0, scale * 1.44269504088896340736f};
    if (A.g % 2 == 0) {
        A.down = 0;
        A.across = 1;
    }
    auto kernel = A.across ? prompt_mma_kernel<HD, true> : prompt_mma_kernel<HD, false>;
    int sms = 0;
    static mfs::PerDevice ready[2];
    cudaError_t e = mfs::op_device(ready[A.across], (const void*)kernel, S::BYTES, &sms);
    if (e == cudaSuccess) {
        const long long most = ((long long)n_tokens / (PT_M + A.down) + n_seqs) * (hq >> A.across);  // blocks there can be
        kernel<<<(unsigned)(most < sms ? most : sms), PT_THREADS, S::BYTES, st>>>(maps[0], maps[1], maps[2], A);
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
    if (n_kv_heads < 1 || n_q_heads < 1 || n_q_heads % n_kv_heads || n_q_heads > MFS_MAX_HEADS)
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
                                      : (head_dim == 128 ? run_f32<128> : run_f32<64>);
    return fn(n_tokens, n_seqs, cu, q, q_stride, n_q_heads, k, k_stride, v, v_stride, n_kv_heads, out, out_stride, scale, window, st);
}
