// A shared prefix under bf16 queries, on the tensor cores.
//
// One CTA per SM takes blocks of up to 256 rows as two tiles of 128 (one where the block has no more) and walks over its tiles
// of 128 positions: scores S = Q K^T and outputs O += P V are tcgen05 MMAs with accumulators in tensor memory (S 2 x 128
// columns, O 2 x head_dim).  Each row tile has four warps with one row per thread, which take the row's maximum without any
// exchange and write the weights back over the scores as bf16, the second product's A operand; while one tile is in its
// softmax the tensor cores work for the other.  The weights are taken against the maximum in use so far; only where a tile's
// own is more than 2^8 larger is O rescaled first.
//
// A bf16 cache's K and V tiles come by TMA, a box for each run of rows that lie in one page, where pages are whole groups of
// eight rows, the layout's unit; else, and where a tile reaches past the prefix, four warps copy them row by row.  An 8-bit
// cache's tiles go through those warps' registers, where each value becomes the bf16 that it is exactly.  Rows past the
// prefix are zeros, so nothing that lies there is seen.
//
// What bounds it: a step over 128 positions takes 3.3 k cycles, 2.7 k of them the tensor core's turns with 32 MMAs (a score
// product reads both operands from shared memory at its full rate), the rest the MMA warp's waits between them; 256 sequences
// of 64 query heads on 8 kv heads of 128 behind 32768 positions about 220 us of the call's 260 us, 1.2 PFLOP/s.  Over codes a step takes
// 6.5 k cycles: the conversions share the issue slots with the softmax, and the weights' second parts take 16 MMAs more (5.8 k without
// them).  A call of few steps is its start and end: 7.5 k cycles
// to the first part (launch, places, the first fetch of the code), 5.7 k until the queries are there, 1.5 k until the first scores,
// 7 k to write 128 KB of outputs: 64 sequences behind 7000 positions, three steps a CTA, 17 us.
//
// Over a bf16 cache the weights are rounded to bf16 (2^-8 of each at most), since the MMA takes both operands of a product in one
// type and the values are bf16; the sums take them unrounded.  Over codes, whose one-token attention keeps 11 bits of each, they are the
// sum of two such parts (2^-16): the second lies where the rest of the scores was, and takes products of its own.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>

#include "mfs_shared.cuh"

// A test build may have every CTA lose one tile of its ring (never fill it), so that waits run out.
#ifndef MFS_SHARED_LOST_TILE
#define MFS_SHARED_LOST_TILE -1
#endif

namespace {

constexpr int SM_M = 128;                     // rows of a row tile, positions of a tile
// Warps 0-3, 4-7: softmax of the two row tiles; 8: MMA; from 9 on: loads; the last one: the parts.  An 8-bit cache takes more
// warps to load it; without, the softmax has more registers.
template <bool QUANT>
struct SmWarps {
    static constexpr int THREADS = QUANT ? 512 : 384, LOADERS = QUANT ? 4 : 2, RL = SM_M / (32 * LOADERS);  // RL: rows of a tile a lane has
};

template <int HD>
struct SmShape {
    static constexpr int BOX = SM_M * 128;        // 128 rows of 64 elements, 128-byte swizzle
    static constexpr int TILE = BOX * (HD / 64);  // a 128-row tile of Q, K or V
};

// The ring's stages; codes on their way to the warps that turn them into bf16: two tiles of 32 rows for each.
template <int HD, bool QUANT>
struct SmRing {
    static constexpr int TILE = SmShape<HD>::TILE, STAGES = QUANT ? (HD == 128 ? 4 : 7) : HD == 128 ? 5 : 8;
    static constexpr int RAW = 32 * HD, RAWS = QUANT ? SmWarps<QUANT>::LOADERS * 2 * RAW : 0;
    static constexpr int BYTES = 1024 + 2 * TILE + STAGES * TILE + RAWS;
    static_assert(BYTES <= 230400 && STAGES * TILE >= SM_M * HD * 4, "a row tile's outputs leave through the ring");
};

struct SmBars {
    uint64_t kv_full[8], kv_empty[8], q_full[2], s_full[2], p_full[2], o_full[2], tail[2], drained;
    uint32_t tmem;
    int abort;  // a wait gave up
    int more, bad;
    ShPart part;
    ShParts parts;  // the last warp's, between the parts
};

template <int THREADS>
__device__ __forceinline__ void sm_sync() { asm volatile("bar.sync 0, %0;" ::"n"(THREADS) : "memory"); }

// Sixteen codes under `by` as bf16
__device__ __forceinline__ void codes_bf16(uint4 w, float by, uint4& a, uint4& b)
{
    const unsigned in[4] = {w.x, w.y, w.z, w.w};
    unsigned out[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        unsigned lo, hi;
        e4m3_f16(in[i], lo, hi);
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo)), y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        out[2 * i] = pack_bf16(x.x * by, x.y * by);
        out[2 * i + 1] = pack_bf16(y.x * by, y.y * by);
    }
    a = make_uint4(out[0], out[1], out[2], out[3]);
    b = make_uint4(out[4], out[5], out[6], out[7]);
}

template <int HD, bool QUANT>
__global__ void __launch_bounds__(SmWarps<QUANT>::THREADS, 1) shared_prefix_mma(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                                                                  const __grid_constant__ ShArgs A)
{
    using S = SmShape<HD>;
    using R = SmRing<HD, QUANT>;
    constexpr int STAGES = R::STAGES, THREADS = SmWarps<QUANT>::THREADS, LOADERS = SmWarps<QUANT>::LOADERS, RL = SmWarps<QUANT>::RL;
    constexpr int DEALER = THREADS / 32 - 1;
    extern __shared__ char sm_raw[];
    __shared__ SmBars B;
    char* base = (char*)(((uintptr_t)sm_raw + 1023) & ~(uintptr_t)1023);
    char* sq = base;
    char* ring = base + 2 * S::TILE;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 0) {
        B.abort = 0;
        for (int i = 0; i < STAGES; ++i) {
            bar_init(&B.kv_full[i], 32 * LOADERS);
            bar_init(&B.kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&B.q_full[i], SM_M);
            bar_init(&B.s_full[i], 1);
            bar_init(&B.p_full[i], SM_M);
            bar_init(&B.o_full[i], 1);
            bar_init(&B.tail[i], 1);
        }
        bar_init(&B.drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&B.tmem)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == 10) {  // the call's queries into L2, a share of them by each CTA, before anyone knows which are its own
        const unsigned per = A.hq * (HD * 2 / 128), lines = A.n_seqs * per;
        for (unsigned i = blockIdx.x * 32 + lane; i < lines; i += gridDim.x * 32)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(A.q + (long long)(i / per) * A.q_stride * 2 + (i % per) * 128) : "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, B.tmem, 0);  // columns: S of tile 0, S of tile 1, O of tile 0, O of tile 1

    // registers: 512 threads x 128 or 384 x 168 at launch; the softmax warps take more, the others less
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(QUANT ? 64 : 88));
        unsigned done = 0, asked = 0;  // tiles of the ring that earlier parts had; and all that were asked for by TMA or before such
        bool ok = true;
        // MMA
        constexpr uint32_t id_s = (1u << 4) | (1u << 7) | (1u << 10) | ((SM_M >> 3) << 17) | ((SM_M >> 4) << 24);
        constexpr uint32_t id_o = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((HD >> 3) << 17) | ((SM_M >> 4) << 24);
        unsigned tails = 0;  // tiles that reach past the prefix, after boxed ones
        unsigned leader = 0, p_par = 0, q_par = 0;  // bit x: of row tile x
        if (warp == 8) asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(leader));
        auto signal = [&](uint64_t* bar) {
            if (leader) commit(bar);
        };
        for (bool begun = false;; begun = true) {
            if (warp == DEALER) {
                ShPart p;
                ShParts parts;
                bool more;
                if (begun) {
                    more = B.more;
                    parts = B.parts;
                } else {
                    more = parts.start(A, blockIdx.x);
                }
                if (more) {
                    more = parts.next(A, p);
                    __syncwarp();
                    if (lane == 0) {
                        B.parts = parts;
                        B.part = p;
                    }
                }
                __syncwarp();
                if (lane == 0) {
                    B.more = more;
                    B.bad = 0;
                }
            }
            sm_sync<THREADS>();
            if (!B.more) break;
            const ShPart& P = B.part;
            const int nt = __shfl_sync(0xffffffffu, P.upto - P.from, 0), nl = 2 * nt;
            const bool two = __shfl_sync(0xffffffffu, P.w.ns * A.g - P.w.rb * 2 * SM_M, 0) > SM_M;
            ok = ok && !*(volatile int*)&B.abort;
            if (!ok) {
                // an earlier wait gave up: nothing more is done
            } else if (warp == 8) {
                const uint64_t dq = desc(su32(sq), 16), dk = desc(su32(ring), 16), dv = desc(su32(ring), S::BOX);
                auto scores = [&](int x, int slot) {
                    const uint64_t qa = dq + (uint64_t)(x * (S::TILE >> 4)), ka = dk + (uint64_t)(slot * (S::TILE >> 4));
                    const uint32_t d = tm + x * SM_M;
#pragma unroll
                    for (int k = 0; k < HD / 16; ++k) {
                        const uint64_t at = (k / 4) * (S::BOX >> 4) + (k % 4) * 2;
                        if (leader) mma_ss(d, qa + at, ka + at, id_s, k > 0);
                    }
                    signal(&B.s_full[x]);
                };
                auto outputs = [&](int x, int slot, bool first) {
                    const uint64_t va = dv + (uint64_t)(slot * (S::TILE >> 4));
                    const uint32_t d = tm + 2 * SM_M + x * HD, pa = tm + x * SM_M;
                    if (leader) mma_ts(d, pa, va, id_o, !first);
#pragma unroll
                    for (int k = 1; k < SM_M / 16; ++k)
                        if (leader) mma_ts(d, pa + 8 * k, va + (uint64_t)(k * 128), id_o, 1);
                    if constexpr (QUANT) {  // the weights' second parts
#pragma unroll
                        for (int k = 0; k < SM_M / 16; ++k)
                            if (leader) mma_ts(d, pa + SM_M / 2 + 8 * k, va + (uint64_t)(k * 128), id_o, 1);
                    }
                };
                // (the same in all lanes, and known to be: the operands' descriptors then stay in uniform registers, where an MMA
                // takes them; moving them there takes longer than the MMA)
                int m_slot = __shfl_sync(0xffffffffu, (int)(done % STAGES), 0);
                unsigned m_par = __shfl_sync(0xffffffffu, (done / STAGES) & 1, 0);
                auto step = [&]() {
                    if (++m_slot == STAGES) { m_slot = 0; m_par ^= 1; }
                };
                const int nx = two ? 2 : 1;
                if (nt > 0) {
                    ok = bar_wait(&B.kv_full[m_slot], m_par, &B.abort);
#pragma unroll 1
                    for (int x = 0; x < nx && ok; ++x) {
                        ok = bar_wait(&B.q_full[x], q_par >> x & 1, &B.abort);
                        if (!ok) break;
                        q_par ^= 1u << x;
                        fence_after();
                        scores(x, m_slot);
                    }
                    signal(&B.kv_empty[m_slot]);
                    step();
                }
                for (int t = 0; t < nt && ok; ++t) {
                    const bool next = t + 1 < nt;
                    const int vs = m_slot;
                    const unsigned v_par = m_par;
                    step();
                    const int ks = m_slot;
                    if (next) {
                        ok = bar_wait(&B.kv_full[ks], m_par, &B.abort);
                        step();
                    }
                    ok = ok && bar_wait(&B.kv_full[vs], v_par, &B.abort);
#pragma unroll 1
                    for (int x = 0; x < nx && ok; ++x) {
                        ok = bar_wait(&B.p_full[x], p_par >> x & 1, &B.abort);
                        if (!ok) break;
                        p_par ^= 1u << x;
                        fence_after();
                        outputs(x, vs, t == 0);
                        if (!next) signal(&B.o_full[x]);
                        else scores(x, ks);
                    }
                    signal(&B.kv_empty[vs]);
                    if (next) signal(&B.kv_empty[ks]);
                }
            } else if (warp - 9 < LOADERS) {
                // 32 RL rows of each tile, RL a lane: pages are looked up two tiles ahead, offsets and exponents found one ahead.
                // By TMA: the first warp's lanes have a box each.
                const int row0 = 32 * RL * (warp - 9);
                int page[RL], in_page[RL];  // page -1: none or a bad one, -2: past the prefix, or not this lane's
                auto boxed = [&](int t) { return !QUANT && A.box > 0 && (long long)P.w.p - (long long)(P.from + t) * SM_M >= SM_M; };
                auto look_up = [&](int t) {
                    const bool box = boxed(t);
#pragma unroll
                    for (int i = 0; i < RL; ++i) {
                        const int r = row0 + 32 * i + lane * (box ? A.box : 1);
                        const long long p = r < SM_M && !(box && i) ? (long long)(P.from + t) * SM_M + r : P.w.p;
                        const int j = page_of(A.C, (int)min(p, (long long)P.w.p));
                        in_page[i] = (int)p - j * A.C.page_size;
                        page[i] = t >= nt || p >= P.w.p ? -2 : j < A.C.table_width ? __ldg(A.C.table + P.reader * A.C.table_stride + j) : -1;
                    }
                };
                struct Row {
                    long long off[RL];  // bytes; a row without a page has the cache's first, whatever it is
                    unsigned xk, xv;    // 8 bits: the row's exponents; a box: its page and its first row there
                };
                auto resolve = [&]() {
                    Row R;
                    R.xk = QUANT ? 0u : (unsigned)A.C.n_pages;  // (past the last page a box is zeros)
                    R.xv = 0;
#pragma unroll
                    for (int i = 0; i < RL; ++i) {
                        R.off[i] = 0;
                        if (page[i] >= 0 && page[i] < A.C.n_pages) {
                            R.off[i] = ((long long)page[i] * A.C.page_stride + (long long)in_page[i] * A.C.row_stride + (long long)P.w.h * A.C.head_stride) * (QUANT ? 1 : 2);
                            if (QUANT) {
                                const long long x = (long long)page[i] * A.x_page + (long long)in_page[i] * A.x_row + (long long)P.w.h * A.x_head;
                                R.xk = __ldg(A.kx + x);
                                R.xv = __ldg(A.vx + x);
                            } else if (i == 0) {
                                R.xk = page[i];
                                R.xv = in_page[i];
                            }
                        } else if (page[i] != -2) {
                            *(volatile int*)&B.bad = 1;
                        }
                    }
                    return R;
                };
                int slot = done % STAGES, waiting = -1;
                unsigned par = ((done / STAGES) & 1) ^ 1;
                auto landed = [&](int ahead) {  // the copies before the last `ahead` are there: passed on
                    if (ahead) asm volatile("cp.async.wait_group 1;" ::: "memory");
                    else asm volatile("cp.async.wait_group 0;" ::: "memory");
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    bar_arrive(&B.kv_full[waiting]);
                    waiting = -1;
                };
                // 16-byte chunks of a row, rows of an instruction, instructions of 32 rows
                constexpr int CH = QUANT ? HD / 16 : HD / 8, RPI = 32 / CH, NI = 32 / RPI;
                const int ch = lane % CH, sub = lane / CH;
                // codes of tile t's rows (keys or values) on their way to the warp's place n mod 2
                char* raw = ring + STAGES * S::TILE + (warp - 9) * 2 * R::RAW;
                auto fetch = [&](const char* from, int t, int n) {
                    const long long left = (long long)P.w.p - (long long)(P.from + t) * SM_M - row0;
                    const unsigned to = su32(raw + (n & 1) * R::RAW) + lane * 16;
#pragma unroll
                    for (int j = 0; j < NI; ++j) {
                        const unsigned long long o = __shfl_sync(0xffffffffu, (unsigned long long)from, j * RPI + sub) + 16 * ch;
                        copy16(to + j * 512, (const void*)o, j * RPI + sub < left);
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                };
                Row now = {}, then = {};
                if (nt > 0) {
                    look_up(0);
                    now = resolve();
                    look_up(1);
                    if constexpr (QUANT) {
                        fetch(A.C.k + now.off[0], 0, 0);
                        fetch(A.C.v + now.off[0], 0, 1);
                    }
                }
                for (int t = 0; t < nt && ok; ++t) {
                    then = resolve();
                    look_up(t + 2);
                    const long long left = (long long)P.w.p - (long long)(P.from + t) * SM_M - row0;  // of the warp's rows, those of the prefix
#pragma unroll 1
                    for (int kv = 0; kv < 2; ++kv) {
                        const bool box = boxed(t);
                        if (box && warp != 9) {  // the first warp's alone
                            if (++slot == STAGES) { slot = 0; par ^= 1; }
                            continue;
                        }
                        if (!QUANT && A.box > 0 && warp != 9) {
                            // behind boxed tiles these warps have not followed the ring: the first one tells them
                            ok = ok && bar_wait(&B.tail[kv], tails & 1, &B.abort);
                        } else {
                            if (waiting >= 0 && !__all_sync(0xffffffffu, bar_try(&B.kv_empty[slot], par))) landed(0);
                            ok = ok && bar_wait(&B.kv_empty[slot], par, &B.abort);
                            if (ok && !QUANT && A.box > 0 && !box && lane == 0) bar_arrive(&B.tail[kv]);
                        }
                        if (!ok) break;
                        if (MFS_SHARED_LOST_TILE >= 0 && done + 2 * t + kv == (unsigned)MFS_SHARED_LOST_TILE) {
                            if (++slot == STAGES) { slot = 0; par ^= 1; }
                            continue;
                        }
                        char* dst = ring + slot * S::TILE + row0 * 128;
                        if (box) {
                            if (lane == 0) {  // its arrival, and the others'
                                bar_expect(&B.kv_full[slot], S::TILE);
                                asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(su32(&B.kv_full[slot])), "n"(32 * LOADERS - 1) : "memory");
                            }
                            __syncwarp();
                            if (lane * A.box < SM_M) {
#pragma unroll
                                for (int x = 0; x < HD / 64; ++x)
                                    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
                                                 ::"r"(su32(dst + x * S::BOX + lane * A.box * 128)), "l"(kv ? &mv : &mk), "r"(64 * x), "r"(now.xv), "r"(P.w.h), "r"(now.xk),
                                                 "r"(su32(&B.kv_full[slot])) : "memory");
                            }
                            asked = done + 2 * t + kv + 1;
                        } else if constexpr (!QUANT) {
                            // (few instructions for each copy: a warp issues them one behind the other)
                            const unsigned to = su32(dst + (ch / 8) * S::BOX) + sub * 128;
                            unsigned at[8 / RPI];  // of eight rows
#pragma unroll
                            for (int j = 0; j < 8 / RPI; ++j) at[j] = to + j * RPI * 128 + (((ch % 8) ^ (j * RPI + sub)) << 4);
#pragma unroll 1
                            for (int j0 = 0; j0 < 32 * RL; j0 += 8) {
                                const unsigned long long src = (unsigned long long)((kv ? A.C.v : A.C.k) + (j0 < 32 ? now.off[0] : now.off[RL - 1]));
                                unsigned long long o[8 / RPI];
#pragma unroll
                                for (int j = 0; j < 8 / RPI; ++j) o[j] = __shfl_sync(0xffffffffu, src, j0 % 32 + j * RPI + sub) + 16 * ch;
#pragma unroll
                                for (int j = 0; j < 8 / RPI; ++j) copy16(at[j] + j0 * 128, (const void*)o[j], j0 + j * RPI + sub < left);
                            }
                            asm volatile("cp.async.commit_group;" ::: "memory");
                            if (waiting >= 0) landed(1);
                            waiting = slot;
                        } else {
                            asm volatile("cp.async.wait_group 1;" ::: "memory");
                            __syncwarp();
                            // rows of exponent 0 are zeros, codes of NaN among theirs too (0 times NaN would not be)
                            if (__any_sync(0xffffffffu, (kv ? now.xv : now.xk) == 0)) {
                                uint4* mine = reinterpret_cast<uint4*>(raw + kv * R::RAW + lane * HD);
                                if ((kv ? now.xv : now.xk) == 0)
#pragma unroll 1
                                    for (int i = 0; i < HD / 16; ++i) mine[i] = make_uint4(0u, 0u, 0u, 0u);
                                __syncwarp();
                            }
                            const uint4* in = reinterpret_cast<const uint4*>(raw + kv * R::RAW) + lane;
                            const bool odd = ch & 4;  // lanes whose chunks lie in the second box store them in the other order: other banks
#pragma unroll 1
                            for (int j0 = 0; j0 < NI; j0 += 4) {
                                uint4 w[4];
                                float by[4];
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    w[j] = in[32 * (j0 + j)];
                                    by[j] = pow2_of(__shfl_sync(0xffffffffu, kv ? now.xv : now.xk, (j0 + j) * RPI + sub));
                                }
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const int r = (j0 + j) * RPI + sub;
                                    uint4 x, y;
                                    codes_bf16(w[j], by[j], x, y);
                                    char* d = dst + (ch / 4) * S::BOX + r * 128;
                                    const int cx = (2 * ch % 8) ^ (r & 7);
                                    *reinterpret_cast<uint4*>(d + ((odd ? cx ^ 1 : cx) << 4)) = odd ? y : x;
                                    *reinterpret_cast<uint4*>(d + ((odd ? cx : cx ^ 1) << 4)) = odd ? x : y;
                                }
                            }
                            __syncwarp();
                            if (t + 1 < nt) fetch((kv ? A.C.v : A.C.k) + then.off[0], t + 1, kv);
                            else asm volatile("cp.async.commit_group;" ::: "memory");
                            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                            bar_arrive(&B.kv_full[slot]);
                        }
                        if (++slot == STAGES) { slot = 0; par ^= 1; }
                    }
                    now = then;
                }
                if (nt > 0 && !boxed(nt - 1)) ++tails;
                if (waiting >= 0) landed(0);
                asm volatile("cp.async.wait_all;" ::: "memory");
            }
            done += nl;
            sm_sync<THREADS>();
        }
        if (warp == 8) {
            signal(&B.drained);
            if (leader) bar_drain(&B.drained, 0);
        }
        // No copy is in flight when the CTA ends, whichever warp's wait gave up: this one may have asked for all of a last part's
        // tiles without a wait, and not know.  (All waits of the parts are behind the barrier that ended the last one.)
        if (warp == 9 && lane == 0 && *(volatile int*)&B.abort)
            for (unsigned k = asked > STAGES ? asked - STAGES : 0; k < asked; ++k) bar_drain(&B.kv_full[k % STAGES], (k / STAGES) & 1);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(QUANT ? 192 : 208));
        const int x = warp >> 2, row = tid & (SM_M - 1);
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tm + lanes + x * SM_M, to = tm + lanes + 2 * SM_M + x * HD;
        unsigned s_par = 0, o_par = 0;
        bool ok = true;
        // The first turn is a rehearsal while the first part is found: one tile's softmax over whatever tensor memory holds, so
        // that its instructions, whose first fetch takes several times their execution, are there when the scores are.
        for (bool real = false;; real = true) {
            int nt = 1, last = SM_M;  // tiles; positions of the last one
            long long at = -1;        // where the row's results go, in rows; -1: no such row
            if (real) {
                sm_sync<THREADS>();
                if (!B.more) break;
                const ShPart& P = B.part;
                nt = P.upto - P.from;
                const long long left = (long long)P.w.p - (long long)(P.upto - 1) * SM_M;
                last = left < SM_M ? (int)left : SM_M;
                const int rows = P.w.ns * A.g - P.w.rb * 2 * SM_M - x * SM_M;  // of this tile and those behind it
                ok = ok && !*(volatile int*)&B.abort;
                at = -1;
                unsigned long long q = (unsigned long long)A.q;  // the row's query; rows past the last have zeros
                if (row < rows) {
                    const int r = P.w.rb * 2 * SM_M + x * SM_M + row, s = P.w.s0 + r / A.g, h = P.w.h * A.g + r % A.g;
                    at = P.slot == 2 ? (long long)s * A.hq + h : ((long long)blockIdx.x * 2 + P.slot) * (2 * SM_M) + x * SM_M + row;
                    q += ((long long)s * A.q_stride + (long long)h * HD) * 2;
                }
                if (nt > 0 && rows > 0) {
                    // a warp's 32 rows, whole rows at a time, all on their way together
                    constexpr int CH = HD / 8, RPI = 32 / CH;
                    const int ch = lane % CH, sub = lane / CH;
                    uint4 v[CH];
#pragma unroll
                    for (int j = 0; j < CH; ++j) {
                        const unsigned long long from = __shfl_sync(0xffffffffu, q, j * RPI + sub);
                        v[j] = (row & ~31) + j * RPI + sub < rows ? __ldg(reinterpret_cast<const uint4*>(from) + ch) : make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int j = 0; j < CH; ++j) {
                        const int r = (row & ~31) + j * RPI + sub;
                        *reinterpret_cast<uint4*>(sq + x * S::TILE + (ch / 8) * S::BOX + r * 128 + (((ch % 8) ^ (r & 7)) << 4)) = v[j];
                    }
                }
                if (rows <= 0) nt = 0;
            }
            if (nt > 0 && real) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                bar_arrive(&B.q_full[x]);
            }
            float m = -INFINITY;      // the maximum in use (raw scores), exact up to 2^8 in the weights
            uint64_t l2[2] = {0, 0};  // the sum, in four parts
            for (int t = 0; t < nt && ok; ++t) {
                if (real) {
                    ok = bar_wait(&B.s_full[x], s_par, &B.abort);
                    if (!ok) break;
                    s_par ^= 1;
                }
                __syncwarp();
                fence_after();
                uint32_t s[SM_M];
#pragma unroll
                for (int k = 0; k < 4; ++k) tld32(ts + 32 * k, s + 32 * k);
                tld_wait();
                if (__builtin_expect(t == nt - 1 && last < SM_M, 0)) {  // places past the prefix
#pragma unroll
                    for (int k = 0; k < SM_M; ++k)
                        if (k >= last) s[k] = 0xff800000u;
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < SM_M; k += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], __uint_as_float(s[k + e]), __uint_as_float(s[k + 4 + e]));
                const float mt = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
                if (t == 0) {
                    m = mt;
                } else {
                    const bool up = mt > m && !((mt - m) * A.c <= 8.f);
                    if (__any_sync(0xffffffffu, up)) {
                        const float a = !up ? 1.f : m == -INFINITY ? 0.f : ex2((m - mt) * A.c);
                        if (up) m = mt;
                        l2[0] = mul2(l2[0], pair(a, a));
                        l2[1] = mul2(l2[1], pair(a, a));
#pragma unroll 1
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
                    uint32_t p[16], rest[QUANT ? 16 : 1];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const int e = 32 * quarter + 2 * k;
                        float u, w;
                        unpair(fma2(pair(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), cc, bb), u, w);
                        u = ex2(u);
                        w = ex2(w);
                        l2[k & 1] = add2(l2[k & 1], pair(u, w));
                        p[k] = pack_bf16(u, w);
                        if constexpr (QUANT) {
                            unpair(fma2(pair(__uint_as_float(p[k] << 16), __uint_as_float(p[k] & 0xffff0000u)), pair(-1.f, -1.f), pair(u, w)), u, w);
                            rest[k] = pack_bf16(u, w);
                        }
                    }
                    tst16(ts + 16 * quarter, p);
                    if constexpr (QUANT) tst16(ts + SM_M / 2 + 16 * quarter, rest);
                }
                tst_wait();
                fence_before();
                if (real) bar_arrive(&B.p_full[x]);
            }
            if (!real) continue;
            if (nt > 0 && ok) ok = bar_wait(&B.o_full[x], o_par, &B.abort);
            if (nt > 0) o_par ^= 1;
            __syncwarp();
            fence_after();
            float* po = B.part.slot == 2 ? A.row_o : A.part_o;
            if (at >= 0) {
                float l0, l1;
                unpair(add2(l2[0], l2[1]), l0, l1);
                (B.part.slot == 2 ? A.row_ml : A.part_ml)[at] = make_float2(m, ok && !*(volatile int*)&B.bad ? l0 + l1 : NAN);
            }
            // A row leaves by one bulk copy from shared memory, its 16-byte units in the order that lets eight lanes' stores meet
            // different banks; the join knows it.  The first row tile's place is that of the queries, which no product reads
            // any more when its outputs are done, the second one's the ring.
            if (__any_sync(0xffffffffu, at >= 0)) {
                char* mine = (x ? ring : sq) + row * (HD * 4);
#pragma unroll 1
                for (int k = 0; k < HD; k += 32) {
                    uint32_t u[32];
                    if (nt > 0) {
                        tld32(to + k, u);
                        tld_wait();
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) u[e] = 0u;
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *reinterpret_cast<uint4*>(mine + ((((k / 4) + e) ^ (row & 7)) << 4)) = make_uint4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                const bool pieces = B.part.slot != 2;  // then a warp's rows lie one behind the other
                const int n = __popc(__ballot_sync(0xffffffffu, at >= 0)) * (HD * 4);
                __syncwarp();  // the first lane's copy reads what all lanes have written
                if (pieces && lane == 0)
                    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(po + at * HD), "r"(su32(mine)), "r"(n) : "memory");
                else if (!pieces && at >= 0)
                    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(po + at * HD), "r"(su32(mine)), "n"(HD * 4) : "memory");
                asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
            }
            fence_before();
            sm_sync<THREADS>();
        }
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    if (warp == 8) {
        __syncwarp();
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512u));
    }
}

// Tensor maps of a bf16 cache, for boxes of A.box rows; 0: it is copied row by row.
template <int HD>
void prefix_maps(ShArgs& A, CUtensorMap (&maps)[2])
{
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> known{nullptr};
    A.box = 0;
    const Cache& C = A.C;
    if (C.page_size % 8) return;
    PFN_cuTensorMapEncodeTiled_v12000 encode = known.load();
    if (!encode) {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &r) != cudaSuccess || !fn) return;
        known.store(encode = (PFN_cuTensorMapEncodeTiled_v12000)fn);
    }
    const int run = C.page_size & -C.page_size, box = run < SM_M ? run : SM_M;
    // (the strides of dimensions of one place are not used, but have to be sound)
    auto stride = [](long long n, long long s) { return (cuuint64_t)(n > 1 ? s : HD) * 2; };
    const cuuint64_t dim[4] = {(cuuint64_t)HD, (cuuint64_t)C.page_size, (cuuint64_t)C.n_kv_heads, (cuuint64_t)C.n_pages};
    const cuuint64_t str[3] = {stride(C.page_size, C.row_stride), stride(C.n_kv_heads, C.head_stride), stride(C.n_pages, C.page_stride)};
    const cuuint32_t size[4] = {64, (cuuint32_t)box, 1, 1}, es[4] = {1, 1, 1, 1};
    for (int i = 0; i < 3; ++i)
        if (str[i] == 0 || str[i] >= (1ull << 40)) return;
    for (int i = 0; i < 2; ++i)
        if (encode(&maps[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, i ? C.v : C.k, dim, str, size, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return;
    A.box = box;
}

template <int HD, bool QUANT>
cudaError_t prefix_mma(ShArgs& A, cudaStream_t st)
{
    using R = SmRing<HD, QUANT>;
    CUtensorMap maps[2] = {};
    if (!QUANT) prefix_maps<HD>(A, maps);
    int sms = 0;
    static mfs::PerDevice ready;
    const cudaError_t e = mfs::op_device(ready, (const void*)shared_prefix_mma<HD, QUANT>, R::BYTES, &sms);
    if (e != cudaSuccess) return e;
    shared_prefix_mma<HD, QUANT><<<A.ctas, SmWarps<QUANT>::THREADS, R::BYTES, st>>>(maps[0], maps[1], A);
    return cudaGetLastError();
}

}  // namespace
