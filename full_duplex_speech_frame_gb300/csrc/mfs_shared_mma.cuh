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
// The weights are rounded to bf16 (2^-8 of each at most), since the MMA takes both operands of a product in one type and the
// values are bf16; the sums take them unrounded.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>

#include "mfs_shared.cuh"

namespace {

constexpr int SM_LOADERS = 4;
constexpr int SM_M = 128;                     // rows of a row tile, positions of a tile
constexpr int SM_THREADS = 512;               // warps 0-3, 4-7: softmax of the two row tiles; 8: MMA; 9-12: loads; 15: the parts

template <int HD>
struct SmShape {
    static constexpr int BOX = SM_M * 128;        // 128 rows of 64 elements, 128-byte swizzle
    static constexpr int TILE = BOX * (HD / 64);  // a 128-row tile of Q, K or V
    static constexpr int STAGES = HD == 128 ? 5 : 8;
    static constexpr int BYTES = 1024 + 2 * TILE + STAGES * TILE;
};

struct SmBars {
    uint64_t kv_full[8], kv_empty[8], q_full[2], s_full[2], p_full[2], o_full[2], drained;
    uint32_t tmem;
    int abort;  // a wait gave up
    int more, bad;
    ShPart part;
    ShParts parts;  // warp 15's, between the parts
};

__device__ __forceinline__ void sm_sync() { asm volatile("bar.sync 0, %0;" ::"n"(SM_THREADS) : "memory"); }

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
__global__ void __launch_bounds__(SM_THREADS, 1) shared_prefix_mma(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                                                                  const __grid_constant__ ShArgs A)
{
    using S = SmShape<HD>;
    constexpr int STAGES = S::STAGES;
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
            bar_init(&B.kv_full[i], 32 * SM_LOADERS);
            bar_init(&B.kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&B.q_full[i], SM_M);
            bar_init(&B.s_full[i], 1);
            bar_init(&B.p_full[i], SM_M);
            bar_init(&B.o_full[i], 1);
        }
        bar_init(&B.drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&B.tmem)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == 15) {
        ShParts parts;
        const bool more = parts.start(A, blockIdx.x);
        if (lane == 0) {
            B.more = more;
            if (more) B.parts = parts;
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, B.tmem, 0);  // columns: S of tile 0, S of tile 1, O of tile 0, O of tile 1

    // registers: 512 threads x 128 at launch; the softmax warps take more, the others less
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        unsigned done = 0, asked = 0;  // tiles of the ring that earlier parts had; and all that were asked for by TMA or before such
        bool ok = true;
        // MMA
        constexpr uint32_t id_s = (1u << 4) | (1u << 7) | (1u << 10) | ((SM_M >> 3) << 17) | ((SM_M >> 4) << 24);
        constexpr uint32_t id_o = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((HD >> 3) << 17) | ((SM_M >> 4) << 24);
        unsigned leader = 0, p_par[2] = {0, 0}, q_par[2] = {0, 0};
        if (warp == 8) asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(leader));
        auto signal = [&](uint64_t* bar) {
            if (leader) commit(bar);
        };
        for (;;) {
            if (warp == 15) {
                ShPart p;
                bool more = B.more;
                if (more) {
                    ShParts parts = B.parts;
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
            sm_sync();
            if (!B.more) break;
            const ShPart& P = B.part;
            const int nt = P.upto - P.from, nl = 2 * nt;
            const bool two = P.w.ns * A.g - P.w.rb * 2 * SM_M > SM_M;
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
                };
                int slot = done % STAGES;
                unsigned par = (done / STAGES) & 1;
                auto step = [&]() {
                    if (++slot == STAGES) { slot = 0; par ^= 1; }
                };
                const int nx = two ? 2 : 1;
                if (nt > 0) {
                    ok = bar_wait(&B.kv_full[slot], par, &B.abort);
                    for (int x = 0; x < nx && ok; ++x) {
                        ok = bar_wait(&B.q_full[x], q_par[x], &B.abort);
                        if (!ok) break;
                        q_par[x] ^= 1;
                        fence_after();
                        scores(x, slot);
                    }
                    signal(&B.kv_empty[slot]);
                    step();
                }
                for (int t = 0; t < nt && ok; ++t) {
                    const bool next = t + 1 < nt;
                    const int vs = slot;
                    const unsigned v_par = par;
                    step();
                    const int ks = slot;
                    if (next) {
                        ok = bar_wait(&B.kv_full[ks], par, &B.abort);
                        step();
                    }
                    ok = ok && bar_wait(&B.kv_full[vs], v_par, &B.abort);
                    for (int x = 0; x < nx && ok; ++x) {
                        ok = bar_wait(&B.p_full[x], p_par[x], &B.abort);
                        if (!ok) break;
                        p_par[x] ^= 1;
                        fence_after();
                        outputs(x, vs, t == 0);
                        if (!next) signal(&B.o_full[x]);
                        else scores(x, ks);
                    }
                    signal(&B.kv_empty[vs]);
                    if (next) signal(&B.kv_empty[ks]);
                }
            } else if (warp - 9 < SM_LOADERS) {
                // 32 rows of each tile, one a lane: pages are looked up two tiles ahead, offsets and exponents found one ahead.
                // By TMA: the first warp's lanes have a box each.
                const int row0 = 32 * (warp - 9);
                int page, in_page;  // page -1: none or a bad one, -2: past the prefix, or not this lane's
                auto boxed = [&](int t) { return !QUANT && A.box > 0 && (long long)P.w.p - (long long)(P.from + t) * SM_M >= SM_M; };
                auto look_up = [&](int t) {
                    const bool box = boxed(t);
                    const long long p = box && row0 + lane * A.box >= SM_M ? P.w.p : (long long)(P.from + t) * SM_M + row0 + lane * (box ? A.box : 1);
                    const int j = page_of(A.C, (int)min(p, (long long)P.w.p));
                    in_page = (int)p - j * A.C.page_size;
                    page = t >= nt || p >= P.w.p ? -2 : j < A.C.table_width ? __ldg(A.C.table + P.reader * A.C.table_stride + j) : -1;
                };
                struct Row {
                    long long off;  // bytes; a row without a page has the cache's first, whatever it is
                    unsigned xk, xv;  // 8 bits: the row's exponents; a box: its page and its first row there
                };
                auto resolve = [&]() {
                    Row R = {0, (unsigned)A.C.n_pages, 0u};  // (past the last page a box is zeros)
                    if (QUANT) R.xk = 0;
                    if (page >= 0 && page < A.C.n_pages) {
                        R.off = ((long long)page * A.C.page_stride + (long long)in_page * A.C.row_stride + (long long)P.w.h * A.C.head_stride) * (QUANT ? 1 : 2);
                        if (QUANT) {
                            const long long x = (long long)page * A.x_page + (long long)in_page * A.x_row + (long long)P.w.h * A.x_head;
                            R.xk = __ldg(A.kx + x);
                            R.xv = __ldg(A.vx + x);
                        } else {
                            R.xk = page;
                            R.xv = in_page;
                        }
                    } else if (page != -2) {
                        *(volatile int*)&B.bad = 1;
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
                uint4 w[QUANT ? NI : 1];
                auto load = [&](int j, const char* from, int t) {  // codes of instruction j's rows
                    const long long left = (long long)P.w.p - (long long)(P.from + t) * SM_M - row0;
                    const unsigned long long o = __shfl_sync(0xffffffffu, (unsigned long long)from, j * RPI + sub);
                    w[QUANT ? j : 0] = j * RPI + sub < left ? __ldg(reinterpret_cast<const uint4*>(o) + ch) : make_uint4(0u, 0u, 0u, 0u);
                };
                Row now = {0, 0u, 0u}, then = {0, 0u, 0u};
                if (nt > 0) {
                    look_up(0);
                    now = resolve();
                    look_up(1);
                    if constexpr (QUANT) {
#pragma unroll
                        for (int j = 0; j < NI; ++j) load(j, A.C.k + now.off, 0);
                    }
                }
                for (int t = 0; t < nt && ok; ++t) {
                    then = resolve();
                    look_up(t + 2);
                    const long long left = (long long)P.w.p - (long long)(P.from + t) * SM_M - row0;  // of the warp's rows, those of the prefix
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        if (waiting >= 0 && !__all_sync(0xffffffffu, bar_try(&B.kv_empty[slot], par))) landed(0);
                        ok = ok && bar_wait(&B.kv_empty[slot], par, &B.abort);
                        if (!ok) break;
                        char* dst = ring + slot * S::TILE + row0 * 128;
                        if (boxed(t)) {
                            if (warp == 9 && lane == 0) bar_expect(&B.kv_full[slot], S::TILE);  // its arrival
                            __syncwarp();
                            if (warp == 9 && lane * A.box < SM_M) {
#pragma unroll
                                for (int x = 0; x < HD / 64; ++x)
                                    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
                                                 ::"r"(su32(dst + x * S::BOX + lane * A.box * 128)), "l"(kv ? &mv : &mk), "r"(64 * x), "r"(now.xv), "r"(P.w.h), "r"(now.xk),
                                                 "r"(su32(&B.kv_full[slot])) : "memory");
                            }
                            if (warp != 9 || lane != 0) bar_arrive(&B.kv_full[slot]);
                            asked = done + 2 * t + kv + 1;
                        } else if constexpr (!QUANT) {
                            // (few instructions for each copy: a warp issues them one behind the other)
                            const unsigned long long src = (unsigned long long)((kv ? A.C.v : A.C.k) + now.off);
                            const unsigned to = su32(dst + (ch / 8) * S::BOX) + sub * 128;
                            unsigned at[8 / RPI];  // of eight rows
#pragma unroll
                            for (int j = 0; j < 8 / RPI; ++j) at[j] = to + j * RPI * 128 + (((ch % 8) ^ (j * RPI + sub)) << 4);
                            auto copy = [&](auto whole) {
#pragma unroll
                                for (int j0 = 0; j0 < 32; j0 += 8) {
                                    unsigned long long o[8 / RPI];
#pragma unroll
                                    for (int j = 0; j < 8 / RPI; ++j) o[j] = __shfl_sync(0xffffffffu, src, j0 + j * RPI + sub) + 16 * ch;
#pragma unroll
                                    for (int j = 0; j < 8 / RPI; ++j) {
                                        if (decltype(whole)::value)
                                            asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(at[j] + j0 * 128), "l"(o[j]) : "memory");
                                        else
                                            copy16(at[j] + j0 * 128, (const void*)o[j], j0 + j * RPI + sub < left);
                                    }
                                }
                            };
                            if (left >= 32) copy(std::true_type());
                            else copy(std::false_type());
                            asm volatile("cp.async.commit_group;" ::: "memory");
                            if (waiting >= 0) landed(1);
                            waiting = slot;
                        } else {
                            const bool more = kv == 0 || t + 1 < nt;
                            const char* next = kv ? A.C.k + then.off : A.C.v + now.off;
#pragma unroll
                            for (int j = 0; j < NI; ++j) {
                                const int r = j * RPI + sub;
                                const float by = pow2_of(__shfl_sync(0xffffffffu, kv ? now.xv : now.xk, r));
                                uint4 x, y;
                                codes_bf16(w[j], by, x, y);
                                char* d = dst + (ch / 4) * S::BOX + r * 128;
                                *reinterpret_cast<uint4*>(d + (((2 * ch % 8) ^ (r & 7)) << 4)) = x;
                                *reinterpret_cast<uint4*>(d + ((((2 * ch + 1) % 8) ^ (r & 7)) << 4)) = y;
                                if (more) load(j, next, t + kv);
                            }
                            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                            bar_arrive(&B.kv_full[slot]);
                        }
                        if (++slot == STAGES) { slot = 0; par ^= 1; }
                    }
                    now = then;
                }
                if (waiting >= 0) landed(0);
                asm volatile("cp.async.wait_all;" ::: "memory");
            }
            done += nl;
            sm_sync();
        }
        if (warp == 8) {
            signal(&B.drained);
            if (leader) bar_drain(&B.drained, 0);
        }
        if (warp == 9 && lane == 0 && !ok)  // no copy is in flight when the CTA ends, whichever wait gave up
            for (unsigned k = asked > STAGES ? asked - STAGES : 0; k < asked; ++k) bar_drain(&B.kv_full[k % STAGES], (k / STAGES) & 1);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        const int x = warp >> 2, row = tid & (SM_M - 1);
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tm + lanes + x * SM_M, to = tm + lanes + 2 * SM_M + x * HD;
        unsigned s_par = 0, o_par = 0;
        bool ok = true;
        for (;;) {
            sm_sync();
            if (!B.more) break;
            int nt, last;    // tiles; positions of the last one
            long long at;    // where the row's results go, in rows; -1: no such row
            {
                const ShPart& P = B.part;
                nt = P.upto - P.from;
                const long long left = (long long)P.w.p - (long long)(P.upto - 1) * SM_M;
                last = left < SM_M ? (int)left : SM_M;
                const int rows = P.w.ns * A.g - P.w.rb * 2 * SM_M - x * SM_M;  // of this tile and those behind it
                ok = ok && !*(volatile int*)&B.abort;
                at = -1;
                if (row < rows) {
                    const int r = P.w.rb * 2 * SM_M + x * SM_M + row, s = P.w.s0 + r / A.g, h = P.w.h * A.g + r % A.g;
                    at = P.slot == 2 ? (long long)s * A.hq + h : ((long long)blockIdx.x * 2 + P.slot) * (2 * SM_M) + x * SM_M + row;
                    if (nt > 0) {
                        const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const bf16*>(A.q) + (long long)s * A.q_stride + (long long)h * HD);
#pragma unroll
                        for (int c = 0; c < HD / 8; ++c)
                            *reinterpret_cast<uint4*>(sq + x * S::TILE + (c / 8) * S::BOX + row * 128 + (((c % 8) ^ (row & 7)) << 4)) = __ldg(q + c);
                    }
                } else if (nt > 0) {
#pragma unroll
                    for (int c = 0; c < HD / 8; ++c)
                        *reinterpret_cast<uint4*>(sq + x * S::TILE + (c / 8) * S::BOX + row * 128 + (((c % 8) ^ (row & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                }
                if (rows <= 0) nt = 0;
            }
            if (nt > 0) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                bar_arrive(&B.q_full[x]);
            }
            float m = -INFINITY;      // the maximum in use (raw scores), exact up to 2^8 in the weights
            uint64_t l2[2] = {0, 0};  // the sum, in four parts
            for (int t = 0; t < nt && ok; ++t) {
                ok = bar_wait(&B.s_full[x], s_par, &B.abort);
                if (!ok) break;
                s_par ^= 1;
                __syncwarp();
                fence_after();
                uint32_t s[SM_M];
#pragma unroll
                for (int k = 0; k < 4; ++k) tld32(ts + 32 * k, s + 32 * k);
                tld_wait();
                if (t == nt - 1 && last < SM_M) {  // places past the prefix
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
                    tst16(ts + 16 * quarter, p);
                }
                tst_wait();
                fence_before();
                bar_arrive(&B.p_full[x]);
            }
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
            // 32 elements of a row at a time: the eight lanes of eight rows exchange 16-byte units so that a store writes
            // 128 bytes of each of four rows
            const int j = lane & 7;
            if (__any_sync(0xffffffffu, at >= 0)) {
#pragma unroll
                for (int k = 0; k < HD; k += 32) {
                    uint32_t u[8][4];
                    if (nt > 0) {
                        tld32(to + k, &u[0][0]);
                        tld_wait();
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) u[e / 4][e % 4] = 0u;
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
                    for (int y = 0; y < 8; ++y) {
                        const long long to_row = __shfl_sync(0xffffffffu, at, (lane & ~7) + y);
                        if (to_row >= 0) *reinterpret_cast<uint4*>(po + to_row * HD + k + 4 * j) = make_uint4(u[y][0], u[y][1], u[y][2], u[y][3]);
                    }
                }
            }
            fence_before();
            sm_sync();
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
    using S = SmShape<HD>;
    CUtensorMap maps[2] = {};
    if (!QUANT) prefix_maps<HD>(A, maps);
    int sms = 0;
    static mfs::PerDevice ready;
    const cudaError_t e = mfs::op_device(ready, (const void*)shared_prefix_mma<HD, QUANT>, S::BYTES, &sms);
    if (e != cudaSuccess) return e;
    shared_prefix_mma<HD, QUANT><<<A.ctas, SM_THREADS, S::BYTES, st>>>(maps[0], maps[1], A);
    return cudaGetLastError();
}

}  // namespace
