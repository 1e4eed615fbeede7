// A shared prefix under bf16 queries, on the tensor cores.
//
// One CTA per SM takes blocks of up to 256 rows as two tiles of 128 (one where the block has no more) and walks over its tiles
// of 128 positions: scores S = Q K^T and outputs O += P V are tcgen05 MMAs with accumulators in tensor memory (S 2 x 128
// columns, O 2 x head_dim).  Each row tile has four warps with one row per thread, which take the row's maximum without any
// exchange and write the weights back over the scores as bf16, the second product's A operand; while one tile is in its
// softmax the tensor cores work for the other.  The weights are taken against the maximum in use so far; only where a tile's
// own is more than 2^8 larger is O rescaled first.
//
// Three warps fill the ring of K and V tiles, a tile each in turn, in the layout that the MMA reads, row by row, since pages
// may have any size: a bf16 cache by asynchronous copies, an 8-bit one by way of registers, where each value becomes the bf16
// that it is exactly.  Rows past the prefix are zeros, so nothing that lies there is seen.
//
// The weights are rounded to bf16 (2^-8 of each at most), since the MMA takes both operands of a product in one type and the
// values are bf16; the sums take them unrounded.
#pragma once
#include "mfs_shared.cuh"

namespace {

constexpr int SM_M = 128;                     // rows of a row tile, positions of a tile
constexpr int SM_THREADS = 384;               // warps 0-3, 4-7: softmax of the two row tiles; 8: MMA; 9-11: loads (11 also the parts)

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
    ShParts parts;  // warp 11's, between the parts
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
__global__ void __launch_bounds__(SM_THREADS, 1) shared_prefix_mma(const __grid_constant__ ShArgs A)
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
            bar_init(&B.kv_full[i], 32);
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
    if (warp == 11) {
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

    // registers: 384 threads x 168 at launch; the softmax warps take more, the others less
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        unsigned done = 0;  // tiles of the ring that earlier parts had
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
            if (warp == 11) {
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
            } else {
                // the tiles' rows, four a lane: where they lie, -1 for those past the prefix
                long long off[4];
                unsigned exps = 0;  // of the rows, a byte each
                auto look_up = [&](int n) {
                    exps = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const long long p = (long long)(P.from + (n >> 1)) * SM_M + lane + 32 * i;
                        off[i] = -1;
                        int page, row;
                        if (n >= nl || p >= P.w.p) continue;
                        if (!row_place(A.C, P.reader, (int)p, page, row)) {
                            *(volatile int*)&B.bad = 1;
                            continue;
                        }
                        off[i] = (long long)page * A.C.page_stride + (long long)row * A.C.row_stride + (long long)P.w.h * A.C.head_stride;
                        if (QUANT)
                            exps |= (unsigned)__ldg((n & 1 ? A.vx : A.kx) + (long long)page * A.x_page + (long long)row * A.x_row + (long long)P.w.h * A.x_head) << (8 * i);
                    }
                };
                int n = (int)((unsigned)(warp - 9 + 3) - done % 3u) % 3, slot = (done + n) % STAGES, waiting = -1;
                unsigned par = (((done + n) / STAGES) & 1) ^ 1;
                auto landed = [&](int ahead) {  // the copies before the last `ahead` are there: passed on
                    if (ahead) asm volatile("cp.async.wait_group 1;" ::: "memory");
                    else asm volatile("cp.async.wait_group 0;" ::: "memory");
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    bar_arrive(&B.kv_full[waiting]);
                    waiting = -1;
                };
                look_up(n);
                for (; n < nl; n += 3) {
                    if (waiting >= 0 && !__all_sync(0xffffffffu, bar_try(&B.kv_empty[slot], par))) landed(0);
                    ok = bar_wait(&B.kv_empty[slot], par, &B.abort);
                    if (!ok) break;
                    const char* src = n & 1 ? A.C.v : A.C.k;
                    char* dst = ring + slot * S::TILE;
                    if constexpr (!QUANT) {
                        constexpr int CH = HD / 8, RPI = 32 / CH;  // 16-byte chunks of a row, rows of an instruction
                        const int ch = lane % CH;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll 8
                            for (int j = 0; j < 32; j += RPI) {
                                const int in = j + lane / CH, row = 32 * i + in;
                                const long long o = __shfl_sync(0xffffffffu, off[i], in);
                                copy16(su32(dst + (ch / 8) * S::BOX + row * 128 + (((ch % 8) ^ (row & 7)) << 4)), src + (o < 0 ? 0 : (o + 8 * ch) * 2), o >= 0);
                            }
                        asm volatile("cp.async.commit_group;" ::: "memory");
                        if (waiting >= 0) landed(1);
                        waiting = slot;
                    } else {
                        constexpr int CH = HD / 16, RPI = 32 / CH;  // 16-byte chunks of a row's codes
                        const int ch = lane % CH;
                        const unsigned x4 = exps;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint4 w[CH];
#pragma unroll
                            for (int j = 0; j < CH; ++j) {
                                const long long o = __shfl_sync(0xffffffffu, off[i], j * RPI + lane / CH);
                                w[j] = o < 0 ? make_uint4(0u, 0u, 0u, 0u) : __ldg(reinterpret_cast<const uint4*>(src + o + 16 * ch));
                            }
#pragma unroll
                            for (int j = 0; j < CH; ++j) {
                                const int in = j * RPI + lane / CH, row = 32 * i + in;
                                const float by = pow2_of(__shfl_sync(0xffffffffu, x4, in) >> (8 * i) & 255u);
                                uint4 a, b;
                                codes_bf16(w[j], by, a, b);
                                char* d = dst + (ch / 4) * S::BOX + row * 128;
                                *reinterpret_cast<uint4*>(d + (((2 * ch % 8) ^ (row & 7)) << 4)) = a;
                                *reinterpret_cast<uint4*>(d + ((((2 * ch + 1) % 8) ^ (row & 7)) << 4)) = b;
                            }
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        bar_arrive(&B.kv_full[slot]);
                    }
                    look_up(n + 3);
                    slot += 3;
                    if (slot >= STAGES) { slot -= STAGES; par ^= 1; }
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
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
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

template <int HD, bool QUANT>
cudaError_t prefix_mma(const ShArgs& A, cudaStream_t st)
{
    using S = SmShape<HD>;
    int sms = 0;
    static mfs::PerDevice ready;
    const cudaError_t e = mfs::op_device(ready, (const void*)shared_prefix_mma<HD, QUANT>, S::BYTES, &sms);
    if (e != cudaSuccess) return e;
    shared_prefix_mma<HD, QUANT><<<A.ctas, SM_THREADS, S::BYTES, st>>>(A);
    return cudaGetLastError();
}

}  // namespace
