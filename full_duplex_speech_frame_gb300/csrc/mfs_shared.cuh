// The work on shared prefixes: how it is cut and dealt out, for the kernels of mfs_shared.cu.
#pragma once
#include "mfs_quant.cuh"

namespace {

// Where the prefix kernels leave their results, and what the join reads.
struct ShArgs {
    Cache C;
    const int32_t *kv_len, *groups, *prefix_len;
    const char* q;
    char* out;
    long long q_stride, out_stride;
    int n_seqs, n_groups, hq, g, window;
    float c;             // scale * log2(e)
    const uint8_t *kx, *vx;
    long long x_page, x_head, x_row;
    int rows, tile;      // rows of a block, positions of a tile
    int ctas;            // of the prefix kernel
    int box;             // rows that a TMA copy takes, 0: none
    int turned;          // the prefix's results: 16-byte unit c of row r of a block lies at c ^ (r & turned)
    float* part_o;       // [CTA][2][rows][HD]
    float2* part_ml;     // [CTA][2][rows] running maximum (raw score) and sum
    float *row_o, *own_o;    // [n_seqs][hq][HD] of the prefix, where one CTA has it all; of what follows
    float2 *row_ml, *own_ml;
    const int2* own_at;      // [n_seqs][head blocks] the pieces of what follows, if any
    const float* own_part_o; // [CTA][2][gm][HD]
    const float2* own_part_ml;
    int gm, nhb;             // query heads of a head block there, head blocks of a kv head
};

constexpr int SH_MAX_CTAS = 152;  // of the prefix kernel: one for each SM

// What an item costs beside its tiles, in tiles.
constexpr int SH_ITEM = 1;

// A place in the walk through the tiles: group i of sequences s0 .. s0 + ns - 1, block rb of nrb of its rows, kv head h, tile of
// ntiles over p positions.
struct ShWalk {
    int i, s0, ns, p, nrb, rb, h, tile, ntiles;
};

// Group w.i's numbers, for a whole warp or a thread alone (window 0); ntiles 0: nothing to do.
__device__ __forceinline__ void sh_group(const ShArgs& A, ShWalk& w)
{
    group_span(A.groups, w.i, A.n_seqs, w.s0, w.ns);
    w.p = max(__ldg(A.prefix_len + w.i), 0);
    w.nrb = (int)(((long long)w.ns * A.g + A.rows - 1) / A.rows);
    w.ntiles = w.ns > 1 ? (int)(((long long)w.p + A.tile - 1) / A.tile) : 0;
    if (w.ntiles == 0) w.nrb = 0;
}

// Places of group w.i, SH_ITEM more for each item
__device__ __forceinline__ long long sh_places(const ShArgs& A, const ShWalk& w)
{
    return (long long)w.nrb * A.C.n_kv_heads * (w.ntiles ? w.ntiles + SH_ITEM : 0);
}

__device__ __forceinline__ long long sh_total(const ShArgs& A)
{
    long long n = 0;
    ShWalk w;
    for (w.i = threadIdx.x & 31; w.i < A.n_groups; w.i += 32) {
        sh_group(A, w);
        n += sh_places(A, w);
    }
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    return n;
}

// The group that holds place `at`, and where it begins; for a whole warp.  at < total.
__device__ __forceinline__ long long sh_find(const ShArgs& A, long long at, ShWalk& w)
{
    const int lane = threadIdx.x & 31;
    long long first = 0;
    for (int b = 0; b < A.n_groups; b += 32) {
        ShWalk x;
        x.i = b + lane;
        long long v = 0;
        if (x.i < A.n_groups) {
            sh_group(A, x);
            v = sh_places(A, x);
        }
        long long inc = v;
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, first + inc > at);
        if (hit) {
            const int l = __ffs(hit) - 1;
            w.i = b + l;
            first += __shfl_sync(0xffffffffu, inc - v, l);
            sh_group(A, w);
            return first;
        }
        first += __shfl_sync(0xffffffffu, inc, 31);
    }
    w.i = A.n_groups;
    w.ntiles = 0;
    return first;
}

// The first sequence of group w that sees its prefix whole, or -1; for a whole warp.
__device__ __forceinline__ int sh_reader(const ShArgs& A, const ShWalk& w)
{
    for (int b = 0; b < w.ns; b += 32) {
        const int i = b + (threadIdx.x & 31);
        const int len = i < w.ns ? __ldg(A.kv_len + w.s0 + i) : 0;
        const unsigned m = __ballot_sync(0xffffffffu, i < w.ns && len >= w.p && (A.window == 0 || len <= A.window));
        if (m) return w.s0 + b + __ffs(m) - 1;
    }
    return -1;
}

// The number of shares: one per CTA, of one place at least (of 4, 8 and 16 at least, fewer CTAs and more SMs for the own parts
// meanwhile, 64 sequences behind 7000 positions took as long, 15 % and 45 % longer).
__device__ __forceinline__ long long sh_shares(const ShArgs& A, long long total) { return min(total, (long long)A.ctas); }

// A CTA's part of an item: tiles from .. upto - 1; whole: all of them.
struct ShPart {
    ShWalk w;
    int from, upto;
    int reader;  // the sequence through whose table the prefix is read
    int slot;  // of the CTA's pieces, or 2: the item's rows themselves
};

// Walks through a CTA's share, an item's part at a time; one warp's registers.
struct ShParts {
    ShWalk w;
    long long at, end;  // places
    __device__ bool start(const ShArgs& A, int cta)
    {
        const long long total = sh_total(A), shares = sh_shares(A, total);
        if (cta >= shares) return false;
        at = muldiv(cta, total, shares);
        end = muldiv(cta + 1, total, shares);
        const long long first = sh_find(A, at, w), in = at - first;
        const int per = w.ntiles + SH_ITEM;
        const long long item = in >> 32 ? in / per : (unsigned)in / (unsigned)per;
        w.rb = (int)(item >> 32 ? item / A.C.n_kv_heads : (unsigned)item / (unsigned)A.C.n_kv_heads);
        w.h = (int)(item - (long long)w.rb * A.C.n_kv_heads);
        w.tile = (int)(in - item * per) - SH_ITEM;  // -SH_ITEM: at the item's beginning
        return true;
    }
    // the next part that some sequence asks for, for a whole warp; false: no more
    __device__ bool next(const ShArgs& A, ShPart& p)
    {
        while (at < end) {
            const int from = max(w.tile, 0);
            const long long left = end - at;
            const int upto = (int)min((long long)w.ntiles, w.tile + left);
            const bool ends = upto == w.ntiles, begins = w.tile == -SH_ITEM;
            p.w = w;
            p.from = from;
            p.upto = upto;
            p.slot = begins ? (ends ? 2 : 1) : 0;
            at += upto - w.tile;
            w.tile = ends ? -SH_ITEM : upto;
            if (ends && ++w.h == A.C.n_kv_heads) {
                w.h = 0;
                if (++w.rb == w.nrb) {
                    w.rb = 0;
                    do {
                        if (++w.i >= A.n_groups) break;
                        sh_group(A, w);
                    } while (w.ntiles == 0);
                }
            }
            // (a share may end in the room before an item's tiles: a piece of none, for the join)
            p.reader = sh_reader(A, p.w);
            if (p.reader >= 0) return true;
        }
        return false;
    }
};

}  // namespace
