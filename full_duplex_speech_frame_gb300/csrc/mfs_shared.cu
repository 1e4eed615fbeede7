// mfs_shared_attention: one new token per sequence, for groups of sequences whose first positions are the same.
//
// A prefix's keys and values meet all rows of its group at once: a row is a query head of one of the group's sequences,
// n sequences with g query heads to a kv head make n g rows.  Items (group, block of rows, kv head) are cut into tiles of
// positions, all laid end to end with a little room at each item's start, and dealt in equal shares to the CTAs, one each,
// which walk through them with a running maximum, sum and output for each row.  An item that lies in one share leaves its
// rows' results; the pieces of others are left for each CTA, two at most.  What follows the prefix is each sequence's own:
// paged_attention_kernel takes it, with the same split over its length.  The last kernel joins, for each sequence and head,
// its own pieces and the prefix's.
//
// bf16, 8 kv heads of 128, 32 query heads: 64 sequences behind 7000 positions, up to 1000 of their own, 58 us (one by one 236 us; 22 us
// is what its bytes take at the measured copy rate): 17 us the prefix, 28 us the own parts, memory at 70 % of that rate, the
// rest the join, which reads each CTA's pieces, 20 MB.
#include "mfs_shared_mma.cuh"

namespace {

// ------------------------------------------------------------- CUDA cores
//
// What bounds it is the data path of shared memory, which feeds the products, as in the prompt attention's fp32 kernel: 64
// sequences behind 2000 positions, 32 + 8 heads of 128, 88 us (one by one 207 us).  fp32: 256 threads take 16 RT rows (RT 8, 4 or 2) and walk over tiles of 64 positions in shared memory; a thread has RT rows x 4 positions of the scores and RT rows x HD / 16 elements of the output in registers (rows and
// positions 16 apart), with paired products; a row's maximum and sum go over half a warp.  The next tile's keys come while
// the values of this one are summed, and the other way round.

constexpr int SF_KEYS = 64, SF_THREADS = 256;

template <int HD, int RT>
struct SfShape {
    static constexpr int ROWS = 16 * RT, LD = HD + 4, LP = SF_KEYS + 4;
    static constexpr int BYTES = 4 * ((ROWS + 2 * SF_KEYS) * LD + ROWS * LP);
};

template <int HD, int RT>
__global__ void __launch_bounds__(SF_THREADS, 1) shared_prefix_f32(const __grid_constant__ ShArgs A)
{
    using S = SfShape<HD, RT>;
    constexpr int ROWS = S::ROWS, LD = S::LD, LP = S::LP, OC = HD / 16;
    extern __shared__ __align__(16) float sf_raw[];
    float *sq = sf_raw, *sk = sq + ROWS * LD, *sv = sk + SF_KEYS * LD, *sp = sv + SF_KEYS * LD;
    __shared__ ShPart sh_part;
    __shared__ int sh_more, sh_bad;
    __shared__ long long sh_off[2][SF_KEYS];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    ShParts parts;
    bool more = false;
    if (tid < 32) more = parts.start(A, blockIdx.x);
    for (;;) {
        if (tid < 32) {
            ShPart p;
            more = more && parts.next(A, p);
            if (tid == 0) {
                sh_more = more;
                sh_bad = 0;
                if (more) sh_part = p;
            }
        }
        __syncthreads();
        if (!sh_more) break;
        const ShPart P = sh_part;
        const int r0 = P.w.rb * ROWS, rows = min(ROWS, P.w.ns * A.g - r0);

        // where a tile's rows lie: -1 for those past the prefix, -2 for a bad page
        auto look_up = [&](int t) {
            if (t >= P.upto || tid >= SF_KEYS) return;
            const long long p = (long long)t * SF_KEYS + tid;
            long long off = -1;
            int page, row;
            if (p < P.w.p) {
                if (row_place(A.C, P.reader, (int)p, page, row)) {
                    off = (long long)page * A.C.page_stride + (long long)row * A.C.row_stride + (long long)P.w.h * A.C.head_stride;
                } else {
                    sh_bad = 1;
                }
            }
            sh_off[t & 1][tid] = off;
        };
        auto fetch = [&](float* dst, bool key, int t) {
            const char* base = key ? A.C.k : A.C.v;
            for (int i = tid; i < SF_KEYS * (HD / 4); i += SF_THREADS) {
                const int r = i / (HD / 4), c = i % (HD / 4) * 4;
                const long long off = sh_off[t & 1][r];
                copy16(su32(dst + r * LD + c), base + (off < 0 ? 0 : (off + c) * 4), off >= 0);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        look_up(P.from);
        for (int i = tid; i < ROWS * (HD / 4); i += SF_THREADS) {
            const int r = i / (HD / 4), c = i % (HD / 4) * 4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) {
                const int s = P.w.s0 + (r0 + r) / A.g, h = P.w.h * A.g + (r0 + r) % A.g;
                v = __ldg(reinterpret_cast<const float4*>(reinterpret_cast<const float*>(A.q) + (long long)s * A.q_stride + (long long)h * HD + c));
            }
            *reinterpret_cast<float4*>(sq + r * LD + c) = v;
        }
        __syncthreads();
        if (P.upto > P.from) {
            fetch(sk, true, P.from);
            fetch(sv, false, P.from);
        }
        float o[RT][OC], m[RT], l[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int e = 0; e < OC; ++e) o[i][e] = 0.f;
        }
        for (int t = P.from; t < P.upto; ++t) {
            const int valid = (int)min(P.w.p - (long long)t * SF_KEYS, (long long)SF_KEYS);
            asm volatile("cp.async.wait_group 1;" ::: "memory");  // the keys
            look_up(t + 1);
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
            if (t + 1 < P.upto) fetch(sk, true, t + 1);
            else asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                float s[4], mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float a, b;
                    unpair(acc[i][j], a, b);
                    s[j] = a + b;
                    if (tx + 16 * j >= valid) s[j] = -INFINITY;
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
            // (places past the prefix: weights of 0 and values of 0)
#pragma unroll 2
            for (int j = 0; j < SF_KEYS; j += 4) {
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
                        const uint64_t pp = pair(p, p);
#pragma unroll
                        for (int e = 0; e < OC / 2; ++e) {
                            const uint64_t r = fma2(pp, v2[e], pair(o[i][2 * e], o[i][2 * e + 1]));
                            unpair(r, o[i][2 * e], o[i][2 * e + 1]);
                        }
                    }
                }
            }
            __syncthreads();  // all have read the values
            if (t + 1 < P.upto) fetch(sv, false, t + 1);
            else asm volatile("cp.async.commit_group;" ::: "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            float sum = l[i];
            for (int x = 8; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
            const int r = ty + 16 * i;
            if (r >= rows) continue;
            if (sh_bad) sum = NAN;
            long long at = ((long long)blockIdx.x * 2 + P.slot) * ROWS + r;
            if (P.slot == 2) at = (long long)(P.w.s0 + (r0 + r) / A.g) * A.hq + P.w.h * A.g + (r0 + r) % A.g;
            float* po = (P.slot == 2 ? A.row_o : A.part_o) + at * HD;
            if (tx == 0) (P.slot == 2 ? A.row_ml : A.part_ml)[at] = make_float2(m[i], sum);
#pragma unroll
            for (int e = 0; e < OC / 4; ++e)
                *reinterpret_cast<float4*>(po + 4 * tx + 64 * e) = make_float4(o[i][4 * e], o[i][4 * e + 1], o[i][4 * e + 2], o[i][4 * e + 3]);
        }
        __syncthreads();  // before the next part's place is written
    }
}

// -------------------------------------------------------------------- join
//
// HD / 4 threads for each sequence and head: its own pieces and the prefix's, in order, eight at a time, all on their
// way together.  Where they lie follows from the lengths alone, and is found while the kernels before still run.

constexpr int SJ_THREADS = 256, SJ_AHEAD = 8;

template <typename T, int HD>
__global__ void __launch_bounds__(SJ_THREADS) shared_join(const __grid_constant__ ShArgs A)
{
    constexpr int LANES = HD / 4, HEADS = SJ_THREADS / LANES;
    __shared__ long long sh_first, sh_total_places;
    __shared__ ShWalk sh_w;
    __shared__ int sh_p;
    const int s = blockIdx.x, tid = threadIdx.x, e = tid % LANES;
    const int len = __ldg(A.kv_len + s);
    if (tid < 32) {
        const int lo = A.window > 0 && len > A.window ? len - A.window : 0;
        const int p = shared_part(A.groups, A.n_groups, A.prefix_len, A.n_seqs, s, lo, len);
        long long total = 0, first = 0;
        ShWalk w = {};
        if (p > 0) {  // the same for all lanes
            total = sh_total(A);
            w.i = group_of(A.groups, A.n_groups, s);
            ShWalk x;
            for (x.i = tid; x.i < w.i; x.i += 32) {
                sh_group(A, x);
                first += sh_places(A, x);
            }
            for (int o = 16; o; o >>= 1) first += __shfl_xor_sync(0xffffffffu, first, o);
            sh_group(A, w);
        }
        if (tid == 0) {
            sh_first = first;
            sh_total_places = total;
            sh_w = w;
            sh_p = p;
        }
    }
    __syncthreads();
    const ShWalk w = sh_w;
    const int p = sh_p, lo = A.window > 0 && len > A.window ? len - A.window : 0;
    const bool own = len > lo + p;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int h = blockIdx.y * HEADS + tid / LANES; h < A.hq; h += gridDim.y * HEADS) {
        const long long at = (long long)s * A.hq + h;
        // parts: -own_n .. -1: its own, 0 ...: the prefix's (one of either: the row itself)
        int c0 = 0, n = 0, row = 0, unit = e, own_n = 0, own_c0 = 0;
        const int in = h % A.g;
        if (own) {
            const int2 r = A.own_at[((long long)s * A.C.n_kv_heads + h / A.g) * A.nhb + in / A.gm];
            own_c0 = r.x;
            own_n = r.x < 0 ? 1 : r.y - r.x + 1;
        }
        if (p > 0) {
            const long long total = sh_total_places, shares = sh_shares(A, total);
            const int r = (s - w.s0) * A.g + in, per = w.ntiles + SH_ITEM;
            const long long begin = sh_first + ((long long)(r / A.rows) * A.C.n_kv_heads + h / A.g) * per;
            // the last share that begins at or before a place
            auto share_of = [&](long long x) {
                const long long y = (x + 1) * shares - 1;
                static_assert((long long)SH_MAX_CTAS << 24 <= 1ll << 32, "y fits in 32 bits");
                return (int)(total < (1 << 24) ? (unsigned)y / (unsigned)total : y / total);
            };
            c0 = share_of(begin);
            n = share_of(begin + per - 1) - c0 + 1;
            row = r % A.rows;
            unit = e ^ (row & A.turned);
        }
        float m = -INFINITY, l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = -own_n; i0 < n; i0 += SJ_AHEAD) {
            float2 ml[SJ_AHEAD];
            float4 v[SJ_AHEAD];
#pragma unroll
            for (int j = 0; j < SJ_AHEAD; ++j) {
                const int i = i0 + j;
                ml[j] = make_float2(-INFINITY, 0.f);
                v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i >= n) continue;
                long long k = at;
                const float* o = i < 0 ? A.own_o : A.row_o;
                const float2* s_ml = i < 0 ? A.own_ml : A.row_ml;
                if (i < 0 && own_c0 >= 0) {
                    k = ((long long)(own_c0 + i + own_n) * 2 + (i == -own_n)) * A.gm + in % A.gm;
                    o = A.own_part_o;
                    s_ml = A.own_part_ml;
                } else if (i >= 0 && n > 1) {
                    k = ((long long)(c0 + i) * 2 + (i == 0)) * A.rows + row;
                    o = A.part_o;
                    s_ml = A.part_ml;
                }
                ml[j] = s_ml[k];
                v[j] = *reinterpret_cast<const float4*>(o + k * HD + 4 * (i < 0 ? e : unit));
            }
            float mn = m;
#pragma unroll
            for (int j = 0; j < SJ_AHEAD; ++j) mn = fmaxf(mn, ml[j].x);
            const float a = m == mn ? 1.f : exp2f((m - mn) * A.c);
            m = mn;
            l *= a;
            acc = make_float4(acc.x * a, acc.y * a, acc.z * a, acc.w * a);
#pragma unroll
            for (int j = 0; j < SJ_AHEAD; ++j) {
                const float b = ml[j].x == mn ? 1.f : exp2f((ml[j].x - mn) * A.c);
                l = fmaf(ml[j].y, b, l);
                acc = make_float4(fmaf(v[j].x, b, acc.x), fmaf(v[j].y, b, acc.y), fmaf(v[j].z, b, acc.z), fmaf(v[j].w, b, acc.w));
            }
        }
        T* o = reinterpret_cast<T*>(A.out) + (long long)s * A.out_stride + (long long)h * HD + 4 * e;
        if (len <= 0) put4(o, make_float4(0.f, 0.f, 0.f, 0.f), 1.f);
        else put4(o, acc, 1.f / l);
    }
}

// -------------------------------------------------------------------- host

// Rows of the prefix kernel's blocks: 128, or 64 or 32 where groups have so few on average.
int f32_rows(long long rows, int n_groups)
{
    const long long each = rows / (n_groups > 0 ? n_groups : 1);
    return each > 64 ? 128 : each > 32 ? 64 : 32;
}

// Whether sharing could pay: what it saves, at most, is reading the positions that the table has room for, or as many of them as a
// window lets a sequence see that begins at its first, once for each sequence but one of a group.  (Where lengths
// are far below the room it is a loss: 16 sequences of 32 + 32 heads behind 250 positions, room for 750, 34 us, one by one 31.)  Its
// three kernels take about 15 us more than the one-token attention's two.  bf16, 8 kv heads of 128, 32 query heads: 4 sequences behind 7000 positions (86 MB saved) 28.1 us, one by one 24.8; 8 (201 MB) 29.7 and 38.4;
// 64 behind 500 (129 MB) 28.7 and 28.6; fp32, 64 behind 500 (258 MB) 49 and 64; 8 bits, 96 behind 500 to 1000 (193 MB) 32.1 and
// 32.0, 64 behind 2000 (262 MB) 31 and 47, 96 behind 3000 to 6000 (1210 MB) 64 and 123.
bool sharing_pays(const mfs_paged_kv* c, int n_seqs, int n_groups, int window, double row_bytes)
{
    const long long room = (long long)c->table_width * c->page_size, most = window > 0 && window < room ? window : room;
    const double saved = ((double)n_seqs - n_groups) * most * c->n_kv_heads * 2 * row_bytes;
    return n_groups > 0 && saved > (c->dtype == MFS_DTYPE_E4M3 ? 200e6 : 120e6);
}

struct ShSpace {
    size_t own, part_o, part_ml, row_o, row_ml, own_o, own_ml, own_at, bytes;
};

ShSpace sh_space(int hd, int hq, int n_seqs)
{
    ShSpace s;
    const size_t rows = (size_t)n_seqs * hq, most = 256;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t x = at;
        at += (n + 255) & ~(size_t)255;
        return x;
    };
    s.own = take(quant_workspace(hd));
    s.part_o = take((size_t)SH_MAX_CTAS * 2 * most * hd * 4);
    s.part_ml = take((size_t)SH_MAX_CTAS * 2 * most * 8);
    s.row_o = take(rows * hd * 4);
    s.row_ml = take(rows * 8);
    s.own_o = take(rows * hd * 4);
    s.own_ml = take(rows * 8);
    s.own_at = take(rows * 8);  // (head blocks are no more than heads)
    s.bytes = at;
    return s;
}

template <int HD, int RT>
cudaError_t prefix_f32(const ShArgs& A, cudaStream_t st)
{
    using S = SfShape<HD, RT>;
    int sms = 0;
    static mfs::PerDevice ready;
    cudaError_t e = mfs::op_device(ready, (const void*)shared_prefix_f32<HD, RT>, S::BYTES, &sms);
    if (e != cudaSuccess) return e;
    shared_prefix_f32<HD, RT><<<A.ctas, SF_THREADS, S::BYTES, st>>>(A);
    return cudaGetLastError();
}

template <typename K, bool QUANT>
int shared(PaArgs P, ShArgs A, char* ws, cudaStream_t st)
{
    using T = typename K::T;
    constexpr int HD = K::HD;
    const char* op = "shared_attention";
    const ShSpace sp = sh_space(HD, A.hq, A.n_seqs);
    A.part_o = (float*)(ws + sp.part_o);
    A.part_ml = (float2*)(ws + sp.part_ml);
    A.row_o = (float*)(ws + sp.row_o);
    A.row_ml = (float2*)(ws + sp.row_ml);
    A.own_o = P.own_o = (float*)(ws + sp.own_o);
    A.own_ml = P.own_ml = (float2*)(ws + sp.own_ml);
    A.own_at = P.own_at = (int2*)(ws + sp.own_at);
    A.own_part_o = (const float*)(ws + sp.own);
    A.own_part_ml = pa_part_ml<K>(ws + sp.own);
    A.gm = K::GM;
    A.nhb = (A.g + K::GM - 1) / K::GM;
    int sms = 0;
    static mfs::PerDevice known;
    cudaError_t e = mfs::op_device(known, nullptr, 0, &sms);
    if (e != cudaSuccess) return mfs::op_launched(op, e);
    A.ctas = sms < SH_MAX_CTAS ? sms : SH_MAX_CTAS;
    if constexpr (sizeof(T) == 2) {
        A.rows = 2 * SM_M;
        A.tile = SM_M;
        A.turned = 7;
        e = prefix_mma<HD, QUANT>(A, st);
    } else {
        A.rows = f32_rows((long long)A.n_seqs * A.g, A.n_groups);
        A.tile = SF_KEYS;
        e = A.rows == 128 ? prefix_f32<HD, 8>(A, st) : A.rows == 64 ? prefix_f32<HD, 4>(A, st) : prefix_f32<HD, 2>(A, st);
    }
    if (e != cudaSuccess) return mfs::op_launched(op, e);
    if (const int rc = attention<K>(P, ws + sp.own, st, op)) return rc;
    cudaLaunchConfig_t cfg = {};
    // a block takes eight (sixteen) heads of a sequence at a time, and all of them where the sequences are enough to fill the SMs
    const int turns = (A.hq - 1) / (SJ_THREADS / (HD / 4)) + 1, most = 4 * sms / A.n_seqs + 1;
    cfg.gridDim = dim3((unsigned)A.n_seqs, (unsigned)(turns < most ? turns : most));
    cfg.blockDim = dim3(SJ_THREADS);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return mfs::op_launched(op, cudaLaunchKernelEx(&cfg, shared_join<T, HD>, A));
}

// 0: go on, 1: nothing to do, else an error's code
int shared_checked(const char* op, PaArgs& P, ShArgs& A, int n_groups, const int32_t* groups, const int32_t* prefix_len)
{
    if (!groups || (n_groups && !prefix_len)) return mfs::op_fail(MFS_E_ARG, op, "null groups or prefix_len");
    P.groups = groups;
    P.prefix_len = prefix_len;
    P.n_groups = n_groups;
    A.C = P.C;
    A.kv_len = P.kv_len; A.groups = groups; A.prefix_len = prefix_len;
    A.q = P.q; A.out = P.out;
    A.q_stride = P.q_stride; A.out_stride = P.out_stride;
    A.n_seqs = P.n_seqs; A.n_groups = n_groups; A.hq = P.hq; A.g = P.g; A.window = P.window;
    A.c = P.c;
    A.kx = P.kx; A.vx = P.vx;
    A.x_page = P.x_page; A.x_head = P.x_head; A.x_row = P.x_row;
    return 0;
}

}  // namespace

extern "C" size_t mfs_shared_attention_workspace(const mfs_paged_kv* cache, int n_q_heads, int n_seqs)
{
    if (mfs::paged_kv_problem(cache) || n_q_heads < 1 || n_q_heads > MFS_MAX_HEADS || n_seqs < 0) return 0;
    return sh_space(cache->head_dim, n_q_heads, n_seqs).bytes;
}

extern "C" size_t mfs_quant_shared_attention_workspace(const mfs_quant_kv* cache, int dtype, int n_q_heads, int n_seqs)
{
    if (mfs::quant_kv_problem(cache) || (dtype != MFS_DTYPE_F32 && dtype != MFS_DTYPE_BF16) || n_q_heads < 1 || n_q_heads > MFS_MAX_HEADS || n_seqs < 0)
        return 0;
    return dtype == MFS_DTYPE_F32 ? quant_workspace(cache->kv.head_dim) : sh_space(cache->kv.head_dim, n_q_heads, n_seqs).bytes;
}

extern "C" int mfs_shared_attention(const mfs_paged_kv* cache, int n_seqs, const int32_t* kv_len, int n_groups, const int32_t* groups,
                                    const int32_t* prefix_len, const void* q, long long q_stride, int n_q_heads, void* out,
                                    long long out_stride, float scale, int window, void* workspace, size_t workspace_bytes, void* cuda_stream)
{
    const char* op = "shared_attention";
    if (const char* why = mfs::paged_kv_problem(cache)) return mfs::op_fail(MFS_E_ARG, op, why);
    if (n_groups < 0) return mfs::op_fail(MFS_E_ARG, op, "need n_groups >= 0");
    PaArgs P = {};
    ShArgs A = {};
    P.C = cache_of(cache);
    const int hd = cache->head_dim;
    int rc = pa_checked(op, P, cache->dtype, hd, n_seqs, kv_len, q, q_stride, n_q_heads, out, out_stride, scale, window, workspace, workspace_bytes,
                        mfs_shared_attention_workspace(cache, n_q_heads, n_seqs));
    if (!rc) rc = shared_checked(op, P, A, n_groups, groups, prefix_len);
    if (rc) return rc < 0 ? rc : MFS_OK;
    cudaStream_t st = (cudaStream_t)cuda_stream;
    char* ws = (char*)workspace;
    if (!sharing_pays(cache, n_seqs, n_groups, window, hd * (cache->dtype == MFS_DTYPE_BF16 ? 2.0 : 4.0)))
        return mfs_paged_attention(cache, n_seqs, kv_len, q, q_stride, n_q_heads, out, out_stride, scale, window, ws, workspace_bytes, cuda_stream);
    if (cache->dtype == MFS_DTYPE_BF16) return hd == 128 ? shared<PaKindBf16<128, true>, false>(P, A, ws, st) : shared<PaKindBf16<64, true>, false>(P, A, ws, st);
    auto fn = hd == 128 ? (P.g == 1 ? shared<PaKindF32<128, 1, true>, false> : P.g <= 4 ? shared<PaKindF32<128, 4, true>, false> : shared<PaKindF32<128, 8, true>, false>)
                        : (P.g == 1 ? shared<PaKindF32<64, 1, true>, false> : P.g <= 4 ? shared<PaKindF32<64, 4, true>, false> : shared<PaKindF32<64, 8, true>, false>);
    return fn(P, A, ws, st);
}

extern "C" int mfs_quant_shared_attention(const mfs_quant_kv* cache, int dtype, int n_seqs, const int32_t* kv_len, int n_groups,
                                          const int32_t* groups, const int32_t* prefix_len, const void* q, long long q_stride, int n_q_heads,
                                          void* out, long long out_stride, float scale, int window, void* workspace, size_t workspace_bytes,
                                          void* cuda_stream)
{
    const char* op = "shared_attention";
    if (const char* why = mfs::quant_kv_problem(cache)) return mfs::op_fail(MFS_E_ARG, op, why);
    if (n_groups < 0) return mfs::op_fail(MFS_E_ARG, op, "need n_groups >= 0");
    PaArgs P = quant_args(cache);
    ShArgs A = {};
    const int hd = cache->kv.head_dim;
    int rc = pa_checked(op, P, dtype, hd, n_seqs, kv_len, q, q_stride, n_q_heads, out, out_stride, scale, window, workspace, workspace_bytes,
                        mfs_quant_shared_attention_workspace(cache, dtype, n_q_heads, n_seqs));
    if (!rc) rc = shared_checked(op, P, A, n_groups, groups, prefix_len);
    if (rc) return rc < 0 ? rc : MFS_OK;
    cudaStream_t st = (cudaStream_t)cuda_stream;
    char* ws = (char*)workspace;
    // fp32 queries: the CUDA cores would take longer for a prefix's products than the one-token attention, whose products of
    // codes run on the matrix units, takes to read it for each sequence (32 behind 4000, 32 + 8 heads of 128: 98 and 59 us)
    if (dtype == MFS_DTYPE_F32 || !sharing_pays(&cache->kv, n_seqs, n_groups, window, hd + 1.0))
        return mfs_quant_attention(cache, dtype, n_seqs, kv_len, q, q_stride, n_q_heads, out, out_stride, scale, window, ws, workspace_bytes, cuda_stream);
    auto fn = P.g <= 8 ? (hd == 128 ? shared<PaKindE4m3<bf16, 128, 1, true>, true> : shared<PaKindE4m3<bf16, 64, 1, true>, true>)
                       : (hd == 128 ? shared<PaKindE4m3<bf16, 128, 2, true>, true> : shared<PaKindE4m3<bf16, 64, 2, true>, true>);
    return fn(P, A, ws, st);
}
