"""mfs_shared_attention on the GPU against the 64-bit definition of each sequence's own attention."""
import numpy as np
import pytest

from tests import _quant as Q
from tests import _serving as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mfs():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from full_duplex_speech_frame_gb300 import mfs as m
    return m


def _torch():
    import torch
    return torch


def _dt(name):
    return {"bf16": _torch().bfloat16, "f32": _torch().float32}[name]


def _normal(rng, *shape, dtype="f32", scale=1.0):
    return _torch().from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(_dt(dtype)).cuda()


def _i32(x):
    return _torch().tensor(x, dtype=_torch().int32, device="cuda")


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _tables(rng, sizes, prefix, lens, page, outside=0):
    """Tables of sequences in groups (sizes[i] sequences behind prefix[i] positions, then `outside` alone): whole pages of a
    prefix are shared, a last page that it fills in part is each sequence's own.  -> table, pages, (page, page, rows) copies."""
    n = sum(sizes) + outside
    need = [max(1, -(-x // page)) for x in lens]
    table = np.full((n, max(need) + 1), -1)
    at, s, copies = 0, 0, []
    order = rng.permutation(sum(need) + sum(-(-p // page) for p in prefix) + 5)
    for g, size in enumerate(sizes):
        whole = prefix[g] // page
        common = order[at:at + whole]
        at += whole
        first = None
        for _ in range(size):
            m = min(whole, need[s])
            table[s, :m] = common[:m]
            table[s, m:need[s]] = order[at:at + need[s] - m]
            at += need[s] - m
            if prefix[g] % page and need[s] > whole:  # the rest of the prefix, the same in each
                if first is None:
                    first = table[s, whole]
                else:
                    copies.append((first, table[s, whole], prefix[g] % page))
            s += 1
    for _ in range(outside):
        table[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
        s += 1
    return table, len(order), copies


def _wide(table, groups, page, hkv, hd, dtype, quant):
    """The table with room for so many positions that sharing them is tried (it is not where it could not pay)."""
    row = hd + 1 if quant else hd * (2 if dtype == "bf16" else 4)
    positions = 260e6 / (max(1, len(table) - groups) * hkv * 2 * row)
    return np.pad(table, ((0, 0), (0, int(positions / page) + 1)), constant_values=-1)


def _cache(mfs, rng, table, pages, copies, hkv, page, hd, dtype, quant):
    torch = _torch()
    if quant:
        pools = []
        for _ in "kv":
            c = rng.integers(0, 256, (pages, hkv, page, hd)).astype(np.uint8)
            c[(c & 127) == 127] -= 1
            pools.append(torch.from_numpy(c).cuda())
        for _ in "kv":
            pools.append(torch.from_numpy(rng.integers(117, 121, (pages, hkv, page)).astype(np.uint8)).cuda())
        cache = mfs.QuantKV(*pools, _i32(table))
        parts = (cache.k, cache.v, cache.k_exp, cache.v_exp)
    else:
        cache = mfs.PagedKV(_normal(rng, pages, hkv, page, hd, dtype=dtype), _normal(rng, pages, hkv, page, hd, dtype=dtype), _i32(table))
        parts = (cache.k, cache.v)
    for a, b, rows in copies:
        for t in parts:
            t[int(b), :, :rows] = t[int(a), :, :rows]
    return cache


def _rows(cache, table, s, lo, hi, quant):
    """-> keys, values [n, heads, hd], codes and exponents of the values (or None)."""
    page = cache.k.shape[2]
    g, r = table[s][np.arange(lo, hi) // page], np.arange(lo, hi) % page
    if not quant:
        return _HOST[id(cache)][0][g, :, r], _HOST[id(cache)][1][g, :, r], None, None
    kc, kx, vc, vx = (_HOST[id(cache)][i][g, :, r] for i in range(4))
    return Q.values(kc, kx), Q.values(vc, vx), vc, vx


_HOST = {}


def _check(cache, table, q, out, lens, window, dtype, quant, scale=None, heads=None, seqs=None, nan=()):
    qs, got, hq, hkv, hd = _np(q), _np(out), q.shape[1], cache.k.shape[1], q.shape[2]
    _HOST.clear()
    _HOST[id(cache)] = [t.cpu().numpy() for t in (cache.k, cache.k_exp, cache.v, cache.v_exp)] if quant else [_np(cache.k), _np(cache.v)]
    scale = hd ** -0.5 if scale is None else scale
    for s in (range(len(lens)) if seqs is None else seqs):
        if s in nan:
            assert np.isnan(got[s]).all(), s
            continue
        lo = max(0, lens[s] - window) if window else 0
        k, v, vc, vx = _rows(cache, table, s, lo, max(lo, lens[s]), quant)
        for h in (range(hq) if heads is None else heads):
            j = h * hkv // hq
            ref, weighted, size = S.attend(qs[s, h], k[:, j], v[:, j], scale)
            lost = Q.lost_weights(qs[s, h], k[:, j], vc[:, j], vx[:, j], scale) if quant else 0.0
            tol = Q.shared_tolerance(ref, weighted, size, len(k), hd, dtype == "bf16", quant, lost)
            far = np.abs(got[s, h] - ref)
            assert (far <= tol).all(), (s, h, (far / tol).max(), far.max())


def _case(mfs, seed, sizes, prefix, lens, hq, hkv, hd, page, dtype, quant, window=0, outside=0, scale=None, wide=True, **kw):
    torch = _torch()
    rng = np.random.default_rng(seed)
    table, pages, copies = _tables(rng, sizes, prefix, lens, page, outside)
    if wide:
        table = _wide(table, len(sizes), page, hkv, hd, dtype, quant)
    cache = _cache(mfs, rng, table, pages, copies, hkv, page, hd, dtype, quant)
    n = len(lens)
    q = _normal(rng, n, hq + 1, hd, dtype=dtype)[:, :hq]
    out = torch.full((n, hq + 2, hd), 7.0, dtype=_dt(dtype), device="cuda")
    groups = _i32(np.cumsum([0] + sizes).tolist())
    mfs.mfs_shared_attention(cache, q, _i32(lens), groups, _i32(prefix), out[:, :hq], window=window, scale=scale)
    assert (out[:, hq:] == 7).all()
    out = out[:, :hq]
    _check(cache, table, q, out, lens, window, dtype, quant, scale=scale, **kw)
    again = torch.empty_like(out)
    mfs.mfs_shared_attention(cache, q, _i32(lens), groups, _i32(prefix), again, window=window, scale=scale)
    assert torch.equal(out, again) or torch.isnan(out).any()
    return cache, table, q, groups, out


KINDS = [("bf16", False), ("f32", False), ("bf16", True), ("f32", True)]


@pytest.mark.parametrize("dtype,quant", KINDS)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("prefix", [0, 1, 63, 64, 65, 127, 128, 129, 255, 1000])
def test_prefix_lengths(mfs, dtype, quant, hd, prefix):
    """One group; sequences that end with the prefix, one and more positions behind it."""
    lens = [prefix + x for x in (0, 1, 2, 33, 300)]
    _case(mfs, prefix, [5], [prefix], lens, 6, 2, hd, 16, dtype, quant)


@pytest.mark.parametrize("dtype,quant", KINDS)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (4, 4), (8, 1), (12, 2), (40, 2)])
@pytest.mark.parametrize("page", [1, 16, 48, 128])
def test_heads_and_pages(mfs, dtype, quant, hq, hkv, page):
    """Groups of every kind: pairs, one of 40 sequences (rows of several blocks for wide groups), uneven prefixes, prefixes that end
    inside a page, groups of one sequence, of none, and sequences of no group."""
    sizes, prefix = [2, 1, 0, 40, 3], [200, 77, 50, 300, 31]
    rng = np.random.default_rng(page)
    lens = [p + int(x) for n, p in zip(sizes, prefix) for x in rng.integers(0, 90, n)] + [55, 0]
    _case(mfs, hq * 100 + page, sizes, prefix, lens, hq, hkv, 64, page, dtype, quant, outside=2, heads=sorted({0, 1 % hq, hq // 2, hq - 1}))


@pytest.mark.parametrize("dtype,quant", KINDS)
def test_sequences_that_do_not_see_the_prefix_whole(mfs, dtype, quant):
    """Lengths of 0, inside the prefix and at its end; with windows that begin inside it, behind it, at its first position."""
    lens = [0, 1, 99, 150, 151, 152, 170, 250, 300, 301, 302, 420]
    for window in (0, 1, 100, 151, 250, 300, 1000):
        _case(mfs, window, [12], [151], lens, 4, 2, 64, 16, dtype, quant, window=window)


@pytest.mark.parametrize("dtype,quant", KINDS)
def test_many_rows_and_long_prefixes(mfs, dtype, quant):
    """Rows of three and more blocks; a prefix whose items cross many CTAs; both."""
    lens = [4000 + 3 * i for i in range(90)]
    _case(mfs, 1, [90], [4000], lens, 8, 1, 128, 32, dtype, quant, heads=[0, 5, 7], seqs=[0, 1, 15, 16, 31, 32, 33, 63, 64, 88, 89])
    _case(mfs, 2, [2], [30000], [30000, 30500], 2, 1, 64, 64, dtype, quant)
    lens = [500 + i % 9 for i in range(300)]
    _case(mfs, 3, [100] * 3, [500] * 3, lens, 4, 4, 64, 16, dtype, quant, heads=[1], seqs=list(range(0, 300, 17)))


@pytest.mark.parametrize("dtype,quant", KINDS)
def test_many_sequences(mfs, dtype, quant):
    """More sequences than a block keeps numbers of, with own parts of none to two positions."""
    sizes, prefix = [1400, 100], [150, 90]
    lens = [prefix[0] + i % 3 for i in range(1400)] + [prefix[1] + i % 2 for i in range(100)]
    _case(mfs, 15, sizes, prefix, lens, 2, 1, 64, 16, dtype, quant, seqs=[0, 1, 2, 700, 1022, 1023, 1024, 1025, 1399, 1400, 1499])


@pytest.mark.parametrize("dtype,quant", KINDS)
@pytest.mark.parametrize("page", [8, 24, 7])
def test_strided_pools(mfs, dtype, quant, page):
    """Pools with the heads innermost and room between rows, in pages that are and are not whole groups of eight rows."""
    torch = _torch()
    rng = np.random.default_rng(16)
    lens, prefix, hkv, hd = [300, 320, 301, 299], 299, 3, 64
    cache, table, q, groups, out = _case(mfs, 16, [4], [prefix], lens, 6, hkv, hd, page, dtype, quant)
    room = 16 if quant else 8
    strided = []
    for src in (cache.k, cache.v):
        x = torch.zeros(src.shape[0], page, hkv, hd + room, dtype=src.dtype, device="cuda").permute(0, 2, 1, 3)[..., :hd]
        x.copy_(src)
        strided.append(x)
    if quant:
        for src in (cache.k_exp, cache.v_exp):
            x = torch.zeros(src.shape[0], page, hkv + 2, dtype=torch.uint8, device="cuda").permute(0, 2, 1)[:, :hkv]
            x.copy_(src)
            strided.append(x)
        other = mfs.QuantKV(strided[0].view(torch.float8_e4m3fn), strided[1].view(torch.float8_e4m3fn), strided[2], strided[3], cache.table)
    else:
        other = mfs.PagedKV(*strided, cache.table)
    got = torch.empty_like(out)
    mfs.mfs_shared_attention(other, q, _i32(lens), groups, _i32([prefix]), got)
    assert torch.equal(got, out)
    one = torch.empty_like(out)
    mfs.mfs_paged_attention(other, q, _i32(lens), one)
    mfs.mfs_paged_attention(cache, q, _i32(lens), got)
    assert torch.equal(one, got)


@pytest.mark.parametrize("dtype,quant", KINDS)
def test_many_groups(mfs, dtype, quant):
    """More groups than a warp has lanes, pairs and threes, with their own prefixes."""
    rng = np.random.default_rng(5)
    sizes = [2 + i % 2 for i in range(70)]
    prefix = [int(x) for x in rng.integers(0, 200, 70)]
    lens = [p + int(x) for n, p in zip(sizes, prefix) for x in rng.integers(1, 40, n)]
    _case(mfs, 5, sizes, prefix, lens, 4, 2, 64, 16, dtype, quant, heads=[0, 3], seqs=list(range(0, len(lens), 7)))


@pytest.mark.parametrize("dtype,quant", KINDS)
@pytest.mark.parametrize("scale", [1e-3, 1.0, 20.0])
def test_scores_of_any_size(mfs, dtype, quant, scale):
    _case(mfs, 6, [6], [400], [400 + 30 * i for i in range(6)], 4, 1, 64, 16, dtype, quant, scale=scale)


@pytest.mark.parametrize("dtype,quant", KINDS)
def test_the_same_as_one_by_one(mfs, dtype, quant):
    """Where nothing can be shared the bits are mfs_paged_attention's; elsewhere the two agree within both tolerances."""
    torch = _torch()
    lens = [300, 310, 290, 500]
    cache, table, q, groups, out = _case(mfs, 7, [4], [250], lens, 4, 2, 64, 16, dtype, quant, wide=False)
    one = torch.empty_like(out)
    mfs.mfs_paged_attention(cache, q, _i32(lens), one)
    assert torch.equal(out, one)  # a table with room for so little is not shared
    cache, table, q, groups, out = _case(mfs, 7, [4], [250], lens, 4, 2, 64, 16, dtype, quant)
    mfs.mfs_paged_attention(cache, q, _i32(lens), one)
    got = torch.empty_like(out)
    for g, p in (([0, 1, 2, 3, 4], [250] * 4), ([0, 4], [0]), ([0, 0], [250]), ([0, 4], [600])):
        mfs.mfs_shared_attention(cache, q, _i32(lens), _i32(g), _i32(p), got)
        # a sequence's own part goes through the same kernel; its join divides once more: two roundings of 2^-24, and the type's
        assert ((got.float() - one.float()).abs() <= (2.0 ** -22 + (2.0 ** -7 if dtype == "bf16" else 0)) * one.float().abs()).all()
    mfs.mfs_shared_attention(cache, q, _i32(lens), _i32([0]), _i32([]), got)
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("dtype,quant", KINDS)
def test_rows_that_are_not_seen(mfs, dtype, quant):
    """NaN behind the sequences, in the prefix's last page past it, and in pages of no one: no influence."""
    torch = _torch()
    lens, prefix = [70, 75, 69, 130], 69
    cache, table, q, groups, out = _case(mfs, 8, [4], [prefix], lens, 4, 2, 64, 16, dtype, quant)
    seen = np.zeros((cache.k.shape[0], 16), bool)
    for s, n in enumerate(lens):
        for p in range(n):
            seen[table[s, p // 16], p % 16] = True
    dark = torch.from_numpy(~seen).cuda()[:, None, :].expand(-1, 2, -1)
    for t in (cache.k, cache.v):
        t[dark] = 0x7f if quant else float("nan")
    if quant:
        for t in (cache.k_exp, cache.v_exp):
            t[dark] = 255
    again = torch.empty_like(out)
    mfs.mfs_shared_attention(cache, q, _i32(lens), groups, _i32([prefix]), again)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype,quant", KINDS)
def test_nan_and_infinite_rows_that_are_seen(mfs, dtype, quant):
    """A NaN value in the prefix reaches its column of all sequences that see it, a NaN key all of their heads; one in a
    sequence's own part reaches it alone."""
    torch = _torch()
    lens, prefix = [200, 180, 160, 40], 160
    for where, hit in ((33, [0, 1, 2, 3]), (45, [0, 1, 2]), (170, [0])):
        for which in "kv":
            cache, table, q, groups, out = _case(mfs, 9, [4], [prefix], lens, 4, 2, 64, 16, dtype, quant)
            bad = getattr(cache, which)
            if where < prefix:
                s = 0
            else:
                s = hit[0]
            bad[int(table[s, where // 16]), 1, where % 16, 7] = 0x7f if quant else float("nan")
            if where == 33 or where == 45:
                for other in (1, 2, 3):
                    if table[other, where // 16] >= 0:
                        assert table[other, where // 16] == table[0, where // 16]
            again = torch.empty_like(out)
            mfs.mfs_shared_attention(cache, q, _i32(lens), groups, _i32([prefix]), again)
            want = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
            for s in hit:
                if which == "k":
                    want[s, 2:] = True
                else:
                    want[s, 2:, 7] = True
            assert torch.equal(torch.isnan(again), want), (where, which)
            assert torch.equal(again[~want], out[~want])


@pytest.mark.parametrize("dtype,quant", KINDS)
def test_queries_that_are_not_finite(mfs, dtype, quant):
    torch = _torch()
    lens = [200, 180, 160]
    cache, table, q, groups, out = _case(mfs, 10, [3], [150], lens, 4, 2, 64, 16, dtype, quant)
    for bad in (float("nan"), float("inf")):
        q2 = q.clone()
        q2[1, 2, 3] = bad
        again = torch.empty_like(out)
        mfs.mfs_shared_attention(cache, q2, _i32(lens), groups, _i32([150]), again)
        keep = torch.ones(3, 4, dtype=torch.bool)
        keep[1, 2] = False
        assert torch.equal(again[keep], out[keep])
        if bad != bad:
            assert torch.isnan(again[1, 2]).all()


@pytest.mark.parametrize("dtype,quant", KINDS)
def test_bad_pages_give_nan(mfs, dtype, quant):
    """A page outside the pool, or a table too narrow, in a group's prefix: NaN for those that share it; in one sequence's
    own part: for that one."""
    torch = _torch()
    lens, prefix = [200, 180, 160, 300, 310], [150, 280]
    cache, table, q, groups, out = _case(mfs, 11, [3, 2], prefix, lens, 4, 2, 64, 16, dtype, quant)
    for s, j, hit in ((0, 3, [0, 1, 2]), (1, 10, [1]), (3, 0, [3, 4])):
        for value in (-1, cache.k.shape[0]):
            bad = table.copy()
            bad[hit if len(hit) > 1 else s, j] = value
            cache.table.copy_(_i32(bad))
            got = torch.empty_like(out)
            mfs.mfs_shared_attention(cache, q, _i32(lens), groups, _i32(prefix), got)
            for i in range(5):
                assert torch.isnan(got[i]).all() if i in hit else torch.equal(got[i], out[i]), (s, j, i)


@pytest.mark.parametrize("dtype,quant", KINDS)
def test_captured_streams_and_aliases(mfs, dtype, quant):
    torch = _torch()
    lens, prefix = [700 + 11 * i for i in range(20)], 640
    cache, table, q, groups, out = _case(mfs, 12, [20], [prefix], lens, 4, 2, 64, 16, dtype, quant, seqs=[0])
    q, lens, prefix = q.contiguous(), _i32(lens), _i32([prefix])
    ws = mfs.mfs_shared_attention_workspace(cache, 4, 20)
    got = torch.empty_like(out)

    def step():
        mfs.mfs_shared_attention(cache, q, lens, groups, prefix, got, workspace=ws)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    q.copy_(_normal(np.random.default_rng(3), *q.shape, dtype=dtype))
    lens.sub_(5)
    prefix.sub_(129)
    step()
    want = got.clone()
    got.zero_()
    graph.replay()
    assert torch.equal(got, want)
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.empty_like(q) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, o in zip(streams, outs):
            mfs.mfs_shared_attention(cache, q, lens, groups, prefix, o, stream=st.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    mfs.mfs_shared_attention(cache, q, lens, groups, prefix, q)  # out may be q
    assert torch.equal(q, want)


@pytest.mark.parametrize("quant", [False, True])
def test_a_session_from_prompt_to_shared_steps(mfs, quant):
    """As a server runs it: a persona's prompt enters the cache once, six sessions share its pages, each appends its own
    frames, and every frame's attention goes over prompt and own frames; positions rotate on from the prompt's."""
    torch = _torch()
    rng = np.random.default_rng(13)
    hq, hkv, hd, page, n, prompt, frames = 8, 2, 64, 16, 6, 160, 5
    own = -(-frames // page)
    table = np.array([list(range(prompt // page)) + [prompt // page + s * own + j for j in range(own)] for s in range(n)])
    pages = prompt // page + n * own
    table = _wide(table, 1, page, hkv, hd, "bf16", quant)
    if quant:
        cache = mfs.QuantKV(*(torch.zeros(pages, hkv, page, hd, dtype=torch.uint8, device="cuda") for _ in "kv"),
                            *(torch.zeros(pages, hkv, page, dtype=torch.uint8, device="cuda") for _ in "kv"), _i32(table))
    else:
        cache = mfs.PagedKV(*(torch.zeros(pages, hkv, page, hd, dtype=torch.bfloat16, device="cuda") for _ in "kv"), _i32(table))
    rope = mfs.Rope("interleaved", dims=32, factor=2.0, original=100.0)
    pk, pv = (_normal(rng, prompt, hkv, hd, dtype="bf16") for _ in "kv")
    mfs.mfs_kv_append(cache, pk, pv, _i32([0, prompt]), _i32([prompt]), rope=rope)
    keys, vals = [[], []], [[], []]
    cu, groups, plen = _i32(list(range(n + 1))), _i32([0, n]), _i32([prompt])
    for f in range(frames):
        q, k, v = (_normal(rng, n, h, hd, dtype="bf16") for h in (hq, hkv, hkv))
        lens = _i32([prompt + f + 1] * n)
        qr, out = torch.empty_like(q), torch.empty_like(q)
        mfs.mfs_kv_append(cache, k, v, cu, lens, q=q, q_out=qr, rope=rope)
        mfs.mfs_shared_attention(cache, qr, lens, groups, plen, out)
        _check(cache, table, qr, out, [prompt + f + 1] * n, 0, "bf16", quant, seqs=[0, n - 1])
        want = Q.rotate(_np(q[1]), prompt + f, layout="interleaved", dims=32, factor=2.0, original=100.0)
        assert np.allclose(_np(qr[1]), want, rtol=2.0 ** -8, atol=2.0 ** -18)
    back = torch.empty(n * frames, hkv, hd, dtype=torch.bfloat16, device="cuda"), torch.empty(n * frames, hkv, hd, dtype=torch.bfloat16, device="cuda")
    mfs.mfs_kv_read(cache, _i32([frames * s for s in range(n + 1)]), _i32([prompt + frames] * n), *back)
    assert torch.isfinite(back[0]).all()
    near = (_np(back[1].view(n, frames, hkv, hd)[:, -1]) - _np(v))
    assert (np.abs(near) <= 2.0 ** -4 * np.abs(_np(v)) + 2.0 ** -17 * 448).all() if quant else (near == 0).all()
