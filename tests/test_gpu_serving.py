"""The serving operators on the GPU (mfs_sample_rows, mfs_kv_append, mfs_paged_attention, mfs_prompt_attention)
against their 64-bit definitions."""
import numpy as np
import pytest

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


def _f32(x):
    return _torch().tensor(x, dtype=_torch().float32, device="cuda")


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


# ------------------------------------------------------------------ sampling

SETTINGS = [(0.7, 25, 1.0, 0.0), (0.8, 250, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (1.3, 0, 1.0, 0.05), (0.9, 40, 0.8, 0.02), (1.0, 0, 1.0, 0.0),
            (0.0, 0, 1.0, 0.0), (0.5, 1, 0.5, 0.5), (0.05, 100, 0.999, 0.0), (30.0, 0, 0.37, 0.0)]


def _sample(mfs, logits, u, t, k, p, m, **kw):
    out = _torch().full((logits.shape[0],), -7, dtype=_torch().int32, device="cuda")
    mfs.mfs_sample_rows(logits, _f32(u), out, temperature=_f32(t), top_k=_i32(k), top_p=_f32(p), min_p=_f32(m), **kw)
    return out.cpu().numpy()


@pytest.mark.parametrize("cols", [1, 2, 31, 129, 2048, 4099, 32000, 50001, 131071])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sample_rows_matches_the_definition(mfs, cols, dtype):
    """Every setting on normal logits of three widths; rows are strided and start at odd addresses."""
    rng = np.random.default_rng(cols)
    rows = 3 * len(SETTINGS)
    wide = _normal(rng, rows, cols + 5, dtype=dtype)
    wide *= _torch().linspace(0.3, 6.0, rows, device="cuda")[:, None].to(wide.dtype)
    x = wide[:, 3:3 + cols]
    u = rng.random(rows).astype(np.float32)
    t, k, p, m = (np.array([s[i] for s in SETTINGS] * 3) for i in range(4))
    got = _sample(mfs, x, u, t, k, p, m)
    xs = _np(x)
    want = [S.sample_row(xs[r], u[r], np.float32(t[r]), k[r], np.float32(p[r]), np.float32(m[r])) for r in range(rows)]
    assert got.tolist() == want


@pytest.mark.parametrize("n", [3, 1000, 40000])
def test_sample_rows_at_the_borders_of_equal_weights(mfs, n):
    """Equal logits: column floor(u n), for uniforms next to the borders j / n (the nearest fp32 on either side)."""
    j = np.unique(np.linspace(0, n - 1, 64).astype(np.int64))
    u = (j / n).astype(np.float32)
    u = np.concatenate([u, np.nextafter(u, np.float32(0)), np.nextafter(u, np.float32(1))])
    u = u[(u >= 0) & (u < 1)]
    x = _f32(np.full((len(u), n), 0.37))
    one, zero = np.ones(len(u)), np.zeros(len(u))
    # u is a fraction of powers of two: floor(u n) in whole numbers
    want = [int(int(float(v) * 2 ** 60) * n >> 60) for v in u]
    assert _sample(mfs, x, u, one, zero, one, zero).tolist() == want
    # the first half by top-k, and by top-p (the shortest prefix with sum >= half)
    h = (n + 1) // 2
    want = [int(int(float(v) * 2 ** 60) * h >> 60) for v in u]
    assert _sample(mfs, x, u, one, zero + h, one, zero).tolist() == want
    assert _sample(mfs, x, u, one, zero, one * 0.5, zero).tolist() == want


def test_sample_rows_decides_close_borders(mfs):
    """Uniforms within a few fp32 steps of a border between unequal weights: fp32 sums would leave them open."""
    rng = np.random.default_rng(3)
    n, rows = 700, 256
    x = rng.standard_normal(n).astype(np.float32)
    w = np.exp(x.astype(np.float64) - x.max())
    c = np.cumsum(w) / w.sum()
    j = rng.integers(0, n - 1, rows)
    u = c[j].astype(np.float32)
    for _ in range(2):
        u = np.where(rng.random(rows) < 0.5, np.nextafter(u, np.float32(1)), np.nextafter(u, np.float32(0)))
    gap = np.abs(c[None] - u.astype(np.float64)[:, None]).min(1)
    assert gap.min() > 1e-11  # the definition itself decides
    logits = _f32(np.tile(x, (rows, 1)))
    one, zero = np.ones(rows), np.zeros(rows)
    want = np.searchsorted(c, u.astype(np.float64), side="right")
    assert _sample(mfs, logits, u, one, zero, one, zero).tolist() == want.tolist()
    # the same borders as top-p: the cut has to fall on the right column
    order = np.argsort(-x, kind="stable")
    cs = np.cumsum(w[order]) / w.sum()
    p = cs[j].astype(np.float32)
    last = np.full(rows, np.nextafter(np.float32(1), np.float32(0)))
    got = _sample(mfs, logits, last, one, zero, p, zero)
    want = [S.sample_row(x, last[r], 1.0, 0, p[r], 0.0) for r in range(rows)]
    assert got.tolist() == want


def test_sample_rows_special_rows(mfs):
    inf, nan = np.inf, np.nan
    cases = [  # logits, u, T, k, p, m
        ([nan, nan, nan], 0.5, 1, 0, 1, 0), ([nan, -inf, -inf], 0.9, 1, 0, 1, 0), ([-inf, 0, -inf], 0.99, 1, 0, 1, 0),
        ([0, inf, 1, inf], 0.7, 1, 0, 1, 0), ([0, inf, 1, inf], 0.2, 1, 2, 0.4, 0), ([nan, 2, nan, 2], 0.6, 1, 0, 1, 0),
        ([1, 2, 3], 0.5, nan, 0, 1, 0), ([1, 2, 3], 0.5, -1, 0, 1, 0), ([3, 2, 3], 0.5, 0, 0, 1, 0), ([1, 2, 3], 0.999, inf, 0, 1, 0),
        ([1, 2, 3], 0.99, 1e-30, 0, 1, 0), ([1, 2, 3], 0.0, 1, 50, 1, 0), ([1, 2, 3], 0.0, 1, 0, 0, 0), ([1, 2, 3], 0.0, 1, 0, -1, 0),
        ([1, 2, 3], 0.0, 1, 0, 1, 1), ([1, 3, 3], 0.9, 1, 0, 1, 7), ([1, 2, 3], 1.0, 1, 0, 1, 0), ([1, 2, 3], -0.5, 1, 0, 1, 0),
        ([1, 2, 3], nan, 1, 0, 1, 0), ([-0.0, 0.0, -0.0], 0.4, 1, 2, 1, 0), ([0, -200, -200], 0.9999999, 1, 0, 1, 0),
        ([3e38, -3e38, 1], 0.5, 1, 0, 1, 0), ([1, 2, 3], 0.2, 1, 0, nan, nan), ([1e-40, 2e-40, 0], 0.9, 1, 1, 1, 0)]
    for row, u, t, k, p, m in cases:
        got = _sample(mfs, _f32([row]), [u], [t], [k], [p], [m])[0]
        # NaN settings switch their filter off
        want = S.sample_row(np.array(row, np.float32), 0.0 if u != u else u, t, k, 1.0 if p != p else p, 0.0 if m != m else m)
        assert got == want, (row, u, t, k, p, m, got, want)


def test_sample_rows_defaults_streams_and_capture(mfs):
    torch = _torch()
    rng = np.random.default_rng(5)
    x, u = _normal(rng, 40, 3001), _f32(rng.random(40))
    out = torch.full((40,), -7, dtype=torch.int32, device="cuda")
    mfs.mfs_sample_rows(x[:0], u, out)
    assert (out == -7).all()
    mfs.mfs_sample_rows(x, u, out)
    want = [S.sample_row(_np(x)[r], float(u[r])) for r in range(40)]
    assert out.tolist() == want
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2 = torch.full((40,), -7, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    mfs.mfs_sample_rows(x, u, out2, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, out2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mfs.mfs_sample_rows(x, u, out2)
    x.copy_(_normal(rng, 40, 3001))
    g.replay()
    torch.cuda.synchronize()
    assert out2.tolist() == [S.sample_row(_np(x)[r], float(u[r])) for r in range(40)]


# --------------------------------------------------------------- paged cache

def _pool(rng, pages, heads, page, hd, dtype, layout="head"):
    """k and v pools: page-major with heads outside ("head") or rows outside ("row"), or one allocation for both ("both")."""
    if layout == "row":
        return tuple(_normal(rng, pages, page, heads, hd, dtype=dtype).transpose(1, 2) for _ in range(2))
    if layout == "both":
        kv = _normal(rng, pages, 2, heads, page, hd, dtype=dtype)
        return kv[:, 0], kv[:, 1]
    return tuple(_normal(rng, pages, heads, page, hd, dtype=dtype) for _ in range(2))


def _table(rng, lens, page, spare=2, extra=3):
    """Shuffled distinct pages; entries past a sequence's length hold rubbish."""
    need = [-(-max(0, n) // page) for n in lens]
    order = rng.permutation(sum(need) + spare)
    t = rng.integers(-2**31, 2**31 - 1, (len(lens), max(need + [0]) + extra)).astype(np.int32)
    at = 0
    for s, c in enumerate(need):
        t[s, :c] = order[at:at + c]
        at += c
    return t, sum(need) + spare


@pytest.mark.parametrize("hq,hkv,hd,page,dtype,rope,layout", [
    (4, 4, 64, 16, "f32", "interleaved", "head"), (8, 2, 128, 16, "bf16", "half", "head"), (6, 2, 64, 1, "bf16", "interleaved", "row"),
    (32, 32, 128, 48, "bf16", "interleaved", "both"), (3, 1, 128, 7, "f32", "half", "row"), (5, 5, 64, 64, "bf16", None, "head")])
def test_kv_append(mfs, hq, hkv, hd, page, dtype, rope, layout):
    torch = _torch()
    rng = np.random.default_rng(hq * 100 + hd + page)
    new = [3, 0, 1, 17, 40, 1]
    past = [0, 5, 2999, 16, 7, 1 << 20]
    total = [a + b for a, b in zip(past, new)]
    lens = [n if n < 10000 else 40 for n in total]
    table, pages = _table(rng, lens, page)
    if page < 1000:  # the far sequence reaches one page only: a table row as wide as its position would be large
        wide = np.full((len(new), total[-1] // page + 1), -9, np.int32)
        wide[:, :min(table.shape[1], wide.shape[1])] = table[:, :wide.shape[1]]
        wide[-1] = -1
        wide[-1, (total[-1] - 1) // page] = table[-1, 0]
        table = wide
    n, tail = sum(new), 4
    qkv = _normal(rng, n + tail, hq + 2 * hkv, hd, dtype=dtype)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    kc, vc = _pool(rng, pages, hkv, page, hd, dtype, layout)
    k0, v0 = _np(kc), _np(vc)
    cache = mfs.PagedKV(kc, vc, torch.from_numpy(table).cuda())
    q_out = torch.full((n + tail, hq, hd), 7.0, dtype=_dt(dtype), device="cuda")
    k_out = torch.full((n + tail, hkv, hd), 7.0, dtype=_dt(dtype), device="cuda")
    mfs.mfs_kv_append(cache, k, v, _i32(np.cumsum([0] + new).tolist()), _i32(total), q=q, q_out=q_out, k_out=k_out, rope=rope, theta=10000.0)
    qn, kn, vn = _np(q), _np(k), _np(v)
    t = 0
    # fp32: the angle in 64 bits is reduced to +-pi and rounded once (2^-24 pi), cosine and sine within 2^-22, two products and a
    # sum (3 x 2^-24), each relative to |x_a| + |x_b| <= 2 max|x|: 2 * (3.2 + 4 + 3) 2^-24 max|x|; bf16: besides one rounding, 2^-8
    bound = 2.0 ** -24 * 21 * np.abs(_np(qkv)).max()
    rel = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    if rope is None:
        bound = rel = 0.0
    for s, c in enumerate(new):
        for p in range(past[s], total[s]):
            for got, src in ((_np(q_out[t]), qn[t]), (_np(k_out[t]), kn[t])):
                want = S.rotate(src, p, rope, 10000.0)
                assert (np.abs(got - want) <= bound + rel * np.abs(want)).all()
            pg = table[s, p // page]
            assert np.array_equal(_np(kc[pg, :, p % page]), _np(k_out[t])) and np.array_equal(_np(vc[pg, :, p % page]), vn[t])
            k0[pg, :, p % page], v0[pg, :, p % page] = _np(k_out[t]), vn[t]
            t += 1
    assert np.array_equal(k0, _np(kc)) and np.array_equal(v0, _np(vc))  # no other row changed
    assert (q_out[n:] == 7).all() and (k_out[n:] == 7).all()          # rows of no sequence


def test_kv_append_in_place_and_bad_pages(mfs):
    """q and k rotated in place; tokens whose page is outside the pool, whose position is outside the table or
    negative are rotated and not written."""
    torch = _torch()
    rng = np.random.default_rng(9)
    hq, hkv, hd, page = 4, 2, 64, 4
    kc, vc = _pool(rng, 3, hkv, page, hd, "f32")
    k0, v0 = kc.clone(), vc.clone()
    table = _i32([[0, 3], [-1, 1], [2, 2], [0, 1]])  # no two tokens reach the same row
    new, total = [2, 6, 3, 2], [2, 8, 10, 1]  # 3: no such page; -1; positions 8, 9 past the table; position -1
    table[0, 0] = 3
    n = sum(new)
    q, k, v = (_normal(rng, n, h, hd) for h in (hq, hkv, hkv))
    qn, kn = _np(q), _np(k)
    mfs.mfs_kv_append(mfs.PagedKV(kc, vc, table), k, v, _i32(np.cumsum([0] + new).tolist()), _i32(total), q=q, q_out=q, k_out=k, theta=500.0)
    t, changed = 0, set()
    for s, c in enumerate(new):
        for p in range(total[s] - c, total[s]):
            assert np.abs(_np(q[t]) - S.rotate(qn[t], p, "interleaved", 500.0)).max() < 1e-5
            assert np.abs(_np(k[t]) - S.rotate(kn[t], p, "interleaved", 500.0)).max() < 1e-5
            pg = int(table[s, p // page]) if 0 <= p < 8 else -1
            if 0 <= pg < 3:
                assert torch.equal(kc[pg, :, p % page], k[t]) and torch.equal(vc[pg, :, p % page], v[t])
                changed.add((pg, p % page))
            t += 1
    for pg in range(3):
        for r in range(page):
            if (pg, r) not in changed:
                assert torch.equal(kc[pg, :, r], k0[pg, :, r]) and torch.equal(vc[pg, :, r], v0[pg, :, r])
    assert len(changed) == 4 + 1 + 1


def _check_decode(mfs, rng, lens, hq, hkv, hd, page, dtype, layout="head", window=0, scale=None, qscale=1.0, check=None):
    torch = _torch()
    table, pages = _table(rng, lens, page)
    kc, vc = _pool(rng, pages, hkv, page, hd, dtype, layout)
    k, v = _np(kc), _np(vc)
    # every row that must not be read becomes NaN
    used = np.zeros((pages, page), bool)
    for s, n in enumerate(lens):
        for p in range(max(0, n - window) if window else 0, n):
            used[table[s, p // page], p % page] = True
    stale = torch.from_numpy(~used).cuda()
    for c in (kc, vc):
        c.masked_fill_(stale[:, None, :, None], float("nan"))
    n = len(lens)
    wide = _normal(rng, n, hq + 2, hd, dtype=dtype, scale=qscale)
    q = wide[:, :hq]
    out = torch.full((n + 2, hq, hd), 7.0, dtype=_dt(dtype), device="cuda")
    cache = mfs.PagedKV(kc, vc, torch.from_numpy(table).cuda())
    kw = {} if scale is None else dict(scale=scale)
    mfs.mfs_paged_attention(cache, q, _i32(lens), out[:n], window=window, **kw)
    got, qn = _np(out), _np(q)
    assert (got[n:] == 7).all()
    sc, g = hd ** -0.5 if scale is None else scale, hq // hkv
    for s in (range(n) if check is None else check):
        lo = max(0, lens[s] - window) if window else 0
        rows_k, rows_v = S.kv_rows(k, table[s], page, lo, lens[s]), S.kv_rows(v, table[s], page, lo, lens[s])
        for h in range(hq):
            ref, weighted, size = S.attend(qn[s, h], rows_k[:, h // g], rows_v[:, h // g], sc)
            tol = S.attention_tolerance(ref, weighted, size, max(1, lens[s] - lo), hd, dtype == "bf16")
            assert (np.abs(got[s, h] - ref) <= tol).all(), (s, h, lens[s], np.abs(got[s, h] - ref).max(), tol.min())
    return cache, q, out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hkv,hd,page,layout", [(4, 4, 64, 16, "head"), (8, 2, 128, 16, "row"), (6, 2, 64, 1, "both"), (3, 1, 128, 7, "head"),
                                                   (40, 2, 64, 48, "row"), (32, 32, 128, 64, "head"), (34, 1, 128, 33, "both")])
def test_paged_attention(mfs, hq, hkv, hd, page, layout, dtype):
    """Lengths 0, 1, around pages and tiles, and some hundred; rows behind each length are NaN."""
    rng = np.random.default_rng(hq + hd + page)
    _check_decode(mfs, rng, [0, 1, page, page + 1, 63, 64, 65, 127, 129, 300, -3, 515], hq, hkv, hd, page, dtype, layout)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window", [1, 2, 64, 100, 4000])
def test_paged_attention_window(mfs, window, dtype):
    rng = np.random.default_rng(window)
    _check_decode(mfs, rng, [0, 1, 63, 64, 100, 101, 165, 700], 8, 2, 64, 16, dtype, window=window)


@pytest.mark.parametrize("dtype,hq,hkv,hd", [("bf16", 8, 2, 128), ("f32", 2, 2, 64), ("bf16", 1, 1, 64)])
def test_paged_attention_long(mfs, dtype, hq, hkv, hd):
    """One long sequence among short ones: the split over the length, and its join."""
    rng = np.random.default_rng(17)
    _check_decode(mfs, rng, [5, 20011, 0, 64], hq, hkv, hd, 32, dtype)


def test_paged_attention_many_sequences(mfs):
    rng = np.random.default_rng(18)
    lens = (rng.integers(0, 40, 1500)).tolist()
    _check_decode(mfs, rng, lens, 4, 2, 64, 8, "bf16", check=range(0, 1500, 37))


def test_paged_attention_large_scores(mfs):
    """Scores of some hundreds: one key takes almost all the weight, and the running maximum moves a lot."""
    rng = np.random.default_rng(19)
    for dtype in ("f32", "bf16"):
        _check_decode(mfs, rng, [300, 1000, 77], 4, 1, 64, 16, dtype, qscale=30.0)
        _check_decode(mfs, rng, [300, 1000, 77], 4, 1, 64, 16, dtype, scale=1e-6)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_paged_attention_bad_pages_give_nan(mfs, dtype):
    torch = _torch()
    rng = np.random.default_rng(20)
    kc, vc = _pool(rng, 4, 2, 16, 64, dtype)
    table = _i32([[0, 1], [0, 4], [-1, 1], [2, 3]])
    q = _normal(rng, 4, 4, 64, dtype=dtype)
    out = torch.zeros_like(q)
    mfs.mfs_paged_attention(mfs.PagedKV(kc, vc, table), q, _i32([20, 20, 20, 40]), out)  # 40: past the table
    o = _np(out)
    assert np.isfinite(o[0]).all() and np.isnan(o[1:]).all()
    mfs.mfs_paged_attention(mfs.PagedKV(kc, vc, table), q, _i32([20, 16, 20, 32]), out, window=4)
    o = _np(out)
    assert np.isfinite(o).all()  # the bad entries are outside the windows now


def test_paged_attention_far_offsets(mfs):
    """Pages whose offsets pass 32 bits."""
    torch = _torch()
    rng = np.random.default_rng(21)
    pages, hkv, page, hd = 9000, 8, 256, 128  # 2.36e9 elements
    kc = torch.empty(pages, hkv, page, hd, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    table = _i32([[8999, 0, 8500], [8300, 8998, 1]])
    n = [600, 513]
    k, v = _normal(rng, sum(n), hkv, hd, dtype="bf16"), _normal(rng, sum(n), hkv, hd, dtype="bf16")
    cache = mfs.PagedKV(kc, vc, table)
    mfs.mfs_kv_append(cache, k, v, _i32([0, n[0], sum(n)]), _i32(n), rope=None)
    q = _normal(rng, 2, 16, hd, dtype="bf16")
    out = torch.empty_like(q)
    mfs.mfs_paged_attention(cache, q, _i32(n), out)
    at = 0
    for s in range(2):
        for h in (0, 7, 15):
            ref, weighted, size = S.attend(_np(q[s, h]), _np(k[at:at + n[s], h // 2]), _np(v[at:at + n[s], h // 2]), hd ** -0.5)
            assert (np.abs(_np(out[s, h]) - ref) <= S.attention_tolerance(ref, weighted, size, n[s], hd, True)).all()
        at += n[s]


def test_paged_attention_is_repeatable_and_captured(mfs):
    torch = _torch()
    rng = np.random.default_rng(22)
    lens = [3000, 1, 777, 0, 12000]
    cache, q, out = _check_decode(mfs, rng, lens, 8, 2, 128, 16, "bf16", check=[0, 1, 3])
    a = out[:5].clone()
    ws = mfs.mfs_paged_attention_workspace(cache, 8)
    kv = _i32(lens)
    b = torch.empty_like(a)
    for _ in range(3):
        ws.fill_(255)  # what a workspace holds before does not matter
        mfs.mfs_paged_attention(cache, q, kv, b, workspace=ws)
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mfs.mfs_paged_attention(cache, q, kv, b, workspace=ws)
    kv.copy_(_i32([10, 1, 30, 2999, 11]))  # lengths are read when the graph runs
    cache.table[3, :200] = 0
    g.replay()
    want = torch.empty_like(b)
    mfs.mfs_paged_attention(cache, q, kv, want)
    assert torch.equal(b, want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    b.zero_()
    torch.cuda.synchronize()
    mfs.mfs_paged_attention(cache, q, kv, b, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(b, want)


# ------------------------------------------------------------------- prompts

def _check_prompt(mfs, rng, lens, hq, hkv, hd, dtype, window=0, scale=None, qscale=1.0, tail=3, rows=None, poison=False):
    torch = _torch()
    n = sum(lens) + tail
    qkv = _normal(rng, n, hq + 2 * hkv, hd, dtype=dtype)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    q *= qscale
    if tail:
        qkv[n - tail:] = float("nan")  # rows behind the last sequence
    qn, kn, vn = _np(q), _np(k), _np(v)
    out = torch.full((n, hq, hd), 7.0, dtype=_dt(dtype), device="cuda")
    kw = {} if scale is None else dict(scale=scale)
    mfs.mfs_prompt_attention(q, k, v, _i32(np.cumsum([0] + lens).tolist()), out, window=window, **kw)
    got = _np(out)
    assert (got[n - tail:] == 7).all()
    sc, g, b = hd ** -0.5 if scale is None else scale, hq // hkv, 0
    for c in lens:
        picked = range(c) if rows is None or c <= rows else sorted(set(rng.integers(0, c, rows).tolist() + [0, 1, c - 1, c - 2, c // 2]))
        for i in picked:
            lo = max(0, i - window + 1) if window else 0
            for h in (range(hq) if c < 40 else {0, hq // 2, hq - 1}):
                ref, weighted, size = S.attend(qn[b + i, h], kn[b + lo:b + i + 1, h // g], vn[b + lo:b + i + 1, h // g], sc)
                tol = S.attention_tolerance(ref, weighted, size, i + 1 - lo, hd, dtype == "bf16")
                assert (np.abs(got[b + i, h] - ref) <= tol).all(), (c, i, h, np.abs(got[b + i, h] - ref).max(), tol.min())
        b += c
    return q, k, v, out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hkv,hd", [(4, 4, 64), (8, 2, 128), (6, 2, 64), (3, 1, 128)])
def test_prompt_attention(mfs, hq, hkv, hd, dtype):
    rng = np.random.default_rng(hq + hd)
    _check_prompt(mfs, rng, [1, 0, 2, 33, 127, 0, 128, 129, 1, 257, 64], hq, hkv, hd, dtype, rows=40)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("window", [1, 2, 64, 100, 128, 300, 5000])
def test_prompt_attention_window(mfs, window, hd, dtype):
    rng = np.random.default_rng(window + hd)
    _check_prompt(mfs, rng, [700, 3, 129, 511], 4, 2, hd, dtype, window=window, rows=60)


@pytest.mark.parametrize("dtype,hd", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_prompt_attention_long(mfs, dtype, hd):
    rng = np.random.default_rng(31)
    _check_prompt(mfs, rng, [3001, 10, 2000], 4, 1, hd, dtype, rows=40)
    _check_prompt(mfs, rng, [2500], 2, 2, hd, dtype, rows=40, tail=0)


def test_prompt_attention_large_scores(mfs):
    rng = np.random.default_rng(32)
    for dtype in ("f32", "bf16"):
        _check_prompt(mfs, rng, [500, 260], 2, 1, 64, dtype, qscale=30.0, rows=80)
        _check_prompt(mfs, rng, [300], 2, 1, 128, dtype, scale=1e-6, rows=80)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_prompt_attention_does_not_see_masked_places(mfs, bad, hd, dtype):
    """A key and a value that are NaN or infinite change no row before them, outside their window, or of another sequence."""
    torch = _torch()
    rng = np.random.default_rng(33)
    lens, window = [200, 450, 300], 150
    n = sum(lens)
    q, k, v = (_normal(rng, n, 2, hd, dtype=dtype) for _ in range(3))
    cu = _i32(np.cumsum([0] + lens).tolist())
    for w in (0, window):
        clean, got = torch.empty_like(q), torch.empty_like(q)
        mfs.mfs_prompt_attention(q, k, v, cu, clean, window=w)
        for which in ("v", "k"):
            at = 200 + 170
            kk, vv = k.clone(), v.clone()
            (vv if which == "v" else kk)[at, 1, 5] = bad
            mfs.mfs_prompt_attention(q, kk, vv, cu, got, window=w)
            touched = torch.zeros(n, dtype=torch.bool)
            touched[at:min(650, at + w) if w else 650] = True
            assert torch.equal(got[:, 0], clean[:, 0])
            assert torch.equal(got[~touched, 1], clean[~touched, 1])
            if which == "v":  # and it reaches the rows that do see it, in its own column
                assert not torch.isfinite(got[touched, 1, 5]).any()
                same = [c for c in range(hd) if c != 5]
                far = (got[touched][:, 1][:, same].float() - clean[touched][:, 1][:, same].float()).abs().max()
                assert float(far) <= 0.05


def test_prompt_attention_capture_and_lengths_on_the_device(mfs):
    torch = _torch()
    rng = np.random.default_rng(34)
    q, k, v = (_normal(rng, 600, 4, 128, dtype="bf16") for _ in range(3))
    cu = _i32([0, 100, 600])
    out = torch.empty_like(q)
    mfs.mfs_prompt_attention(q, k, v, cu, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mfs.mfs_prompt_attention(q, k, v, cu, out)
    cu.copy_(_i32([0, 333, 500]))
    out.fill_(7)
    g.replay()
    want = torch.full_like(out, 7)
    mfs.mfs_prompt_attention(q, k, v, cu, want)
    assert torch.equal(out, want) and (out[500:] == 7).all() and (out[:500] != 7).any()


# ------------------------------------------------------- a run of them together

@pytest.mark.parametrize("dtype,hd,rope,window", [("bf16", 128, "interleaved", 0), ("f32", 64, "half", 90), ("bf16", 64, "half", 50)])
def test_prompts_then_tokens_through_the_paged_cache(mfs, dtype, hd, rope, window):
    """Two prompts enter the cache and are attended to, then tokens follow one by one: every output equals the attention over
    the sequence's whole history, rotated at its positions; then a token is drawn from logits made of the outputs."""
    torch = _torch()
    rng = np.random.default_rng(hd + window)
    hq, hkv, page, steps, lens = 8, 2, 16, 5, [130, 41]
    n = sum(lens)
    table, pages = _table(rng, [x + steps for x in lens], page)
    kc, vc = _pool(rng, pages, hkv, page, hd, dtype)
    cache = mfs.PagedKV(kc, vc, torch.from_numpy(table).cuda())
    hist_k, hist_v = [[], []], [[], []]

    def keep(s, k, v, p):
        hist_k[s].append(S.rotate(_np(k), p, rope, 10000.0))
        hist_v[s].append(_np(v))

    def check(s, i, q, got):
        lo = max(0, i - window + 1) if window else 0
        k, v = np.stack(hist_k[s])[lo:i + 1], np.stack(hist_v[s])[lo:i + 1]
        for h in range(hq):
            qr = S.rotate(_np(q)[h], i, rope, 10000.0)
            ref, weighted, size = S.attend(qr, k[:, h // 4], v[:, h // 4], hd ** -0.5)
            tol = S.attention_tolerance(ref, weighted, size, i + 1, hd, dtype == "bf16")
            # the rotated q and k are rounded to the cache's type: each moves a score by half a step of at most `size`, a weight by as much
            tol = tol + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -22) * 4 * size * weighted
            assert (np.abs(_np(got)[h] - ref) <= tol).all()

    q, k, v = (_normal(rng, n, h, hd, dtype=dtype) for h in (hq, hkv, hkv))
    q_out, k_out, out = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q)
    cu = _i32([0, lens[0], n])
    mfs.mfs_kv_append(cache, k, v, cu, _i32(lens), q=q, q_out=q_out, k_out=k_out, rope=rope)
    mfs.mfs_prompt_attention(q_out, k_out, v, cu, out, window=window)
    t = 0
    for s in range(2):
        for p in range(lens[s]):
            keep(s, k[t + p], v[t + p], p)
        for p in (0, 1, lens[s] // 2, lens[s] - 1):
            check(s, p, q[t + p], out[t + p])
        t += lens[s]
    ws = mfs.mfs_paged_attention_workspace(cache, hq)
    head = _normal(rng, hq * hd, 501)
    tokens = torch.empty(2, dtype=torch.int32, device="cuda")
    for step in range(1, steps + 1):
        q, k, v = (_normal(rng, 2, h, hd, dtype=dtype) for h in (hq, hkv, hkv))
        kv_len = _i32([x + step for x in lens])
        q_out, o = torch.empty_like(q), torch.empty_like(q)
        mfs.mfs_kv_append(cache, k, v, _i32([0, 1, 2]), kv_len, q=q, q_out=q_out, rope=rope)
        mfs.mfs_paged_attention(cache, q_out, kv_len, o, window=window, workspace=ws)
        logits = o.float().reshape(2, -1) @ head
        u = _f32(rng.random(2))
        mfs.mfs_sample_rows(logits, u, tokens, temperature=_f32([0.7, 0.9]), top_k=_i32([25, 0]), top_p=_f32([1.0, 0.9]))
        for s in range(2):
            keep(s, k[s], v[s], lens[s] + step - 1)
            check(s, lens[s] + step - 1, q[s], o[s])
            want = S.sample_row(_np(logits[s]), float(u[s]), *[(np.float32(0.7), 25, 1.0), (np.float32(0.9), 0, np.float32(0.9))][s])
            assert int(tokens[s]) == want


# ------------------------------------------------------- refusals of the binding

def test_binding_refuses_tensors_that_do_not_fit(mfs):
    torch = _torch()
    f = dict(device="cuda", dtype=torch.bfloat16)
    kc, table, kv, cu = torch.zeros(4, 2, 16, 64, **f), torch.zeros(2, 2, dtype=torch.int32, device="cuda"), _i32([1, 1]), _i32([0, 1, 2])
    cache = mfs.PagedKV(kc, kc.clone(), table)
    q, k = torch.zeros(2, 4, 64, **f), torch.zeros(2, 2, 64, **f)

    def refused(call, *a, **kw):
        with pytest.raises(mfs.MfsError) as e:
            call(*a, **kw)
        assert e.value.status == "MFS_E_ARG"

    refused(mfs.PagedKV, kc, kc.float(), table)
    refused(mfs.PagedKV, kc, kc[:3], table)
    refused(mfs.PagedKV, kc, kc.transpose(1, 2).contiguous().transpose(1, 2), table)
    refused(mfs.PagedKV, kc, kc, table.long())
    refused(mfs.PagedKV, kc, kc, table.t()[:, :2].contiguous().t())
    refused(mfs.PagedKV, kc.half(), kc.half(), table)
    append, attend, prompt, sample = mfs.mfs_kv_append, mfs.mfs_paged_attention, mfs.mfs_prompt_attention, mfs.mfs_sample_rows
    refused(append, cache, k, k[:1], cu, kv)
    refused(append, cache, k.float(), k.float(), cu, kv)
    refused(append, cache, k, k, cu[:2], kv)
    refused(append, cache, k, k, cu, _i32([1, 1, 1]))
    refused(append, cache, k, k, cu, kv, q=q)
    refused(append, cache, k, k, cu, kv, q=q, q_out=q[:, :2])
    refused(append, cache, k, k, cu.cpu(), kv)
    refused(append, cache, k, k, cu, kv, rope="both")
    refused(append, cache, k, k, cu, kv, theta=0.0)
    refused(append, cache, torch.zeros(2, 64, 2, **f).transpose(1, 2), k, cu, kv)
    refused(attend, cache, q, kv[:1], q)
    refused(attend, cache, torch.zeros(3, 4, 64, **f), _i32([1, 1, 1]), torch.zeros(3, 4, 64, **f))
    refused(attend, cache, q[:, :3], kv, q[:, :3])
    refused(attend, cache, q, kv, q, window=-1)
    refused(attend, cache, q, kv, q, scale=0.0)
    refused(attend, cache, q, kv, q, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    refused(prompt, q, k, k.float(), cu, q)
    refused(prompt, q, k, k, cu.float(), q)
    refused(prompt, q[:, :3], k, k, cu, torch.empty_like(q[:, :3]))
    refused(prompt, torch.zeros(2, 4, 32, **f), torch.zeros(2, 2, 32, **f), torch.zeros(2, 2, 32, **f), cu, torch.zeros(2, 4, 32, **f))
    x, u, out = torch.zeros(2, 8, device="cuda"), _f32([0, 0]), _i32([0, 0])
    refused(sample, x.half(), u, out)
    refused(sample, x, u[:1], out)
    refused(sample, x, u, out.long())
    refused(sample, x, u, out, top_k=_f32([1, 1]))
    refused(sample, x.t(), u, out)
    refused(sample, x[:, :0], u, out)


# ------------------------------------------------------------- calls at the edges

def test_sample_rows_of_extreme_shapes(mfs):
    """Many short rows; one row of the most columns; a row too wide for shared memory with each filter."""
    rng = np.random.default_rng(41)
    x = _normal(rng, 5000, 50, scale=2.0)
    u = rng.random(5000).astype(np.float32)
    t, k, p, m = np.full(5000, 0.9), rng.integers(0, 60, 5000), rng.random(5000).astype(np.float32) * 1.2, rng.random(5000).astype(np.float32) * 0.2
    xs = _np(x)
    assert _sample(mfs, x, u, t, k, p, m).tolist() == [S.sample_row(xs[r], u[r], np.float32(0.9), k[r], p[r], m[r]) for r in range(5000)]
    for cols, dtype in ((1 << 22, "bf16"), (500_001, "f32")):
        x = _normal(rng, 1, cols, dtype=dtype, scale=3.0)
        xs = _np(x)[0]
        for t, k, p, m in ((1.0, 0, 1.0, 0.0), (0.8, 40, 0.9, 0.0), (1.0, 0, 0.8, 0.0), (1.2, 3000, 1.0, 0.0), (1.0, 0, 1.0, 0.01)):
            assert _sample(mfs, x, [0.37], [t], [k], [p], [m])[0] == S.sample_row(xs, np.float32(0.37), np.float32(t), k, np.float32(p), np.float32(m))


@pytest.mark.parametrize("cols", [700, 40000])
def test_sample_rows_of_ties_and_flat_rows(mfs, cols):
    """Few distinct logits, so that borders fall among equal ones; temperatures from almost 0 to infinity."""
    rng = np.random.default_rng(cols)
    rows = 60
    x = _torch().from_numpy(rng.integers(-3, 3, (rows, cols)).astype(np.float32)).cuda()
    u = rng.random(rows).astype(np.float32)
    t = np.array([1e-20, 0.01, 0.5, 1.0, 40.0, np.inf] * 10)
    k = np.array([0, 1, 7, 300, 600, cols // 3, cols, cols + 5, 0, 0] * 6)
    p = np.array([1.0, 0.5, 0.99, 0.2] * 15).astype(np.float32)
    m = np.array([0.0, 0.0, 0.1] * 20).astype(np.float32)
    xs = _np(x)
    want = [S.sample_row(xs[r], u[r], np.float32(t[r]), k[r], p[r], m[r]) for r in range(rows)]
    assert _sample(mfs, x, u, t, k, p, m).tolist() == want


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_paged_attention_over_its_own_queries(mfs, dtype):
    """out may be q; the table may be shared by all sequences (stride 0) and the pages too."""
    torch = _torch()
    rng = np.random.default_rng(43)
    kc, vc = _pool(rng, 64, 2, 16, 128, dtype)
    table = torch.randperm(64, device="cuda").to(torch.int32)[None].expand(5, 64)
    cache = mfs.PagedKV(kc, vc, table)
    q = _normal(rng, 5, 8, 128, dtype=dtype)
    kv = _i32([1000, 3, 517, 0, 1024])
    want = torch.empty_like(q)
    mfs.mfs_paged_attention(cache, q, kv, want)
    k = _np(kc)[table[0].cpu().numpy()].transpose(0, 2, 1, 3).reshape(-1, 2, 128)
    v = _np(vc)[table[0].cpu().numpy()].transpose(0, 2, 1, 3).reshape(-1, 2, 128)
    for s, n in ((0, 1000), (4, 1024)):
        ref, weighted, size = S.attend(_np(q[s, 5]), k[:n, 1], v[:n, 1], 128 ** -0.5)
        assert (np.abs(_np(want[s, 5]) - ref) <= S.attention_tolerance(ref, weighted, size, n, 128, dtype == "bf16")).all()
    mfs.mfs_paged_attention(cache, q, kv, q)
    assert torch.equal(q, want)


def test_calls_on_two_streams_at_once(mfs):
    """Prompts, tokens and sampling on two streams, each with outputs and a workspace of its own, repeated."""
    torch = _torch()
    rng = np.random.default_rng(44)
    kc, vc = _pool(rng, 300, 4, 16, 128, "bf16")
    cache = mfs.PagedKV(kc, vc, torch.arange(300, dtype=torch.int32, device="cuda").reshape(3, 100))
    q, kv = _normal(rng, 3, 16, 128, dtype="bf16"), _i32([1600, 100, 900])
    pq, pk, pv, cu = _normal(rng, 1500, 16, 128, dtype="bf16"), _normal(rng, 1500, 4, 128, dtype="bf16"), _normal(rng, 1500, 4, 128, dtype="bf16"), _i32([0, 400, 1500])
    x, u = _normal(rng, 200, 33000, scale=3.0), _f32(rng.random(200))
    p = torch.full((200,), 0.9, device="cuda")

    def run(stream):
        a, b, c = torch.empty_like(q), torch.empty_like(pq), torch.empty(200, dtype=torch.int32, device="cuda")
        ws = mfs.mfs_paged_attention_workspace(cache, 16)
        torch.cuda.synchronize()
        return a, b, c, lambda: (mfs.mfs_paged_attention(cache, q, kv, a, workspace=ws, stream=stream), mfs.mfs_prompt_attention(pq, pk, pv, cu, b, stream=stream),
                                 mfs.mfs_sample_rows(x, u, c, top_p=p, stream=stream))

    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    one, two = run(s1.cuda_stream), run(s2.cuda_stream)
    one[3]()
    torch.cuda.synchronize()
    want = [t.clone() for t in one[:3]]
    for _ in range(10):
        one[3]()
        two[3]()
    torch.cuda.synchronize()
    for t in (one, two):
        assert all(torch.equal(a, b) for a, b in zip(t[:3], want))


def test_prompt_attention_many_short_sequences(mfs):
    """Padded batches: far more entries in cu than sequences with tokens, and hundreds of short ones."""
    rng = np.random.default_rng(45)
    lens = np.zeros(700, int)
    lens[::3] = rng.integers(1, 9, len(lens[::3]))
    for dtype in ("bf16", "f32"):
        _check_prompt(mfs, rng, lens.tolist(), 4, 2, 64, dtype)


@pytest.mark.parametrize("hd,dtype", [(64, "bf16"), (128, "f32")])
def test_paged_attention_at_the_largest_length(mfs, hd, dtype):
    """2^31 - 1 positions, a window of the last 1001: the last tile ends past the largest int.  Every
    page of the sequence is the same one, so the window's rows are its rows 64534 .. 65534."""
    torch, rng = _torch(), np.random.RandomState(3)
    k, v = _normal(rng, 1, 1, 65536, hd, dtype=dtype), _normal(rng, 1, 1, 65536, hd, dtype=dtype)
    k[:, :, 65535] = v[:, :, 65535] = float("nan")
    q = _normal(rng, 1, 4, hd, dtype=dtype)
    out = torch.full_like(q, -7.0)
    table = torch.zeros(1, 32768, dtype=torch.int32, device="cuda")
    mfs.mfs_paged_attention(mfs.PagedKV(k, v, table), q, _i32([2**31 - 1]), out, window=1001)
    keys, vals, qs = _np(k)[0, 0, 64534:65535], _np(v)[0, 0, 64534:65535], _np(q)[0]
    scores = qs @ keys.T * hd ** -0.5
    w = np.exp(scores - scores.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    ref = w @ vals
    size = (np.abs(qs) @ np.abs(keys).T * hd ** -0.5).max()
    assert (np.abs(_np(out)[0] - ref) <= S.attention_tolerance(ref, w @ np.abs(vals), size, 1001, hd, dtype == "bf16")).all()


def test_numbers_past_an_int_are_refused(mfs):
    import torch
    q = torch.zeros(1, 2, 64, device="cuda")
    c = mfs.PagedKV(torch.zeros(1, 2, 16, 64, device="cuda"), torch.zeros(1, 2, 16, 64, device="cuda"),
                    torch.zeros(1, 1, dtype=torch.int32, device="cuda"))
    n = torch.ones(2, dtype=torch.int32, device="cuda")
    for window in (-1, 2**31, 2**32 + 5):
        with pytest.raises(mfs.MfsError, match="window"):
            mfs.mfs_paged_attention(c, q, n[:1], torch.empty_like(q), window=window)
        with pytest.raises(mfs.MfsError, match="window"):
            mfs.mfs_prompt_attention(q, q, q, n, torch.empty_like(q), window=window)
    one = torch.zeros(1, device="cuda")
    with pytest.raises(mfs.MfsError, match="too many"):
        mfs.mfs_sample_rows(one[:, None].expand(2**32 + 1, 1), one, torch.zeros(1, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("hq,hkv,hd,lens", [(1, 1, 128, [333]), (8, 8, 64, [300]), (4, 2, 128, [150] * 12), (32, 8, 64, [300, 1, 299]),
                                            (3, 1, 64, [33] * 70), (32, 8, 128, [700, 600])])
def test_prompt_attention_fp32_row_tiles(mfs, hq, hkv, hd, lens):
    """Few rows, many short sequences and many rows, so that row tiles of every size are chosen."""
    _check_prompt(mfs, np.random.default_rng(71), lens, hq, hkv, hd, "f32", rows=12)
    _check_prompt(mfs, np.random.default_rng(72), lens, hq, hkv, hd, "f32", window=37, rows=12)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hkv,hd", [(2, 2, 128), (10, 2, 64), (24, 2, 128)])
def test_paged_attention_of_tiny_and_long_sequences_together(mfs, hq, hkv, hd, dtype):
    """Hundreds of sequences of one to three positions around a few long ones: shares that hold many items, one,
    a part of one, or nothing."""
    rng = np.random.default_rng(hq + hd)
    lens = [1] * 400 + [0, 3001, 2, 0] + [3] * 300 + [700, 1, 0, 650]
    check = [0, 1, 399, 400, 401, 402, 403, 404, 405, 555, 700, 703, 704, 705, 706, 707]
    _check_decode(mfs, rng, lens, hq, hkv, hd, 16, dtype, check=check)
    _check_decode(mfs, rng, [40] * 61 + [1], hq, hkv, hd, 16, dtype, window=33)


@pytest.mark.parametrize("cols,dtype", [(16384, "f32"), (32000, "f32"), (40003, "bf16")])
def test_sample_rows_many_long_rows(mfs, cols, dtype):
    """More rows than half the SMs, each too long for half an SM's shared memory: one CTA to a row."""
    rng = np.random.default_rng(cols + 1)
    rows = 9 * len(SETTINGS)
    x = _normal(rng, rows, cols + 1, dtype=dtype, scale=2.5)[:, 1:]
    u = rng.random(rows).astype(np.float32)
    t, k, p, m = (np.array([s[i] for s in SETTINGS] * 9) for i in range(4))
    got = _sample(mfs, x, u, t, k, p, m)
    xs = _np(x)
    assert got.tolist() == [S.sample_row(xs[r], u[r], np.float32(t[r]), k[r], np.float32(p[r]), np.float32(m[r])) for r in range(rows)]
    flat = _torch().from_numpy(rng.integers(-2, 2, (rows, cols)).astype(np.float32)).to(_dt(dtype)).cuda()
    got, fs = _sample(mfs, flat, u, t, k, p, m), _np(flat)
    assert got.tolist() == [S.sample_row(fs[r], u[r], np.float32(t[r]), k[r], np.float32(p[r]), np.float32(m[r])) for r in range(rows)]


@pytest.mark.parametrize("how", ["infinite", "overflowing"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hkv,hd", [(4, 4, 64), (8, 2, 128), (6, 2, 64), (3, 1, 128), (40, 2, 64)])
def test_paged_attention_scores_of_minus_infinity(mfs, hq, hkv, hd, dtype, how):
    """Keys whose score is -infinity (an infinite element, or products past the largest fp32) weigh nothing, wherever they
    lie in their tile, share or sequence; a sequence that has no other keys gives NaN.  The same alone and in a batch."""
    torch = _torch()
    rng = np.random.default_rng(51 + hq + hd)
    page, big = 16, 1e20
    where = [(1, [0]), (17, [16]), (33, [32]), (40, range(32)), (65, range(64)), (300, range(299)), (300, range(1, 300)), (50, range(50)),
             (3001, range(2990)), (3001, range(100, 3001)), (3001, [0, 1500, 3000]), (3001, range(3001)), (20, [])]
    lens = [n for n, _ in where]
    table, pages = _table(rng, lens, page)
    kc, vc = _pool(rng, pages, hkv, page, hd, dtype)
    q = _normal(rng, len(lens), hq, hd, dtype=dtype)
    q[:, :, 5] = big if how == "overflowing" else q[:, :, 5].abs() + 0.125
    if how == "overflowing":
        kc[:, :, :, 5] = 0
    for s, (_, gone) in enumerate(where):
        for p in gone:
            kc[table[s, p // page], :, p % page, 5] = -big if how == "overflowing" else -np.inf
    cache = mfs.PagedKV(kc, vc, torch.from_numpy(table).cuda())
    out, k, v, qn = torch.empty_like(q), _np(kc), _np(vc), _np(q)
    mfs.mfs_paged_attention(cache, q, _i32(lens), out)
    alone = torch.empty_like(q)
    for s, n in enumerate(lens):
        mfs.mfs_paged_attention(mfs.PagedKV(kc, vc, cache.table[s:s + 1]), q[s:s + 1], _i32([n]), alone[s:s + 1])
    for s, (n, gone) in enumerate(where):
        seen = sorted(set(range(n)) - set(gone))
        rows_k, rows_v = S.kv_rows(k, table[s], page, 0, n)[seen], S.kv_rows(v, table[s], page, 0, n)[seen]
        for got in (_np(out[s]), _np(alone[s])):
            if not seen:
                assert np.isnan(got).all(), (s, n)
                continue
            for h in range(hq):
                ref, weighted, size = S.attend(qn[s, h], rows_k[:, h * hkv // hq], rows_v[:, h * hkv // hq], hd ** -0.5)
                tol = S.attention_tolerance(ref, weighted, size, n, hd, dtype == "bf16")
                assert (np.abs(got[h] - ref) <= tol).all(), (s, n, h)


def test_default_workspace_on_the_null_stream(mfs):
    """stream=0 with no workspace, beside other streams that allocate and write: each call has its own results."""
    torch = _torch()
    rng = np.random.default_rng(52)
    cache = mfs.PagedKV(*_pool(rng, 300, 2, 16, 128, "bf16"), torch.arange(300, dtype=torch.int32, device="cuda")[None])
    q, kv = _normal(rng, 1, 8, 128, dtype="bf16"), _i32([4800])
    want, others = torch.empty_like(q), [torch.cuda.Stream() for _ in range(33)]
    mfs.mfs_paged_attention(cache, q, kv, want)
    size = mfs.mfs_paged_attention_workspace(cache, 8).numel()
    torch.cuda.synchronize()
    outs = [torch.zeros_like(q) for _ in others]
    torch.cuda.synchronize()
    for out, side in zip(outs, others):
        mfs.mfs_paged_attention(cache, q, kv, out, stream=0)
        with torch.cuda.stream(side):
            torch.empty(size, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for out in outs)


@pytest.mark.parametrize("hq,hkv", [(4, 2), (8, 2), (6, 2), (10, 2)])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_prompt_attention_bad_values_among_grouped_heads(mfs, bad, hd, hq, hkv):
    """A NaN or infinite value reaches exactly the rows of its kv head's query heads that see it, in its own column, and
    as itself; every other element is what it is without it."""
    torch = _torch()
    rng = np.random.default_rng(35)
    lens, g = [200, 450, 300], hq // hkv
    n = sum(lens)
    q, k, v = (_normal(rng, n, h, hd, dtype="bf16") for h in (hq, hkv, hkv))
    cu = _i32(np.cumsum([0] + lens).tolist())
    qn, kn, vn = _np(q), _np(k), _np(v)
    for w in (0, 150):
        clean, got, again = (torch.empty_like(q) for _ in range(3))
        mfs.mfs_prompt_attention(q, k, v, cu, clean, window=w)
        for at in (200 + 170, 200 + 3, 200 + 449):  # inside the second sequence, near its start, its last token
            vv = v.clone()
            vv[at, 1, 5] = bad
            mfs.mfs_prompt_attention(q, k, vv, cu, got, window=w)
            mfs.mfs_prompt_attention(q, k, vv, cu, again, window=w)
            assert torch.equal(got.view(torch.int16), again.view(torch.int16))
            end = min(650, at + w) if w else 650
            touched = torch.zeros(n, dtype=torch.bool)
            touched[at:end] = True
            assert torch.equal(got[:, :g], clean[:, :g]) and torch.equal(got[~touched], clean[~touched])
            column = _np(got[at:end, g:, 5])
            assert np.isnan(column).all() if bad != bad else (column == bad).all()
            for i in {at, at + 1, (at + end) // 2, end - 1} - {650}:
                lo = max(200, i - w + 1) if w else 200
                for h in range(g, hq):
                    ref, weighted, size = S.attend(qn[i, h], kn[lo:i + 1, 1], vn[lo:i + 1, 1], hd ** -0.5)
                    tol = S.attention_tolerance(ref, weighted, size, i + 1 - lo, hd, True)
                    off = np.abs(_np(got[i, h]) - ref) <= tol
                    off[5] = True
                    assert off.all(), (at, i, h)


@pytest.mark.parametrize("hq,hkv,hd,dtype", [(2, 2, 64, "bf16"), (2, 2, 128, "bf16"), (4, 2, 128, "bf16"), (8, 2, 64, "bf16"), (3, 1, 64, "f32")])
def test_prompt_attention_infinite_scores_beside_bad_values(mfs, hq, hkv, hd, dtype):
    """An infinite key next to an infinite value: rows whose score is +infinity there are NaN, rows whose score is
    -infinity do not see that key, and have the infinity in the value's column."""
    torch = _torch()
    rng = np.random.default_rng(36)
    n, at, g, b = 330, 140, hq // hkv, hkv - 1
    q, k, v = (_normal(rng, n, h, hd, dtype=dtype) for h in (hq, hkv, hkv))
    k[at + 3, b, 5] = float("inf")
    v[at, b, 7] = float("inf")
    k[0, b, 9] = float("-inf")  # and a first key that some rows do not see
    out = torch.empty_like(q)
    mfs.mfs_prompt_attention(q, k, v, _i32([0, n]), out)
    qn, kn, vn, got = _np(q), _np(k), _np(v), _np(out)
    vn[at, b, 7] = 0
    for i in (at - 1, at, at + 2, at + 3, at + 4, at + 20, 255, 256, n - 1):
        for h in range(b * g, hq):
            plus = qn[i, h, 9] < 0 or (i >= at + 3 and qn[i, h, 5] > 0)
            if plus:
                assert np.isnan(got[i, h]).all(), (i, h)
                continue
            keys = [j for j in range(1, i + 1) if j != at + 3]
            ref, weighted, size = S.attend(qn[i, h], kn[keys, b], vn[keys, b], hd ** -0.5)
            off = np.abs(got[i, h] - ref) <= S.attention_tolerance(ref, weighted, size, i + 1, hd, dtype == "bf16")
            if i >= at:
                assert got[i, h, 7] == np.inf
                off[7] = True
            assert off.all(), (i, h)
    # rows that see nothing but keys of score -infinity
    q, k = torch.ones_like(q), torch.ones_like(k)
    k[:129, :, 3] = float("-inf")
    mfs.mfs_prompt_attention(q, k, v, _i32([0, n]), out)
    got = _np(out)
    assert np.isnan(got[:129]).all() and np.isfinite(got[129:, 0, 8]).all() and (got[at:, hq - 1, 7] == np.inf).all()


@pytest.mark.parametrize("hq,hkv,hd", [(2, 1, 64), (1, 1, 128)])
def test_prompt_attention_bad_values_cost_no_pass_over_the_prompt(mfs, hq, hkv, hd):
    """What rows that see a bad value take besides does not grow with the prompt."""
    torch = _torch()
    rng = np.random.default_rng(37)
    n = 16384
    q, k, v = (_normal(rng, n, h, hd, dtype="bf16") for h in (hq, hkv, hkv))
    cu, clean, got = _i32([0, n]), torch.empty_like(q), torch.empty_like(q)

    def milliseconds(values, out):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        mfs.mfs_prompt_attention(q, k, values, cu, out)
        a.record()
        mfs.mfs_prompt_attention(q, k, values, cu, out)
        b.record()
        b.synchronize()
        return a.elapsed_time(b)

    fast = milliseconds(v, clean)
    v[n - 120, 0, 3] = float("nan")
    slow = milliseconds(v, got)
    assert torch.equal(got[:n - 120], clean[:n - 120]) and torch.isnan(got[n - 120:, :, 3]).all()
    # keys of the last 128-row tile by 32 rows a warp, some microseconds each: a millisecond; 32 passes over all keys take a hundred
    assert slow <= 2 * fast + 10, (fast, slow)


def test_sample_rows_of_the_most_columns_with_a_light_tail(mfs):
    """One column outweighs 4194303 others of 0.49 2^-39 of it each, 3.7e-6 of the total together: the draw and the border of
    top-p fall into the tail at the place that the definition gives, to the stated distance in weight."""
    import math
    from fractions import Fraction as F
    cols = 1 << 22
    tail = np.float32(math.log(0.49) - 39 * math.log(2))
    w, n = F(math.exp(float(tail))), cols - 1
    far = [1.0 - j * 2.0 ** -24 for j in (1, 7, 20, 30, 41, 55, 60)]  # fp32 numbers; 62 of these steps are the tail
    x = np.full(cols, tail, np.float32)
    x[0] = 0
    # a border may be missed by (2^-40 + cols 2^-60) of the total; each column weighs w, and a rounding of the place down
    miss = (2.0 ** -40 + cols * 2.0 ** -60) / float(w) + 1

    def column(u, kept):  # the first one at which 1 + c w exceeds u (1 + kept w)
        return math.floor((F(u) * (1 + kept * w) - 1) / w) + 1

    rows = _f32(np.tile(x, (len(far), 1)))
    one, zero = np.ones(len(far)), np.zeros(len(far))
    got = _sample(mfs, rows, np.array(far, np.float32), one, zero, one, zero)
    assert (np.abs(got - np.array([column(u, n) for u in far])) <= miss).all(), got
    last = 1.0 - 2.0 ** -24
    got = _sample(mfs, rows, np.full(len(far), last, np.float32), one, zero, np.array(far, np.float32), zero)
    kept = [math.ceil((F(p) * (1 + n * w) - 1) / w) for p in far]  # the shortest prefix of at least p
    assert (np.abs(got - np.array([max(0, column(last, m)) for m in kept])) <= 2 * miss).all(), got


def test_kv_append_of_two_tokens_on_one_row(mfs):
    """Two sequences whose tables share a page and reach the same row of it: every 16 bytes of that row are one of the two
    tokens', and no other row changes."""
    torch = _torch()
    rng = np.random.default_rng(53)
    kc, vc = _pool(rng, 3, 2, 16, 128, "bf16")
    k0, v0 = kc.clone(), vc.clone()
    k, v = _normal(rng, 2, 2, 128, dtype="bf16"), _normal(rng, 2, 2, 128, dtype="bf16")
    mfs.mfs_kv_append(mfs.PagedKV(kc, vc, _i32([[1], [1]])), k, v, _i32([0, 1, 2]), _i32([6, 6]), rope=None)
    for pool, old, new in ((kc, k0, k), (vc, v0, v)):
        parts, either = pool[1, :, 5].reshape(2, 16, 8), new.reshape(2, 2, 16, 8)
        assert ((parts == either[0]).all(-1) | (parts == either[1]).all(-1)).all()
        pool[1, :, 5] = old[1, :, 5]
        assert torch.equal(pool, old)


def test_sample_rows_at_the_ends_of_temperature(mfs):
    """Temperatures next to 0 (below 1.5e-30 they count as that) with logits as small; temperatures near the largest fp32
    number with logits whose difference is past it (which counts as infinite), in short rows and long ones."""
    u = np.linspace(0, 0.999, 23).astype(np.float32)
    one = np.ones(len(u))
    x = np.array([0, 1e-30, 2e-30, -1e-30, -4e-31], np.float32)
    for t in (1e-45, 1e-38, 1.4e-30, 1.6e-30, 1e-29):
        for k, p, m in ((0, 1.0, 0.0), (3, 1.0, 0.0), (0, 0.6, 0.0), (0, 1.0, 0.3)):
            got = _sample(mfs, _f32(np.tile(x, (len(u), 1))), u, one * t, one * k, one * p, one * m)
            want = [S.sample_row(x, v, max(np.float32(t), np.float32(1.5e-30)), k, np.float32(p), np.float32(m)) for v in u]
            assert got.tolist() == want, (t, k, p, m)
    rng = np.random.default_rng(54)
    big = np.float32(3e38)
    for x in (np.array([big, -big, 1, 2.9e38], np.float32), rng.choice(np.array([big, -big, 0, 1e38, -2e37], np.float32), 5000),
              rng.choice(np.array([big, -big, 1e38], np.float32), 40000)):
        seen = np.where(x == -big, -np.inf, x)
        n = len(x)
        for k, p, m in ((0, 1.0, 0.0), (2, 1.0, 0.0), (n - 1, 1.0, 0.0), (n * 9 // 10, 0.99, 0.0), (0, 0.7, 0.0), (0, 1.0, 0.4)):
            got = _sample(mfs, _f32(np.tile(x, (len(u), 1))), u, one * big, one * k, one * p, one * m)
            assert got.tolist() == [S.sample_row(seen, v, big, k, np.float32(p), np.float32(m)) for v in u], (n, k, p, m)
    # equal weights besides, so that the draws next to their borders are decided by the second pass
    x = np.where(rng.random(3000) < 0.4, big, -big)
    heavy = np.nonzero(x > 0)[0]
    n = len(heavy)
    v = (rng.integers(0, n, 60) / n).astype(np.float32)
    v = np.concatenate([v, np.nextafter(v, np.float32(0)), np.nextafter(v, np.float32(1))])
    v = v[(v >= 0) & (v < 1)]
    got = _sample(mfs, _f32(np.tile(x, (len(v), 1))), v, np.full(len(v), big), np.zeros(len(v)), np.ones(len(v)), np.zeros(len(v)))
    assert got.tolist() == [int(heavy[int(float(a) * 2 ** 60) * n >> 60]) for a in v]


@pytest.mark.parametrize("hq,hkv,hd", [(4, 2, 64), (4, 2, 128), (3, 1, 128), (2, 2, 64)])
@pytest.mark.parametrize("window", [0, 3, 40, 200])
def test_prompt_attention_many_bad_values(mfs, window, hq, hkv, hd):
    """NaN in every value from a token on, and NaN, infinities of either sign and both in neighbouring columns of some tokens:
    each element is what the values that its row sees make it."""
    torch = _torch()
    rng = np.random.default_rng(38)
    n, inf, nan = 420, float("inf"), float("nan")
    q, k, v = (_normal(rng, n, h, hd, dtype="bf16") for h in (hq, hkv, hkv))
    cu, clean, got = _i32([0, n]), torch.empty_like(q), torch.empty_like(q)
    mfs.mfs_prompt_attention(q, k, v, cu, clean, window=window)
    for bad in ([(130, 4, nan), (131, 5, inf), (140, 4, inf), (150, 5, -inf), (131, 20, -inf), (290, 20, -inf), (291, 21, nan), (292, 20, nan),
                 (3, 9, inf), (3, 8, -inf), (260, 9, inf), (255, hd - 1, inf), (256, hd - 2, nan), (256, hd - 1, nan), (257, hd - 1, -inf)],
                [(t, slice(None), nan) for t in range(200, n)], [(t, slice(None), nan) for t in range(37)], [(t, slice(None), inf) for t in range(260, 275)]):
        vv = v.clone()
        for t, c, x in bad:
            vv[t, hkv - 1, c] = x
        mfs.mfs_prompt_attention(q, k, vv, cu, got, window=window)
        add = torch.zeros(n, hd)  # what the bad values that a row sees add to it
        for t, c, x in bad:
            add[t:min(n, t + window) if window else n, c] += x
        want, g = clean.cpu().float(), hq // hkv
        want[:, -g:] += add[:, None]
        assert torch.equal(torch.nan_to_num(got.cpu().float(), nan=7e7), torch.nan_to_num(want, nan=7e7))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("hq,hkv,hd", [(4, 2, 64), (8, 1, 128), (2, 2, 128)])
def test_paged_attention_bad_keys_and_values_stay_with_their_rows(mfs, hq, hkv, hd, bad, dtype):
    """A NaN key, or one whose score is +infinity, makes its sequence's heads of that kv head NaN; a NaN or infinite value
    reaches its own column of them; every other output is what it is without them."""
    torch = _torch()
    rng = np.random.default_rng(55)
    page, lens = 16, [5, 700, 33, 3001, 64]
    table, pages = _table(rng, lens, page)
    kc, vc = _pool(rng, pages, hkv, page, hd, dtype)
    q, g = _normal(rng, 5, hq, hd, dtype=dtype), hq // hkv
    q[:, :, 5] = q[:, :, 5].abs() + 0.125
    cache, kv = mfs.PagedKV(kc, vc, torch.from_numpy(table).cuda()), _i32(lens)
    clean, got = torch.empty_like(q), torch.empty_like(q)
    mfs.mfs_paged_attention(cache, q, kv, clean)
    for s, p in ((1, 0), (1, 333), (2, 32), (3, 1700), (4, 63)):
        at = (int(table[s, p // page]), hkv - 1, p % page, 5)
        for pool, columns in ((kc, slice(None)), (vc, slice(5, 6))):
            was = pool[at].item()
            pool[at] = bad
            mfs.mfs_paged_attention(cache, q, kv, got)
            pool[at] = was
            hit = torch.zeros_like(got, dtype=torch.bool)
            hit[s, hq - g:, columns] = True
            assert torch.equal(got[~hit], clean[~hit])
            assert torch.isnan(got[hit]).all() if pool is kc or bad != bad else (got[hit] == bad).all()
