"""The 8-bit cache on the GPU (mfs_kv_append into it, mfs_kv_read, mfs_paged_attention over it) and partial and scaled
rotations, against their 64-bit definitions."""
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


def _bytes(t):
    return t.view(_torch().uint8).cpu().numpy()


def _quant_pool(mfs, rng, pages, hkv, page, hd, table, spread=12, strided=False):
    """A cache of random finite codes and exponents over `spread` binades; strided: rows with room between them, heads innermost."""
    torch = _torch()
    if strided:
        k, v = (torch.empty(pages, page, hkv, hd + 16, dtype=torch.uint8, device="cuda").permute(0, 2, 1, 3)[..., :hd] for _ in "kv")
        kx, vx = (torch.empty(pages, page, hkv + 3, dtype=torch.uint8, device="cuda").permute(0, 2, 1)[:, :hkv] for _ in "kv")
    else:
        k, v = (torch.empty(pages, hkv, page, hd, dtype=torch.uint8, device="cuda") for _ in "kv")
        kx, vx = (torch.empty(pages, hkv, page, dtype=torch.uint8, device="cuda") for _ in "kv")
    for t in (k, v):
        c = rng.integers(0, 256, t.shape).astype(np.uint8)
        c[(c & 127) == 127] -= 1
        t.copy_(torch.from_numpy(c))
    for t in (kx, vx):
        t.copy_(torch.from_numpy(rng.integers(127 - 8 - spread // 2, 127 - 8 + spread - spread // 2, t.shape).astype(np.uint8)))
    return mfs.QuantKV(k, v, kx, vx, _i32(table))


def _codes(cache, s, lo, hi):
    """Positions lo .. hi - 1 of sequence s: codes and exponents of the keys [hi - lo, heads, hd], then of the values."""
    table, page = cache.table.cpu().numpy(), cache.k.shape[2]
    g, r = table[s][np.arange(lo, hi) // page], np.arange(lo, hi) % page
    return [_bytes(x)[g, :, r] for x in (cache.k, cache.k_exp, cache.v, cache.v_exp)]


def _history(cache, s, lo, hi):
    """Positions lo .. hi - 1 of sequence s as the codes stand for them: keys and values [hi - lo, heads, hd]."""
    kc, kx, vc, vx = _codes(cache, s, lo, hi)
    return Q.values(kc, kx), Q.values(vc, vx)


def _check_attention(got, q, codes, scale, bf16, g):
    """Heads got, q [hq, hd] against codes (_codes())."""
    kc, kx, vc, vx = codes
    k, v = Q.values(kc, kx), Q.values(vc, vx)
    for h in range(len(q)):
        ref, weighted, size = S.attend(q[h], k[:, h // g], v[:, h // g], scale)
        lost = Q.lost_weights(q[h], k[:, h // g], vc[:, h // g], vx[:, h // g], scale)
        tol = Q.attention_tolerance(ref, weighted, size, len(k), q.shape[-1], bf16, lost)
        far = np.abs(got[h] - ref)
        assert (far <= tol).all(), (h, (far / tol).max(), far.max())


# -------------------------------------------------------------------- append

ROPES = [dict(layout="interleaved"), dict(layout="half"), dict(layout=None), dict(layout="half", dims=32), dict(layout="interleaved", dims=48),
         dict(layout="half", dims=64, factor=8.0), dict(layout="interleaved", factor=4.0, original=4096.0, low=1.0, high=32.0, magnitude=1.2),
         dict(layout="half", dims=16, theta=500.0, factor=2.0, original=8192.0, low=0.0, high=0.5, magnitude=0.5)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rope", ROPES, ids=str)
@pytest.mark.parametrize("hd,hq,hkv,page", [(64, 5, 5, 1), (128, 6, 2, 16), (128, 1, 1, 48)])
def test_append_into_8_bits(mfs, dtype, rope, hd, hq, hkv, page):
    """Sequences of 0, 1, 3 and 37 new tokens at far and near positions, strided parts of one projection's output; all
    other rows of the cache stay as they were."""
    torch = _torch()
    rng = np.random.default_rng(hd + page)
    new, past = [3, 0, 37, 1], [0, 9, 4000, 131071]
    n, total = sum(new), [a + b for a, b in zip(new, past)]
    width = max(-(-t // page) for t in total)
    table, at = np.full((4, width), -5), 0
    for i, (a, b) in enumerate(zip(past, total)):
        for j in range(a // page, -(-b // page)):
            table[i, j] = at
            at += 1
    cache = _quant_pool(mfs, rng, at, hkv, page, hd, table, strided=page == 16)
    before = [_bytes(t).copy() for t in (cache.k, cache.v, cache.k_exp, cache.v_exp)]
    qkv = _normal(rng, n + 2, hq + 2 * hkv, hd, dtype=dtype)  # two tokens behind the last sequence
    qkv *= torch.exp2(torch.randint(-20, 20, (n + 2, hq + 2 * hkv, 1), device="cuda").float()).to(qkv.dtype)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    k[1, 0] = 0  # a row of zeros
    v[2, 0, 1:] = 0
    q_out, k_out = torch.full((n + 2, hq, hd), 7.0, dtype=q.dtype, device="cuda"), torch.full((n + 2, hkv, hd), 7.0, dtype=q.dtype, device="cuda")
    mfs.mfs_kv_append(cache, k, v, _i32(np.cumsum([0] + new).tolist()), _i32(total), q=q, q_out=q_out, k_out=k_out, rope=mfs.Rope(**rope))
    after = [_bytes(t) for t in (cache.k, cache.v, cache.k_exp, cache.v_exp)]
    rounding = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    touched = np.zeros(before[2].shape, bool)
    t = 0
    for s in range(4):
        for p in range(past[s], total[s]):
            for x, out, heads in ((q, q_out, hq), (k, k_out, hkv)):
                want, slack = Q.rotate(_np(x[t]), p, **rope), Q.rotation_slack(_np(x[t]), **rope)
                assert (np.abs(_np(out[t]) - want) <= slack * (1 + rounding) + rounding * np.abs(want)).all()
            g, r = table[s, p // page], p % page
            touched[g, :, r] = True
            for h in range(hkv):
                Q.check_row(after[0][g, h, r], after[2][g, h, r], Q.rotate(_np(k[t, h]), p, **rope), Q.rotation_slack(_np(k[t, h]), **rope))
                x = _np(v[t, h])
                b = Q.exponent(x)
                assert after[3][g, h, r] == b and (Q.values(after[1][g, h, r], b) == Q.nearest(x, b)).all()
            t += 1
    assert (q_out[n:] == 7).all() and (k_out[n:] == 7).all()
    for a, b in zip(before, after):
        assert (a[~touched] == b[~touched]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd", [64, 128])
def test_rows_at_the_borders(mfs, dtype, hd):
    """Largest values at and next to a border of the exponent, ties, tiny, subnormal, huge and not finite ones, in keys
    (not rotated) and values."""
    torch = _torch()
    t = _dt(dtype)
    tops = [448.0, 450.0, 447.0, 1.0, 0.875, 0.87890625, 1.75, 2.0 ** -126 * 448, 2.0 ** -127, 2.0 ** -133, 3.3e38, 2.0 ** 127, -448.0, -3.5, 2.0 ** -140]
    ladder = np.array([1.0625, 1.1875, 1.3125, -1.0625, 17.0, 18.0, 19.0, 0.001953125, 0.0009765625, 0.00146484375, 0.0029296875, 0.0, -0.0])
    rows = []
    for x in tops:
        r = np.zeros(hd)
        r[3] = x
        r[8:8 + len(ladder)] = ladder * abs(x) / 448.0
        rows.append(r)
    n = len(rows)
    x = torch.from_numpy(np.array(rows)).to(t)[:, None].cuda().contiguous()
    page = 5
    cache = mfs.QuantKV(*(torch.zeros(n, 1, page, hd, dtype=torch.uint8, device="cuda") for _ in "kv"),
                        *(torch.zeros(n, 1, page, dtype=torch.uint8, device="cuda") for _ in "kv"), _i32([list(range(n))]))
    mfs.mfs_kv_append(cache, x, -x, _i32([0, n]), _i32([n]), rope=None)
    back, back_v = torch.empty(n, 1, hd, device="cuda"), torch.empty(n, 1, hd, device="cuda")
    mfs.mfs_kv_read(cache, _i32([0, n]), _i32([n]), back, back_v)
    k, v = _history(cache, 0, 0, n)
    for i in range(n):
        want = _np(x[i, 0])
        b = Q.exponent(want)
        assert _bytes(cache.k_exp)[i // page, 0, i % page] == b
        assert (k[i, 0] == Q.nearest(want, b)).all() and (v[i, 0] == -k[i, 0]).all()
        assert (_np(back[i, 0]) == k[i, 0].astype(np.float32)).all() and (_np(back_v[i, 0]) == v[i, 0].astype(np.float32)).all()
    # (3.3e38 is 1.94 2^127, nearest to 2 x 2^127 among the codes: past fp32, which reads it as infinite)
    want = torch.cat([back, back_v], 1)
    want[n // 2] = float("nan")
    for bad in (np.nan, np.inf, -np.inf):
        x[n // 2, 0, hd - 1] = bad
        mfs.mfs_kv_append(cache, x, -x, _i32([0, n]), _i32([n]), rope=None)
        mfs.mfs_kv_read(cache, _i32([0, n]), _i32([n]), back, back_v)
        assert np.array_equal(torch.cat([back, back_v], 1).cpu().numpy(), want.cpu().numpy(), equal_nan=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rope", ROPES[3:], ids=str)
def test_rotations_of_the_plain_cache(mfs, dtype, rope):
    torch = _torch()
    rng = np.random.default_rng(11)
    hd, hq, hkv, page, n, past = 128, 4, 2, 16, 21, 70000
    width = -(-(past + n) // page)
    table = np.full((1, width), -1)
    table[0, past // page:] = np.arange(width - past // page)
    pool = lambda: _normal(rng, width - past // page, hkv, page, hd, dtype=dtype)
    cache = mfs.PagedKV(pool(), pool(), _i32(table))
    q, k, v = (_normal(rng, n, h, hd, dtype=dtype) for h in (hq, hkv, hkv))
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    mfs.mfs_kv_append(cache, k, v, _i32([0, n]), _i32([past + n]), q=q, q_out=q_out, k_out=k_out, rope=mfs.Rope(**rope))
    back = torch.empty_like(k), torch.empty_like(v)
    mfs.mfs_kv_read(cache, _i32([0, n]), _i32([past + n]), *back)
    assert torch.equal(back[0], k_out) and torch.equal(back[1], v)
    rounding = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for t in range(n):
        for x, out in ((q, q_out), (k, k_out)):
            want, slack = Q.rotate(_np(x[t]), past + t, **rope), Q.rotation_slack(_np(x[t]), **rope)
            assert (np.abs(_np(out[t]) - want) <= slack * (1 + rounding) + rounding * np.abs(want)).all()


def test_a_whole_rotation_is_the_named_one(mfs):
    """Rope() of all of the head, unscaled, gives the bits of the named layout, in both caches."""
    torch = _torch()
    rng = np.random.default_rng(12)
    for layout in ("interleaved", "half"):
        outs = []
        for rope in (layout, mfs.Rope(layout)):
            k = _normal(np.random.default_rng(1), 9, 2, 64)
            cache = mfs.PagedKV(torch.zeros(2, 2, 16, 64, device="cuda"), torch.zeros(2, 2, 16, 64, device="cuda"), _i32([[1, 0]]))
            mfs.mfs_kv_append(cache, k, k, _i32([0, 9]), _i32([20]), rope=rope, k_out=k)
            quant = _quant_pool(mfs, np.random.default_rng(2), 2, 2, 16, 64, [[1, 0]])
            mfs.mfs_kv_append(quant, k, k, _i32([0, 9]), _i32([20]), rope=rope)
            outs.append([cache.k, k, quant.k, quant.k_exp])
        for a, b in zip(*outs):
            assert torch.equal(a, b)


def test_append_skips_what_has_no_page(mfs):
    """Pages outside the pool, positions past the table and negative ones: nothing is written, the queries are rotated."""
    torch = _torch()
    rng = np.random.default_rng(13)
    cache = _quant_pool(mfs, rng, 3, 2, 4, 64, [[0, 3], [-1, 2]])
    before = [_bytes(t).copy() for t in (cache.k, cache.v, cache.k_exp, cache.v_exp)]
    k = _normal(rng, 12, 2, 64)
    k_out = torch.zeros_like(k)
    # sequence 0: positions 3 .. 8 (3 in page 0, 4 - 7 in page 3 of 3, 8 past the table); sequence 1: -2 .. 3 (a page of -1)
    mfs.mfs_kv_append(cache, k, k, _i32([0, 6, 12]), _i32([9, 4]), k_out=k_out, rope=None)
    assert torch.equal(k_out, k)
    after = [_bytes(t) for t in (cache.k, cache.v, cache.k_exp, cache.v_exp)]
    for a, b in zip(before, after):
        a[0, :, 3] = b[0, :, 3]
        assert (a == b).all()
    out = torch.zeros(12, 2, 64, device="cuda"), torch.zeros(12, 2, 64, device="cuda")
    mfs.mfs_kv_read(cache, _i32([0, 6, 12]), _i32([9, 4]), *out)
    for o in out:
        assert torch.isfinite(o[0]).all() and torch.isnan(o[1:]).all()


# ---------------------------------------------------------------------- read

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd,hkv,page", [(64, 1, 1), (64, 5, 16), (128, 2, 48), (128, 8, 128)])
@pytest.mark.parametrize("quant", [True, False])
def test_read_back(mfs, dtype, hd, hkv, page, quant):
    torch = _torch()
    rng = np.random.default_rng(hd + hkv)
    lens, new = [0, 1, 300, 17, 129], [0, 1, 300, 5, 100]
    need = [-(-n // page) for n in lens]
    order = rng.permutation(sum(need))
    table, at = np.full((5, max(need)), -1), 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    if quant:
        cache = _quant_pool(mfs, rng, sum(need), hkv, page, hd, table, spread=60, strided=page == 16)
        cache.k_exp[:, :, 0] = 0
    else:
        cache = mfs.PagedKV(_normal(rng, sum(need), hkv, page, hd, dtype=dtype), _normal(rng, sum(need), hkv, page, hd, dtype=dtype), _i32(table))
    n = sum(new)
    wide = torch.full((n + 3, 2 * hkv, hd), 7.0, dtype=_dt(dtype), device="cuda")
    k, v = wide[:, :hkv], wide[:, hkv:]
    mfs.mfs_kv_read(cache, _i32(np.cumsum([0] + new).tolist()), _i32(lens), k, v)
    assert (wide[n:] == 7).all()
    t = 0
    for s in range(5):
        if quant:
            want = _history(cache, s, lens[s] - new[s], lens[s])
        else:
            want = tuple(S.kv_rows(_np(x), table[s], page, lens[s] - new[s], lens[s]) for x in (cache.k, cache.v))
        assert (_np(k[t:t + new[s]]) == want[0]).all() and (_np(v[t:t + new[s]]) == want[1]).all()
        t += new[s]


# ----------------------------------------------------------------- attention

def _attend_case(mfs, rng, lens, hq, hkv, hd, page, dtype, window=0, scale=None, spread=4, strided=False, q_scale=1.0, check=None):
    torch = _torch()
    need = [max(1, -(-n // page)) for n in lens]
    order = rng.permutation(sum(need))
    table, at = np.full((len(lens), max(need)), -1), 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    cache = _quant_pool(mfs, rng, sum(need), hkv, page, hd, table, spread=spread, strided=strided)
    qw = _normal(rng, len(lens), hq + 1, hd, dtype=dtype, scale=q_scale)
    q = qw[:, :hq]
    out = torch.full((len(lens), hq, hd), 7.0, dtype=_dt(dtype), device="cuda")
    kw = {} if scale is None else dict(scale=scale)
    mfs.mfs_paged_attention(cache, q, _i32(lens), out, window=window, **kw)
    again = torch.empty_like(out)
    mfs.mfs_paged_attention(cache, q, _i32(lens), again, window=window, **kw)
    assert torch.equal(out, again) or torch.isnan(out).any()
    got, qs = _np(out), _np(q)
    for s in (range(len(lens)) if check is None else check):
        lo = max(0, lens[s] - window) if window else 0
        _check_attention(got[s], qs[s], _codes(cache, s, lo, lens[s]), hd ** -0.5 if scale is None else scale, dtype == "bf16", hq // hkv)
    return cache, q, out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 5), (6, 2), (8, 1), (16, 1), (20, 1), (34, 2)])
@pytest.mark.parametrize("page", [1, 16, 48])
def test_attention_over_8_bits(mfs, dtype, hd, hq, hkv, page):
    """Lengths of zero and one, next to the tile's 32 and past it, with random codes (the weights spread over many binades)."""
    rng = np.random.default_rng(hq * 100 + page)
    _attend_case(mfs, rng, [0, 1, 2, 31, 32, 33, 63, 65, 200, 777], hq, hkv, hd, page, dtype, strided=page == 16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 31, 32, 100, 1 << 30])
def test_attention_over_8_bits_in_a_window(mfs, dtype, window):
    _attend_case(mfs, np.random.default_rng(window), [0, 1, 30, 32, 100, 101, 500], 4, 2, 64, 16, dtype, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_over_8_bits_long_and_ragged(mfs, dtype, hd):
    """Items that cross blocks, and shares with many items."""
    rng = np.random.default_rng(4)
    _attend_case(mfs, rng, [20011], 4, 1, hd, 64, dtype)
    _attend_case(mfs, rng, [3, 9000] + [1 + 7 * i for i in range(150)], 4, 2, hd, 16, dtype, check=[0, 1, 2, 50, 151])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_scale,scale", [(1e-30, 1e28), (1e15, 1e-16), (1e-3, 100.0), (300.0, 0.01), (1.0, 30.0)])
def test_attention_over_8_bits_extreme_scales(mfs, dtype, q_scale, scale):
    """Queries far from 1 (their power of two), and scores so large that one weight is all."""
    _attend_case(mfs, np.random.default_rng(8), [200, 33], 4, 2, 64, 16, dtype, q_scale=q_scale, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_of_any_size(mfs, dtype):
    """Values whose rows differ by 2^60: weights below 2^-60 still count, whatever order the rows come in."""
    for seed in range(3):
        _attend_case(mfs, np.random.default_rng(20 + seed), [300, 40], 3, 1, 64, 16, dtype, spread=60, q_scale=2.0 ** -26)


def test_rows_that_are_not_seen(mfs):
    """NaN codes and exponents of 255 in rows past the length, before the window and in pages of no one: no influence."""
    torch = _torch()
    for dtype in ("bf16", "f32"):
        rng = np.random.default_rng(5)
        cache, q, out = _attend_case(mfs, rng, [70, 45], 4, 2, 64, 16, dtype, window=33)
        table = cache.table.cpu().numpy()
        for s, n in ((0, 70), (1, 45)):
            for j in range(table.shape[1]):
                for r in range(16):
                    p = 16 * j + r
                    if table[s, j] >= 0 and not n - 33 <= p < n:
                        for t in (cache.k, cache.v):
                            t[int(table[s, j]), :, r] = 0x7f
                        for t in (cache.k_exp, cache.v_exp):
                            t[int(table[s, j]), :, r] = 255
        again = torch.empty_like(out)
        mfs.mfs_paged_attention(cache, q, _i32([70, 45]), again, window=33)
        assert torch.equal(out, again)


def test_nan_codes_that_are_seen(mfs):
    torch = _torch()
    for dtype in ("bf16", "f32"):
        rng = np.random.default_rng(6)
        for which in "kv":
            cache, q, out = _attend_case(mfs, rng, [70, 45], 4, 2, 64, 16, dtype)
            g = int(cache.table[0, 1])
            getattr(cache, which)[g, 1, 5, 7] = 0xff  # position 21 of sequence 0, kv head 1
            again = torch.empty_like(out)
            mfs.mfs_paged_attention(cache, q, _i32([70, 45]), again)
            want = out.clone()
            if which == "k":
                want[0, 2:] = float("nan")
            else:
                want[0, 2:, 7] = float("nan")
            assert torch.equal(torch.isnan(again), torch.isnan(want)) and torch.equal(again[~torch.isnan(want)], out[~torch.isnan(want)])


def test_queries_that_are_not_finite(mfs):
    """A NaN or an infinity in one head's query reaches that head alone."""
    torch = _torch()
    for dtype in ("bf16", "f32"):
        for bad in (float("nan"), float("inf")):
            rng = np.random.default_rng(7)
            cache, q, out = _attend_case(mfs, rng, [70, 45], 4, 2, 64, 16, dtype)
            q[1, 2, 3] = bad
            again = torch.empty_like(out)
            mfs.mfs_paged_attention(cache, q, _i32([70, 45]), again)
            keep = torch.ones(2, 4, dtype=torch.bool)
            keep[1, 2] = False
            assert torch.equal(again[keep], out[keep])
            if bad != bad:
                assert torch.isnan(again[1, 2]).all()


def test_zero_rows(mfs):
    """A query of zeros weighs all alike; rows of zeros (exponent 0, whatever the codes) are keys and values of 0."""
    torch = _torch()
    for dtype in ("bf16", "f32"):
        rng = np.random.default_rng(9)
        cache = _quant_pool(mfs, rng, 4, 1, 16, 64, [[0, 1, 2, 3]])
        cache.k_exp[1], cache.v_exp[1] = 0, 0
        q = _normal(rng, 1, 2, 64, dtype=dtype)
        q[0, 0] = 0
        out = torch.empty_like(q)
        for n in (16, 32, 50):
            mfs.mfs_paged_attention(cache, q, _i32([n]), out)
            _check_attention(_np(out[0]), _np(q[0]), _codes(cache, 0, 0, n), 0.125, dtype == "bf16", 2)
        cache.v_exp[:] = 0
        mfs.mfs_paged_attention(cache, q, _i32([64]), out)
        assert (out == 0).all()


def test_bad_pages_give_nan(mfs):
    torch = _torch()
    rng = np.random.default_rng(10)
    cache = _quant_pool(mfs, rng, 4, 1, 16, 64, [[0, 4, 1], [2, 3, -1]])
    q = _normal(rng, 2, 2, 64, dtype="bf16")
    out = torch.empty_like(q)
    for lens, bad in (([16, 32], [False, False]), ([17, 32], [True, False]), ([10, 33], [False, True]), ([10, 49], [False, True])):
        mfs.mfs_paged_attention(cache, q, _i32(lens), out)
        assert [bool(torch.isnan(out[s]).all()) for s in range(2)] == bad


def test_attention_over_8_bits_captured_and_on_streams(mfs):
    """A captured append, read and attention replayed on new data give the bits of the plain calls; two streams with a
    workspace each run side by side."""
    torch = _torch()
    rng = np.random.default_rng(14)
    n, hq, hkv, hd = 6, 8, 2, 128
    cache = _quant_pool(mfs, rng, n * 40, hkv, 16, hd, rng.permutation(n * 40).reshape(n, 40))
    lens, cu = _i32([5, 100, 633, 17, 2, 300]), _i32(list(range(n + 1)))
    q, k, v = (_normal(rng, n, h, hd, dtype="bf16") for h in (hq, hkv, hkv))
    qr, out, bk, bv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = mfs.mfs_paged_attention_workspace(cache, hq)

    def step():
        mfs.mfs_kv_append(cache, k, v, cu, lens, q=q, q_out=qr, rope=mfs.Rope("half", dims=64))
        mfs.mfs_paged_attention(cache, qr, lens, out, workspace=ws)
        mfs.mfs_kv_read(cache, cu, lens, bk, bv)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (q, k, v):
        t.copy_(_normal(rng, *t.shape, dtype="bf16"))
    step()
    want = [t.clone() for t in (qr, out, bk, bv)]
    for t in (qr, out, bk, bv):
        t.zero_()
    graph.replay()
    for a, b in zip(want, (qr, out, bk, bv)):
        assert torch.equal(a, b)
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.empty_like(q) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, o in zip(streams, outs):
            mfs.mfs_paged_attention(cache, qr, lens, o, stream=st.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[1]) and torch.equal(outs[1], want[1])
    mfs.mfs_paged_attention(cache, qr, lens, qr)  # out may be q
    assert torch.equal(qr, want[1])


def test_far_positions_of_a_large_pool(mfs):
    """Element offsets past 2^31: pages at the end of a pool of 2.4 GB."""
    torch = _torch()
    hkv, hd, page = 4, 128, 64
    pages = 2_400_000_000 // (hkv * hd * page)
    codes = torch.zeros(pages, hkv, page, hd, dtype=torch.uint8, device="cuda")
    exps = torch.zeros(pages, hkv, page, dtype=torch.uint8, device="cuda")
    cache = mfs.QuantKV(codes, codes, exps, exps, _i32([[pages - 1, pages - 3]]))
    rng = np.random.default_rng(15)
    k = _normal(rng, 100, hkv, hd)
    mfs.mfs_kv_append(cache, k, k, _i32([0, 100]), _i32([100]), rope=None)
    assert not bool(codes[:pages - 3].any())
    back = torch.empty_like(k), torch.empty_like(k)
    mfs.mfs_kv_read(cache, _i32([0, 100]), _i32([100]), *back)
    ks = _np(k)
    want = np.array([[Q.nearest(ks[t, h], Q.exponent(ks[t, h])) for h in range(hkv)] for t in range(100)])
    assert (_np(back[0]) == want).all() and (_np(back[1]) == want).all()
    q = _normal(rng, 1, hkv, hd)
    out = torch.empty_like(q)
    mfs.mfs_paged_attention(cache, q, _i32([100]), out)
    codes, exps = codes[pages - 3:], exps[pages - 3:]
    small = mfs.QuantKV(codes, codes, exps, exps, _i32([[2, 0]]))
    _check_attention(_np(out[0]), _np(q[0]), _codes(small, 0, 0, 100), hd ** -0.5, False, 1)
