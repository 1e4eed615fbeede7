"""Rows of the 8-bit cache whose exponent is 0 are zeros, whatever their codes: NaN among those changes nothing."""
import numpy as np
import pytest

from tests import test_gpu_shared as H
from tests.test_gpu_quant import _dt, _i32, _normal, _quant_pool, _torch, mfs  # noqa: F401

pytestmark = pytest.mark.gpu


def _cleared(mfs, rng, cache, rows):  # noqa: F811
    """Exponents of 0 in `rows` ((which, page, row), of all heads); -> a twin whose codes are zeros there, while the cache's
    are anything, every third NaN."""
    torch = _torch()
    twin = mfs.QuantKV(cache.k.clone(), cache.v.clone(), cache.k_exp.clone(), cache.v_exp.clone(), cache.table)
    for which, page, row in rows:
        codes = rng.integers(0, 256, cache.k.shape[1::2]).astype(np.uint8)
        codes[:, ::3] = np.where(codes[:, ::3] & 1, 0x7f, 0xff)
        getattr(cache, which)[page, :, row] = torch.from_numpy(codes).cuda()
        getattr(twin, which)[page, :, row] = 0
        getattr(cache, which + "_exp")[page, :, row] = 0
        getattr(twin, which + "_exp")[page, :, row] = 0
    return twin


#: keys alone, values alone, both, the last row that is seen, a whole page, the next tile's first row
ROWS = [("k", 0, 3), ("v", 0, 5), ("k", 1, 7), ("v", 1, 7), ("k", 2, 2), ("v", 2, 2), ("v", 2, 0)] + [(w, 3, r) for w in "kv" for r in range(16)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd", [64, 128])
def test_read_back(mfs, dtype, hd):  # noqa: F811
    torch = _torch()
    rng = np.random.default_rng(hd)
    cache = _quant_pool(mfs, rng, 4, 3, 16, hd, [[0, 1, 3, 2]])
    twin = _cleared(mfs, rng, cache, ROWS)
    got, want = ([torch.full((64, 3, hd), 7.0, dtype=_dt(dtype), device="cuda") for _ in "kv"] for _ in range(2))
    mfs.mfs_kv_read(cache, _i32([0, 64]), _i32([64]), *got)
    mfs.mfs_kv_read(twin, _i32([0, 64]), _i32([64]), *want)
    for a, b in zip(got, want):
        assert torch.equal(a, b) and not torch.isnan(a).any()
    assert not got[0][32:48].any() and not got[1][32:48].any()  # the page of zeros


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (12, 1)])
def test_attention(mfs, dtype, hd, hq, hkv):  # noqa: F811
    torch = _torch()
    rng = np.random.default_rng(hd + hq)
    cache = _quant_pool(mfs, rng, 4, hkv, 16, hd, [[0, 1, 3, 2]] * 5)
    twin = _cleared(mfs, rng, cache, ROWS)
    q = _normal(rng, 5, hq, hd, dtype=dtype)
    got, want = torch.empty_like(q), torch.empty_like(q)
    lens = _i32([4, 24, 33, 51, 64])
    for window in (0, 20):
        mfs.mfs_paged_attention(cache, q, lens, got, window=window)
        mfs.mfs_paged_attention(twin, q, lens, want, window=window)
        assert torch.equal(got, want) and torch.isfinite(got).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd", [64, 128])
def test_shared_prefix(mfs, dtype, hd):  # noqa: F811
    """In the prefix (its first tile, its second, its last row) and in a sequence's own part."""
    torch = _torch()
    lens, prefix = [200, 180, 160, 300], 152
    cache, table, q, groups, out = H._case(mfs, 18, [4], [prefix], lens, 4, 2, hd, 16, dtype, True)
    at = [("k", 5), ("v", 9), ("k", 100), ("v", 100), ("k", 128), ("v", 129), ("v", 151)]
    rows = [(w, int(table[0, p // 16]), p % 16) for w, p in at] + [(w, int(table[3, 170 // 16]), 170 % 16) for w in "kv"]
    twin = _cleared(mfs, np.random.default_rng(1), cache, rows)
    got, want = torch.empty_like(out), torch.empty_like(out)
    mfs.mfs_shared_attention(cache, q, _i32(lens), groups, _i32([prefix]), got)
    mfs.mfs_shared_attention(twin, q, _i32(lens), groups, _i32([prefix]), want)
    assert torch.equal(got, want) and torch.isfinite(got).all() and not torch.equal(got, out)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_queries_that_are_not_finite(mfs, dtype, bad):  # noqa: F811
    """Such a query's products with keys of zeros are NaN, as with any others; the heads beside it are right."""
    torch = _torch()
    rng = np.random.default_rng(3)
    for hq in (4, 12):
        cache = _quant_pool(mfs, rng, 3, 1, 16, 64, [[0, 1, 2]] * 2)
        cache.k_exp[:] = 0
        q = _normal(rng, 2, hq, 64, dtype=dtype)
        want, got = torch.empty_like(q), torch.empty_like(q)
        mfs.mfs_paged_attention(cache, q, _i32([40, 3]), want)
        q[1, 2, 9] = bad
        mfs.mfs_paged_attention(cache, q, _i32([40, 3]), got)
        keep = torch.ones(2, hq, dtype=torch.bool)
        keep[1, 2] = False
        assert torch.isnan(got[1, 2]).all() and torch.isfinite(want).all() and torch.equal(got[keep], want[keep])
