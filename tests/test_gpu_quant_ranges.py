"""One-token attention over the 8-bit cache at the ends of what its rows and calls can hold: keys and queries whose products are
of ordinary size although they are not, queries of zeros under small scales, values next to the smallest normal number."""
import numpy as np
import pytest

from tests import _quant as Q
from tests import _serving as S
from tests.test_gpu_quant import _check_attention, _codes, _i32, _normal, _np, _quant_pool, _torch, mfs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq", [2, 12])
@pytest.mark.parametrize("key,query,scale", [(108, 0, 2.0 ** -108), (116, -116, 1.0), (116, -60, 2.0 ** -56), (-100, 100, 1.0), (-112, 118, 0.01),
                                             (60, 60, 1e-36)])
def test_keys_of_any_size(mfs, dtype, hq, key, query, scale):  # noqa: F811
    """Keys about 2^key, queries about 2^query: scores within fp32, and within +-100 times the scale."""
    torch = _torch()
    rng = np.random.default_rng(31)
    cache = _quant_pool(mfs, rng, 5, 1, 16, 64, [[4, 2, 0, 1, 3]] * 3)
    cache.k_exp.copy_(torch.from_numpy(rng.integers(127 - 10 + key, 127 - 6 + key, tuple(cache.k_exp.shape)).astype(np.uint8)))
    q = _normal(rng, 3, hq, 64, dtype=dtype, scale=2.0 ** query)
    out = torch.empty_like(q)
    lens = [77, 33, 1]
    mfs.mfs_paged_attention(cache, q, _i32(lens), out, scale=scale)
    for s, n in enumerate(lens):
        _check_attention(_np(out[s]), _np(q[s]), _codes(cache, s, 0, n), float(np.float32(scale)), dtype == "bf16", hq)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1.0, 1e-9, 1e-20, 1e-38])
def test_a_query_of_zeros_under_any_scale(mfs, dtype, scale):  # noqa: F811
    """Heads of zeros among others: the mean of the values, also where the last tile is not full."""
    torch = _torch()
    rng = np.random.default_rng(32)
    cache = _quant_pool(mfs, rng, 5, 2, 16, 64, [[4, 2, 0, 1, 3]] * 4)
    q = _normal(rng, 4, 6, 64, dtype=dtype)
    q[:, 1::2] = 0
    out = torch.empty_like(q)
    lens = [77, 32, 31, 1]
    mfs.mfs_paged_attention(cache, q, _i32(lens), out, scale=scale)
    for s, n in enumerate(lens):
        _check_attention(_np(out[s]), _np(q[s]), _codes(cache, s, 0, n), float(np.float32(scale)), dtype == "bf16", 3)


def test_orthogonal_huge_keys(mfs):  # noqa: F811
    """A large element of the query against codes of zero in huge keys: scores of 0, not 0 times infinity."""
    torch = _torch()
    rng = np.random.default_rng(33)
    for dtype in ("bf16", "f32"):
        cache = _quant_pool(mfs, rng, 3, 1, 16, 64, [[0, 1, 2]])
        cache.k[..., 5] = 0
        cache.k_exp[:] = 240
        q = torch.zeros(1, 1, 64, device="cuda")
        q[0, 0, 5] = 1e38
        q = q.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
        out = torch.empty_like(q)
        mfs.mfs_paged_attention(cache, q, _i32([45]), out)
        _check_attention(_np(out[0]), _np(q[0]), _codes(cache, 0, 0, 45), 0.125, dtype == "bf16", 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [2, 3, 40])
def test_values_next_to_the_smallest(mfs, dtype, n):  # noqa: F811
    """Values about 2^-118 (exponents 1 to 4) keep their precision.  The tolerance is attention_tolerance()'s without its floor of
    1e-30, which is far above them; outputs below 2^-126 are rounded to steps of 2^-149 (bf16: 2^-133)."""
    torch = _torch()
    rng = np.random.default_rng(34 + n)
    cache = _quant_pool(mfs, rng, 6, 1, 8, 64, [[4, 2, 0, 1, 3]] * 8)
    cache.v_exp.copy_(torch.from_numpy(rng.integers(1, 5, tuple(cache.v_exp.shape)).astype(np.uint8)))
    cache.k_exp[:] = 115
    q = _normal(rng, 8, 4, 64, dtype=dtype, scale=0.1)
    out = torch.empty_like(q)
    mfs.mfs_paged_attention(cache, q, _i32([n] * 8), out)
    got, qs = _np(out), _np(q)
    for s in range(8):
        kc, kx, vc, vx = _codes(cache, s, 0, n)
        k, v = Q.values(kc, kx)[:, 0], Q.values(vc, vx)[:, 0]
        for h in range(4):
            ref, weighted, size = S.attend(qs[s, h], k, v, 0.125)
            lost = Q.lost_weights(qs[s, h], k, vc[:, 0], vx[:, 0], 0.125)
            tol = Q.attention_tolerance(ref, weighted, size, n, 64, dtype == "bf16", lost) - 1e-30 + (2.0 ** -133 if dtype == "bf16" else 2.0 ** -148)
            assert (np.abs(got[s, h] - ref) <= tol).all(), (s, h, (np.abs(got[s, h] - ref) / tol).max())
