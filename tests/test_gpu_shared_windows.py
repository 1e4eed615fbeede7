"""Windows and shared prefixes: a window bounds what sharing can save, whatever room the table has."""
import numpy as np
import pytest

from tests import test_gpu_shared as H
from tests.test_gpu_shared import KINDS, _i32, _torch, mfs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,quant", KINDS)
def test_a_short_window_is_not_shared(mfs, dtype, quant):  # noqa: F811
    """A table with room for much sharing under a window that leaves little: the bits are mfs_paged_attention's."""
    torch = _torch()
    lens = [250, 260, 290, 400]
    cache, table, q, groups, out = H._case(mfs, 50, [4], [250], lens, 4, 2, 64, 16, dtype, quant, window=300)
    one = torch.empty_like(out)
    mfs.mfs_paged_attention(cache, q, _i32(lens), one, window=300)
    assert torch.equal(out, one)


@pytest.mark.parametrize("dtype,quant", KINDS)
def test_a_long_window_is_shared(mfs, dtype, quant):  # noqa: F811
    """40 sequences, enough for sharing under a window of 2800: it begins before the prefix of 2700, at its first position, inside it and behind it."""
    lens = [2699, 2700, 2701, 2799, 2800, 2801, 2802, 2900, 5499, 5500, 5501, 5600] + [2700 + 2 * i for i in range(28)]
    _, _, _, _, out = H._case(mfs, 51, [40], [2700], lens, 16, 8, 128, 64, dtype, quant, window=2800, heads=[0, 9, 15], seqs=list(range(13)) + [39])
    assert np.isfinite(out.float().cpu().numpy()).all()


@pytest.mark.parametrize("quant", [False, True])
def test_a_view_of_a_wide_table(mfs, quant):  # noqa: F811
    """A cache of a view as wide as the longest sequence needs: the choice goes by the view, whatever the table's own width."""
    torch = _torch()
    lens = [250, 260, 290, 400]
    cache, table, q, groups, out = H._case(mfs, 52, [4], [250], lens, 4, 2, 64, 16, "bf16", quant)
    view = cache.table[:, :25]
    narrow = mfs.QuantKV(cache.k, cache.v, cache.k_exp, cache.v_exp, view) if quant else mfs.PagedKV(cache.k, cache.v, view)
    got, one = torch.empty_like(out), torch.empty_like(out)
    mfs.mfs_shared_attention(narrow, q, _i32(lens), groups, _i32([250]), got)
    mfs.mfs_paged_attention(cache, q, _i32(lens), one)
    assert torch.equal(got, one)
