"""Behind a shared prefix an 8-bit cache's outputs are as precise as the one-token attention's over the same codes."""
import numpy as np
import pytest

from tests import _quant as Q
from tests import _serving as S
from tests import test_gpu_shared as H
from tests.test_gpu_shared import _np, mfs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("prefix", [2, 3, 5, 30, 129, 1000])
def test_weights_keep_their_bits(mfs, hd, prefix):  # noqa: F811
    """The prefix's weights are two bf16 parts: what the first leaves, at most 2^-8 of it, is rounded by 2^-8, so 2^-16 in all.
    What follows the prefix has fp16 weights (2^-11).  So the one-token attention's tolerance holds: 2^-11 of the weighted sizes, and the
    output's own rounding."""
    lens = [prefix + x for x in (0, 0, 0, 1, 2, 40)]
    cache, table, q, groups, out = H._case(mfs, 40 + prefix, [6], [prefix], lens, 8, 2, hd, 16, "bf16", True)
    got, qs = _np(out), _np(q)
    for s, n in enumerate(lens):
        k, v, vc, vx = H._rows(cache, table, s, 0, n, True)
        for h in range(8):
            ref, weighted, size = S.attend(qs[s, h], k[:, h // 4], v[:, h // 4], hd ** -0.5)
            lost = Q.lost_weights(qs[s, h], k[:, h // 4], vc[:, h // 4], vx[:, h // 4], hd ** -0.5)
            tol = Q.attention_tolerance(ref, weighted, size, n, hd, True, lost)
            far = np.abs(got[s, h] - ref)
            assert (far <= tol).all(), (s, h, (far / tol).max())
