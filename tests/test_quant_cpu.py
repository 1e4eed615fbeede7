"""The 8-bit cache's operators, the shared prefixes' and the rotations refuse bad calls on the host, before anything is launched
(no GPU needed: the pointers are never touched), and the binding refuses tensors that are not what it passes on."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from tests import _quant as Q
from tests.test_serving_cpu import BAD_CACHES, FAKE, _cache, mfs  # noqa: F401


def _quant(mfs, **kw):  # noqa: F811
    c = mfs.mfs_quant_kv(kv=_cache(mfs, dtype=2), k_exp=FAKE + 3, v_exp=FAKE + 5, exp_page_stride=32, exp_head_stride=16, exp_row_stride=1)
    for k, v in kw.items():
        setattr(c if hasattr(c, k) else c.kv, k, v)
    return c


def _rope(mfs, **kw):  # noqa: F811
    r = mfs.Rope("half", dims=32, factor=2.0, original=4096.0).c
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def _append(mfs, cache=None, quant=True, rope=None, dtype=1, **kw):  # noqa: F811
    a = dict(n=3, n_seqs=2, cu=FAKE, kv_len=FAKE, q=FAKE, qs=256, hq=4, q_out=FAKE, qos=256, k=FAKE, ks=128, k_out=FAKE, kos=128, v=FAKE, vs=128)
    a.update(kw)
    if quant:
        return mfs._lib.mfs_quant_append(cache if cache is not None else _quant(mfs), dtype, *a.values(), rope, None)
    return mfs._lib.mfs_kv_append_rope(cache if cache is not None else _cache(mfs), *a.values(), rope, None)


BAD_APPENDS = [dict(n=-1), dict(n_seqs=-1), dict(cu=None), dict(kv_len=None), dict(k=None), dict(v=None), dict(q_out=None), dict(q=None),
               dict(hq=0), dict(hq=65536), dict(qs=255), dict(qs=248), dict(ks=64), dict(vs=130), dict(kos=124), dict(k=FAKE + 2), dict(v=FAKE + 4)]
BAD_ROPES = [dict(layout=3), dict(layout=-1), dict(dims=8), dict(dims=24), dict(dims=80), dict(dims=-16), dict(theta=0.0), dict(theta=float("nan")),
             dict(theta=float("inf")), dict(factor=0.0), dict(factor=-2.0), dict(factor=float("nan")), dict(magnitude=0.0),
             dict(magnitude=float("inf")), dict(original=-1.0), dict(original=float("nan")), dict(low=5.0), dict(low=-1.0), dict(high=1.0),
             dict(high=float("inf")), dict(low=float("nan"))]


@pytest.mark.parametrize("quant", [True, False])
@pytest.mark.parametrize("bad", BAD_APPENDS)
def test_append_refusals(mfs, quant, bad):  # noqa: F811
    assert _append(mfs, quant=quant, **bad) == -1
    assert mfs.mfs_last_error(None).startswith("kv_append: ")


@pytest.mark.parametrize("quant", [True, False])
@pytest.mark.parametrize("bad", BAD_ROPES)
def test_rope_refusals(mfs, quant, bad):  # noqa: F811
    assert _append(mfs, quant=quant, rope=_rope(mfs, **bad)) == -1
    assert mfs.mfs_last_error(None).startswith("kv_append: ")


def test_ropes_that_are_fine(mfs):  # noqa: F811
    for r in (None, _rope(mfs), _rope(mfs, dims=0), _rope(mfs, dims=64), _rope(mfs, original=0.0, low=9.0, high=1.0), _rope(mfs, layout=0, theta=-1.0)):
        assert _append(mfs, rope=r, n=0) == 0 and _append(mfs, quant=False, rope=r, n_seqs=0) == 0


BAD_QUANT = [b for b in BAD_CACHES if "dtype" not in b] + [dict(dtype=1), dict(dtype=0), dict(k_exp=None), dict(v_exp=None), dict(exp_page_stride=-1),
                                                          dict(exp_head_stride=-1), dict(exp_row_stride=-1), dict(row_stride=72)]


@pytest.mark.parametrize("bad", BAD_QUANT)
def test_bad_caches_are_refused(mfs, bad):  # noqa: F811
    c = _quant(mfs, **bad)
    assert _append(mfs, c) == -1 and _read(mfs, c) == -1 and _attend(mfs, c) == -1 and _share(mfs, c) == -1
    assert mfs._lib.mfs_quant_attention_workspace(c, 1, 4) == 0 and mfs._lib.mfs_quant_shared_attention_workspace(c, 1, 4, 2) == 0


def test_plain_calls_refuse_the_codes(mfs):  # noqa: F811
    c = _cache(mfs, dtype=2)
    assert _append(mfs, c, quant=False) == -1 and _read(mfs, c, quant=False) == -1 and _share(mfs, c, quant=False) == -1
    assert mfs._lib.mfs_shared_attention_workspace(c, 4, 2) == 0


@pytest.mark.parametrize("dtype", [2, -1, 3])
def test_dtypes_are_refused(mfs, dtype):  # noqa: F811
    assert _append(mfs, dtype=dtype) == -1 and _read(mfs, dtype=dtype) == -1 and _attend(mfs, dtype=dtype) == -1 and _share(mfs, dtype=dtype) == -1
    assert mfs._lib.mfs_quant_attention_workspace(_quant(mfs), dtype, 4) == 0


def _read(mfs, cache=None, quant=True, dtype=1, **kw):  # noqa: F811
    a = dict(n=3, n_seqs=2, cu=FAKE, kv_len=FAKE, k=FAKE, ks=128, v=FAKE, vs=128)
    a.update(kw)
    if quant:
        return mfs._lib.mfs_quant_read(cache if cache is not None else _quant(mfs), dtype, *a.values(), None)
    return mfs._lib.mfs_kv_read(cache if cache is not None else _cache(mfs), *a.values(), None)


@pytest.mark.parametrize("quant", [True, False])
@pytest.mark.parametrize("bad", [dict(n=-1), dict(n_seqs=-1), dict(cu=None), dict(kv_len=None), dict(k=None), dict(v=None), dict(ks=120), dict(vs=130),
                                 dict(k=FAKE + 8), dict(v=FAKE + 2)])
def test_read_refusals(mfs, quant, bad):  # noqa: F811
    assert _read(mfs, quant=quant, **bad) == -1
    assert mfs.mfs_last_error(None).startswith("kv_read: ")


def _attend(mfs, cache=None, dtype=1, **kw):  # noqa: F811
    a = dict(n=2, kv_len=FAKE, q=FAKE, qs=256, hq=4, out=FAKE, os=256, scale=0.125, window=0, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return mfs._lib.mfs_quant_attention(cache if cache is not None else _quant(mfs), dtype, *a.values(), None)


BAD_ATTENTION = [dict(n=-1), dict(window=-1), dict(hq=3), dict(hq=0), dict(hq=65538), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                 dict(scale=float("inf")), dict(kv_len=None), dict(q=None), dict(out=None), dict(ws=None), dict(wsb=0), dict(ws=FAKE + 8),
                 dict(qs=252), dict(os=192), dict(q=FAKE + 2), dict(out=FAKE + 8)]


@pytest.mark.parametrize("bad", BAD_ATTENTION)
def test_attention_refusals(mfs, bad):  # noqa: F811
    assert _attend(mfs, **bad) == -1
    assert mfs.mfs_last_error(None).startswith("paged_attention: ")


def _share(mfs, cache=None, quant=True, dtype=1, **kw):  # noqa: F811
    a = dict(n=2, kv_len=FAKE, ng=1, groups=FAKE, prefix=FAKE, q=FAKE, qs=256, hq=4, out=FAKE, os=256, scale=0.125, window=0, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    if quant:
        return mfs._lib.mfs_quant_shared_attention(cache if cache is not None else _quant(mfs), dtype, *a.values(), None)
    return mfs._lib.mfs_shared_attention(cache if cache is not None else _cache(mfs), *a.values(), None)


@pytest.mark.parametrize("quant", [True, False])
@pytest.mark.parametrize("bad", BAD_ATTENTION + [dict(ng=-1), dict(groups=None), dict(prefix=None)])
def test_shared_attention_refusals(mfs, quant, bad):  # noqa: F811
    assert _share(mfs, quant=quant, **bad) == -1
    assert mfs.mfs_last_error(None).startswith("shared_attention: ")


def test_workspaces_are_stated_and_checked(mfs):  # noqa: F811
    lib, c, q = mfs._lib, _cache(mfs), _quant(mfs)
    for t in (0, 1):
        need = lib.mfs_quant_attention_workspace(q, t, 4)
        assert need >= 16 and _attend(mfs, dtype=t, wsb=need - 1) == -1
        need = lib.mfs_quant_shared_attention_workspace(q, t, 4, 2)
        assert need > 16 and _share(mfs, dtype=t, wsb=need - 1) == -1
        assert lib.mfs_quant_shared_attention_workspace(q, t, 4, 3) >= need
    need = lib.mfs_shared_attention_workspace(c, 4, 2)
    assert need > 16 and _share(mfs, quant=False, wsb=need - 1) == -1
    assert lib.mfs_shared_attention_workspace(c, 0, 2) == 0 and lib.mfs_shared_attention_workspace(c, 4, -1) == 0


def test_nothing_to_do_is_ok(mfs):  # noqa: F811
    for quant in (True, False):
        assert _append(mfs, quant=quant, n=0) == 0 and _read(mfs, quant=quant, n=0) == 0 and _read(mfs, quant=quant, n_seqs=0) == 0
        assert _share(mfs, quant=quant, n=0) == 0
    assert _attend(mfs, n=0) == 0


def test_layouts_match_the_header(mfs, tmp_path):  # noqa: F811
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "probe.c"
    src.write_text('#include <stdio.h>\n#include "mfs.h"\nint main(void){printf("%zu %zu %zu %zu %zu %zu %zu\\n", sizeof(mfs_quant_kv),'
                   ' offsetof(mfs_quant_kv, k_exp), offsetof(mfs_quant_kv, exp_row_stride), sizeof(mfs_rope), offsetof(mfs_rope, dims),'
                   ' offsetof(mfs_rope, theta), offsetof(mfs_rope, magnitude)); return 0;}\n')
    exe = tmp_path / "probe"
    subprocess.check_call(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    c, r = mfs.mfs_quant_kv, mfs.mfs_rope
    assert got == [ctypes.sizeof(c), c.k_exp.offset, c.exp_row_stride.offset, ctypes.sizeof(r), r.dims.offset, r.theta.offset, r.magnitude.offset]


def test_binding_refuses(mfs):  # noqa: F811
    import torch
    codes, exps, table = torch.zeros(4, 2, 16, 64, dtype=torch.uint8), torch.zeros(4, 2, 16, dtype=torch.uint8), torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(mfs.MfsError, match="CUDA"):
        mfs.QuantKV(codes, codes, exps, exps, table)
    with pytest.raises(mfs.MfsError, match="codes"):
        mfs.QuantKV(codes.float(), codes.float(), exps, exps, table)
    with pytest.raises(mfs.MfsError, match="rope"):
        mfs.Rope("spiral")


def test_the_definition_by_hand():
    """The 8-bit form itself: exponents at the borders, ties to even, subnormal codes."""
    assert Q.E4M3[0x7e] == 448 and Q.E4M3[0x08] == 2.0 ** -6 and Q.E4M3[0x01] == 2.0 ** -9 and Q.E4M3[0xb8] == -1 and np.isnan(Q.E4M3[0x7f])
    assert [Q.exponent(np.array([x])) for x in (448.0, 448.1, 224.0, 224.1, 1.75, 0.0, 2.0 ** -140)] == [127, 128, 126, 127, 119, 0, 1]
    got = Q.nearest(np.array([1.0625, 1.1875, 17.0, 19.0, 2.0 ** -10, 2.0 ** -10 * 1.01, 3 * 2.0 ** -10, 448.0]), 127)
    assert got.tolist() == [1.0, 1.25, 16.0, 20.0, 0.0, 2.0 ** -9, 2.0 ** -8, 448.0]
    # a rotation slowed by 4 between 1 and 3 turns over 100 positions: 2 pi 100 f = 2 turns keeps half its speed
    f = 10000.0 ** (-2.0 / 4)
    r = Q.rotate(np.array([0.0, 0.0, 1.0, 0.0]), 7, "interleaved", original=2 * 2 * np.pi / f, low=1.0, high=3.0, factor=4.0)
    assert np.allclose(r[2:], [np.cos(7 * f * 0.625), np.sin(7 * f * 0.625)])
