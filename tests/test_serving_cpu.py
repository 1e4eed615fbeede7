"""The serving operators refuse bad calls on the host, before anything is launched (no GPU needed:
the pointers are never touched), and the binding refuses tensors that are not what it passes on."""
import ctypes

import numpy as np
import pytest

from tests import _serving as S


@pytest.fixture(scope="module")
def mfs():
    from full_duplex_speech_frame_gb300 import mfs as m
    return m


FAKE = 1 << 20  # a 16-byte aligned address that no refused call may touch


def _sample(mfs, **kw):
    a = dict(logits=FAKE, dtype=0, rows=2, cols=10, ld=10, t=None, k=None, p=None, m=None, u=FAKE, out=FAKE, st=None)
    a.update(kw)
    return mfs._lib.mfs_sample_rows(*a.values())


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(cols=0), dict(cols=(1 << 22) + 1, ld=1 << 23), dict(ld=9), dict(dtype=2),
                                 dict(logits=None), dict(u=None), dict(out=None), dict(logits=FAKE + 2)])
def test_sample_rows_refusals(mfs, bad):
    assert _sample(mfs, **bad) == -1
    assert mfs.mfs_last_error(None).startswith("sample_rows: ")


def test_no_rows_is_nothing(mfs):
    assert _sample(mfs, rows=0, logits=None, u=None, out=None) == 0


def _cache(mfs, **kw):
    c = mfs.mfs_paged_kv(k=FAKE, v=FAKE, table=FAKE, table_width=4, table_stride=4, n_pages=8, page_size=16, n_kv_heads=2,
                         head_dim=64, dtype=1, page_stride=2048, head_stride=1024, row_stride=64)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [dict(k=None), dict(v=None), dict(table=None), dict(table_width=0), dict(table_stride=-1), dict(n_pages=0), dict(page_size=0),
              dict(page_size=65537), dict(n_kv_heads=0), dict(head_dim=96), dict(dtype=2), dict(page_stride=-64), dict(row_stride=60),
              dict(head_stride=1028), dict(k=FAKE + 8)]


def _append(mfs, cache=None, **kw):
    a = dict(n=3, n_seqs=2, cu=FAKE, kv_len=FAKE, q=FAKE, qs=256, hq=4, q_out=FAKE, qos=256, k=FAKE, ks=128, k_out=FAKE, kos=128,
             v=FAKE, vs=128, rope=1, theta=1e4, st=None)
    a.update(kw)
    return mfs._lib.mfs_kv_append(cache if cache is not None else _cache(mfs), *a.values())


@pytest.mark.parametrize("bad", [dict(n=-1), dict(n_seqs=-1), dict(cu=None), dict(kv_len=None), dict(k=None), dict(v=None), dict(q_out=None),
                                 dict(q=None), dict(hq=0), dict(qs=255), dict(qs=248), dict(ks=64), dict(vs=130), dict(kos=124), dict(k=FAKE + 2),
                                 dict(v=FAKE + 4), dict(rope=3), dict(theta=0.0), dict(theta=-1.0), dict(theta=float("nan")),
                                 dict(theta=float("inf"))])
def test_kv_append_refusals(mfs, bad):
    assert _append(mfs, **bad) == -1
    assert mfs.mfs_last_error(None).startswith("kv_append: ")


def _attend(mfs, cache=None, **kw):
    a = dict(n=2, kv_len=FAKE, q=FAKE, qs=256, hq=4, out=FAKE, os=256, scale=0.125, window=0, ws=FAKE, wsb=1 << 30, st=None)
    a.update(kw)
    return mfs._lib.mfs_paged_attention(cache if cache is not None else _cache(mfs), *a.values())


@pytest.mark.parametrize("bad", [dict(n=-1), dict(window=-1), dict(hq=3), dict(hq=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                                 dict(scale=float("inf")), dict(kv_len=None), dict(q=None), dict(out=None), dict(ws=None), dict(wsb=0),
                                 dict(ws=FAKE + 8), dict(qs=252), dict(os=192), dict(q=FAKE + 2), dict(out=FAKE + 8)])
def test_paged_attention_refusals(mfs, bad):
    assert _attend(mfs, **bad) == -1
    assert mfs.mfs_last_error(None).startswith("paged_attention: ")


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_bad_caches_are_refused(mfs, bad):
    c = _cache(mfs, **bad)
    assert _append(mfs, c) == -1 and _attend(mfs, c) == -1
    assert mfs._lib.mfs_kv_append(None, *([0] * 2), *([None] * 3), 0, 0, None, 0, None, 0, None, 0, None, 0, 0, 1.0, None) == -1


def _prompt(mfs, **kw):
    a = dict(dtype=1, n=5, n_seqs=2, cu=FAKE, q=FAKE, qs=256, hq=4, k=FAKE, ks=128, v=FAKE, vs=128, hkv=2, hd=64, out=FAKE, os=256,
             scale=0.125, window=0, st=None)
    a.update(kw)
    return mfs._lib.mfs_prompt_attention(*a.values())


@pytest.mark.parametrize("bad", [dict(dtype=2), dict(hd=80), dict(n=-1), dict(n_seqs=-1), dict(window=-1), dict(hkv=3), dict(hkv=0), dict(hq=0),
                                 dict(scale=0.0), dict(scale=float("nan")), dict(cu=None), dict(q=None), dict(k=None), dict(v=None), dict(out=None),
                                 dict(qs=248), dict(ks=132), dict(vs=120), dict(os=260), dict(q=FAKE + 8), dict(out=FAKE + 2)])
def test_prompt_attention_refusals(mfs, bad):
    assert _prompt(mfs, **bad) == -1
    assert mfs.mfs_last_error(None).startswith("prompt_attention: ")


def test_heads_past_the_limit_are_refused(mfs):
    n = 65536
    c = _cache(mfs, n_kv_heads=n, head_stride=64, row_stride=64 * n, page_stride=64 * n * 16)
    assert _append(mfs, c, ks=64 * n, vs=64 * n, k_out=None) == -1 and "heads" in mfs.mfs_last_error(None)
    assert _attend(mfs, c, hq=n, qs=64 * n, os=64 * n) == -1 and "heads" in mfs.mfs_last_error(None)
    c = _cache(mfs)
    assert _append(mfs, c, hq=n, qs=64 * n, qos=64 * n) == -1 and "heads" in mfs.mfs_last_error(None)
    assert _attend(mfs, c, hq=n, qs=64 * n, os=64 * n) == -1 and "heads" in mfs.mfs_last_error(None)
    assert _prompt(mfs, hq=n, qs=64 * n, os=64 * n) == -1 and "heads" in mfs.mfs_last_error(None)


def test_nothing_to_do_is_ok(mfs):
    assert _append(mfs, n=0) == 0 and _append(mfs, n_seqs=0) == 0
    assert _attend(mfs, n=0) == 0
    assert _prompt(mfs, n=0) == 0 and _prompt(mfs, n_seqs=0) == 0


def test_workspace_size_is_stated(mfs):
    c = _cache(mfs)
    assert mfs._lib.mfs_paged_attention_workspace(c, 4) >= 16


def test_paged_kv_layout_matches_header(mfs, tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "probe.c"
    src.write_text('#include <stdio.h>\n#include "mfs.h"\nint main(void){printf("%zu %zu %zu %zu %zu\\n", sizeof(mfs_paged_kv),'
                   ' offsetof(mfs_paged_kv, table_width), offsetof(mfs_paged_kv, table_stride), offsetof(mfs_paged_kv, dtype),'
                   ' offsetof(mfs_paged_kv, row_stride)); return 0;}\n')
    exe = tmp_path / "probe"
    subprocess.check_call(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    c = mfs.mfs_paged_kv
    assert got == [ctypes.sizeof(c), c.table_width.offset, c.table_stride.offset, c.dtype.offset, c.row_stride.offset]


def test_binding_refuses_host_tensors(mfs):
    import torch
    z = torch.zeros(4, 2, 16, 64)
    t = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(mfs.MfsError, match="CUDA"):
        mfs.PagedKV(z, z, t)
    with pytest.raises(mfs.MfsError, match="CUDA"):
        mfs.mfs_sample_rows(torch.zeros(2, 8), torch.zeros(2), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(mfs.MfsError, match="CUDA"):
        mfs.mfs_prompt_attention(z[0], z[0], z[0], t[0], z[0])


def test_sampling_definition_by_hand():
    """The oracle itself: weights 1, 1/2, 1/4 at columns 2, 0, 1 (T = 1 / ln 2 makes e^(-1/T) one half)."""
    t = 1 / np.log(2)
    x = [-1.0, -2.0, 0.0]
    assert [S.sample_row(x, u, t) for u in (0.0, 0.28, 0.29, 0.42, 0.43, 0.99)] == [0, 0, 1, 1, 2, 2]
    assert [S.sample_row(x, u, t, top_k=2) for u in (0.0, 0.33, 0.34)] == [0, 0, 2]
    assert S.sample_row(x, 0.0, t, top_p=0.5) == 2 and S.sample_row(x, 0.0, t, top_p=0.6) == 0
    assert S.sample_row(x, 0.0, t, min_p=0.6) == 2 and S.sample_row(x, 0.0, t, min_p=0.4) == 0
    assert S.sample_row([np.nan, np.nan], 0.3) == 0 and S.sample_row([np.nan, -np.inf], 0.3) == 1
    assert S.sample_row([0.0, np.inf, np.inf], 0.6) == 2


@pytest.mark.parametrize("stream,owner", [(None, "current"), (0, "default of dev"), (77, "external 77 on dev")])
def test_default_workspace_is_of_the_stream_that_runs(mfs, monkeypatch, stream, owner):
    """A workspace made for a call comes from the pool of the call's stream, the null stream's among them: torch takes a
    null handle given to ExternalStream for none and hands out another stream."""
    import contextlib
    import types

    import torch
    now, made, ran = ["current"], [], []

    @contextlib.contextmanager
    def on(s):
        now.append(s)
        yield
        now.pop()

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: f"external {handle} on {device}")
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: f"default of {device}")

    def workspace(cache, heads):
        made.append(now[-1])
        return torch.empty(16, dtype=torch.uint8)

    monkeypatch.setattr(mfs, "mfs_paged_attention_workspace", workspace)
    monkeypatch.setattr(mfs, "_enqueue", lambda dev, stream, fn, *args: ran.append(stream))
    cache = types.SimpleNamespace(_is=(-1, torch.float32, 2, 64), n_seqs=3, device="dev", c=None)
    q = torch.zeros(3, 4, 64)
    mfs.mfs_paged_attention(cache, q, torch.ones(3, dtype=torch.int32), torch.empty_like(q), stream=stream)
    assert made == [owner] and ran == [stream] and now == ["current"]
