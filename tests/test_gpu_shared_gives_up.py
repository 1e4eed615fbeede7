"""The shared prefixes' tensor-core kernel when one of its waits runs out, in a build whose every CTA loses one tile of its ring
(never fills it) and waits 20 ms at most: the call ends, what it could not compute is NaN, and the rest is right."""
import ctypes
import subprocess
import time

import numpy as np
import pytest

from tests.test_gpu_shared import _cache, _i32, _normal, _tables, _torch, _wide, mfs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def losing(mfs, tmp_path_factory):  # noqa: F811
    """The library built from the same sources but for one that loses tile 2 of each CTA's ring (the keys of its second tile)."""
    import glob
    import os

    from full_duplex_speech_frame_gb300.build import ARCH, BUILD, CSRC, FLAGS, NVCC
    where = tmp_path_factory.mktemp("losing_shared")
    obj, lib = str(where / "shared.o"), str(where / "lose.so")
    subprocess.check_call([NVCC] + FLAGS + ["-DMFS_SHARED_LOST_TILE=2", "-DMFS_PROMPT_WAIT_NS=20000000ull", "-c", os.path.join(CSRC, "mfs_shared.cu"),
                          "-o", obj])
    rest = [o for o in glob.glob(os.path.join(BUILD, "*.o")) if "mfs_shared.cu" not in o]
    subprocess.check_call([NVCC] + ARCH + ["-shared", "-o", lib, obj] + rest + ["-lcudart"])
    so = ctypes.CDLL(lib)
    for name in ("mfs_shared_attention", "mfs_quant_shared_attention"):
        getattr(so, name).argtypes, getattr(so, name).restype = getattr(mfs._lib, name).argtypes, ctypes.c_int
    return so


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("page", [16, 3])
@pytest.mark.parametrize("hd", [64, 128])
def test_what_misses_a_tile_is_nan(mfs, losing, quant, page, hd):  # noqa: F811
    """Two groups of two sequences on one kv head: the first one's prefix is long enough that every CTA loses a tile of it;
    the second group's fits in one tile, and two more sequences share nothing."""
    torch = _torch()
    rng = np.random.default_rng(5)
    sizes, prefix, lens = [2, 2], [128 * 800, 100], [128 * 800 + 3, 128 * 800, 130, 140, 77, 500]
    table, pages, copies = _tables(rng, sizes, prefix, lens, page, 2)
    cache = _cache(mfs, rng, _wide(table, 2, page, 1, hd, "bf16", quant), pages, copies, 1, page, hd, "bf16", quant)
    q = _normal(rng, 6, 4, hd, dtype="bf16")
    want, out, after = torch.empty_like(q), torch.full_like(q, 7.0), torch.empty_like(q)
    groups, plen, kv_len = _i32([0, 2, 4]), _i32(prefix), _i32(lens)
    mfs.mfs_shared_attention(cache, q, kv_len, groups, plen, want)
    ws = mfs.mfs_shared_attention_workspace(cache, 4, 6)
    torch.cuda.synchronize()
    t = time.monotonic()
    args = (6, kv_len.data_ptr(), 2, groups.data_ptr(), plen.data_ptr(), q.data_ptr(), 4 * hd, 4, out.data_ptr(), 4 * hd, hd ** -0.5, 0, ws.data_ptr(),
            ws.nbytes, torch.cuda.current_stream().cuda_stream)
    rc = losing.mfs_quant_shared_attention(ctypes.byref(cache.c), 1, *args) if quant else losing.mfs_shared_attention(ctypes.byref(cache.c), *args)
    assert rc == 0
    torch.cuda.synchronize()
    assert time.monotonic() - t < 20.0
    assert torch.isnan(out[:2]).all() and torch.equal(out[4:], want[4:])
    assert all(torch.isnan(out[s]).all() or torch.equal(out[s], want[s]) for s in (2, 3))  # behind a CTA that gave up, or not
    mfs.mfs_shared_attention(cache, q, kv_len, groups, plen, after)
    assert torch.equal(after, want)
