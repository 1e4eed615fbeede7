"""The shared prefixes' tensor-core kernel when a wait runs out although the warp that loads has asked for all of its part without
one: the block still waits for the copies it asked for before it ends.  The build loses the keys of each block's second tile and
waits 200 ms at most, and no part has more tiles than the ring: the products' warp gives up after 200 ms, and the wait for the
copies, which here meets the lost one, takes 200 ms more."""
import ctypes
import subprocess
import time

import numpy as np
import pytest

from tests.test_gpu_shared import _cache, _i32, _normal, _tables, _torch, _wide, mfs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def losing(mfs, tmp_path_factory):  # noqa: F811
    import glob
    import os

    from full_duplex_speech_frame_gb300.build import ARCH, BUILD, CSRC, FLAGS, NVCC
    where = tmp_path_factory.mktemp("losing_last")
    obj, lib = str(where / "shared.o"), str(where / "lose.so")
    subprocess.check_call([NVCC] + FLAGS + ["-DMFS_SHARED_LOST_TILE=2", "-DMFS_PROMPT_WAIT_NS=200000000ull", "-c", os.path.join(CSRC, "mfs_shared.cu"),
                          "-o", obj])
    rest = [o for o in glob.glob(os.path.join(BUILD, "*.o")) if "mfs_shared.cu" not in o]
    subprocess.check_call([NVCC] + ARCH + ["-shared", "-o", lib, obj] + rest + ["-lcudart"])
    so = ctypes.CDLL(lib)
    so.mfs_shared_attention.argtypes, so.mfs_shared_attention.restype = mfs._lib.mfs_shared_attention.argtypes, ctypes.c_int
    return so


@pytest.mark.parametrize("hd", [64, 128])
def test_copies_are_waited_for(mfs, losing, hd):  # noqa: F811
    """303 tiles of a pair's prefix and the room at its start are two places for each of 152 blocks: four tiles of the ring,
    which has five or eight."""
    torch = _torch()
    rng = np.random.default_rng(17)
    page, prefix = 16, 128 * 303
    lens = [prefix + 3, prefix]
    table, pages, copies = _tables(rng, [2], [prefix], lens, page)
    cache = _cache(mfs, rng, _wide(table, 1, page, 1, hd, "bf16", False), pages, copies, 1, page, hd, "bf16", False)
    q = _normal(rng, 2, 4, hd, dtype="bf16")
    want, out, after = torch.empty_like(q), torch.full_like(q, 7.0), torch.empty_like(q)
    groups, plen, kv_len = _i32([0, 2]), _i32([prefix]), _i32(lens)
    mfs.mfs_shared_attention(cache, q, kv_len, groups, plen, want)
    ws = mfs.mfs_shared_attention_workspace(cache, 4, 2)
    torch.cuda.synchronize()
    t = time.monotonic()
    rc = losing.mfs_shared_attention(ctypes.byref(cache.c), 2, kv_len.data_ptr(), 1, groups.data_ptr(), plen.data_ptr(), q.data_ptr(), 4 * hd, 4,
                                     out.data_ptr(), 4 * hd, hd ** -0.5, 0, ws.data_ptr(), ws.nbytes, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    t = time.monotonic() - t
    assert 0.39 < t < 10.0, t
    assert torch.isnan(out).all()
    mfs.mfs_shared_attention(cache, q, kv_len, groups, plen, after)
    assert torch.equal(after, want) and torch.isfinite(want).all()
