"""The bf16 prompt kernel when one of its waits runs out, in a build whose every CTA loses one tile of its ring (never asks
for it) and waits 20 ms at most: the call ends, the rows that it could not compute are NaN, and the others are right."""
import ctypes
import subprocess
import time

import numpy as np
import pytest

from tests.test_gpu_serving import _i32, _normal, _torch, mfs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def losing(mfs, tmp_path_factory):  # noqa: F811
    """losing(n): mfs_prompt_attention of a build that loses tile n of each CTA (keys and values in turn)."""
    import os

    from full_duplex_speech_frame_gb300.build import CSRC, FLAGS, NVCC
    made, where = {}, tmp_path_factory.mktemp("losing")
    (where / "errors.cu").write_text("namespace mfs { void set_thread_error(const char*) {} }\n")

    def entry(n):
        if n not in made:
            lib = str(where / f"lose{n}.so")
            subprocess.check_call([NVCC] + FLAGS + [f"-DMFS_PROMPT_LOST_TILE={n}", "-DMFS_PROMPT_WAIT_NS=20000000ull", "-shared",
                                  "-o", lib, os.path.join(CSRC, "mfs_prompt.cu"), str(where / "errors.cu"), "-lcudart"])
            fn = ctypes.CDLL(lib).mfs_prompt_attention
            fn.argtypes, fn.restype = mfs._lib.mfs_prompt_attention.argtypes, ctypes.c_int
            made[n] = fn
        return made[n]

    return entry


def _run(mfs, losing, lost, lens, hq, hkv, hd):  # noqa: F811
    """(the stalled call's output, the right one)"""
    torch = _torch()
    rng = np.random.default_rng(61)
    n = sum(lens)
    q, k, v = (_normal(rng, n, h, hd, dtype="bf16") for h in (hq, hkv, hkv))
    cu, want, out = _i32(np.cumsum([0] + lens).tolist()), torch.empty_like(q), torch.full_like(q, 7.0)
    mfs.mfs_prompt_attention(q, k, v, cu, want)
    torch.cuda.synchronize()
    t = time.monotonic()
    assert losing(lost)(1, n, len(lens), cu.data_ptr(), q.data_ptr(), hq * hd, hq, k.data_ptr(), hkv * hd, v.data_ptr(), hkv * hd, hkv, hd,
                        out.data_ptr(), hq * hd, hd ** -0.5, 0, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert time.monotonic() - t < 10.0
    after = torch.empty_like(q)
    mfs.mfs_prompt_attention(q, k, v, cu, after)
    assert torch.equal(after, want)
    return out, want


@pytest.mark.parametrize("hq,hkv,hd", [(4, 2, 64), (4, 2, 128), (3, 1, 64), (2, 2, 128)])
@pytest.mark.parametrize("lost", [0, 1, 4])
def test_rows_that_miss_a_tile_are_nan(mfs, losing, lost, hq, hkv, hd):  # noqa: F811
    """One block to a CTA: the t-th tile of keys is tile 2 t of its ring, and the values behind it."""
    torch = _torch()
    out, want = _run(mfs, losing, lost, [700], hq, hkv, hd)
    paired = hq // hkv % 2 == 0
    for r0 in range(0, 700, 128):
        rows, ref = out[r0:r0 + 128], want[r0:r0 + 128]
        for h in range(hq):
            nan, right = bool(torch.isnan(rows[:, h]).all()), torch.equal(rows[:, h], ref[:, h])
            if 2 * (r0 // 128 + 1) > lost:
                assert nan, (r0, h)
            elif paired or 2 * (r0 // 256 * 2 + 2) <= lost:  # the whole block has its tiles
                assert right, (r0, h)
            else:
                assert nan or right, (r0, h)


@pytest.mark.parametrize("hq,hkv,hd,lens", [(32, 16, 64, [300] * 20), (64, 32, 128, [130, 1, 260] * 8), (27, 9, 128, [300, 520] * 9), (16, 16, 64, [40] * 300)])
@pytest.mark.parametrize("lost", [0, 3, 10])
def test_no_row_is_left_as_it_was(mfs, losing, lost, hq, hkv, hd, lens):  # noqa: F811
    """Several blocks to a CTA, waiting, dealt out or not yet: each row and head is right or NaN, and with the first tile lost
    every one is NaN."""
    torch = _torch()
    out, want = _run(mfs, losing, lost, lens, hq, hkv, hd)
    nan, right = torch.isnan(out).all(-1), (out == want).all(-1)
    assert (nan | right).all() and nan.any()
    if lost == 0:
        assert nan.all()
