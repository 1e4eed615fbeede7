"""Python binding of the C ABI in include/mfs.h (ctypes; argument marshalling only).

Every step of the frame step runs in the CUDA library ``libmfs.so``; this module
only converts arguments.  There is no fallback: if the library is missing the
import fails with the command that builds it.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
# MFS_LIBRARY selects another build of the same library (same ABI).
LIB_PATH = os.environ.get("MFS_LIBRARY") or os.path.join(_HERE, "libmfs.so")

MFS_OK = 0
STATUS = {-1: "MFS_E_ARG", -2: "MFS_E_SLOT", -3: "MFS_E_TOKEN", -4: "MFS_E_RANGE", -5: "MFS_E_STATE",
          -6: "MFS_E_CUDA", -7: "MFS_E_DEVICE", -8: "MFS_E_NOMEM"}
MFS_DTYPE_F32, MFS_DTYPE_BF16 = 0, 1
MFS_MAX_SLOTS = 64
MFS_ROPE = {None: 0, "interleaved": 1, "half": 2}


class MfsError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"{STATUS.get(code, code)}: {message}")
        self.code = code
        self.status = STATUS.get(code, str(code))


class mfs_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "d", "n_layers", "n_heads", "head_dim", "ffn", "text_vocab", "card", "n_q", "window", "max_pos",
        "dep_d", "dep_layers", "dep_heads", "dep_head_dim", "dep_ffn", "dep_steps")] + [
        ("delays", ctypes.c_int * 17), ("rope_theta", ctypes.c_double), ("eps", ctypes.c_double),
        ("weight_dtype", ctypes.c_int), ("kv_dtype", ctypes.c_int), ("max_slots", ctypes.c_int)]


class mfs_paged_kv(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("table", ctypes.c_void_p), ("table_width", ctypes.c_int),
                ("table_stride", ctypes.c_longlong)] + [(n, ctypes.c_int) for n in (
                    "n_pages", "page_size", "n_kv_heads", "head_dim", "dtype")] + [
                        (n, ctypes.c_longlong) for n in ("page_stride", "head_stride", "row_stride")]


def _load_library():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -c 'import __graft_entry__ as g; g.build()'` "
                          "(or python full_duplex_speech_frame_gb300/build.py)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, ci, i32p = ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p
    ll, pkv = ctypes.c_longlong, ctypes.POINTER(mfs_paged_kv)
    sig = {
        "mfs_create": (ci, [ctypes.POINTER(mfs_config), vp, ctypes.POINTER(vp)]),
        "mfs_destroy": (None, [vp]),
        "mfs_last_error": (ctypes.c_char_p, [vp]),
        "mfs_load_weights": (ci, [vp, ctypes.c_char_p, vp, ctypes.c_size_t, ci]),
        "mfs_step": (ci, [vp, ci, i32p, i32p, i32p, i32p]),
        "mfs_step_device": (ci, [vp, ci, i32p, vp, vp, vp]),
        "mfs_sync": (ci, [vp]),
        "mfs_prefill": (ci, [vp, ci, i32p, ci, i32p]),
        "mfs_reset_slot": (ci, [vp, ci]),
        "mfs_position": (ci, [vp, ci]),
        "mfs_read_debug": (ci, [vp, vp, vp, vp, vp]),
        "mfs_set_ring_mask_oldest": (ci, [vp, ci]),
        "mfs_debug_set_seq": (ci, [vp, ctypes.c_uint32]),
        "mfs_set_mode": (ci, [vp, ci]),
        "mfs_launches_per_step": (ci, [vp]),
        "mfs_set_skip_settled": (ci, [vp, ci]),
        "mfs_set_wait_limit": (ci, [vp, ci]),
        "mfs_debug_stall": (ci, [vp, ci]),
        "mfs_set_sampling": (ci, [vp, ci, ctypes.c_float, ci, ctypes.c_float, ci]),
        "mfs_step_sampled": (ci, [vp, ci, i32p, i32p, vp, i32p, i32p]),
        "mfs_set_timing": (ci, [vp, ci]),
        "mfs_kernel_time": (ci, [vp, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int)]),
        "mfs_phase_times": (ci, [vp, vp, ci]),
        "mfs_argmax_rows_noalloc": (ci, [vp, ci, ci, ctypes.c_longlong, vp, vp]),
        "mfs_rvq_encode": (ci, [vp, vp, ci, ci, vp, ci, vp, vp]),
        "mfs_sample_rows": (ci, [vp, ci, ci, ci, ll, vp, vp, vp, vp, vp, vp, vp]),
        "mfs_kv_append": (ci, [pkv, ci, ci, vp, vp, vp, ll, ci, vp, ll, vp, ll, vp, ll, vp, ll, ci, ctypes.c_double, vp]),
        "mfs_paged_attention_workspace": (ctypes.c_size_t, [pkv, ci]),
        "mfs_paged_attention": (ci, [pkv, ci, vp, vp, ll, ci, vp, ll, ctypes.c_float, ci, vp, ctypes.c_size_t, vp]),
        "mfs_prompt_attention": (ci, [ci, ci, ci, vp, vp, ll, ci, vp, ll, vp, ll, ci, ci, vp, ll, ctypes.c_float, ci, vp]),
        "mfs_slot_state_bytes": (ctypes.c_size_t, [vp]),
        "mfs_export_slot": (ci, [vp, ci, vp, ctypes.c_size_t]),
        "mfs_import_slot": (ci, [vp, ci, vp, ctypes.c_size_t]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


_lib = _load_library()


def exported_symbols() -> Sequence[str]:
    return [n for n in dir(_lib) if n.startswith("mfs_")]


class Ctx:
    """Owner of an ``mfs_ctx*``; destroyed with ``mfs_destroy``."""

    def __init__(self, handle: int, cfg: mfs_config):
        self.handle = ctypes.c_void_p(handle)
        self.cfg = cfg
        self.last_n = 0

    def __del__(self):
        if getattr(self, "handle", None) and self.handle.value:
            _lib.mfs_destroy(self.handle)
            self.handle = ctypes.c_void_p(None)


def _check(ctx: Optional[Ctx], rc: int) -> None:
    if rc != MFS_OK:
        h = ctx.handle if ctx is not None else None
        raise MfsError(rc, (_lib.mfs_last_error(h) or b"").decode())


def make_config(d, n_layers, n_heads, head_dim, ffn, text_vocab, card, window, max_pos, dep_d, dep_layers,
                dep_heads, dep_head_dim, dep_ffn, delays, rope_theta=10000.0, eps=1e-8,
                weight_dtype="bf16", kv_dtype="bf16", max_slots=1, n_q=16, dep_steps=16) -> mfs_config:
    c = mfs_config()
    for k, v in dict(d=d, n_layers=n_layers, n_heads=n_heads, head_dim=head_dim, ffn=ffn, text_vocab=text_vocab,
                     card=card, n_q=n_q, window=window, max_pos=max_pos, dep_d=dep_d, dep_layers=dep_layers,
                     dep_heads=dep_heads, dep_head_dim=dep_head_dim, dep_ffn=dep_ffn, dep_steps=dep_steps,
                     max_slots=max_slots).items():
        setattr(c, k, int(v))
    c.delays[:] = [int(x) for x in delays]
    c.rope_theta = float(rope_theta)
    c.eps = float(eps)
    c.weight_dtype = MFS_DTYPE_BF16 if weight_dtype == "bf16" else MFS_DTYPE_F32
    c.kv_dtype = MFS_DTYPE_BF16 if kv_dtype == "bf16" else MFS_DTYPE_F32
    return c


def config_from_shape(shape) -> mfs_config:
    """An mfs_config from any object with the config's field names as attributes
    (dtypes as the strings "bf16" / "f32")."""
    s = shape
    return make_config(d=s.d, n_layers=s.n_layers, n_heads=s.n_heads, head_dim=s.head_dim, ffn=s.ffn,
                       text_vocab=s.text_vocab, card=s.card, window=s.window, max_pos=s.max_pos,
                       dep_d=s.dep_d, dep_layers=s.dep_layers, dep_heads=s.dep_heads,
                       dep_head_dim=s.dep_head_dim, dep_ffn=s.dep_ffn, delays=s.delays,
                       rope_theta=s.rope_theta, eps=s.eps, weight_dtype=s.weight_dtype,
                       kv_dtype=s.kv_dtype, max_slots=s.max_slots, n_q=s.n_q, dep_steps=s.dep_steps)


def context_with_weights(shape, weights) -> "Ctx":
    """A context for `shape` with every named tensor of `weights` loaded."""
    ctx = mfs_create(config_from_shape(shape))
    for name, arr in weights.items():
        mfs_load_weights(ctx, name, arr)
    return ctx


def _current_stream():
    try:
        import torch
        if torch.cuda.is_available():
            return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    except ImportError:
        pass
    return None


def mfs_create(cfg: mfs_config, stream=None) -> Ctx:
    out = ctypes.c_void_p()
    st = _current_stream() if stream is None else ctypes.c_void_p(stream)
    rc = _lib.mfs_create(ctypes.byref(cfg), st, ctypes.byref(out))
    _check(None, rc)
    return Ctx(out.value, cfg)


def mfs_destroy(ctx: Ctx) -> None:
    if ctx.handle.value:
        _lib.mfs_destroy(ctx.handle)
        ctx.handle = ctypes.c_void_p(None)


def mfs_last_error(ctx: Optional[Ctx]) -> str:
    return (_lib.mfs_last_error(ctx.handle if ctx else None) or b"").decode()


def mfs_load_weights(ctx: Ctx, name: str, src) -> None:
    """src: a C-contiguous numpy array (host) or a contiguous CUDA torch tensor."""
    if isinstance(src, np.ndarray):
        src = np.ascontiguousarray(src)
        rc = _lib.mfs_load_weights(ctx.handle, name.encode(), src.ctypes.data, src.nbytes, 0)
    else:
        assert src.is_cuda and src.is_contiguous()
        rc = _lib.mfs_load_weights(ctx.handle, name.encode(), src.data_ptr(),
                                   src.numel() * src.element_size(), 1)
    _check(ctx, rc)


def _i32(a) -> np.ndarray:
    return np.ascontiguousarray(a, dtype=np.int32)


def mfs_step(ctx: Ctx, slots, in_codes):
    """Returns (text_tok [n], codes [n, 16]) as int32 numpy arrays."""
    slots = _i32(slots).reshape(-1)
    n = slots.size
    codes_in = _i32(in_codes).reshape(n, 17)
    text = np.empty(n, np.int32)
    codes = np.empty((n, 16), np.int32)
    rc = _lib.mfs_step(ctx.handle, n, slots.ctypes.data, codes_in.ctypes.data, text.ctypes.data, codes.ctypes.data)
    _check(ctx, rc)
    ctx.last_n = n
    return text, codes


def mfs_set_sampling(ctx: Ctx, slot: int, text_temp: float, text_topk: int, audio_temp: float, audio_topk: int) -> None:
    _check(ctx, _lib.mfs_set_sampling(ctx.handle, int(slot), float(text_temp), int(text_topk), float(audio_temp),
                                      int(audio_topk)))


def mfs_step_sampled(ctx: Ctx, slots, in_codes, uniforms):
    """mfs_step with uniforms [n, 17] in [0, 1) for the slots' sampling heads."""
    slots = _i32(slots).reshape(-1)
    n = slots.size
    codes_in = _i32(in_codes).reshape(n, 17)
    unif = np.ascontiguousarray(uniforms, dtype=np.float32).reshape(n, 17)
    text = np.empty(n, np.int32)
    codes = np.empty((n, 16), np.int32)
    rc = _lib.mfs_step_sampled(ctx.handle, n, slots.ctypes.data, codes_in.ctypes.data, unif.ctypes.data,
                               text.ctypes.data, codes.ctypes.data)
    _check(ctx, rc)
    ctx.last_n = n
    return text, codes


def mfs_step_device(ctx: Ctx, slots, d_in_codes, d_text=None, d_codes=None) -> None:
    """d_* are contiguous int32 CUDA tensors; returns without waiting."""
    slots = _i32(slots).reshape(-1)
    n = slots.size
    rc = _lib.mfs_step_device(ctx.handle, n, slots.ctypes.data, d_in_codes.data_ptr(),
                              d_text.data_ptr() if d_text is not None else None,
                              d_codes.data_ptr() if d_codes is not None else None)
    _check(ctx, rc)
    ctx.last_n = n


def mfs_sync(ctx: Ctx) -> None:
    _check(ctx, _lib.mfs_sync(ctx.handle))


def mfs_prefill(ctx: Ctx, slots, codes) -> None:
    """codes [n, T, 17] int, every entry >= 0."""
    slots = _i32(slots).reshape(-1)
    n = slots.size
    codes = _i32(codes)
    T = codes.shape[1] if codes.ndim == 3 else codes.size // (17 * n)
    codes = codes.reshape(n, T, 17)
    _check(ctx, _lib.mfs_prefill(ctx.handle, n, slots.ctypes.data, T, codes.ctypes.data))


def mfs_reset_slot(ctx: Ctx, slot: int) -> None:
    _check(ctx, _lib.mfs_reset_slot(ctx.handle, int(slot)))


def mfs_position(ctx: Ctx, slot: int) -> int:
    rc = _lib.mfs_position(ctx.handle, int(slot))
    if rc < 0:
        _check(ctx, rc)
    return rc


def mfs_export_slot(ctx: Ctx, slot: int) -> np.ndarray:
    """The slot's state as a uint8 buffer (layout in include/mfs.h)."""
    buf = np.empty(_lib.mfs_slot_state_bytes(ctx.handle), np.uint8)
    _check(ctx, _lib.mfs_export_slot(ctx.handle, int(slot), buf.ctypes.data, buf.nbytes))
    return buf


def mfs_import_slot(ctx: Ctx, slot: int, buf: np.ndarray) -> None:
    buf = np.ascontiguousarray(buf, dtype=np.uint8)
    _check(ctx, _lib.mfs_import_slot(ctx.handle, int(slot), buf.ctypes.data, buf.nbytes))


def mfs_read_debug(ctx: Ctx, n: Optional[int] = None) -> dict:
    n = ctx.last_n if n is None else n
    c = ctx.cfg
    out = {"text_logits": np.empty((n, c.text_vocab), np.float32),
           "dep_logits": np.empty((n, 16, c.card), np.float32),
           "text_argmax": np.empty(n, np.int32), "code_argmax": np.empty((n, 16), np.int32)}
    rc = _lib.mfs_read_debug(ctx.handle, out["text_logits"].ctypes.data, out["dep_logits"].ctypes.data,
                             out["text_argmax"].ctypes.data, out["code_argmax"].ctypes.data)
    _check(ctx, rc)
    return out


def mfs_set_ring_mask_oldest(ctx: Ctx, on: bool) -> None:
    """Attend to W - 1 keys once the ring is full (the masked-oldest-slot window variant)."""
    _check(ctx, _lib.mfs_set_ring_mask_oldest(ctx.handle, 1 if on else 0))


def mfs_debug_set_seq(ctx: Ctx, seq: int) -> None:
    """Testing: the next step takes sequence number seq + 1 (see include/mfs.h)."""
    _check(ctx, _lib.mfs_debug_set_seq(ctx.handle, int(seq) & 0xFFFFFFFF))


def mfs_set_mode(ctx: Ctx, mode: int) -> None:
    _check(ctx, _lib.mfs_set_mode(ctx.handle, int(mode)))


def mfs_set_skip_settled(ctx: Ctx, on: bool) -> None:
    """Skip trailing depformer substeps whose outputs are all supplied (include/mfs.h)."""
    _check(ctx, _lib.mfs_set_skip_settled(ctx.handle, int(bool(on))))


def mfs_set_wait_limit(ctx: Ctx, ms: int) -> None:
    _check(ctx, _lib.mfs_set_wait_limit(ctx.handle, int(ms)))


def mfs_debug_stall(ctx: Ctx, slot: int) -> None:
    """Raises MfsError(MFS_E_DEVICE) when the device's bounded waits work (include/mfs.h)."""
    _check(ctx, _lib.mfs_debug_stall(ctx.handle, int(slot)))


def mfs_launches_per_step(ctx: Ctx) -> int:
    return _lib.mfs_launches_per_step(ctx.handle)


def mfs_set_timing(ctx: Ctx, flags) -> None:
    """flags: bit 0 = event timing of each step's kernel, bit 1 = per-phase timer stamps."""
    _check(ctx, _lib.mfs_set_timing(ctx.handle, int(flags)))


def mfs_phase_times(ctx: Ctx) -> np.ndarray:
    """Diagnostic timer values of the last step(s), [phases + 1, 8] (see include/mfs.h)."""
    buf = np.zeros(16384, np.uint64)
    rc = _lib.mfs_phase_times(ctx.handle, buf.ctypes.data, buf.size)
    if rc < 0:
        _check(ctx, rc)
    return buf[:rc].reshape(-1, 8).copy()


def mfs_kernel_time(ctx: Ctx):
    """(summed kernel milliseconds, steps timed) since the previous call."""
    ms, n = ctypes.c_double(), ctypes.c_int()
    _check(ctx, _lib.mfs_kernel_time(ctx.handle, ctypes.byref(ms), ctypes.byref(n)))
    return ms.value, n.value


def mfs_argmax_rows_noalloc(logits, out, stream=None) -> None:
    """Greedy argmax of each row of a 2-D fp32 CUDA tensor into an int32 CUDA tensor,
    with no device allocation (see include/mfs.h); enqueued on `stream` (default:
    torch's current stream)."""
    import torch
    assert logits.is_cuda and logits.dtype == torch.float32 and logits.dim() == 2 and logits.stride(1) == 1
    assert out.is_cuda and out.dtype == torch.int32 and out.is_contiguous() and out.numel() >= logits.shape[0]
    rows, cols = logits.shape
    st = _current_stream() if stream is None else ctypes.c_void_p(stream)
    rc = _lib.mfs_argmax_rows_noalloc(logits.data_ptr(), rows, cols, logits.stride(0), out.data_ptr(), st)
    _check(None, rc)


def mfs_rvq_encode(z_sem, z_ac, codebooks, codes, stream=None) -> None:
    """Mimi split RVQ encode on CUDA tensors: z_sem, z_ac [T, D] fp32, codebooks [8, Cb, D]
    fp32 -> codes [T, 8] int32 (see include/mfs.h); enqueued on `stream`."""
    import torch
    for t in (z_sem, z_ac, codebooks):
        assert t.is_cuda and t.dtype == torch.float32 and t.is_contiguous()
    assert codes.is_cuda and codes.dtype == torch.int32 and codes.is_contiguous()
    T, D = z_sem.shape
    st = _current_stream() if stream is None else ctypes.c_void_p(stream)
    rc = _lib.mfs_rvq_encode(z_sem.data_ptr(), z_ac.data_ptr(), T, D, codebooks.data_ptr(), codebooks.shape[1],
                             codes.data_ptr(), st)
    _check(None, rc)


# ------------------------------------------------- operators on device tensors
# These calls take microseconds on the GPU, so their checks build nothing that is not needed.

def _refuse(message: str):
    raise MfsError(-1, message)


def _window(w: int) -> int:
    if not 0 <= w <= 0x7fffffff:
        _refuse(f"window {w} outside [0, 2^31)")
    return w


def _dtype_code(t) -> int:
    import torch
    if t.dtype is torch.bfloat16:
        return MFS_DTYPE_BF16
    if t.dtype is not torch.float32:
        _refuse(f"dtype {t.dtype}: need float32 or bfloat16")
    return MFS_DTYPE_F32


def _array(t, what: str, n: int, dtype, dev: int):
    """Data pointer of a contiguous 1-D tensor of at least n elements on CUDA device `dev` (None: null)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.dim() != 1 or t.numel() < n or t.get_device() != dev or not (t.is_contiguous() or n <= 1):
        _refuse(f"{what}: need a contiguous {dtype} tensor of {n} elements on cuda:{dev}")
    return t.data_ptr()


def _rows(t, what: str, n: int, heads: int, head_dim: int, dtype, dev: int):
    """(data pointer, token stride) of a [tokens, heads, head_dim] tensor whose heads are dense."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != (n, heads, head_dim):
        _refuse(f"{what}: need {dtype} [{n}, {heads}, {head_dim}] on cuda:{dev}")
    stride = t.stride()
    if stride[2] != 1 or (heads > 1 and stride[1] != head_dim):
        _refuse(f"{what}: need dense heads")
    return t.data_ptr(), stride[0] if n > 1 else heads * head_dim


def _enqueue(dev: int, stream, fn, *args) -> None:
    """Call a library function (its last argument: the stream) with CUDA device `dev` current."""
    import torch
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    if torch._C._cuda_getDevice() == dev:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, stream)
    if rc != MFS_OK:
        _check(None, rc)


def mfs_sample_rows(logits, uniforms, tokens, temperature=None, top_k=None, top_p=None, min_p=None, stream=None) -> None:
    """Draw tokens[r] (int32) from row r of the 2-D CUDA tensor logits (fp32 or bf16, unit column
    stride) with uniforms[r]: temperature, min-p, top-k and top-p from per-row CUDA tensors, or
    None (see include/mfs.h); enqueued on `stream` (default: torch's current stream)."""
    import torch
    if not logits.is_cuda or logits.dim() != 2:
        _refuse("logits: need a 2-D CUDA tensor")
    rows, cols = logits.shape
    if cols > 1 and logits.stride(1) != 1:
        _refuse("logits: need unit column stride")
    if rows > 0x7fffffff or cols > 0x7fffffff:
        _refuse("logits: too many rows or columns")
    dev, f32, i32 = logits.get_device(), torch.float32, torch.int32
    _enqueue(dev, stream, _lib.mfs_sample_rows, logits.data_ptr(), _dtype_code(logits), rows, cols,
             logits.stride(0) if rows > 1 else cols, _array(temperature, "temperature", rows, f32, dev),
             _array(top_k, "top_k", rows, i32, dev), _array(top_p, "top_p", rows, f32, dev),
             _array(min_p, "min_p", rows, f32, dev), _array(uniforms, "uniforms", rows, f32, dev),
             _array(tokens, "tokens", rows, i32, dev))


class PagedKV:
    """One layer's paged key/value cache (mfs_paged_kv): k, v [n_pages, n_kv_heads, page_size,
    head_dim] CUDA tensors of equal strides with dense rows, table [n_seqs, pages] int32.  Keeps the
    tensors; what they hold may change between calls."""

    def __init__(self, k, v, table):
        import torch
        if not k.is_cuda or k.dim() != 4 or v.shape != k.shape or v.dtype != k.dtype or v.device != k.device:
            _refuse("cache: need k and v [n_pages, n_kv_heads, page_size, head_dim] of one type on one CUDA device")
        if k.stride(3) != 1 or v.stride(3) != 1 or any(k.shape[i] > 1 and k.stride(i) != v.stride(i) for i in range(3)):
            _refuse("cache: need dense rows, and equal strides in k and v")
        if table.dim() != 2 or table.dtype != torch.int32 or table.device != k.device or (table.shape[1] > 1 and table.stride(1) != 1):
            _refuse("cache: need an int32 table [n_seqs, pages] with unit column stride on the cache's device")
        if max(*k.shape, *table.shape) > 0x7fffffff:
            _refuse("cache: too many pages")
        self.k, self.v, self.table = k, v, table
        self.device, self.n_seqs = k.device, table.shape[0]
        stride = [k.stride(i) if k.shape[i] > 1 else 0 for i in range(3)]
        self.c = mfs_paged_kv(k=k.data_ptr(), v=v.data_ptr(), table=table.data_ptr(), table_width=table.shape[1],
                              table_stride=table.stride(0) if table.shape[0] > 1 else 0, n_pages=k.shape[0], page_size=k.shape[2],
                              n_kv_heads=k.shape[1], head_dim=k.shape[3], dtype=_dtype_code(k), page_stride=stride[0],
                              head_stride=stride[1], row_stride=stride[2])
        # what each call compares its tensors with
        self._is = (k.get_device(), k.dtype, k.shape[1], k.shape[3])


def mfs_kv_append(cache: PagedKV, k, v, cu, kv_len, q=None, q_out=None, k_out=None, rope="interleaved", theta=10000.0,
                  stream=None) -> None:
    """Write the tokens' keys (rotated) and values k, v [tokens, n_kv_heads, head_dim] into the cache at
    their positions, and their rotated queries q [tokens, n_q_heads, head_dim] and keys into q_out and
    k_out.  cu [n_seqs + 1], kv_len [n_seqs]: int32 CUDA tensors; kv_len counts the new tokens.
    rope: "interleaved", "half" or None (see include/mfs.h)."""
    import torch
    dev, dtype, hkv, hd = cache._is
    n, n_seqs, i32 = k.size(0), kv_len.size(0), torch.int32
    if rope not in MFS_ROPE:
        _refuse(f"rope: one of {list(MFS_ROPE)}")
    if (q is None) != (q_out is None):
        _refuse("q and q_out go together")
    if n_seqs > cache.n_seqs:
        _refuse("the cache's table has fewer rows than kv_len")
    kp, ks = _rows(k, "k", n, hkv, hd, dtype, dev)
    vp, vs = _rows(v, "v", n, hkv, hd, dtype, dev)
    op, os_ = (None, 0) if k_out is None else _rows(k_out, "k_out", n, hkv, hd, dtype, dev)
    qp, qs, hq, xp, xs = None, 0, 0, None, 0
    if q is not None:
        hq = q.size(1)
        qp, qs = _rows(q, "q", n, hq, hd, dtype, dev)
        xp, xs = _rows(q_out, "q_out", n, hq, hd, dtype, dev)
    _enqueue(dev, stream, _lib.mfs_kv_append, cache.c, n, n_seqs, _array(cu, "cu", n_seqs + 1, i32, dev),
             _array(kv_len, "kv_len", n_seqs, i32, dev), qp, qs, hq, xp, xs, kp, ks, op, os_, vp, vs, MFS_ROPE[rope], theta)


def mfs_paged_attention_workspace(cache: PagedKV, n_q_heads: int):
    """A workspace tensor for mfs_paged_attention of this cache (see include/mfs.h on sharing it)."""
    import torch
    return torch.empty(_lib.mfs_paged_attention_workspace(cache.c, n_q_heads), dtype=torch.uint8, device=cache.device)


def mfs_paged_attention(cache: PagedKV, q, kv_len, out, scale=None, window=0, workspace=None, stream=None) -> None:
    """Attention of one new token per sequence, q and out [n_seqs, n_q_heads, head_dim], over the cache's
    first kv_len[s] positions (the last `window` of them if it is not 0).  scale: default
    head_dim ** -0.5.  workspace: default one of its own for this call."""
    import torch
    dev, dtype, _, hd = cache._is
    n, hq = q.size(0), q.size(1)
    if n > cache.n_seqs:
        _refuse("the cache's table has fewer rows than q")
    qp, qs = _rows(q, "q", n, hq, hd, dtype, dev)
    op, os_ = _rows(out, "out", n, hq, hd, dtype, dev)
    if workspace is None:
        if stream is None:
            workspace = mfs_paged_attention_workspace(cache, hq)
        else:  # from the pool of the stream that uses it, so that it is not handed out again too early
            # (ExternalStream takes the null stream's handle for none given)
            own = torch.cuda.ExternalStream(stream, device=cache.device) if stream else torch.cuda.default_stream(cache.device)
            with torch.cuda.stream(own):
                workspace = mfs_paged_attention_workspace(cache, hq)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        _refuse("workspace: need a contiguous tensor on the cache's device")
    _enqueue(dev, stream, _lib.mfs_paged_attention, cache.c, n, _array(kv_len, "kv_len", n, torch.int32, dev), qp, qs, hq, op, os_,
             hd ** -0.5 if scale is None else scale, _window(window), workspace.data_ptr(), workspace.nbytes)


def mfs_prompt_attention(q, k, v, cu, out, scale=None, window=0, stream=None) -> None:
    """Causal attention of packed prompts: q, out [tokens, n_q_heads, head_dim], k, v [tokens, n_kv_heads,
    head_dim] CUDA tensors (fp32 or bf16), sequence s = tokens cu[s] .. cu[s + 1] - 1; the last `window`
    keys of each row if it is not 0.  scale: default head_dim ** -0.5 (see include/mfs.h)."""
    import torch
    if not q.is_cuda or q.dim() != 3 or k.dim() != 3 or cu.dim() != 1 or cu.size(0) < 1:
        _refuse("need CUDA tensors [tokens, heads, head_dim] and cu [n_seqs + 1]")
    (n, hq, hd), hkv, n_seqs, dev, dtype = q.shape, k.size(1), cu.size(0) - 1, q.get_device(), q.dtype
    qp, qs = _rows(q, "q", n, hq, hd, dtype, dev)
    kp, ks = _rows(k, "k", n, hkv, hd, dtype, dev)
    vp, vs = _rows(v, "v", n, hkv, hd, dtype, dev)
    op, os_ = _rows(out, "out", n, hq, hd, dtype, dev)
    _enqueue(dev, stream, _lib.mfs_prompt_attention, _dtype_code(q), n, n_seqs, _array(cu, "cu", n_seqs + 1, torch.int32, dev), qp, qs, hq,
             kp, ks, vp, vs, hkv, hd, op, os_, hd ** -0.5 if scale is None else scale, _window(window))
