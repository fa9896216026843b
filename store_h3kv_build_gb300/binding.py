"""Thin Python binding over ``libh3kv.so`` (the C ABI in ``include/h3kv.h``).

Argument marshalling only: torch tensors are used for device memory and the
current CUDA stream, their pointers and sizes go through ctypes, and every
step of the computation runs in the library's CUDA kernels.  Importing this
module loads the library and raises ImportError if it has not been built
(``python -m store_h3kv_build_gb300.build_lib``); there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libh3kv.so")
if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m store_h3kv_build_gb300.build_lib`")
_lib = ctypes.CDLL(LIB_PATH)

HEAD_DIM = 128
DEFAULT_KV_BLOCK = 16384
KV_TILE = 128
H3KV_STATIC_SCRATCH_BYTES = 32 * 1024 * 1024  # the fixed scratch of h3kv_attend_staged_static

H3KV_OK = 0
H3KV_ERR_INVALID_ARG = 1
H3KV_ERR_UNSUPPORTED = 2
H3KV_ERR_CUDA = 3
H3KV_ERR_DEVICE_TIMEOUT = 4
H3KV_ERR_DEVICE_DATA = 5
PAGE_SIZES = (16, 32, 64, 128)
TREE_MAX_NODES = 64


class h3kv_store(ctypes.Structure):  # noqa: N801 - mirrors the C struct name
    _fields_ = [
        ("k_codes", ctypes.c_void_p),
        ("v_codes", ctypes.c_void_p),
        ("k_scales", ctypes.c_void_p),
        ("v_scales", ctypes.c_void_p),
        ("heads", ctypes.c_int32),
        ("seq", ctypes.c_int64),
        ("head_dim", ctypes.c_int32),
        ("scale_group", ctypes.c_int32),
    ]


class h3kv_store_f8(ctypes.Structure):  # noqa: N801 - mirrors the C struct name
    _fields_ = [
        ("k_codes", ctypes.c_void_p),
        ("v_codes_t", ctypes.c_void_p),
        ("k_scales", ctypes.c_void_p),
        ("v_scales", ctypes.c_void_p),
        ("k_mean", ctypes.c_void_p),
        ("heads", ctypes.c_int32),
        ("seq", ctypes.c_int64),
        ("head_dim", ctypes.c_int32),
    ]


class h3kv_store_fp4(ctypes.Structure):  # noqa: N801 - mirrors the C struct name
    _fields_ = [
        ("k_codes", ctypes.c_void_p),
        ("v_codes", ctypes.c_void_p),
        ("k_scales", ctypes.c_void_p),
        ("v_scales", ctypes.c_void_p),
        ("heads", ctypes.c_int32),
        ("seq", ctypes.c_int64),
        ("head_dim", ctypes.c_int32),
    ]


class h3kv_rows(ctypes.Structure):  # noqa: N801 - mirrors the C struct name
    _fields_ = [
        ("data", ctypes.c_void_p),
        ("head_stride", ctypes.c_int64),
        ("row_stride", ctypes.c_int64),
    ]


class h3kv_paged_store(ctypes.Structure):  # noqa: N801 - mirrors the C struct name
    _fields_ = [
        ("k_codes", ctypes.c_void_p),
        ("v_codes", ctypes.c_void_p),
        ("k_scales", ctypes.c_void_p),
        ("v_scales", ctypes.c_void_p),
        ("pages", ctypes.c_int32),
        ("kv_heads", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
    ]


_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_rows, _paged = ctypes.POINTER(h3kv_rows), ctypes.POINTER(h3kv_paged_store)
_SIGS = {
    "h3kv_abi_version": (ctypes.c_uint32, []),
    "h3kv_store_bytes": (ctypes.c_size_t, [_i32, _i64, _i32]),
    "h3kv_build_store": (ctypes.c_int, [_vp, _vp, _i32, _i64, _i32, ctypes.POINTER(h3kv_store), _vp]),
    "h3kv_attend": (ctypes.c_int, [_vp, _i64, ctypes.POINTER(h3kv_store), _i32, _i32, _f32, _vp, _vp]),
    "h3kv_attend_exact": (ctypes.c_int, [_vp, _i64, _vp, _vp, _i32, _i64, _i32, _i32, _i32, _f32, _vp, _vp]),
    "h3kv_sync_status": (ctypes.c_int, [_vp]),
    "h3kv_staging_bytes": (ctypes.c_size_t, [_i32, _i32]),
    "h3kv_attend_staged_static": (ctypes.c_int, [_vp, _i64, ctypes.POINTER(h3kv_store), _i32, _i32, _f32, _vp,
                                                 _vp]),
    "h3kv_attend_staged": (ctypes.c_int, [_vp, _i64, ctypes.POINTER(h3kv_store), _i32, _i32, _f32, _vp, _vp,
                                          ctypes.c_size_t, _vp, _vp]),
    "h3kv_hostio_scratch_bytes": (ctypes.c_size_t, [_i32, _i32]),
    "h3kv_attend_hostio": (ctypes.c_int, [_vp, _i64, ctypes.POINTER(h3kv_store), _i32, _i32, _f32, _vp, _vp,
                                          ctypes.c_size_t, _vp]),
    "h3kv_f8_v_stride": (ctypes.c_int64, [_i64]),
    "h3kv_store_f8_bytes": (ctypes.c_size_t, [_i32, _i64, _i32]),
    "h3kv_build_store_f8": (ctypes.c_int, [_vp, _vp, _i32, _i64, _i32, ctypes.POINTER(h3kv_store_f8), _vp]),
    "h3kv_attend_f8": (ctypes.c_int, [_vp, _i64, ctypes.POINTER(h3kv_store_f8), _i32, _i32, _f32, _vp, _vp]),
    "h3kv_store_fp4_bytes": (ctypes.c_size_t, [_i32, _i64, _i32]),
    "h3kv_build_store_fp4": (ctypes.c_int, [_vp, _vp, _i32, _i64, _i32, ctypes.POINTER(h3kv_store_fp4), _vp]),
    "h3kv_attend_fp4": (ctypes.c_int, [_vp, _i64, ctypes.POINTER(h3kv_store_fp4), _i32, _i32, _f32, _vp, _vp]),
    "h3kv_set_wait_timeout_ns": (ctypes.c_int, [ctypes.c_uint64]),
    "h3kv_selftest_wait_timeout": (ctypes.c_int, [ctypes.c_uint64, _vp]),
    "h3kv_selftest_tmem_ld_max": (ctypes.c_int, [ctypes.POINTER(ctypes.c_int32), _vp]),
    "h3kv_attend_launch_count": (ctypes.c_int64, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32]),
    "h3kv_debug_withhold_p": (ctypes.c_int, [ctypes.c_int32]),
    "h3kv_strerror": (ctypes.c_char_p, [ctypes.c_int]),
    "h3kv_paged_store_bytes": (ctypes.c_size_t, [_i32, _i32, _i32, _i32]),
    "h3kv_paged_append": (ctypes.c_int, [_rows, _rows, _vp, _i64, _paged, _vp]),
    "h3kv_paged_read": (ctypes.c_int, [_paged, _vp, _i64, _rows, _rows, _vp]),
    "h3kv_paged_copy": (ctypes.c_int, [_paged, _vp, _vp, _i64, _vp]),
    "h3kv_paged_keep": (ctypes.c_int, [_paged, _vp, _i64, _vp, _vp, _i32, _vp, _i64, _vp, _vp]),
    "h3kv_attend_tree_workspace_bytes": (ctypes.c_size_t, [_i32, _i32, _i64, _i32]),
    "h3kv_attend_tree": (ctypes.c_int, [_rows, _i32, _i64, _paged, _vp, _i64, _vp, _vp, _i32, _vp, _f32, _rows, _vp,
                                        _vp, ctypes.c_size_t, _vp]),
    "h3kv_attend_prompt": (ctypes.c_int, [_rows, _i32, _i64, _rows, _rows, _i32, _i64, _vp, _vp, _i32, _i32, _f32,
                                          _rows, _vp, _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args
    globals()[_name] = _fn

EXPORTED = tuple(_SIGS)


class H3kvError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {h3kv_strerror(status).decode()} (status {status})")


def check(status: int, where: str = "h3kv") -> None:
    if status != H3KV_OK:
        raise H3kvError(status, where)


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _need(t, name: str, dtype, shape=None) -> None:
    """Argument check: the library reads and writes raw contiguous buffers of
    the sizes its arguments imply, so a strided view, another dtype or a
    buffer of another shape would be read as garbage or written past its end."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(int(x) for x in shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(int(x) for x in shape)}")


def _need_rows(t, name: str, heads: int | None = None) -> None:
    """bf16 [heads, rows, 128] input (Q, K or V)."""
    _need(t, name, torch.bfloat16)
    if t.dim() != 3 or t.shape[2] != HEAD_DIM:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [heads, rows, {HEAD_DIM}]")
    if heads is not None and t.shape[0] != heads:
        raise ValueError(f"{name}: {t.shape[0]} heads, the store has {heads}")


def _need_out(out, Q) -> None:
    _need(out, "out", torch.float32, Q.shape)


def _stream(stream=None) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _on(stream=None):
    """Context for the device tensors the binding allocates for a call
    (outputs, stores, scratch): the call's stream, so that PyTorch's caching
    allocator hands a freed block to new work only after that stream's work
    on it -- a scratch dropped when the call returns is still in use there."""
    return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()


class Store:
    """A kvi8r store held in torch tensors: int8 codes [heads, seq, 128] and
    fp16 scales [heads, seq] for K and for V."""

    def __init__(self, k_codes, v_codes, k_scales, v_scales):
        self.k_codes, self.v_codes = k_codes, v_codes
        self.k_scales, self.v_scales = k_scales, v_scales
        self.heads, self.seq = int(k_codes.shape[0]), int(k_codes.shape[1])
        # [heads, seq] scales: one per row; [heads, seq, 4]: one per 32 values
        self.scale_group = 32 if k_scales.dim() == 3 else 0

    @classmethod
    def empty(cls, heads: int, seq: int, device="cuda", host: bool = False, scale_group: int = 0) -> "Store":
        """Uninitialised store buffers.  ``host=True`` places them in pinned
        host memory: on a Grace-Blackwell node the kernels read (and the
        store build writes) them directly over NVLink-C2C, so the whole
        sequence's K/V need not occupy HBM."""
        if host:
            kw = dict(pin_memory=True)
        else:
            kw = dict(device=device)
        # every buffer allocated with its own pin_memory request: empty_like
        # of a pinned tensor is pageable, and h3kv_attend_staged refuses a
        # store with pageable buffers
        sshape = (heads, seq, HEAD_DIM // 32) if scale_group == 32 else (heads, seq)
        kc, vc = (torch.empty((heads, seq, HEAD_DIM), dtype=torch.int8, **kw) for _ in range(2))
        ks, vs = (torch.empty(sshape, dtype=torch.float16, **kw) for _ in range(2))
        return cls(kc, vc, ks, vs)

    @property
    def in_host_memory(self) -> bool:
        return not self.k_codes.is_cuda

    def c_struct(self) -> h3kv_store:
        H, L = self.heads, self.seq
        _need(self.k_codes, "store.k_codes", torch.int8, (H, L, HEAD_DIM))
        _need(self.v_codes, "store.v_codes", torch.int8, (H, L, HEAD_DIM))
        sshape = (H, L, HEAD_DIM // 32) if self.scale_group == 32 else (H, L)
        _need(self.k_scales, "store.k_scales", torch.float16, sshape)
        _need(self.v_scales, "store.v_scales", torch.float16, sshape)
        return h3kv_store(_ptr(self.k_codes), _ptr(self.v_codes), _ptr(self.k_scales), _ptr(self.v_scales),
                          self.heads, self.seq, HEAD_DIM, self.scale_group)

    def nbytes(self) -> int:
        return int(h3kv_store_bytes(self.heads, self.seq, HEAD_DIM))


def build_store(K: torch.Tensor, V: torch.Tensor, out: Store | None = None, stream=None,
                scale_group: int = 0) -> Store:
    """h3kv_build_store on bf16 K, V [heads, seq, 128] (CUDA, contiguous);
    scale_group 32 gives one scale per 32 rotated values."""
    _need_rows(K, "K")
    _need_rows(V, "V")
    if V.shape != K.shape:
        raise ValueError(f"V: shape {tuple(V.shape)}, K has {tuple(K.shape)}")
    heads, seq = int(K.shape[0]), int(K.shape[1])
    with _on(stream):
        out = Store.empty(heads, seq, K.device, scale_group=scale_group) if out is None else out
    st = out.c_struct()
    check(h3kv_build_store(_ptr(K), _ptr(V), heads, seq, int(K.shape[2]), ctypes.byref(st), _stream(stream)),
          "h3kv_build_store")
    return out


def attend(Q: torch.Tensor, store: Store, q_chunk: int = 16384, kv_block: int = 0, softmax_scale: float = 0.0,
           out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """h3kv_attend: kvi8r attention of bf16 Q [heads, q_seq, 128] over `store`
    -> fp32 [heads, q_seq, 128]."""
    _need_rows(Q, "Q", store.heads)
    q_seq = int(Q.shape[1])
    with _on(stream):
        out = torch.empty(Q.shape, dtype=torch.float32, device=Q.device) if out is None else out
    _need_out(out, Q)
    st = store.c_struct()
    check(h3kv_attend(_ptr(Q), q_seq, ctypes.byref(st), int(q_chunk), int(kv_block), float(softmax_scale),
                      _ptr(out), _stream(stream)), "h3kv_attend")
    return out


def staging_bytes_double(heads: int, kv_block: int) -> int:
    """Staging bytes with room for two kv_blocks (h3kv_attend_staged then
    copies the next block while attending the current one)."""
    need = int(h3kv_staging_bytes(int(heads), int(kv_block)))
    return (need + 255) // 256 * 256 + need


def attend_staged(Q: torch.Tensor, store: Store, q_chunk: int = 16384, kv_block: int = 0,
                  softmax_scale: float = 0.0, out: torch.Tensor | None = None, staging: torch.Tensor | None = None,
                  state: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """h3kv_attend_staged: kvi8r attention over a store held outside HBM (e.g.
    ``Store.empty(..., host=True)``), staged through HBM one kv_block at a
    time.  ``staging`` (uint8, >= h3kv_staging_bytes; with
    ``staging_bytes_double`` bytes two blocks are staged and the next block's
    copy overlaps the current block's attention) and ``state`` (fp32 [heads,
    q_seq, 2]) are device scratch; they are created here if not given (the
    staging with room for two blocks)."""
    _need_rows(Q, "Q", store.heads)
    dev = Q.device
    heads, q_seq = int(Q.shape[0]), int(Q.shape[1])
    with _on(stream):
        out = torch.empty(Q.shape, dtype=torch.float32, device=dev) if out is None else out
        if staging is None:
            staging = torch.empty(max(staging_bytes_double(store.heads, int(kv_block)), 16), dtype=torch.uint8,
                                  device=dev)
        if state is None:
            state = torch.empty((heads, q_seq, 2), dtype=torch.float32, device=dev)
    _need_out(out, Q)
    _need(staging, "staging", torch.uint8)
    _need(state, "state", torch.float32, (int(Q.shape[0]), int(Q.shape[1]), 2))
    st = store.c_struct()
    check(h3kv_attend_staged(_ptr(Q), q_seq, ctypes.byref(st), int(q_chunk), int(kv_block), float(softmax_scale),
                             _ptr(out), _ptr(staging), staging.numel() * staging.element_size(), _ptr(state),
                             _stream(stream)), "h3kv_attend_staged")
    return out


def attend_hostio(Q_host: torch.Tensor, store: Store, q_chunk: int = 16384, kv_block: int = 0,
                  softmax_scale: float = 0.0, out: torch.Tensor | None = None, scratch: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """h3kv_attend_hostio: kvi8r attention of bf16 Q in (pinned) host memory
    over a device store, streamed through HBM per query chunk; the fp32
    output lands in host memory (``out``, pinned, created here if not
    given).  ``scratch`` (uint8 device, >= h3kv_hostio_scratch_bytes) is
    created here if not given."""
    _need_rows(Q_host, "Q_host", store.heads)
    heads, q_seq = int(Q_host.shape[0]), int(Q_host.shape[1])
    if out is None:
        out = torch.empty(Q_host.shape, dtype=torch.float32, pin_memory=True)
    if scratch is None:
        dev = store.k_codes.device
        with _on(stream):
            scratch = torch.empty(max(int(h3kv_hostio_scratch_bytes(heads, int(q_chunk))), 16), dtype=torch.uint8,
                                  device=dev)
    _need_out(out, Q_host)
    _need(scratch, "scratch", torch.uint8)
    st = store.c_struct()
    check(h3kv_attend_hostio(_ptr(Q_host), q_seq, ctypes.byref(st), int(q_chunk), int(kv_block),
                             float(softmax_scale), _ptr(out), _ptr(scratch), scratch.numel(), _stream(stream)),
          "h3kv_attend_hostio")
    return out


def attend_exact(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, q_chunk: int = 16384, kv_block: int = 0,
                 softmax_scale: float = 0.0, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """h3kv_attend_exact: softmax attention on bf16 Q, K, V -> fp32."""
    _need_rows(K, "K")
    _need_rows(V, "V")
    if V.shape != K.shape:
        raise ValueError(f"V: shape {tuple(V.shape)}, K has {tuple(K.shape)}")
    _need_rows(Q, "Q", int(K.shape[0]))
    with _on(stream):
        out = torch.empty(Q.shape, dtype=torch.float32, device=Q.device) if out is None else out
    _need_out(out, Q)
    check(h3kv_attend_exact(_ptr(Q), int(Q.shape[1]), _ptr(K), _ptr(V), int(K.shape[0]), int(K.shape[1]),
                            int(K.shape[2]), int(q_chunk), int(kv_block), float(softmax_scale), _ptr(out),
                            _stream(stream)), "h3kv_attend_exact")
    return out


K_BLOCK_F8 = 64


class StoreF8:
    """A kvf8s store held in torch tensors: e4m3 K codes [heads, seq, 128]
    (uint8), channel-major e4m3 V codes [heads, 128, v_stride], fp32 K block
    scales [heads, ceil(seq / 64)], fp32 V channel scales and K means
    [heads, 128]."""

    def __init__(self, k_codes, v_codes_t, k_scales, v_scales, k_mean, seq: int):
        self.k_codes, self.v_codes_t = k_codes, v_codes_t
        self.k_scales, self.v_scales, self.k_mean = k_scales, v_scales, k_mean
        self.heads, self.seq = int(k_codes.shape[0]), int(seq)

    @classmethod
    def empty(cls, heads: int, seq: int, device="cuda") -> "StoreF8":
        vstride = int(h3kv_f8_v_stride(seq))
        nblk = (seq + K_BLOCK_F8 - 1) // K_BLOCK_F8
        kc = torch.empty((heads, seq, HEAD_DIM), dtype=torch.uint8, device=device)
        vt = torch.empty((heads, HEAD_DIM, vstride), dtype=torch.uint8, device=device)
        ks = torch.empty((heads, nblk), dtype=torch.float32, device=device)
        vs = torch.empty((heads, HEAD_DIM), dtype=torch.float32, device=device)
        km = torch.empty((heads, HEAD_DIM), dtype=torch.float32, device=device)
        return cls(kc, vt, ks, vs, km, seq)

    def c_struct(self) -> h3kv_store_f8:
        H, L = self.heads, self.seq
        _need(self.k_codes, "store.k_codes", torch.uint8, (H, L, HEAD_DIM))
        _need(self.v_codes_t, "store.v_codes_t", torch.uint8, (H, HEAD_DIM, int(h3kv_f8_v_stride(L))))
        _need(self.k_scales, "store.k_scales", torch.float32, (H, (L + K_BLOCK_F8 - 1) // K_BLOCK_F8))
        _need(self.v_scales, "store.v_scales", torch.float32, (H, HEAD_DIM))
        _need(self.k_mean, "store.k_mean", torch.float32, (H, HEAD_DIM))
        return h3kv_store_f8(_ptr(self.k_codes), _ptr(self.v_codes_t), _ptr(self.k_scales), _ptr(self.v_scales),
                             _ptr(self.k_mean), self.heads, self.seq, HEAD_DIM)

    def nbytes(self) -> int:
        return int(h3kv_store_f8_bytes(self.heads, self.seq, HEAD_DIM))


def build_store_f8(K: torch.Tensor, V: torch.Tensor, out: StoreF8 | None = None, stream=None) -> StoreF8:
    """h3kv_build_store_f8 on bf16 K, V [heads, seq, 128] (CUDA, contiguous)."""
    _need_rows(K, "K")
    _need_rows(V, "V")
    if V.shape != K.shape:
        raise ValueError(f"V: shape {tuple(V.shape)}, K has {tuple(K.shape)}")
    heads, seq = int(K.shape[0]), int(K.shape[1])
    with _on(stream):
        out = StoreF8.empty(heads, seq, K.device) if out is None else out
    st = out.c_struct()
    check(h3kv_build_store_f8(_ptr(K), _ptr(V), heads, seq, int(K.shape[2]), ctypes.byref(st), _stream(stream)),
          "h3kv_build_store_f8")
    return out


def attend_f8(Q: torch.Tensor, store: StoreF8, q_chunk: int = 16384, kv_block: int = 0, softmax_scale: float = 0.0,
              out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """h3kv_attend_f8: kvf8s attention of bf16 Q [heads, q_seq, 128] -> fp32."""
    _need_rows(Q, "Q", store.heads)
    q_seq = int(Q.shape[1])
    with _on(stream):
        out = torch.empty(Q.shape, dtype=torch.float32, device=Q.device) if out is None else out
    _need_out(out, Q)
    st = store.c_struct()
    check(h3kv_attend_f8(_ptr(Q), q_seq, ctypes.byref(st), int(q_chunk), int(kv_block), float(softmax_scale),
                         _ptr(out), _stream(stream)), "h3kv_attend_f8")
    return out


class StoreFp4:
    """A kvfp4 store held in torch tensors: packed e2m1 codes [heads, seq, 64]
    (uint8, element 2i in the low nibble of byte i) and e4m3 block scales
    [heads, seq, 8] (uint8) for K and for V."""

    def __init__(self, k_codes, v_codes, k_scales, v_scales):
        self.k_codes, self.v_codes = k_codes, v_codes
        self.k_scales, self.v_scales = k_scales, v_scales
        self.heads, self.seq = int(k_codes.shape[0]), int(k_codes.shape[1])

    @classmethod
    def empty(cls, heads: int, seq: int, device="cuda") -> "StoreFp4":
        kc = torch.empty((heads, seq, HEAD_DIM // 2), dtype=torch.uint8, device=device)
        ks = torch.empty((heads, seq, HEAD_DIM // 16), dtype=torch.uint8, device=device)
        return cls(kc, torch.empty_like(kc), ks, torch.empty_like(ks))

    def c_struct(self) -> h3kv_store_fp4:
        H, L = self.heads, self.seq
        _need(self.k_codes, "store.k_codes", torch.uint8, (H, L, HEAD_DIM // 2))
        _need(self.v_codes, "store.v_codes", torch.uint8, (H, L, HEAD_DIM // 2))
        _need(self.k_scales, "store.k_scales", torch.uint8, (H, L, HEAD_DIM // 16))
        _need(self.v_scales, "store.v_scales", torch.uint8, (H, L, HEAD_DIM // 16))
        return h3kv_store_fp4(_ptr(self.k_codes), _ptr(self.v_codes), _ptr(self.k_scales), _ptr(self.v_scales),
                              self.heads, self.seq, HEAD_DIM)

    def nbytes(self) -> int:
        return int(h3kv_store_fp4_bytes(self.heads, self.seq, HEAD_DIM))


def build_store_fp4(K: torch.Tensor, V: torch.Tensor, out: StoreFp4 | None = None, stream=None) -> StoreFp4:
    """h3kv_build_store_fp4 on bf16 K, V [heads, seq, 128] (CUDA, contiguous)."""
    _need_rows(K, "K")
    _need_rows(V, "V")
    if V.shape != K.shape:
        raise ValueError(f"V: shape {tuple(V.shape)}, K has {tuple(K.shape)}")
    heads, seq = int(K.shape[0]), int(K.shape[1])
    with _on(stream):
        out = StoreFp4.empty(heads, seq, K.device) if out is None else out
    st = out.c_struct()
    check(h3kv_build_store_fp4(_ptr(K), _ptr(V), heads, seq, int(K.shape[2]), ctypes.byref(st), _stream(stream)),
          "h3kv_build_store_fp4")
    return out


def attend_fp4(Q: torch.Tensor, store: StoreFp4, q_chunk: int = 16384, kv_block: int = 0,
               softmax_scale: float = 0.0, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """h3kv_attend_fp4: kvfp4 attention of bf16 Q [heads, q_seq, 128] -> fp32."""
    _need_rows(Q, "Q", store.heads)
    q_seq = int(Q.shape[1])
    with _on(stream):
        out = torch.empty(Q.shape, dtype=torch.float32, device=Q.device) if out is None else out
    _need_out(out, Q)
    st = store.c_struct()
    check(h3kv_attend_fp4(_ptr(Q), q_seq, ctypes.byref(st), int(q_chunk), int(kv_block), float(softmax_scale),
                          _ptr(out), _stream(stream)), "h3kv_attend_fp4")
    return out


# ------------------------------------------------------- serving operators --
def _need_strided(t, name: str, heads: int | None = None, rows: int | None = None) -> h3kv_rows:
    """bf16 [heads, rows, 128] whose 128 values are contiguous; heads and rows
    may lie at any stride that is a multiple of 8 elements (a projection's
    output [rows, heads, 128] is passed as its transpose(0, 1))."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name}: dtype {t.dtype}, expected torch.bfloat16")
    shape = t.shape
    if len(shape) != 3 or shape[2] != HEAD_DIM:
        raise ValueError(f"{name}: shape {tuple(shape)}, expected [heads, rows, {HEAD_DIM}]")
    h, r, _ = shape
    if heads is not None and h != heads:
        raise ValueError(f"{name}: {h} heads, expected {heads}")
    if rows is not None and r != rows:
        raise ValueError(f"{name}: {r} rows, expected {rows}")
    hs, rs, inner = t.stride()
    ptr = t.data_ptr()
    if (inner != 1 or ptr % 16) and h and r:
        raise ValueError(f"{name}: the last dimension must be contiguous" if inner != 1
                         else f"{name}: must be 16-byte aligned")
    # the stride of a dimension of one entry is never used
    if h <= 1:
        hs = 0
    elif (hs % 8 or hs < HEAD_DIM) and r:
        raise ValueError(f"{name}: stride {hs} of dimension 0 must be a multiple of 8, at least {HEAD_DIM}")
    if r <= 1:
        rs = 0
    elif (rs % 8 or rs < HEAD_DIM) and h:
        raise ValueError(f"{name}: stride {rs} of dimension 1 must be a multiple of 8, at least {HEAD_DIM}")
    return h3kv_rows(ptr, hs, rs)


def _need_index(t, name: str, shape=None, dtype=torch.int32) -> None:
    # (the long way round only for the message of a refusal)
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_contiguous()
            and (shape is None or t.shape == shape)):
        _need(t, name, dtype, shape)


def _need_apart(out, **inputs) -> None:
    """An output may not share memory with an input that other CTAs still
    read; tensors of one storage are refused where their extents meet."""
    if out is None or out.numel() == 0:
        return

    def extent(t):
        last = sum((n - 1) * abs(st) for n, st in zip(t.shape, t.stride()))
        return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()

    a0, a1 = extent(out)
    for name, t in inputs.items():
        if t is None or t.numel() == 0:
            continue
        b0, b1 = extent(t)
        if a0 < b1 and b0 < a1 and t.device == out.device:
            raise ValueError(f"out: shares memory with {name}")


def _check_apart(status: int, where: str, outs: dict, ins: dict) -> None:
    """check() of a call that refuses outputs over its inputs or over one
    another; says which where that is why."""
    if status == H3KV_ERR_INVALID_ARG:
        outs = {n: t for n, t in outs.items() if t is not None}
        for i, t in enumerate(outs.values()):
            others = {"another output" if n == "out" else n: x for n, x in list(outs.items())[:i]}
            _need_apart(t, **ins, **others)
    check(status, where)


def _one_device(stream, first, *others) -> int:
    """The index of the CUDA device that every tensor of a call (and the
    stream) is on."""
    dev = first.get_device()
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors must lie on one CUDA device: {first.device} and {t.device}")
    if dev < 0:
        raise ValueError(f"tensors must lie on one CUDA device: {first.device}")
    if stream is not None and stream.device.index != dev:
        raise ValueError(f"stream of {stream.device}, tensors on cuda:{dev}")
    return dev


# The current stream's handle without building a Stream object (a tenth of the
# time of torch.cuda.current_stream), where this PyTorch has the call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = torch.cuda.current_device


def _handle(dev: int, stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream


def _on_device(dev: int, call, *args, **kw):
    """The call again with `dev` as the current device."""
    with torch.cuda.device(dev):
        return call(*args, **kw)


def _new(stream, like: torch.Tensor, shape, dtype) -> torch.Tensor:
    """An uninitialised tensor on `like`'s device, allocated on the call's
    stream (see _on).  (torch.empty: new_empty takes twice its time.)"""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _new_rows(stream, like: torch.Tensor, heads: int, rows: int) -> tuple[torch.Tensor, h3kv_rows]:
    """A bf16 [heads, rows, 128] result and its C struct."""
    out = _new(stream, like, (heads, rows, HEAD_DIM), torch.bfloat16)
    return out, h3kv_rows(out.data_ptr(), rows * HEAD_DIM if heads > 1 else 0, HEAD_DIM if rows > 1 else 0)


@functools.lru_cache(maxsize=256)
def _tree_workspace_bytes(q_heads: int, kv_heads: int, nodes: int, seqs: int) -> int:
    return max(h3kv_attend_tree_workspace_bytes(q_heads, kv_heads, nodes, seqs), 32)


class PagedStore:
    """A kvi8r cache in pages, held in torch tensors: int8 codes [pages,
    kv_heads, page_size, 128] and fp16 scales [pages, kv_heads, page_size]
    for K and for V.  Pool row r is slot r % page_size of page
    r // page_size.  The four buffers are checked once and stay the same."""

    __slots__ = ("_buffers", "_struct", "_ref", "pages", "kv_heads", "page_size")

    def __init__(self, k_codes, v_codes, k_scales, v_scales):
        _need(k_codes, "k_codes", torch.int8)
        if k_codes.dim() != 4 or k_codes.shape[3] != HEAD_DIM:
            raise ValueError(f"k_codes: shape {tuple(k_codes.shape)}, expected [pages, kv_heads, page_size, {HEAD_DIM}]")
        shape = self.pages, self.kv_heads, self.page_size = tuple(int(x) for x in k_codes.shape[:3])
        if self.page_size not in PAGE_SIZES:
            raise ValueError(f"page_size {self.page_size}, expected one of {PAGE_SIZES}")
        _need(v_codes, "v_codes", torch.int8, (*shape, HEAD_DIM))
        _need(k_scales, "k_scales", torch.float16, shape)
        _need(v_scales, "v_scales", torch.float16, shape)
        self._buffers = (k_codes, v_codes, k_scales, v_scales)
        if len({t.device for t in self._buffers}) != 1:
            raise ValueError("the four buffers must lie on one device")
        self._struct = h3kv_paged_store(*(t.data_ptr() for t in self._buffers), *shape, HEAD_DIM)
        self._ref = ctypes.byref(self._struct)

    k_codes = property(lambda self: self._buffers[0])
    v_codes = property(lambda self: self._buffers[1])
    k_scales = property(lambda self: self._buffers[2])
    v_scales = property(lambda self: self._buffers[3])

    @classmethod
    def empty(cls, pages: int, kv_heads: int, page_size: int = 64, device="cuda") -> "PagedStore":
        """Uninitialised pages: a row holds something once it is appended."""
        kc, vc = (torch.empty((pages, kv_heads, page_size, HEAD_DIM), dtype=torch.int8, device=device)
                  for _ in range(2))
        ks, vs = (torch.empty((pages, kv_heads, page_size), dtype=torch.float16, device=device) for _ in range(2))
        return cls(kc, vc, ks, vs)

    def tensors(self) -> dict:
        return dict(zip(("k_codes", "v_codes", "k_scales", "v_scales"), self._buffers))

    def nbytes(self) -> int:
        return int(h3kv_paged_store_bytes(self.pages, self.kv_heads, self.page_size, HEAD_DIM))


def paged_append(K: torch.Tensor, V: torch.Tensor, store: PagedStore, rows: torch.Tensor, stream=None) -> None:
    """h3kv_paged_append: row i of bf16 K, V [kv_heads, n, 128] rotated,
    quantised and written to pool row rows[i] (int32 [n]; negative: left
    out).  No pool row may be named twice."""
    k = _need_strided(K, "K", store.kv_heads)
    n = K.shape[1]
    v = _need_strided(V, "V", store.kv_heads, n)
    _need_index(rows, "rows", (n,))
    dev = _one_device(stream, K, V, rows, store._buffers[0])
    if _current_device() != dev:
        return _on_device(dev, paged_append, K, V, store, rows, stream)
    st = h3kv_paged_append(ctypes.byref(k), ctypes.byref(v), rows.data_ptr(), n, store._ref, _handle(dev, stream))
    if st != H3KV_OK:
        _check_apart(st, "h3kv_paged_append", store.tensors(), dict(K=K, V=V, rows=rows))


def paged_read(store: PagedStore, rows: torch.Tensor, K: torch.Tensor | None = None, V: torch.Tensor | None = None,
               stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """h3kv_paged_read: pool rows rows[i] (int32 [n]; negative: a row of
    zeros) dequantised, un-rotated and rounded to bf16 [kv_heads, n, 128]."""
    _need_index(rows, "rows")
    if rows.dim() != 1:
        raise ValueError(f"rows: shape {tuple(rows.shape)}, expected [n]")
    n = rows.shape[0]
    dev = _one_device(stream, rows, K, V, store._buffers[0])
    if _current_device() != dev:
        return _on_device(dev, paged_read, store, rows, K, V, stream)
    if K is None:
        K, k = _new_rows(stream, rows, store.kv_heads, n)
    else:
        k = _need_strided(K, "K", store.kv_heads, n)
        _need_apart(K, rows=rows, **store.tensors())
    if V is None:
        V, v = _new_rows(stream, rows, store.kv_heads, n)
    else:
        v = _need_strided(V, "V", store.kv_heads, n)
        _need_apart(V, rows=rows, **store.tensors())
    if k.data == v.data and n and store.kv_heads:
        raise ValueError("out: K shares memory with V")
    st = h3kv_paged_read(store._ref, rows.data_ptr(), n, ctypes.byref(k), ctypes.byref(v), _handle(dev, stream))
    if st != H3KV_OK:
        _check_apart(st, "h3kv_paged_read", dict(K=K, V=V), {})
    return K, V


def paged_copy(store: PagedStore, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
    """h3kv_paged_copy: page src[i] copied to page dst[i] (int32 [n]; a pair
    with a negative entry is left out).  No page may be a dst twice, or both a
    dst and a src."""
    _need_index(src, "src")
    if src.dim() != 1:
        raise ValueError(f"src: shape {tuple(src.shape)}, expected [n]")
    _need_index(dst, "dst", src.shape)
    dev = _one_device(stream, src, dst, store._buffers[0])
    if _current_device() != dev:
        return _on_device(dev, paged_copy, store, src, dst, stream)
    st = h3kv_paged_copy(store._ref, src.data_ptr(), dst.data_ptr(), src.shape[0], _handle(dev, stream))
    if st != H3KV_OK:
        _check_apart(st, "h3kv_paged_copy", store.tensors(), dict(src=src, dst=dst))


def _need_table(page_table, lengths, cu_nodes) -> int:
    _need_index(cu_nodes, "cu_nodes")
    shape = cu_nodes.shape
    if len(shape) != 1 or shape[0] < 1:
        raise ValueError(f"cu_nodes: shape {tuple(shape)}, expected [seqs + 1]")
    seqs = shape[0] - 1
    _need_index(lengths, "lengths", (seqs,))
    _need_index(page_table, "page_table")
    if page_table.dim() != 2 or page_table.shape[0] != seqs:
        raise ValueError(f"page_table: shape {tuple(page_table.shape)}, expected [{seqs}, max_pages]")
    return seqs


def paged_keep(store: PagedStore, page_table: torch.Tensor, lengths: torch.Tensor, cu_nodes: torch.Tensor,
               keep: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """h3kv_paged_keep: of each sequence's last cu_nodes[i+1] - cu_nodes[i]
    cached rows (at most 64), those with keep (uint8 or bool [nodes]) set move
    up behind the rows before them, in order -> the lengths that are left
    (int32 [seqs]).  The pages of those rows belong to that sequence alone."""
    seqs = _need_table(page_table, lengths, cu_nodes)
    if not (isinstance(keep, torch.Tensor) and keep.dtype is torch.bool):
        _need_index(keep, "keep", dtype=torch.uint8)
    if keep.dim() != 1 or not keep.is_contiguous():
        raise ValueError(f"keep: shape {tuple(keep.shape)}, expected contiguous [nodes]")
    dev = _one_device(stream, page_table, lengths, cu_nodes, keep, out, store._buffers[0])
    if _current_device() != dev:
        return _on_device(dev, paged_keep, store, page_table, lengths, cu_nodes, keep, out, stream)
    if out is None:
        out = _new(stream, lengths, (seqs,), torch.int32)
    else:
        _need_index(out, "out", (seqs,))
        _need_apart(out, lengths=lengths, cu_nodes=cu_nodes, page_table=page_table, keep=keep)
    st = h3kv_paged_keep(store._ref, page_table.data_ptr(), page_table.shape[1], lengths.data_ptr(),
                         cu_nodes.data_ptr(), seqs, keep.data_ptr(), keep.shape[0], out.data_ptr(),
                         _handle(dev, stream))
    if st != H3KV_OK:
        _check_apart(st, "h3kv_paged_keep", dict(store.tensors(), out=out),
                     dict(page_table=page_table, lengths=lengths, cu_nodes=cu_nodes, keep=keep))
    return out


def attend_tree(Q: torch.Tensor, store: PagedStore, page_table: torch.Tensor, lengths: torch.Tensor,
                cu_nodes: torch.Tensor, parents: torch.Tensor | None = None, softmax_scale: float = 0.0,
                out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """h3kv_attend_tree: bf16 Q [q_heads, nodes, 128], the drafted nodes of
    sequence i in rows cu_nodes[i] .. cu_nodes[i+1]-1 (at most 64), attends
    over the sequence's lengths[i] cached rows, the last of which are the
    nodes themselves -> bf16 like Q.  A node sees the rows before the drafted
    ones and its own path to the root by ``parents`` (int32 [nodes]; None: a
    plain run of tokens).  ``lse`` (fp32 [q_heads, nodes]) takes the
    log-sum-exp of the scores.  ``workspace`` (uint8, >=
    h3kv_attend_tree_workspace_bytes) is created here if not given."""
    q = _need_strided(Q, "Q")
    heads, nodes, _ = Q.shape
    if store.kv_heads < 1 or heads % store.kv_heads != 0:
        raise ValueError(f"Q: {heads} heads, not a multiple of the store's {store.kv_heads}")
    seqs = _need_table(page_table, lengths, cu_nodes)
    if parents is not None:
        _need_index(parents, "parents", (nodes,))
    if lse is not None:
        _need_index(lse, "lse", (heads, nodes), torch.float32)
    dev = _one_device(stream, Q, page_table, lengths, cu_nodes, parents, out, lse, workspace, store._buffers[0])
    if _current_device() != dev:
        return _on_device(dev, attend_tree, Q, store, page_table, lengths, cu_nodes, parents, softmax_scale, out, lse,
                          workspace, stream)
    if workspace is None:
        workspace = _new(stream, Q, (_tree_workspace_bytes(heads, store.kv_heads, nodes, seqs),), torch.uint8)
    else:
        _need_index(workspace, "workspace", dtype=torch.uint8)
    if out is None:
        out, o = _new_rows(stream, Q, heads, nodes)
    else:
        o = _need_strided(out, "out", heads, nodes)
        _need_apart(out, Q=Q, lse=lse, workspace=workspace)
    st = h3kv_attend_tree(ctypes.byref(q), heads, nodes, store._ref, page_table.data_ptr(), page_table.shape[1],
                          lengths.data_ptr(), cu_nodes.data_ptr(), seqs, 0 if parents is None else parents.data_ptr(),
                          softmax_scale, ctypes.byref(o), 0 if lse is None else lse.data_ptr(),
                          workspace.data_ptr(), workspace.numel(), _handle(dev, stream))
    if st != H3KV_OK:
        _check_apart(st, "h3kv_attend_tree", dict(out=out, lse=lse, workspace=workspace),
                     dict(Q=Q, page_table=page_table, lengths=lengths, cu_nodes=cu_nodes, parents=parents,
                          **store.tensors()))
    return out


def attend_prompt(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, cu_q: torch.Tensor,
                  cu_k: torch.Tensor | None = None, causal: bool = True, softmax_scale: float = 0.0,
                  out: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """h3kv_attend_prompt: bf16 Q [q_heads, q_rows, 128] over bf16 K, V
    [kv_heads, k_rows, 128], sequences packed by cu_q and cu_k (int32
    [seqs + 1]; cu_k None: cu_q), causal from the last row back or not ->
    bf16 like Q.  ``lse`` (fp32 [q_heads, q_rows]) takes the log-sum-exp of
    the scores.  Rows of no sequence are left as they are in ``out``."""
    q, k = _need_strided(Q, "Q"), _need_strided(K, "K")
    heads, rows, _ = Q.shape
    kv_heads, k_rows, _ = K.shape
    v = _need_strided(V, "V", kv_heads, k_rows)
    if kv_heads < 1 or heads % kv_heads != 0:
        raise ValueError(f"Q: {heads} heads, not a multiple of K's {kv_heads}")
    _need_index(cu_q, "cu_q")
    shape = cu_q.shape
    if len(shape) != 1 or shape[0] < 1:
        raise ValueError(f"cu_q: shape {tuple(shape)}, expected [seqs + 1]")
    if cu_k is None:
        cu_k = cu_q
    else:
        _need_index(cu_k, "cu_k", shape)
    if lse is not None:
        _need_index(lse, "lse", (heads, rows), torch.float32)
    dev = _one_device(stream, Q, K, V, cu_q, cu_k, out, lse)
    if _current_device() != dev:
        return _on_device(dev, attend_prompt, Q, K, V, cu_q, cu_k, causal, softmax_scale, out, lse, stream)
    if out is None:
        out, o = _new_rows(stream, Q, heads, rows)
    else:
        o = _need_strided(out, "out", heads, rows)
        _need_apart(out, Q=Q, K=K, V=V, lse=lse)
    st = h3kv_attend_prompt(ctypes.byref(q), heads, rows, ctypes.byref(k), ctypes.byref(v), kv_heads, k_rows,
                            cu_q.data_ptr(), cu_k.data_ptr(), shape[0] - 1, bool(causal), softmax_scale,
                            ctypes.byref(o), 0 if lse is None else lse.data_ptr(), _handle(dev, stream))
    if st != H3KV_OK:
        _check_apart(st, "h3kv_attend_prompt", dict(out=out, lse=lse), dict(Q=Q, K=K, V=V, cu_q=cu_q, cu_k=cu_k))
    return out


def sync_status(stream=None) -> None:
    """Synchronise the stream and raise if a kernel recorded a wait timeout or
    an index out of range."""
    check(h3kv_sync_status(_stream(stream)), "h3kv_sync_status")
