"""Thin Python binding of libpagedkv (argument marshalling only).

Same names as the C ABI in ``include/pagedkv.h``. Device arguments are torch
CUDA tensors (PyTorch supplies device memory and streams); every step of the
path runs in the library's kernels. A missing library or a non-zero status
raises: there is no fallback. The calls that a step makes once a layer hand
plain arguments to the library through _marshal.so (csrc/python/marshal.cpp),
the others, and whatever is not plain, through ctypes; without that module, or
with one that was built against another torch or Python, all of them do, at 5 us
or so a call more.
"""

from __future__ import annotations

import ctypes
import os
import warnings

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpagedkv.so")

KVP_OK = 0
KVP_ERR_INVALID_ARG = -1
KVP_ERR_CUDA = -2
KVP_ERR_OUT_OF_PAGES = -3
KVP_ERR_BAD_INDEX = -4
KVP_ERR_TIMEOUT = -5

KVP_F32, KVP_BF16 = 0, 1
KVP_BLOCK_TABLE, KVP_RAW_LOCATIONS = 0, 1
KVP_ROTARY_HALF, KVP_ROTARY_INTERLEAVED = 0, 1
KVP_ROTARY_MAX_AXES = 8
KVP_ROTARY_PLAIN, KVP_ROTARY_LINEAR, KVP_ROTARY_NTK, KVP_ROTARY_BY_PARTS = 0, 1, 2, 3

_ERR_NAMES = {
    KVP_ERR_INVALID_ARG: "KVP_ERR_INVALID_ARG",
    KVP_ERR_CUDA: "KVP_ERR_CUDA",
    KVP_ERR_OUT_OF_PAGES: "KVP_ERR_OUT_OF_PAGES",
    KVP_ERR_BAD_INDEX: "KVP_ERR_BAD_INDEX",
    KVP_ERR_TIMEOUT: "KVP_ERR_TIMEOUT",
}

# Every symbol the header declares, with its C signature.
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_ll, _d = ctypes.c_longlong, ctypes.c_double
_ip = ctypes.POINTER(ctypes.c_int)
_szp = ctypes.POINTER(ctypes.c_size_t)
SIGNATURES = {
    "kv_pool_create": [_i, _i, _i, _i, _i, _i, _vp, _vp, ctypes.POINTER(_vp)],
    "kv_pool_destroy": [_vp],
    "store_cache": [_vp, _i, _vp, _vp, _vp, _i, _vp],
    "page_table_write": [_vp, _i, _i, _vp, _vp, _vp, _i, _i, _vp, _vp],
    "copy_pages": [_vp, _vp, _vp, _i, _vp],
    "paged_decode_attention_workspace_size": [_vp, _i, _i, _szp],
    "paged_decode_attention": [_vp, _i, _vp, _i, _i, _vp, _i, _i, _i, _vp, _vp, _i, _i, _f, _vp, _vp, _sz, _vp],
    "paged_verify_attention_workspace_size": [_vp, _i, _i, _i, _szp],
    "paged_verify_attention": [_vp, _i, _vp, _i, _i, _i, _vp, _i, _i, _i, _vp, _vp, _i, _i, _f, _vp, _vp, _sz, _vp],
    "paged_prefill_attention": [_vp, _i, _vp, _i, _i, _i, _vp, _vp, _i, _i, _i, _vp, _vp, _i, _i, _f, _vp, _vp],
    "paged_decode_attention_noalloc": [_vp, _i, _vp, _i, _i, _vp, _i, _i, _i, _vp, _vp, _i, _i, _f, _vp, _vp],
    "store_cache_and_attention": [_vp, _i, _vp, _vp, _vp, _vp, _i, _i, _vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _i,
                                  _i, _i, _f, _vp, _vp, _sz, _vp],
    "kv_latent_pool_create": [_i, _i, _i, _i, _i, _i, _vp, _vp, ctypes.POINTER(_vp)],
    "kvp_rotary_frequencies": [_i, _d, _i, _d, _d, _d, _d, _vp],
    "rotary_store_cache": [_vp, _i, _vp, _ll, _ll, _i, _vp, _ll, _vp, _ll, _vp, _vp, _i, _vp, _i, _i, _f, _vp, _ll, _ll,
                           _vp],
    "rotary_store_latent": [_vp, _i, _vp, _ll, _ll, _i, _vp, _ll, _vp, _ll, _vp, _vp, _i, _vp, _i, _i, _f, _vp, _ll, _ll,
                            _vp],
    "kv_fp4_pool_create": [_i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, ctypes.POINTER(_vp)],
    "rotary_store_cache_axes": [_vp, _i, _vp, _ll, _ll, _i, _vp, _ll, _vp, _ll, _vp, _ll, _vp, _i, _vp, _vp, _i, _i, _i, _f,
                                _vp, _ll, _ll, _vp],
    "rotary_store_latent_axes": [_vp, _i, _vp, _ll, _ll, _i, _vp, _ll, _vp, _ll, _vp, _ll, _vp, _i, _vp, _vp, _i, _i, _i, _f,
                                 _vp, _ll, _ll, _vp],
    "rotary_store_fp4": [_vp, _i, _vp, _ll, _ll, _i, _vp, _ll, _vp, _ll, _vp, _ll, _vp, _i, _vp, _vp, _i, _i, _i, _f, _vp, _ll,
                         _ll, _vp],
    "load_cache_fp4": [_vp, _i, _vp, _i, _vp, _vp, _vp],
    "paged_fp4_attention_workspace_size": [_vp, _i, _i, _i, _i, _szp],
    "paged_fp4_attention": [_vp, _i, _vp, _i, _i, _i, _vp, _vp, _i, _i, _i, _vp, _vp, _i, _i, _i, _f, _vp, _vp, _sz, _vp],
    "paged_latent_attention_workspace_size": [_vp, _i, _i, _i, _szp],
    "paged_latent_attention": [_vp, _i, _vp, _i, _i, _i, _vp, _vp, _i, _i, _i, _vp, _vp, _i, _i, _f, _vp, _vp, _sz, _vp],
    "latent_prefill_attention": [_vp, _ll, _ll, _vp, _ll, _ll, _vp, _ll, _vp, _ll, _ll, _vp, _vp, _i, _i, _i, _i, _i, _i,
                                 _i, _i, _i, _f, _vp, _vp, _vp],
    "gather_indices": [_vp, _vp, _i, _i, _i, _vp, _vp, _i, _i, _i, _vp, _i, _vp],
    "kvp_sync_error": [_vp, _vp, _ip],
    "kvp_selftest_wait": [ctypes.c_longlong, _i, _vp, _vp],
    "kvp_pool_set_timing_events": [_vp, _vp, _vp],
    "kvp_host_create": [_i, _i, _i, _vp, ctypes.POINTER(_vp)],
    "kvp_host_destroy": [_vp],
    "kvp_host_new": [_vp, _i],
    "kvp_host_fork": [_vp, _i, _i, _vp, _vp, _vp, _i, _ip],
    "kvp_host_release": [_vp, _i],
    "kvp_host_append": [_vp, _vp, _i, _vp, _vp, _vp, _vp, _i, _ip, _vp, _vp, _ip],
    "kvp_host_trim": [_vp, _i, _i, _vp, _vp, _vp, _i, _ip],
    "kvp_host_trim_sinks": [_vp, _i, _i, _i, _vp, _vp, _vp, _i, _ip],
    "kvp_host_rewind": [_vp, _i, _i, _vp, _vp, _vp, _i, _ip],
    "kvp_host_used": [_vp, _ip],
    "kvp_host_length": [_vp, _i, _ip, _ip],
    "kvp_host_block_row": [_vp, _i, _vp, _i, _ip],
    "kvp_host_refcounts": [_vp, _vp, _i],
    "kvp_host_free_list": [_vp, _vp, _i, _ip],
    "kvp_dev_pages_bytes": [_i, _i, _szp],
    "kvp_dev_pages_create": [_i, _i, _i, _vp, _sz, _vp, _i, _i, _i, ctypes.POINTER(_vp)],
    "kvp_dev_pages_destroy": [_vp],
    "kvp_dev_pages_init": [_vp, _vp, _vp],
    "kvp_dev_new": [_vp, _vp, _i, _vp],
    "kvp_dev_append": [_vp, _vp, _vp, _i, _vp, _i, _vp, _vp, _vp, _vp, _vp],
    "kvp_dev_trim": [_vp, _vp, _vp, _i, _i, _i, _vp],
    "kvp_dev_release": [_vp, _vp, _i, _vp],
    "kvp_dev_sync_error": [_vp, _vp, _ip],
    "kvp_dev_fork": [_vp, _vp, _vp, _i, _vp],
    "kvp_dev_rewind": [_vp, _vp, _vp, _i, _vp],
    "kvp_verify_step_device_io": [_vp, _vp, _vp, _i, _i, _i, _vp, _i, _i, _i, _i, _i, _f, _vp, _vp, _vp, _vp, _vp,
                                  _vp, _vp, _vp, _vp, _vp, _i, _vp, _sz, _vp],
    "copy_pages_device_count": [_vp, _vp, _vp, _vp, _i, _vp],
    "kvp_decode_step_device": [_vp, _vp, _vp, _i, _i, _i, _vp, _i, _i, _i, _i, _f, _vp, _vp, _vp, _vp, _vp, _vp,
                               _vp, _i, _vp, _sz, _vp],
    "kvp_decode_step_device_io": [_vp, _vp, _vp, _i, _i, _i, _vp, _i, _i, _i, _i, _f, _vp, _vp, _vp, _vp, _vp, _vp,
                                  _vp, _vp, _vp, _i, _vp, _sz, _vp],
    "kvp_decode_step": [_vp, _vp, _vp, _i, _i, _i, _vp, _i, _i, _i, _i, _f, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                        _i, _vp, _sz, _vp, _vp],
}


class StepInfo(ctypes.Structure):
    _fields_ = [("n_table_writes", ctypes.c_int), ("n_copies", ctypes.c_int), ("n_trim_writes", ctypes.c_int),
                ("meta_ints", ctypes.c_int)]

_lib = None
_addresses = {}


class KvpError(RuntimeError):
    def __init__(self, code, what):
        super().__init__(f"{what}: {_ERR_NAMES.get(code, code)}")
        self.code = code


class OutOfPages(KvpError):
    pass


def lib():
    """Load libpagedkv.so (built by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
        L = ctypes.CDLL(LIB_PATH)
        for name, args in SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        _addresses.clear()
        _lib = L
    return _lib


_marshal = None  # the module, or False: none that fits


def _native():
    """The argument marshalling in C++ (_marshal.so, built with the library); None where another library stands in for it, and,
    with a warning, where there is no module that fits this torch and Python."""
    global _marshal
    if lib() is not _lib:
        return None
    if _marshal is None:
        from .build import marshal_for

        try:
            from . import _marshal as m

            why = None if m.built_for == marshal_for() else f"built for {m.built_for}, not {marshal_for()}"
        except (ImportError, AttributeError) as e:
            why = str(e)
        if why:
            warnings.warn(f"_marshal.so is not used ({why}), every call goes through ctypes: build it (python -c "
                          "'import __graft_entry__ as g; g.build()')", RuntimeWarning, stacklevel=3)
        _marshal = False if why else m
    return _marshal or None


def _address(what):
    """The address of a function of the library."""
    a = _addresses.get(what)
    if a is None:
        a = _addresses[what] = ctypes.cast(getattr(lib(), what), ctypes.c_void_p).value
    return a


def _check(code, what):
    if code == KVP_ERR_OUT_OF_PAGES:
        raise OutOfPages(code, what)
    if code != KVP_OK:
        raise KvpError(code, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(t, dtype=None, name="tensor"):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _elsewhere(t, index, name):
    """The refusal of what is no tensor on the CUDA device of that index."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    raise ValueError(f"{name} must be on device {index}, got {t.device}")


def _on(t, index, dtype, name):
    """_dev, on the CUDA device of that index."""
    if not isinstance(t, torch.Tensor) or t.get_device() != index:
        _elsewhere(t, index, name)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


_TORCH_DTYPE = {KVP_F32: torch.float32, KVP_BF16: torch.bfloat16}


class Pool:
    """A kvp_pool over a caller-owned KV buffer (kept alive here)."""

    def __init__(self, kv_buffer, page_size, dtype, error_word=None):
        _dev(kv_buffer, name="kv_buffer")
        if kv_buffer.dim() != 6 or kv_buffer.shape[0] != 2 or kv_buffer.shape[3] != page_size:
            raise ValueError("kv_buffer must be (2, layers, num_pages, page_size, kv_heads, head_dim)")
        if kv_buffer.dtype != _TORCH_DTYPE[dtype]:
            raise TypeError("kv_buffer dtype does not match")
        _, self.num_layers, self.num_pages, self.page_size, self.kv_heads, self.head_dim = kv_buffer.shape
        self.dtype = dtype
        self.kv_buffer = kv_buffer
        self.device_index = kv_buffer.get_device()
        self.error_word = (torch.zeros(1, dtype=torch.int32, device=kv_buffer.device)
                           if error_word is None else _dev(error_word, torch.int32, "error_word"))
        h = ctypes.c_void_p()
        _check(lib().kv_pool_create(self.num_pages, page_size, self.kv_heads, self.head_dim, dtype,
                                    self.num_layers, _ptr(kv_buffer), _ptr(self.error_word), ctypes.byref(h)),
               "kv_pool_create")
        self.handle = h

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and _lib is not None:
            _lib.kv_pool_destroy(h)
            self.handle = None


def kv_pool_create(num_pages, page_size, kv_heads, head_dim, dtype, num_layers, kv_buffer=None, device="cuda"):
    """Describe (allocating with torch when ``kv_buffer`` is None) a KV buffer."""
    if kv_buffer is None:
        kv_buffer = torch.empty((2, num_layers, num_pages, page_size, kv_heads, head_dim),
                                dtype=_TORCH_DTYPE[dtype], device=device)
    return Pool(kv_buffer, page_size, dtype)


class LatentPool:
    """A kvp_pool over a caller-owned buffer of latent rows (kept alive here):
    (layers, num_pages, page_size, latent_dim + rope_dim), see
    include/pagedkv.h, kv_latent_pool_create."""

    def __init__(self, buffer, latent_dim, dtype, error_word=None):
        _dev(buffer, _TORCH_DTYPE[dtype], "buffer")
        if buffer.dim() != 4 or not 0 < latent_dim <= buffer.shape[3]:
            raise ValueError("buffer must be (layers, num_pages, page_size, latent_dim + rope_dim)")
        self.num_layers, self.num_pages, self.page_size, width = buffer.shape
        self.latent_dim, self.rope_dim, self.kv_heads, self.head_dim = latent_dim, width - latent_dim, 1, width
        self.dtype = dtype
        self.kv_buffer = buffer
        self.device_index = buffer.get_device()
        self.error_word = (torch.zeros(1, dtype=torch.int32, device=buffer.device)
                           if error_word is None else _on(error_word, self.device_index, torch.int32, "error_word"))
        h = ctypes.c_void_p()
        with torch.cuda.device(buffer.device):
            _check(lib().kv_latent_pool_create(self.num_pages, self.page_size, latent_dim, self.rope_dim, dtype,
                                               self.num_layers, _ptr(buffer), _ptr(self.error_word), ctypes.byref(h)),
                   "kv_latent_pool_create")
        self.handle = h

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and _lib is not None:
            _lib.kv_pool_destroy(h)
            self.handle = None


class Fp4Pool:
    """A kvp_pool over caller-owned codes and block scales (kept alive here), K
    and V in four bits: codes uint8 (layers, num_pages, page_size, kv_heads, 2,
    head_dim / 2), scales uint8 (layers, ceil(slots / 16), kv_heads, 16, 2,
    head_dim / 16); see include/pagedkv.h, kv_fp4_pool_create. ``dtype`` is that
    of what is stored, read and attended; ``k_scale`` and ``v_scale``: powers of
    two, one or one a layer."""

    def __init__(self, codes, scales, dtype, k_scale=1.0, v_scale=1.0, error_word=None):
        _dev(codes, torch.uint8, "codes")
        if codes.dim() != 6 or codes.shape[4] != 2:
            raise ValueError("codes must be (layers, num_pages, page_size, kv_heads, 2, head_dim / 2)")
        self.num_layers, self.num_pages, self.page_size, self.kv_heads, _, half = codes.shape
        self.head_dim = 2 * half
        self.device_index = codes.get_device()
        _on(scales, self.device_index, torch.uint8, "scales")
        groups = -(-self.num_pages * self.page_size // 16)
        if scales.shape != (self.num_layers, groups, self.kv_heads, 16, 2, self.head_dim // 16):
            raise ValueError(f"scales must be {(self.num_layers, groups, self.kv_heads, 16, 2, self.head_dim // 16)}, got "
                             f"{tuple(scales.shape)}")
        if dtype not in _TORCH_DTYPE:
            raise ValueError(f"dtype must be KVP_F32 or KVP_BF16, got {dtype!r}")
        self.dtype, self.codes, self.scales = dtype, codes, scales
        self.error_word = (torch.zeros(1, dtype=torch.int32, device=codes.device)
                           if error_word is None else _on(error_word, self.device_index, torch.int32, "error_word"))
        each = []
        for g, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            g = [float(g)] * self.num_layers if isinstance(g, (int, float)) else [float(x) for x in g]
            if len(g) != self.num_layers:
                raise ValueError(f"{name} must be one number or one a layer")
            each.append((ctypes.c_float * self.num_layers)(*g))
        h = ctypes.c_void_p()
        with torch.cuda.device(codes.device):
            _check(lib().kv_fp4_pool_create(self.num_pages, self.page_size, self.kv_heads, self.head_dim, dtype,
                                            self.num_layers, _ptr(codes), _ptr(scales), *each, _ptr(self.error_word),
                                            ctypes.byref(h)), "kv_fp4_pool_create")
        self.handle = h

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and _lib is not None:
            _lib.kv_pool_destroy(h)
            self.handle = None


def kv_fp4_pool_create(num_pages, page_size, kv_heads, head_dim, dtype, num_layers, k_scale=1.0, v_scale=1.0, device="cuda",
                       zero=False):
    """Describe a four-bit K/V cache, its codes and scales allocated with torch."""
    alloc = torch.zeros if zero else torch.empty
    codes = alloc((num_layers, num_pages, page_size, kv_heads, 2, head_dim // 2), dtype=torch.uint8, device=device)
    scales = alloc((num_layers, -(-num_pages * page_size // 16), kv_heads, 16, 2, head_dim // 16), dtype=torch.uint8,
                   device=device)
    return Fp4Pool(codes, scales, dtype, k_scale, v_scale)


_SCALINGS = {"none": KVP_ROTARY_PLAIN, "linear": KVP_ROTARY_LINEAR, "ntk": KVP_ROTARY_NTK, "by_parts": KVP_ROTARY_BY_PARTS}
_LAYOUTS = {"half": KVP_ROTARY_HALF, "interleaved": KVP_ROTARY_INTERLEAVED}


def rotary_frequencies(rotary_dim, base=10000.0, scaling="none", factor=1.0, original_len=4096, low_turns=1.0,
                       high_turns=32.0):
    """kvp_rotary_frequencies: the pairs' frequencies as turns * 2^64 (list of ints, host)."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}, got {scaling!r}")
    out = (ctypes.c_uint64 * max(1, rotary_dim // 2))()
    _check(lib().kvp_rotary_frequencies(int(rotary_dim), float(base), _SCALINGS[scaling], float(factor),
                                        float(original_len), float(low_turns), float(high_turns), out),
           "kvp_rotary_frequencies")
    return list(out)


def pair_axes(sections, interleave=False):
    """The axis of each pair: sections[a] pairs for axis a, axis after axis or dealt in turn."""
    left = [int(x) for x in sections]
    if not 1 <= len(left) <= KVP_ROTARY_MAX_AXES or min(left) < 0:
        raise ValueError(f"sections must be 1 to {KVP_ROTARY_MAX_AXES} counts, got {sections!r}")
    if not interleave:
        return [a for a, n in enumerate(left) for _ in range(n)]
    out = []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                out.append(a)
                left[a] -= 1
    return out


class RotaryPlan:
    """Frequencies on the device, layout and factor of rotary_store_cache and
    rotary_store_latent. ``layout``: "half" or "interleaved"; ``scaling``:
    "none", "linear", "ntk" or "by_parts" (see include/pagedkv.h,
    kvp_rotary_frequencies); ``attn_factor`` multiplies what is rotated.

    ``sections``: positions of several axes (time, height, width), then int32
    [axes, n] in the calls: how many of the rotary_dim / 2 pairs turn by each
    axis, one axis after another, or dealt to them in turn (``interleave``)
    until each has its share. Pair i's frequency is that of pair i of one axis,
    or (``per_axis``) each axis' pairs have the frequencies of a rotary_dim of
    their own, twice their number."""

    axes, pair_axis = 1, None

    def __init__(self, rotary_dim, base=10000.0, layout="half", scaling="none", factor=1.0, original_len=4096,
                 low_turns=1.0, high_turns=32.0, attn_factor=1.0, device="cuda", sections=None, interleave=False,
                 per_axis=False):
        if layout not in _LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}, got {layout!r}")
        self.rotary_dim, self.layout, self.attn_factor = int(rotary_dim), _LAYOUTS[layout], float(attn_factor)
        freq = lambda dim: rotary_frequencies(dim, base, scaling, factor, original_len, low_turns, high_turns)  # noqa: E731
        pairs = self.rotary_dim // 2
        of_pair = pair_axes(sections, interleave) if sections is not None else [0] * pairs
        if len(of_pair) != pairs:
            raise ValueError(f"the sections must add up to {pairs} pairs, got {list(sections)}")
        f = []  # 0: nothing turns
        if self.rotary_dim and per_axis:
            own = {a: iter(freq(2 * of_pair.count(a))) for a in set(of_pair)}
            f = [next(own[a]) for a in of_pair]
        elif self.rotary_dim:
            f = freq(self.rotary_dim)
        signed = [x - (1 << 64) if x >= 1 << 63 else x for x in f]
        self.freqs = torch.tensor(signed, dtype=torch.int64).to(device)
        if sections is not None and len(sections) > 1:
            self.axes = len(sections)
            self.pair_axis = torch.tensor(of_pair, dtype=torch.uint8).to(device)


def _current_stream():
    """The current stream's handle (torch.cuda.current_stream() builds a Stream object: 3 us a call)."""
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _raw_stream(stream):
    if stream is None:
        return _current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _int32(x, name):
    """An argument that a C int holds (ctypes would cut it down to one)."""
    x = int(x)
    if not -(1 << 31) <= x < 1 << 31:
        raise OverflowError(f"{name} must be an int32, got {x}")
    return x


def _heads_view(t, index, dt, name, heads, width):
    """(address, stride of a token, stride of a head, heads) of a [n, heads, width] view on device ``index`` whose last
    axis is contiguous."""
    if not isinstance(t, torch.Tensor) or t.get_device() != index:
        _elsewhere(t, index, name)
    if t.dtype != dt:
        raise TypeError(f"{name} must be {dt}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != width or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be [n, {'heads' if heads is None else heads}, {width}], got {tuple(shape)}")
    n, h, w = shape
    st, sh, se = t.stride()
    if h <= 1:
        sh = w  # the stride of an axis of one entry says nothing
    if n <= 1:
        st = max(st, (h - 1) * sh + w)
    if se != 1 and w > 1:
        raise ValueError(f"{name}'s last axis must be contiguous")
    return t.data_ptr(), st, sh, h


def _rows_view(t, index, dt, name, n, heads, width):
    """(address, stride of a token) of [n, heads, width] (or, for one head, [n, width]) on device ``index`` with each
    token's row contiguous."""
    if not isinstance(t, torch.Tensor) or t.get_device() != index:
        _elsewhere(t, index, name)
    if t.dtype != dt:
        raise TypeError(f"{name} must be {dt}, got {t.dtype}")
    shape, stride = t.shape, t.stride()
    if len(shape) == 3 and shape[1] == heads and shape[2] == width:
        good = (width == 1 or stride[2] == 1) and (heads == 1 or stride[1] == width)
    else:
        good = heads == 1 and len(shape) == 2 and shape[1] == width and (width == 1 or stride[1] == 1)
    if not good or shape[0] != n:
        raise ValueError(f"{name} must be [{n}, {heads}, {width}] with each token's row contiguous, got {tuple(shape)}")
    return t.data_ptr(), stride[0] if n > 1 else heads * width


def _positions_of(t, index, axes):
    """(address, tokens, distance of two axes) of int32 positions: [n], or [axes, n] for a plan of several axes, whose
    rows may lie apart."""
    if not isinstance(t, torch.Tensor) or t.get_device() != index:
        _elsewhere(t, index, "positions")
    if axes == 1:
        return _on(t, index, torch.int32, "positions").data_ptr(), t.numel(), 0
    if t.dtype != torch.int32:
        raise TypeError(f"positions must be {torch.int32}, got {t.dtype}")
    if t.dim() != 2 or t.shape[0] != axes:
        raise ValueError(f"positions must be [{axes}, n] for a plan of {axes} axes, got {tuple(t.shape)}")
    n = t.shape[1]
    if n > 1 and t.stride(1) != 1:
        raise ValueError("positions' last axis must be contiguous")
    stride = t.stride(0) if n else 0
    if stride < n:
        raise ValueError("positions' axes must not overlap")
    return t.data_ptr(), n, stride


def _rotary_call(what, pool, layer, q, first, second, positions, out_loc, rope, q_out, width, stream, always_axes=False):
    """Marshals the rotary stores: ``first`` and ``second`` are the two row inputs in the order of the C call, each
    (tensor, name, heads, width). With a plan of several axes the call is what + "_axes" (``always_axes``: the call takes
    axes under its own name, and may come without a plan)."""
    dt, dev = _TORCH_DTYPE[pool.dtype], pool.device_index
    axes = 1 if rope is None else getattr(rope, "axes", 1)
    k, v = first[0], second[0]
    native = _native()
    if native is not None:
        on_axes = axes > 1 or always_axes
        name = what if always_axes or axes == 1 else what + "_axes"
        of_plan = ((None, None, 1, 0, 0, 1.0) if rope is None else
                   (rope.freqs, rope.pair_axis, axes, rope.rotary_dim, rope.layout, rope.attn_factor))
        code = native.rotary(_address(name), 1 if on_axes else 0, pool.handle.value, pool.dtype, dev, layer, q, k, first[2],
                             first[3], v, second[2], second[3], positions, out_loc, *of_plan, q_out, width,
                             None if stream is None else _raw_stream(stream))
        if code is not None:
            return _check(code, name)
    layer = _int32(layer, "layer")
    if (k is None) != (v is None):
        raise ValueError(f"{first[1]} and {second[1]} come together")
    freqs = of_pair = rot = layout = pos = apart = 0
    factor = 1.0
    if rope is None:  # rows as they are
        if positions is not None or q is not None:
            raise ValueError("positions and queries need a plan")
        n = _on(out_loc, dev, torch.int32, "out_loc").numel()
    else:
        pos, n, apart = _positions_of(positions, dev, axes)
        if rope.rotary_dim and rope.freqs.get_device() != dev:
            _elsewhere(rope.freqs, dev, "the plan's frequencies")
        freqs, rot, layout, factor = rope.freqs.data_ptr(), rope.rotary_dim, rope.layout, rope.attn_factor
        if axes > 1:
            of_pair = rope.pair_axis.data_ptr()
    if rot > width:
        raise ValueError(f"the plan turns {rot} entries of {width}")
    qp = qt = qh = heads = op = ot = oh = kp = kt = vp = vt = loc = 0
    if q is not None:
        qp, qt, qh, heads = _heads_view(q, dev, dt, "q", None, width)
        op, ot, oh, _ = _heads_view(q_out, dev, dt, "q_out", heads, width)
        if q.shape[0] != n or q_out.shape[0] != n:
            raise ValueError("the queries and their output must hold one row per position")
    elif k is None:
        raise ValueError("neither queries nor keys")
    if k is not None:
        kp, kt = _rows_view(k, dev, dt, first[1], n, first[2], first[3])
        vp, vt = _rows_view(v, dev, dt, second[1], n, second[2], second[3])
        if _on(out_loc, dev, torch.int32, "out_loc").numel() != n:
            raise ValueError("out_loc and positions must have the same length")
        loc = out_loc.data_ptr()
    if axes > 1 or always_axes:
        what = what if always_axes else what + "_axes"
        _check(getattr(lib(), what)(pool.handle, layer, qp, qt, qh, heads, kp, kt, vp, vt, pos, apart, loc, n, freqs, of_pair,
                                    axes, rot, layout, factor, op, ot, oh, _raw_stream(stream)), what)
    else:
        _check(getattr(lib(), what)(pool.handle, layer, qp, qt, qh, heads, kp, kt, vp, vt, pos, loc, n, freqs, rot, layout,
                                    factor, op, ot, oh, _raw_stream(stream)), what)


def rotary_store_cache(pool, layer, q, k, v, positions, out_loc, rope, q_out, stream=None):
    """Rotary positions of a step's q and k, and the store of the rotated k and
    of v, in one launch. q, q_out [n, Hq, D] (any token and head strides;
    q_out may be q), k, v [n, kv_heads, D] (any token stride), positions and
    out_loc int32 [n], ``rope`` a RotaryPlan (of several axes: positions int32
    [axes, n]). q and q_out None: only the store; k, v and out_loc None: only
    q. See include/pagedkv.h."""
    h, d = pool.kv_heads, pool.head_dim
    _rotary_call("rotary_store_cache", pool, layer, q, (k, "k", h, d), (v, "v", h, d), positions, out_loc, rope, q_out, d,
                 stream)


def rotary_store_latent(pool, layer, q_pe, latent, k_pe, positions, out_loc, rope, q_pe_out, stream=None):
    """rotary_store_cache of a LatentPool: q_pe, q_pe_out [n, Hq, rope_dim]
    (q_pe_out usually the tail of the absorbed queries), latent [n,
    latent_dim] and k_pe [n, rope_dim] with any token stride. q_pe and
    q_pe_out None: only the store; latent, k_pe and out_loc None: only q_pe."""
    _rotary_call("rotary_store_latent", pool, layer, q_pe, (latent, "latent", 1, pool.latent_dim),
                 (k_pe, "k_pe", 1, pool.rope_dim), positions, out_loc, rope, q_pe_out, pool.rope_dim, stream)


def rotary_store_fp4(pool, layer, q, k, v, positions, out_loc, rope, q_out, stream=None):
    """rotary_store_cache into a Fp4Pool: the rotated k and v are rounded to four
    bits as they are stored (the rotated k is not rounded before). See
    include/pagedkv.h."""
    if rope is None:
        raise ValueError("rotary_store_fp4 needs a plan (rows as they are: store_cache_fp4)")
    h, d = pool.kv_heads, pool.head_dim
    _rotary_call("rotary_store_fp4", pool, layer, q, (k, "k", h, d), (v, "v", h, d), positions, out_loc, rope, q_out, d, stream,
                 always_axes=True)


def store_cache_fp4(pool, layer, k, v, out_loc, stream=None):
    """store_cache of a Fp4Pool: k, v [n, kv_heads, D] as they are (any token
    stride), rounded to four bits, to the slots out_loc int32 [n]."""
    h, d = pool.kv_heads, pool.head_dim
    if k is None:
        raise ValueError("store_cache_fp4 needs k and v")
    _rotary_call("rotary_store_fp4", pool, layer, None, (k, "k", h, d), (v, "v", h, d), None, out_loc, None, None, d, stream,
                 always_axes=True)


def load_cache_fp4(pool, layer, slots, k_out, v_out, stream=None):
    """The rows of a Fp4Pool at ``slots`` (int32 [n], any order) as the values
    they stand for: k_out, v_out [n, kv_heads, D] contiguous, pool dtype."""
    dt, dev = _TORCH_DTYPE[pool.dtype], pool.device_index
    native = _native()
    if native is not None:
        code = native.load(_address("load_cache_fp4"), pool.handle.value, pool.dtype, dev, layer, slots, k_out, v_out,
                           pool.kv_heads * pool.head_dim, None if stream is None else _raw_stream(stream))
        if code is not None:
            return _check(code, "load_cache_fp4")
    layer = _int32(layer, "layer")
    n = _on(slots, dev, torch.int32, "slots").numel()
    for t, name in ((k_out, "k_out"), (v_out, "v_out")):
        if _on(t, dev, dt, name).numel() != n * pool.kv_heads * pool.head_dim:
            raise ValueError(f"{name} must be [{n}, {pool.kv_heads}, {pool.head_dim}], got {tuple(t.shape)}")
    _check(lib().load_cache_fp4(pool.handle, layer, slots.data_ptr(), n, k_out.data_ptr(), v_out.data_ptr(),
                                _raw_stream(stream)), "load_cache_fp4")


def paged_fp4_attention_workspace_size(pool, batch, chunk, num_q_heads, max_context):
    n = ctypes.c_size_t()
    _check(lib().paged_fp4_attention_workspace_size(pool.handle, batch, chunk, num_q_heads, max_context, ctypes.byref(n)),
           "paged_fp4_attention_workspace_size")
    return n.value


def alloc_fp4_workspace(pool, batch, chunk, num_q_heads, max_context, device="cuda"):
    nbytes = paged_fp4_attention_workspace_size(pool, batch, chunk, num_q_heads, max_context)
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def paged_fp4_attention(pool, layer, q, table, table_mode, context_lens, window, scale, out, workspace, q_lens=None,
                        table_rows=None, stream=None, sinks=0, max_context=None):
    """Attention over a Fp4Pool: q, out [B, C, Hq, D]; query j of request b sits
    at position context_lens[b] - q_lens[b] + j (q_lens None: C) and attends
    causally (decode: C = 1). Rows j >= q_lens[b] are not written.
    ``max_context``: a bound of context_lens (None: what the table holds), the
    one the workspace was made for. See include/pagedkv.h."""
    dt, dev = _TORCH_DTYPE[pool.dtype], pool.device_index
    native = _native()
    if native is not None:
        code = native.attend(_address("paged_fp4_attention"), pool.handle.value, pool.dtype, dev, pool.head_dim, pool.page_size,
                             layer, q, q_lens, table, table_mode, table_rows, context_lens, max_context, window or 0, sinks, scale,
                             out, workspace, None if stream is None else _raw_stream(stream))
        if code is not None:
            return _check(code, "paged_fp4_attention")
    layer, sinks, most = _int32(layer, "layer"), _int32(sinks, "sinks"), (1 << 31) - 1
    window = max(0, min(int(window or 0), most))  # one that no context can fill is none
    _on(q, dev, dt, "q")
    _on(out, dev, dt, "out")
    _on(table, dev, torch.int32, "table")
    _on(context_lens, dev, torch.int32, "context_lens")
    shape = q.shape
    if len(shape) != 4 or shape[3] != pool.head_dim or out.shape != shape:
        raise ValueError("q and out must be [B, C, Hq, D]")
    B, C, Hq, _ = shape
    per = [0, 0]
    for i, (t, nm) in enumerate(((q_lens, "q_lens"), (table_rows, "table_rows"))):
        if t is not None:
            if _on(t, dev, torch.int32, nm).numel() != B:
                raise ValueError(f"{nm} must be [B]")
            per[i] = t.data_ptr()
    if context_lens.numel() != B or table.dim() != 2:
        raise ValueError("context_lens must be [B], table [rows, columns]")
    rows, cols = table.shape
    if max_context is None:
        max_context = cols if table_mode == KVP_RAW_LOCATIONS else cols * pool.page_size
    max_context = max(0, min(int(max_context), most))
    _check(lib().paged_fp4_attention(pool.handle, layer, q.data_ptr(), B, C, Hq, per[0], table.data_ptr(), rows, cols,
                                     table_mode, per[1], context_lens.data_ptr(), max_context, window, sinks,
                                     float(scale), out.data_ptr(), _on(workspace, dev, None, "workspace").data_ptr(),
                                     workspace.nbytes, _raw_stream(stream)), "paged_fp4_attention")


def paged_latent_attention_workspace_size(pool, batch, chunk, num_q_heads):
    n = ctypes.c_size_t()
    _check(lib().paged_latent_attention_workspace_size(pool.handle, batch, chunk, num_q_heads, ctypes.byref(n)),
           "paged_latent_attention_workspace_size")
    return n.value


def alloc_latent_workspace(pool, batch, chunk, num_q_heads, device="cuda"):
    nbytes = paged_latent_attention_workspace_size(pool, batch, chunk, num_q_heads)
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def paged_latent_attention(pool, layer, q, table, table_mode, context_lens, window, scale, out, workspace, q_lens=None,
                           table_rows=None, stream=None, sinks=0):
    """Absorbed latent attention over a LatentPool: q [B, C, Hq, latent_dim +
    rope_dim], out [B, C, Hq, latent_dim]; query j of request b sits at position
    context_lens[b] - q_lens[b] + j (q_lens None: C) and attends causally
    (decode: C = 1). Rows j >= q_lens[b] are not written. See
    include/pagedkv.h."""
    dt, dev = _TORCH_DTYPE[pool.dtype], pool.device_index
    _on(q, dev, dt, "q")
    _on(out, dev, dt, "out")
    _on(table, dev, torch.int32, "table")
    _on(context_lens, dev, torch.int32, "context_lens")
    shape = q.shape
    if len(shape) != 4 or shape[3] != pool.head_dim or out.shape != (*shape[:3], pool.latent_dim):
        raise ValueError("q must be [B, C, Hq, latent_dim + rope_dim] and out [B, C, Hq, latent_dim]")
    B, C, Hq, _ = shape
    per = [0, 0]
    for i, (t, nm) in enumerate(((q_lens, "q_lens"), (table_rows, "table_rows"))):
        if t is not None:
            if _on(t, dev, torch.int32, nm).numel() != B:
                raise ValueError(f"{nm} must be [B]")
            per[i] = t.data_ptr()
    if context_lens.numel() != B:
        raise ValueError("context_lens must be [B]")
    rows, cols = table.shape
    ws_ptr, ws_bytes = (0, 0) if workspace is None else (_on(workspace, dev, None, "workspace").data_ptr(), workspace.nbytes)
    _check(lib().paged_latent_attention(pool.handle, layer, q.data_ptr(), B, C, Hq, per[0], table.data_ptr(), rows, cols,
                                        table_mode, per[1], context_lens.data_ptr(), int(window or 0), int(sinks),
                                        float(scale), out.data_ptr(), ws_ptr, ws_bytes, _raw_stream(stream)),
           "paged_latent_attention")


def latent_prefill_attention(q, k, k_pe, v, q_start, k_start, max_q, scale, out, error_word=None, stream=None):
    """Causal attention of ragged prompts in expanded form: q [total_q, H, dn +
    dr], k [total_k, H, dn], k_pe [total_k, dr] (None when dr is 0), v
    [total_k, H, dv] (views with any token and head strides), out [total_q, H,
    dv] contiguous, q_start/k_start int32 [B + 1]; query j of a request attends
    its keys up to (key rows - query rows) + j. See include/pagedkv.h."""
    dt = q.dtype
    if dt not in (torch.float32, torch.bfloat16):
        raise TypeError(f"q must be float32 or bfloat16, got {dt}")
    dev = q.get_device()
    if dev < 0:
        _elsewhere(q, dev, "q")
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be [tokens, heads, entries]")
    tq, H, width = q.shape
    tk, _, dn = k.shape
    dv = v.shape[2]
    dr = width - dn
    if dr < 0 or (dr > 0) != (k_pe is not None):
        raise ValueError("q must be as wide as k and k_pe together")
    qa = _heads_view(q, dev, dt, "q", None, width)[:3]
    ka = _heads_view(k, dev, dt, "k", H, dn)[:3]
    va = _heads_view(v, dev, dt, "v", H, dv)[:3]
    pa = (0, 0) if k_pe is None else _rows_view(k_pe, dev, dt, "k_pe", tk, 1, dr)
    _on(out, dev, dt, "out")
    _on(q_start, dev, torch.int32, "q_start")
    _on(k_start, dev, torch.int32, "k_start")
    B = q_start.numel() - 1
    if v.shape[0] != tk or out.shape != (tq, H, dv) or B < 0 or k_start.numel() != B + 1:
        raise ValueError("v must hold k's tokens, out be [total_q, H, dv], q_start and k_start [B + 1]")
    if B == 0:
        return
    err = 0 if error_word is None else _on(error_word, dev, torch.int32, "error_word").data_ptr()
    _check(lib().latent_prefill_attention(*qa, *ka, *pa, *va, q_start.data_ptr(), k_start.data_ptr(), B, H, int(max_q), tq,
                                          tk, dn, dr, dv, KVP_F32 if dt == torch.float32 else KVP_BF16, float(scale),
                                          out.data_ptr(), err, _raw_stream(stream)), "latent_prefill_attention")


def store_cache(pool, layer, k, v, out_loc, stream=None):
    _dev(k, _TORCH_DTYPE[pool.dtype], "k")
    _dev(v, _TORCH_DTYPE[pool.dtype], "v")
    _dev(out_loc, torch.int32, "out_loc")
    n = out_loc.numel()
    if k.numel() != n * pool.kv_heads * pool.head_dim or v.numel() != k.numel():
        raise ValueError("k/v must be [n, kv_heads, head_dim]")
    _check(lib().store_cache(pool.handle, layer, _ptr(k), _ptr(v), _ptr(out_loc), n, _stream(stream)), "store_cache")


def page_table_write(table, rows, cols, vals, expand=1, error_word=None, stream=None):
    _dev(table, torch.int32, "table")
    for t, nm in ((rows, "rows"), (cols, "cols"), (vals, "vals")):
        _dev(t, torch.int32, nm)
    n = rows.numel()
    if cols.numel() != n or vals.numel() != n:
        raise ValueError("rows, cols and vals must have the same length")
    _check(lib().page_table_write(_ptr(table), table.shape[0], table.shape[1], _ptr(rows), _ptr(cols), _ptr(vals),
                                  n, expand, _ptr(error_word), _stream(stream)), "page_table_write")


class DevicePages:
    """Device-side page allocation over a caller's device table (see
    include/pagedkv.h, kvp_dev_*). The state buffer is allocated here with
    torch and kept alive; every call is asynchronous on the current stream."""

    def __init__(self, num_pages, page_size, max_requests, table, table_mode, free_stack=None, device="cuda"):
        _dev(table, torch.int32, "table")
        n = ctypes.c_size_t()
        _check(lib().kvp_dev_pages_bytes(num_pages, max_requests, ctypes.byref(n)), "kvp_dev_pages_bytes")
        self.state = torch.zeros(n.value, dtype=torch.uint8, device=device)
        self.table = table
        self.num_pages, self.page_size, self.max_requests = num_pages, page_size, max_requests
        h = ctypes.c_void_p()
        _check(lib().kvp_dev_pages_create(num_pages, page_size, max_requests, _ptr(self.state), n.value, _ptr(table),
                                          table.shape[0], table.shape[1], table_mode, ctypes.byref(h)),
               "kvp_dev_pages_create")
        self.handle = h
        fs = None
        if free_stack is not None:
            fs = torch.as_tensor(list(free_stack), dtype=torch.int32).to(device)
            if fs.numel() != num_pages:
                raise ValueError("free_stack must hold num_pages entries")
        self._free_stack = fs
        _check(lib().kvp_dev_pages_init(h, _ptr(fs), _stream(None)), "kvp_dev_pages_init")

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and _lib is not None:
            _lib.kvp_dev_pages_destroy(h)
            self.handle = None

    def new(self, rids, stream=None):
        _dev(rids, torch.int32, "rids")
        _check(lib().kvp_dev_new(self.handle, _ptr(rids), rids.numel(), _stream(stream)), "kvp_dev_new")

    def append(self, rids, out_loc, cow_src, cow_dst, n_cow, counts=None, lens_out=None, stream=None):
        for t, nm in ((rids, "rids"), (out_loc, "out_loc"), (cow_src, "cow_src"), (cow_dst, "cow_dst"),
                      (n_cow, "n_cow")):
            _dev(t, torch.int32, nm)
        if counts is not None:
            _dev(counts, torch.int32, "counts")
        n = rids.numel()
        if cow_src.numel() < n or cow_dst.numel() < n:
            raise ValueError("cow_src/cow_dst need room for one pair per request")
        if lens_out is not None:
            _dev(lens_out, torch.int32, "lens_out")
        _check(lib().kvp_dev_append(self.handle, _ptr(rids), _ptr(counts), n, _ptr(out_loc), out_loc.numel(),
                                    _ptr(cow_src), _ptr(cow_dst), _ptr(n_cow), _ptr(lens_out), _stream(stream)),
               "kvp_dev_append")

    def trim(self, rids, keep_from=None, sinks=0, window=0, stream=None):
        """Release what the next step cannot read: below keep_from[i] (device
        int32), or, without keep_from, below each request's L + 1 - (window - sinks)."""
        _dev(rids, torch.int32, "rids")
        if keep_from is not None:
            _dev(keep_from, torch.int32, "keep_from")
        _check(lib().kvp_dev_trim(self.handle, _ptr(rids), _ptr(keep_from), rids.numel(), int(window), int(sinks),
                                  _stream(stream)), "kvp_dev_trim")

    def release(self, rids, stream=None):
        _dev(rids, torch.int32, "rids")
        _check(lib().kvp_dev_release(self.handle, _ptr(rids), rids.numel(), _stream(stream)), "kvp_dev_release")

    def fork(self, src, dst, stream=None):
        _dev(src, torch.int32, "src")
        _dev(dst, torch.int32, "dst")
        if src.numel() != dst.numel():
            raise ValueError("src and dst must have the same length")
        _check(lib().kvp_dev_fork(self.handle, _ptr(src), _ptr(dst), src.numel(), _stream(stream)), "kvp_dev_fork")

    def rewind(self, rids, n_back, stream=None):
        """Drop the newest n_back[i] rows of request rids[i] (both device int32)."""
        _dev(rids, torch.int32, "rids")
        _dev(n_back, torch.int32, "n_back")
        if rids.numel() != n_back.numel():
            raise ValueError("rids and n_back must have the same length")
        _check(lib().kvp_dev_rewind(self.handle, _ptr(rids), _ptr(n_back), rids.numel(), _stream(stream)),
               "kvp_dev_rewind")

    def sync_error(self, stream=None):
        e = ctypes.c_int()
        _check(lib().kvp_dev_sync_error(self.handle, _stream(stream), ctypes.byref(e)), "kvp_dev_sync_error")
        return e.value

    def snapshot(self):
        """(free list, reference counts, lengths, released pages, sink pages) read back to the host."""
        P, R = self.num_pages, self.max_requests
        a16 = lambda x: (x + 15) // 16 * 16  # noqa: E731
        st = self.state.cpu()
        hdr = st[:16].view(torch.int32).tolist()
        off = 16
        stack = st[off:off + 4 * P].view(torch.int32).tolist()
        off += a16(4 * P)
        ref = st[off:off + 4 * P].view(torch.int32).tolist()
        off += a16(4 * P)
        arr = []
        for _ in range(3):
            arr.append(st[off:off + 4 * R].view(torch.int32).tolist())
            off += a16(4 * R)
        return stack[:hdr[0]], ref, arr[0], arr[1], arr[2]


def copy_pages_device_count(pool, src, dst, n_dev, stream=None):
    _dev(src, torch.int32, "src")
    _dev(dst, torch.int32, "dst")
    _dev(n_dev, torch.int32, "n_dev")
    _check(lib().copy_pages_device_count(pool.handle, _ptr(src), _ptr(dst), _ptr(n_dev), src.numel(),
                                         _stream(stream)), "copy_pages_device_count")


def copy_pages(pool, src, dst, stream=None):
    _dev(src, torch.int32, "src")
    _dev(dst, torch.int32, "dst")
    if src.numel() != dst.numel():
        raise ValueError("src and dst must have the same length")
    _check(lib().copy_pages(pool.handle, _ptr(src), _ptr(dst), src.numel(), _stream(stream)), "copy_pages")


def paged_decode_attention_workspace_size(pool, batch, num_q_heads):
    n = ctypes.c_size_t()
    _check(lib().paged_decode_attention_workspace_size(pool.handle, batch, num_q_heads, ctypes.byref(n)),
           "paged_decode_attention_workspace_size")
    return n.value


def alloc_workspace(pool, batch, num_q_heads, device="cuda"):
    nbytes = paged_decode_attention_workspace_size(pool, batch, num_q_heads)
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def paged_decode_attention(pool, layer, q, table, table_mode, context_lens, window, scale, out, workspace,
                           table_rows=None, stream=None, sinks=0):
    dt = _TORCH_DTYPE[pool.dtype]
    _dev(q, dt, "q")
    _dev(out, dt, "out")
    _dev(table, torch.int32, "table")
    _dev(context_lens, torch.int32, "context_lens")
    if table_rows is not None:
        _dev(table_rows, torch.int32, "table_rows")
    B, Hq = q.shape[0], q.shape[1]
    if out.shape != q.shape or context_lens.numel() != B:
        raise ValueError("q/out must be [B, Hq, D] and context_lens [B]")
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (_ptr(workspace), workspace.numel() * workspace.element_size())
    _check(lib().paged_decode_attention(pool.handle, layer, _ptr(q), B, Hq, _ptr(table), table.shape[0],
                                        table.shape[1], table_mode, _ptr(table_rows), _ptr(context_lens),
                                        int(window or 0), int(sinks), float(scale), _ptr(out), ws_ptr, ws_bytes,
                                        _stream(stream)), "paged_decode_attention")


def paged_verify_attention_workspace_size(pool, batch, num_q_tokens, num_q_heads):
    n = ctypes.c_size_t()
    _check(lib().paged_verify_attention_workspace_size(pool.handle, batch, num_q_tokens, num_q_heads,
                                                       ctypes.byref(n)), "paged_verify_attention_workspace_size")
    return n.value


def alloc_verify_workspace(pool, batch, num_q_tokens, num_q_heads, device="cuda"):
    nbytes = paged_verify_attention_workspace_size(pool, batch, num_q_tokens, num_q_heads)
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def paged_verify_attention(pool, layer, q, table, table_mode, context_lens, window, scale, out, workspace,
                           table_rows=None, stream=None, sinks=0):
    """Multi-token verify: q/out [B, M, Hq, D]; query j of request b sits at
    position context_lens[b] - M + j and attends causally (see
    include/pagedkv.h)."""
    dt = _TORCH_DTYPE[pool.dtype]
    _dev(q, dt, "q")
    _dev(out, dt, "out")
    _dev(table, torch.int32, "table")
    _dev(context_lens, torch.int32, "context_lens")
    if table_rows is not None:
        _dev(table_rows, torch.int32, "table_rows")
    if q.dim() != 4 or out.shape != q.shape or context_lens.numel() != q.shape[0]:
        raise ValueError("q/out must be [B, M, Hq, D] and context_lens [B]")
    B, M, Hq = q.shape[0], q.shape[1], q.shape[2]
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (_ptr(workspace), workspace.numel() * workspace.element_size())
    _check(lib().paged_verify_attention(pool.handle, layer, _ptr(q), B, M, Hq, _ptr(table), table.shape[0],
                                        table.shape[1], table_mode, _ptr(table_rows), _ptr(context_lens),
                                        int(window or 0), int(sinks), float(scale), _ptr(out), ws_ptr, ws_bytes,
                                        _stream(stream)), "paged_verify_attention")


def paged_prefill_attention(pool, layer, q, table, table_mode, context_lens, window, scale, out, q_lens=None,
                            table_rows=None, stream=None, sinks=0):
    """Chunked prefill: q/out [B, C, Hq, D]; query j of request b sits at
    position context_lens[b] - q_lens[b] + j (q_lens NULL: C) and attends
    causally (see include/pagedkv.h). Rows j >= q_lens[b] are not written."""
    dt = _TORCH_DTYPE[pool.dtype]
    _dev(q, dt, "q")
    _dev(out, dt, "out")
    _dev(table, torch.int32, "table")
    _dev(context_lens, torch.int32, "context_lens")
    for t, nm in ((q_lens, "q_lens"), (table_rows, "table_rows")):
        if t is not None:
            _dev(t, torch.int32, nm)
    if q.dim() != 4 or out.shape != q.shape or context_lens.numel() != q.shape[0]:
        raise ValueError("q/out must be [B, C, Hq, D] and context_lens [B]")
    B, C, Hq = q.shape[0], q.shape[1], q.shape[2]
    _check(lib().paged_prefill_attention(pool.handle, layer, _ptr(q), B, C, Hq, _ptr(q_lens), _ptr(table),
                                         table.shape[0], table.shape[1], table_mode, _ptr(table_rows),
                                         _ptr(context_lens), int(window or 0), int(sinks), float(scale), _ptr(out),
                                         _stream(stream)), "paged_prefill_attention")


def store_cache_and_attention(pool, layer, q, k, v, out_loc, table, table_mode, context_lens, window, scale, out,
                              workspace, table_rows=None, table_writes=None, stream=None, sinks=0):
    """store_cache + paged_decode_attention of one layer in one launch, with
    the step's new-page table writes (rows, cols, vals device int32 tensors)
    applied in the same launch. out_loc[b] must be the slot of request b's
    newest position; see include/pagedkv.h for what the table writes may be."""
    dt = _TORCH_DTYPE[pool.dtype]
    for name, x in (("q", q), ("k", k), ("v", v), ("out", out)):
        _dev(x, dt, name)
    _dev(out_loc, torch.int32, "out_loc")
    _dev(table, torch.int32, "table")
    _dev(context_lens, torch.int32, "context_lens")
    if table_rows is not None:
        _dev(table_rows, torch.int32, "table_rows")
    B, Hq = q.shape[0], q.shape[1]
    if out.shape != q.shape or context_lens.numel() != B or out_loc.numel() != B or k.shape[0] != B:
        raise ValueError("q/out [B, Hq, D], k/v [B, Hkv, D], out_loc and context_lens [B]")
    if table_writes is None:
        tw = (None, None, None, 0)
    else:
        r, c, vals = table_writes
        for name, x in (("rows", r), ("cols", c), ("vals", vals)):
            _dev(x, torch.int32, name)
        tw = (_ptr(r), _ptr(c), _ptr(vals), r.numel())
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (_ptr(workspace), workspace.numel() * workspace.element_size())
    _check(lib().store_cache_and_attention(pool.handle, layer, _ptr(q), _ptr(k), _ptr(v), _ptr(out_loc), B, Hq,
                                           _ptr(table), table.shape[0], table.shape[1], table_mode,
                                           _ptr(table_rows), _ptr(context_lens), *tw, int(window or 0), int(sinks),
                                           float(scale), _ptr(out), ws_ptr, ws_bytes, _stream(stream)),
           "store_cache_and_attention")


def paged_decode_attention_noalloc(pool, layer, q, table, table_mode, context_lens, window, scale, out,
                                   table_rows=None, stream=None, sinks=0):
    """paged_decode_attention without a workspace argument, for callers that
    cannot allocate: the library uses a fixed scratch array of its own (see
    include/pagedkv.h). Overlapping calls on one device must be serialised."""
    dt = _TORCH_DTYPE[pool.dtype]
    _dev(q, dt, "q")
    _dev(out, dt, "out")
    _dev(table, torch.int32, "table")
    _dev(context_lens, torch.int32, "context_lens")
    if table_rows is not None:
        _dev(table_rows, torch.int32, "table_rows")
    B, Hq = q.shape[0], q.shape[1]
    if out.shape != q.shape or context_lens.numel() != B:
        raise ValueError("q/out must be [B, Hq, D] and context_lens [B]")
    _check(lib().paged_decode_attention_noalloc(pool.handle, layer, _ptr(q), B, Hq, _ptr(table), table.shape[0],
                                                table.shape[1], table_mode, _ptr(table_rows), _ptr(context_lens),
                                                int(window or 0), int(sinks), float(scale), _ptr(out),
                                                _stream(stream)),
           "paged_decode_attention_noalloc")


def gather_indices(pool, table, table_mode, context_lens, window, slots_out, table_rows=None, stream=None, sinks=0):
    _dev(table, torch.int32, "table")
    _dev(context_lens, torch.int32, "context_lens")
    _dev(slots_out, torch.int32, "slots_out")
    B = context_lens.numel()
    _check(lib().gather_indices(pool.handle, _ptr(table), table.shape[0], table.shape[1], table_mode,
                                _ptr(table_rows), _ptr(context_lens), B, int(window or 0), int(sinks), _ptr(slots_out),
                                slots_out.shape[1], _stream(stream)), "gather_indices")


def kvp_pool_set_timing_events(pool, before=None, after=None):
    """Record ``before``/``after`` (torch.cuda.Event) around the next attention kernel."""
    b = None if before is None else ctypes.c_void_p(before.cuda_event)
    a = None if after is None else ctypes.c_void_p(after.cuda_event)
    _check(lib().kvp_pool_set_timing_events(pool.handle, b, a), "kvp_pool_set_timing_events")


def kvp_sync_error(pool, stream=None):
    e = ctypes.c_int()
    _check(lib().kvp_sync_error(pool.handle, _stream(stream), ctypes.byref(e)), "kvp_sync_error")
    return e.value


def kvp_selftest_wait(limit_ns, arrive, err, stream=None):
    """One bounded mbarrier wait on the device (kvp_selftest_wait): ``err`` is
    a device int32 tensor that receives KVP_ERR_TIMEOUT when nothing arrives."""
    _check(lib().kvp_selftest_wait(int(limit_ns), int(arrive), _ptr(err), _stream(stream)), "kvp_selftest_wait")


# ---------------------------------------------------------------------------
# Host bookkeeping (pure C++, usable without a GPU).
# ---------------------------------------------------------------------------
def _i32(n):
    return (ctypes.c_int32 * max(1, n))()


class HostPageTable:
    """kvp_host_*: refcounted LIFO free list, block tables with -1 holes,
    fork, lazy copy-on-write, window trim; emits device table writes."""

    def __init__(self, num_pages, page_size, max_requests, free_stack=None):
        self.num_pages, self.page_size, self.max_requests = num_pages, page_size, max_requests
        h = ctypes.c_void_p()
        fs = None
        if free_stack is not None:
            fs = (ctypes.c_int32 * num_pages)(*[int(x) for x in free_stack])
        _check(lib().kvp_host_create(num_pages, page_size, max_requests, fs, ctypes.byref(h)), "kvp_host_create")
        self.handle = h

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and _lib is not None:
            _lib.kvp_host_destroy(h)
            self.handle = None

    def new(self, rid):
        _check(lib().kvp_host_new(self.handle, rid), "kvp_host_new")

    def fork(self, src, dst):
        """Share every page of ``src`` with ``dst``; returns the table writes for dst's row."""
        cap = self.length(src)[0] // self.page_size + 2
        tr, tc, tv = _i32(cap), _i32(cap), _i32(cap)
        n = ctypes.c_int()
        _check(lib().kvp_host_fork(self.handle, src, dst, tr, tc, tv, cap, ctypes.byref(n)), "kvp_host_fork")
        return list(zip(tr[:n.value], tc[:n.value], tv[:n.value]))

    def release(self, rid):
        _check(lib().kvp_host_release(self.handle, rid), "kvp_host_release")

    def append(self, rids):
        """One token for each entry of ``rids`` -> (slots, table writes, cow pairs) as Python lists."""
        rids = [int(r) for r in rids]
        n = len(rids)
        r = (ctypes.c_int32 * max(1, n))(*rids)
        slots, tr, tc, tv, cs, cd = _i32(n), _i32(n), _i32(n), _i32(n), _i32(n), _i32(n)
        ntw, ncow = ctypes.c_int(), ctypes.c_int()
        _check(lib().kvp_host_append(self.handle, r, n, slots, tr, tc, tv, n, ctypes.byref(ntw), cs, cd,
                                     ctypes.byref(ncow)), "kvp_host_append")
        writes = list(zip(tr[:ntw.value], tc[:ntw.value], tv[:ntw.value]))
        cows = list(zip(cs[:ncow.value], cd[:ncow.value]))
        return list(slots[:n]), writes, cows

    def append_into(self, rids, slots, tw, cow):
        """Fast form of :meth:`append` over numpy buffers.

        ``rids`` int32[n]; outputs go to ``slots`` int32[n], ``tw`` int32[3, n]
        (rows, cols, vals) and ``cow`` int32[2, n] (src, dst). Returns the
        numbers of table writes and copy-on-write pairs."""
        n = int(rids.shape[0])
        ntw, ncow = ctypes.c_int(), ctypes.c_int()
        p = lambda a: a.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
        _check(lib().kvp_host_append(self.handle, p(rids), n, p(slots), p(tw[0]), p(tw[1]), p(tw[2]), n,
                                     ctypes.byref(ntw), p(cow[0]), p(cow[1]), ctypes.byref(ncow)), "kvp_host_append")
        return ntw.value, ncow.value

    def trim_into(self, rid, keep_from, tw, cap, sinks=0):
        """Fast form of :meth:`trim`: writes go to ``tw`` int32[3, cap]; returns their number."""
        n = ctypes.c_int()
        p = lambda a: a.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
        _check(lib().kvp_host_trim_sinks(self.handle, rid, int(keep_from), int(sinks), p(tw[0]), p(tw[1]),
                                         p(tw[2]), cap, ctypes.byref(n)), "kvp_host_trim_sinks")
        return n.value

    def trim(self, rid, keep_from, sinks=0):
        """Release the pages no later step reads: below keep_from, except the
        first ceil(sinks / P) pages. Returns the (rid, page, -1) table writes."""
        cap = max(1, self.length(rid)[0] // self.page_size + 1)
        tr, tc, tv = _i32(cap), _i32(cap), _i32(cap)
        n = ctypes.c_int()
        if sinks:
            _check(lib().kvp_host_trim_sinks(self.handle, rid, int(keep_from), int(sinks), tr, tc, tv, cap,
                                             ctypes.byref(n)), "kvp_host_trim_sinks")
        else:
            _check(lib().kvp_host_trim(self.handle, rid, int(keep_from), tr, tc, tv, cap, ctypes.byref(n)),
                   "kvp_host_trim")
        return list(zip(tr[:n.value], tc[:n.value], tv[:n.value]))

    def rewind(self, rid, n):
        """Drop the newest n tokens; returns the (rid, page, -1) table writes
        of the pages let go (tail first)."""
        cap = max(1, self.length(rid)[0] // self.page_size + 1)
        tr, tc, tv = _i32(cap), _i32(cap), _i32(cap)
        k = ctypes.c_int()
        _check(lib().kvp_host_rewind(self.handle, rid, int(n), tr, tc, tv, cap, ctypes.byref(k)), "kvp_host_rewind")
        return list(zip(tr[:k.value], tc[:k.value], tv[:k.value]))

    def used(self):
        u = ctypes.c_int()
        _check(lib().kvp_host_used(self.handle, ctypes.byref(u)), "kvp_host_used")
        return u.value

    def length(self, rid):
        L, d = ctypes.c_int(), ctypes.c_int()
        _check(lib().kvp_host_length(self.handle, rid, ctypes.byref(L), ctypes.byref(d)), "kvp_host_length")
        return L.value, d.value

    def block_row(self, rid):
        L, _ = self.length(rid)
        cap = L // self.page_size + 2
        out = _i32(cap)
        n = ctypes.c_int()
        _check(lib().kvp_host_block_row(self.handle, rid, out, cap, ctypes.byref(n)), "kvp_host_block_row")
        return list(out[:n.value])

    def refcounts(self):
        out = _i32(self.num_pages)
        _check(lib().kvp_host_refcounts(self.handle, out, self.num_pages), "kvp_host_refcounts")
        return list(out[:self.num_pages])

    def free_list(self):
        out = _i32(self.num_pages)
        n = ctypes.c_int()
        _check(lib().kvp_host_free_list(self.handle, out, self.num_pages, ctypes.byref(n)), "kvp_host_free_list")
        return list(out[:n.value])
