"""ctypes binding of libspectre_mix (C ABI in include/spectre_mix.h,
include/dct_mix.h, include/gated_scan.h and include/residual_norm.h).

Argument marshalling only: every step of the mix runs in the library's CUDA
kernels.  The functions carry the C names; :class:`SpectreMix`, :class:`DctMix`,
:class:`GatedScan` and :class:`ResidualNorm` wrap a handle for use with torch
tensors.  Importing this module loads the library and raises if it has not been
built -- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
from typing import Optional, Tuple

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libspectre_mix.so")

SPECTRE_F32 = 0
SPECTRE_BF16 = 1

SPECTRE_OK = 0
SPECTRE_ERR_ARG = -1
SPECTRE_ERR_UNSUPPORTED_L = -2
SPECTRE_ERR_ALIGN = -3
SPECTRE_ERR_CUDA = -4
SPECTRE_ERR_NOMEM = -5
SPECTRE_ERR_DEVICE = -6
SPECTRE_ERR_SCRATCH = -7
SPECTRE_ERR_TIMEOUT = -8

SPECTRE_OPT_TENSOR_CORES = 1
SPECTRE_OPT_NORM = 2
SPECTRE_OPT_COMPLEX_GATE = 3
SPECTRE_OPT_TEST_WAIT_TIMEOUT = 4
SPECTRE_OPT_ROW_TENSOR_CORES = 5
SPECTRE_OPT_GRAPH = 6

# enum spectre_norm, keyed as in the oracle
SPECTRE_NORM = {"post_ln": 0, "pre_ln": 1, "post_rms": 2, "pre_rms": 3}

SPECTRE_SLICE_CUDA_CORES = 0
SPECTRE_SLICE_TENSOR_CORES = 1

# fixed device scratch behind spectre_mix_run_noalloc (SPECTRE_NOALLOC_SCRATCH_BYTES)
SPECTRE_NOALLOC_SCRATCH_BYTES = 64 << 20

GATED_SCAN_GATE = {"sigmoid": 0, "exp": 1}         # enum gated_scan_gate
GATED_SCAN_PER = {"channel": 0, "head": 1}         # enum gated_scan_per
GATED_SCAN_OPT_TEST_WAIT_TIMEOUT = 1               # enum gated_scan_option
RESIDUAL_NORM_OPT_TEST_WAIT_TIMEOUT = 1            # enum residual_norm_option
GATED_SCAN_CHUNK = 128                             # rows between two saved states

# every entry point the header declares, with its ctypes signature
_vp = ctypes.c_void_p
_i = ctypes.c_int
_ll = ctypes.c_longlong
_sz = ctypes.c_size_t


SIGNATURES = {
    "spectre_mix_create": (_i, [ctypes.POINTER(_vp), _i, _i, _i, _i, _i, _i, ctypes.c_float]),
    "spectre_mix_run": (_i, [_vp] * 10),
    "spectre_mix_run_debug": (_i, [_vp] * 11),
    "spectre_mix_run_host": (_i, [_vp] * 10),
    "spectre_mix_run_profiled": (_i, [_vp] * 10 + [_i, _vp]),
    "spectre_mix_run_noalloc": (_i, [_i] * 6 + [ctypes.c_float] + [_vp] * 9),
    "spectre_mix_destroy": (_i, [_vp]),
    "spectre_mix_device_status": (_i, [_vp, _vp]),
    "spectre_mix_set_option": (_i, [_vp, _i, _i]),
    "spectre_mix_slice_pass": (_i, [_vp]),
    "spectre_mix_error_string": (ctypes.c_char_p, [_i]),
    "spectre_mix_workspace_bytes": (ctypes.c_size_t, [_vp]),
    "spectre_mix_plan_info": (_i, [_vp] + [ctypes.POINTER(_i)] * 5),
    "dct_mix_create": (_i, [ctypes.POINTER(_vp), _i, _i, ctypes.c_float]),
    "dct_mix_run": (_i, [_vp, ctypes.c_longlong] + [_vp] * 4 + [ctypes.c_float] + [_vp] * 4),
    "dct_mix_run_debug": (_i, [_vp, ctypes.c_longlong] + [_vp] * 4 + [ctypes.c_float] + [_vp] * 5),
    "dct_mix_run_host": (_i, [_vp, ctypes.c_longlong] + [_vp] * 4 + [ctypes.c_float] + [_vp] * 4),
    "dct_mix_destroy": (_i, [_vp]),
    "gated_scan_create": (_i, [ctypes.POINTER(_vp)] + [_i] * 6),
    "gated_scan_set_option": (_i, [_vp, _i, _i]),
    "gated_scan_workspace_bytes": (_sz, [_vp, _ll, _ll, _i]),
    "gated_scan_run": (_i, [_vp, ctypes.c_char_p, _vp]),
    "gated_scan_backward": (_i, [_vp, ctypes.c_char_p, _vp]),
    "gated_scan_step": (_i, [_vp, _ll, _vp, _ll, _vp, _ll, _vp, _ll, _vp, _vp, _ll, _vp, _i, _vp]),
    "gated_scan_device_status": (_i, [_vp, _vp]),
    "gated_scan_destroy": (_i, [_vp]),
    "residual_norm_create": (_i, [ctypes.POINTER(_vp), _i, _i, _i, ctypes.c_float]),
    "residual_norm_set_option": (_i, [_vp, _i, _i]),
    "residual_norm_run": (_i, [_vp, _ll, _vp, _ll, _vp, _ll, _vp, _vp, _vp, _ll, _vp]),
    "residual_norm_workspace_bytes": (_sz, [_vp, _ll]),
    "residual_norm_backward": (_i, [_vp, _ll, _vp, _ll, _vp, _ll, _vp, _ll, _vp, _vp, _ll, _vp, _vp,
                                    _vp, _sz, _vp]),
    "residual_norm_device_status": (_i, [_vp, _vp]),
    "residual_norm_destroy": (_i, [_vp]),
}


class SpectreMixError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {spectre_mix_error_string(code)} (status {code})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"libspectre_mix.so not found at {LIB_PATH}; build it with "
            "`python -m sub_quadratic_attention_b200.build_lib` (no CPU fallback exists)")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()


def _ptr(t) -> Optional[int]:
    """Device or host address of a tensor, an int address, or None."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors passed to libspectre_mix must be contiguous")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch

        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(code: int, where: str) -> None:
    if code != SPECTRE_OK:
        raise SpectreMixError(code, where)


def spectre_mix_error_string(code: int) -> str:
    return _lib.spectre_mix_error_string(int(code)).decode()


def spectre_mix_create(B: int, L: int, H: int, D: int, F: int, dtype: int, eps: float = 1e-5) -> int:
    h = _vp()
    _check(_lib.spectre_mix_create(ctypes.byref(h), B, L, H, D, F, dtype, eps), "spectre_mix_create")
    return h.value


def spectre_mix_create_status(B: int, L: int, H: int, D: int, F: int, dtype: int,
                              eps: float = 1e-5) -> Tuple[int, Optional[int]]:
    """Raw status and handle (for tests of the error paths)."""
    h = _vp()
    code = _lib.spectre_mix_create(ctypes.byref(h), B, L, H, D, F, dtype, eps)
    return code, h.value


def spectre_mix_run(h: int, q, k, v, x, G, gamma, beta, y, stream=None) -> None:
    _check(_lib.spectre_mix_run(h, _ptr(q), _ptr(k), _ptr(v), _ptr(x), _ptr(G), _ptr(gamma),
                                _ptr(beta), _ptr(y), _stream(stream)), "spectre_mix_run")


def spectre_mix_run_status(h: int, q, k, v, x, G, gamma, beta, y, stream=None) -> int:
    return _lib.spectre_mix_run(h, _ptr(q), _ptr(k), _ptr(v), _ptr(x), _ptr(G), _ptr(gamma),
                                _ptr(beta), _ptr(y), _stream(stream))


def spectre_mix_run_debug(h: int, q, k, v, x, G, gamma, beta, y, out_f32, stream=None) -> None:
    _check(_lib.spectre_mix_run_debug(h, _ptr(q), _ptr(k), _ptr(v), _ptr(x), _ptr(G), _ptr(gamma),
                                      _ptr(beta), _ptr(y), _ptr(out_f32), _stream(stream)),
           "spectre_mix_run_debug")


def spectre_mix_run_host(h: int, q, k, v, x, G, gamma, beta, y, stream=None) -> None:
    _check(_lib.spectre_mix_run_host(h, _ptr(q), _ptr(k), _ptr(v), _ptr(x), _ptr(G), _ptr(gamma),
                                     _ptr(beta), _ptr(y), _stream(stream)), "spectre_mix_run_host")


def spectre_mix_run_profiled(h: int, q, k, v, x, G, gamma, beta, y, events, stream=None) -> None:
    """``events``: launches + 1 ``torch.cuda.Event(enable_timing=True)`` (already
    created), recorded before every kernel launch and after the last."""
    arr = (_vp * len(events))(*[e.cuda_event for e in events])
    _check(_lib.spectre_mix_run_profiled(h, _ptr(q), _ptr(k), _ptr(v), _ptr(x), _ptr(G),
                                         _ptr(gamma), _ptr(beta), _ptr(y),
                                         ctypes.cast(arr, _vp), len(events), _stream(stream)),
           "spectre_mix_run_profiled")


def spectre_mix_run_noalloc_status(B: int, L: int, H: int, D: int, F: int, dtype: int, eps: float,
                                   q, k, v, x, G, gamma, beta, y, stream=None) -> int:
    """One mix with no device allocation (the library's fixed 64 MiB scratch);
    for callers that may not call cudaMalloc.  Returns the raw status."""
    return _lib.spectre_mix_run_noalloc(B, L, H, D, F, dtype, eps, _ptr(q), _ptr(k), _ptr(v),
                                        _ptr(x), _ptr(G), _ptr(gamma), _ptr(beta), _ptr(y),
                                        _stream(stream))


def spectre_mix_run_noalloc(B: int, L: int, H: int, D: int, F: int, dtype: int, eps: float,
                            q, k, v, x, G, gamma, beta, y, stream=None) -> None:
    _check(spectre_mix_run_noalloc_status(B, L, H, D, F, dtype, eps, q, k, v, x, G, gamma, beta,
                                          y, stream), "spectre_mix_run_noalloc")


def spectre_mix_set_option(h: int, option: int, value: int) -> None:
    _check(_lib.spectre_mix_set_option(h, option, value), "spectre_mix_set_option")


def spectre_mix_slice_pass(h: int) -> int:
    """SPECTRE_SLICE_TENSOR_CORES or SPECTRE_SLICE_CUDA_CORES for the plan's runs."""
    st = _lib.spectre_mix_slice_pass(h)
    if st < 0:
        _check(st, "spectre_mix_slice_pass")
    return st


def spectre_mix_device_status(h: int, stream=None) -> int:
    """Synchronise and return SPECTRE_OK or SPECTRE_ERR_TIMEOUT for earlier runs."""
    return _lib.spectre_mix_device_status(h, _stream(stream))


def spectre_mix_destroy(h: Optional[int]) -> None:
    _check(_lib.spectre_mix_destroy(h), "spectre_mix_destroy")


def spectre_mix_workspace_bytes(h: Optional[int]) -> int:
    return int(_lib.spectre_mix_workspace_bytes(h))


def spectre_mix_plan_info(h: int) -> Tuple[int, int, int, int, int]:
    """(R, M, slices per channel, channels per wave, kernel launches per run)."""
    vals = [_i() for _ in range(5)]
    _check(_lib.spectre_mix_plan_info(h, *[ctypes.byref(v) for v in vals]), "spectre_mix_plan_info")
    return tuple(v.value for v in vals)


def check_arguments(B, L, H, C, plan_L, dtype_code, q, k, v, x, G, gamma, beta, y, out=None):
    """Sizes and element types of one run's tensors, checked on the host: the
    library reads raw pointers, so a short buffer would be read out of bounds.
    q, k, v, x, y hold B * L * C values of the plan's type (bf16 or fp32); G
    holds H * (plan_L / 2 + 1) fp32 values (complex64 for a complex gate);
    gamma, beta hold C fp32 values; out (optional) B * L * C fp32 values."""
    import torch

    n = B * L * C
    tok_type = torch.float32 if dtype_code == SPECTRE_F32 else torch.bfloat16
    for name, t in (("q", q), ("k", k), ("v", v), ("x", x), ("y", y)):
        if t.numel() != n or t.dtype != tok_type:
            raise ValueError(f"{name} must hold B * L * C = {n} values of {tok_type}")
    if out is not None and (out.numel() != n or out.dtype != torch.float32):
        raise ValueError(f"out must hold B * L * C = {n} fp32 values")
    nb = plan_L // 2 + 1
    if G.numel() != H * nb or G.dtype not in (torch.float32, torch.complex64, torch.complex128):
        raise ValueError(f"G must be [H, {nb}], fp32 (or complex for a complex gate)")
    for name, t in (("gamma", gamma), ("beta", beta)):
        if t.numel() != C or t.dtype != torch.float32:
            raise ValueError(f"{name} must hold C = {C} fp32 values")


class SpectreMix:
    """A plan for one shape, usable with torch CUDA tensors.

    ``mix(q, k, v, x, G, gamma, beta)`` returns y; pass ``out=`` (fp32
    [B, L, C]) to also receive the pre-LayerNorm mixer output.

    ``block_len``: blockwise mode (walk-through §3.2, ``fft_len``): the mix runs
    within each block of block_len consecutive tokens, as B * L / block_len
    independent sequences of length block_len.  A [B, L, C] tensor is already
    laid out as [B * L / block_len, block_len, C], so only the plan's shape
    changes; G is then [H, block_len / 2 + 1] and F counts the block's bins.
    (The pages leave the exchange between blocks unspecified; none is done.)
    """

    def __init__(self, B: int, L: int, H: int, D: int, F: Optional[int] = None,
                 dtype: str = "bf16", eps: float = 1e-5, tensor_cores: Optional[bool] = None,
                 norm: Optional[str] = None, complex_gate: bool = False,
                 block_len: Optional[int] = None, row_tensor_cores: bool = False,
                 graph: Optional[bool] = None):
        self.B, self.L, self.H, self.D = B, L, H, D
        self.C = H * D
        if block_len is not None and (block_len < 1 or L % block_len):
            raise ValueError("block_len must divide L")
        self.block_len = block_len
        self.plan_B, self.plan_L = (B * (L // block_len), block_len) if block_len else (B, L)
        self.F = self.plan_L // 2 + 1 if F is None else F
        self.dtype_code = SPECTRE_F32 if dtype in ("f32", "float32", "fp32") else SPECTRE_BF16
        self.eps = eps
        self.handle = spectre_mix_create(self.plan_B, self.plan_L, H, D, self.F, self.dtype_code, eps)
        if tensor_cores is not None:   # None keeps the library's default (on)
            spectre_mix_set_option(self.handle, SPECTRE_OPT_TENSOR_CORES, 1 if tensor_cores else 0)
        if norm is not None:           # None keeps the default, "post_ln": LayerNorm(out + x)
            spectre_mix_set_option(self.handle, SPECTRE_OPT_NORM, SPECTRE_NORM[norm])
        self.complex_gate = complex_gate
        if complex_gate:               # G: complex [H, L/2+1] (a relative-position phase)
            spectre_mix_set_option(self.handle, SPECTRE_OPT_COMPLEX_GATE, 1)
        if row_tensor_cores:           # the row pass on the tensor cores (where it applies)
            spectre_mix_set_option(self.handle, SPECTRE_OPT_ROW_TENSOR_CORES, 1)
        if graph is not None:          # None keeps the library's default
            spectre_mix_set_option(self.handle, SPECTRE_OPT_GRAPH, 1 if graph else 0)
        self._gate_ref = None

    def _check_shapes(self, q, k, v, x, G, gamma, beta, y, out):
        check_arguments(self.B, self.L, self.H, self.C, self.plan_L, self.dtype_code,
                        q, k, v, x, G, gamma, beta, y, out)

    def _gate(self, G):
        """G as the library reads it: a real gate as given, a complex one as its
        (re, im) fp32 pairs.  The converted tensor stays referenced until the
        next call, since runs are asynchronous."""
        if G.is_complex():
            if not self.complex_gate:
                raise ValueError("a complex G needs a plan made with complex_gate=True")
            import torch

            G = torch.view_as_real(G.to(torch.complex64)).contiguous()
        elif self.complex_gate:
            raise ValueError("this plan expects a complex G")
        self._gate_ref = G
        return G

    def __call__(self, q, k, v, x, G, gamma, beta, y=None, out=None, stream=None):
        import torch

        if y is None:
            y = torch.empty_like(x)
        self._check_shapes(q, k, v, x, G, gamma, beta, y, out)
        G = self._gate(G)
        if out is None:
            spectre_mix_run(self.handle, q, k, v, x, G, gamma, beta, y, stream)
        else:
            spectre_mix_run_debug(self.handle, q, k, v, x, G, gamma, beta, y, out, stream)
        return y

    def run_host(self, q, k, v, x, G, gamma, beta, y, stream=None):
        self._check_shapes(q, k, v, x, G, gamma, beta, y, None)
        G = self._gate(G)
        spectre_mix_run_host(self.handle, q, k, v, x, G, gamma, beta, y, stream)
        return y

    @property
    def workspace_bytes(self) -> int:
        return spectre_mix_workspace_bytes(self.handle)

    @property
    def plan(self) -> Tuple[int, int, int, int, int]:
        return spectre_mix_plan_info(self.handle)

    @property
    def slice_pass(self) -> str:
        """'tensor_cores' or 'cuda_cores': the slice pass runs of this plan launch."""
        sp = spectre_mix_slice_pass(self.handle)
        return "tensor_cores" if sp == SPECTRE_SLICE_TENSOR_CORES else "cuda_cores"

    def close(self) -> None:
        if self.handle is not None:
            h, self.handle = self.handle, None
            spectre_mix_destroy(h)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------------------
# per-token DCT mix with spectral-entropy routing (include/dct_mix.h)
# ---------------------------------------------------------------------------
def dct_mix_create_status(d: int, dtype: int, eps: float = 1e-5) -> Tuple[int, Optional[int]]:
    h = _vp()
    code = _lib.dct_mix_create(ctypes.byref(h), d, dtype, eps)
    return code, h.value


def dct_mix_create(d: int, dtype: int, eps: float = 1e-5) -> int:
    code, h = dct_mix_create_status(d, dtype, eps)
    _check(code, "dct_mix_create")
    return h


def dct_mix_run(h: int, T: int, x, w, gamma, beta, tau: float, y, H, route, stream=None) -> None:
    _check(_lib.dct_mix_run(h, T, _ptr(x), _ptr(w), _ptr(gamma), _ptr(beta), tau, _ptr(y),
                            _ptr(H), _ptr(route), _stream(stream)), "dct_mix_run")


def dct_mix_run_debug(h: int, T: int, x, w, gamma, beta, tau: float, y, H, route, mix,
                      stream=None) -> None:
    _check(_lib.dct_mix_run_debug(h, T, _ptr(x), _ptr(w), _ptr(gamma), _ptr(beta), tau, _ptr(y),
                                  _ptr(H), _ptr(route), _ptr(mix), _stream(stream)),
           "dct_mix_run_debug")


def dct_mix_run_host(h: int, T: int, x, w, gamma, beta, tau: float, y, H, route,
                     stream=None) -> None:
    _check(_lib.dct_mix_run_host(h, T, _ptr(x), _ptr(w), _ptr(gamma), _ptr(beta), tau, _ptr(y),
                                 _ptr(H), _ptr(route), _stream(stream)), "dct_mix_run_host")


def dct_mix_destroy(h: Optional[int]) -> None:
    _check(_lib.dct_mix_destroy(h), "dct_mix_destroy")


def check_dct_arguments(d, dtype_code, x, w, gamma, beta, y, H, route, mix=None) -> int:
    """Sizes and types of one DCT-mix run's tensors; returns T (token rows).
    x and y hold T * d values of the plan's type; w, gamma, beta d fp32
    values; H T fp32 values; route T uint8 values; mix (optional) T * d fp32."""
    import torch

    if x.numel() % d:
        raise ValueError(f"x must hold whole rows of d = {d} values")
    T = x.numel() // d
    tok_type = torch.float32 if dtype_code == SPECTRE_F32 else torch.bfloat16
    for name, t in (("x", x), ("y", y)):
        if t.numel() != T * d or t.dtype != tok_type:
            raise ValueError(f"{name} must hold T * d = {T * d} values of {tok_type}")
    for name, t in (("w", w), ("gamma", gamma), ("beta", beta)):
        if t.numel() != d or t.dtype != torch.float32:
            raise ValueError(f"{name} must hold d = {d} fp32 values")
    if H.numel() != T or H.dtype != torch.float32:
        raise ValueError(f"H must hold T = {T} fp32 values")
    if route.numel() != T or route.dtype != torch.uint8:
        raise ValueError(f"route must hold T = {T} uint8 values")
    if mix is not None and (mix.numel() != T * d or mix.dtype != torch.float32):
        raise ValueError(f"mix must hold T * d = {T * d} fp32 values")
    return T


class DctMix:
    """A DCT-mix plan for token rows of length d (Chiaroscuro Attention
    summary: the orthonormal Type-II DCT of each token, its normalised
    spectral entropy H, the route H <= tau, and LayerNorm(x + iDCT(DCT(x) * w))).

    ``mix(x, w, gamma, beta, tau)`` takes x [..., d] on the GPU and returns
    (y, H, route) shaped [..., d], [...], [...]; pass ``mix_out=`` (fp32, the
    shape of x) to also receive iDCT(DCT(x) * w).
    """

    def __init__(self, d: int, dtype: str = "bf16", eps: float = 1e-5):
        self.d = d
        self.dtype_code = SPECTRE_F32 if dtype in ("f32", "float32", "fp32") else SPECTRE_BF16
        self.eps = eps
        self.handle = dct_mix_create(d, self.dtype_code, eps)

    def __call__(self, x, w, gamma, beta, tau: float, y=None, H=None, route=None, mix_out=None,
                 stream=None):
        import torch

        lead = tuple(x.shape[:-1])
        if y is None:
            y = torch.empty_like(x)
        if H is None:
            H = torch.empty(lead, dtype=torch.float32, device=x.device)
        if route is None:
            route = torch.empty(lead, dtype=torch.uint8, device=x.device)
        T = check_dct_arguments(self.d, self.dtype_code, x, w, gamma, beta, y, H, route, mix_out)
        if mix_out is None:
            dct_mix_run(self.handle, T, x, w, gamma, beta, tau, y, H, route, stream)
        else:
            dct_mix_run_debug(self.handle, T, x, w, gamma, beta, tau, y, H, route, mix_out, stream)
        return y, H, route

    def run_host(self, x, w, gamma, beta, tau: float, y, H, route, stream=None):
        T = check_dct_arguments(self.d, self.dtype_code, x, w, gamma, beta, y, H, route)
        dct_mix_run_host(self.handle, T, x, w, gamma, beta, tau, y, H, route, stream)
        return y, H, route

    def close(self) -> None:
        if self.handle is not None:
            h, self.handle = self.handle, None
            dct_mix_destroy(h)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------------------
# operators of rows: the gated linear recurrence (include/gated_scan.h) and the
# residual norm (include/residual_norm.h)
# ---------------------------------------------------------------------------
def _dtype_code(name: str, what: str) -> int:
    if name in ("f32", "float32", "fp32"):
        return SPECTRE_F32
    if name in ("bf16", "bfloat16"):
        return SPECTRE_BF16
    raise ValueError(f"{what} must be 'f32' or 'bf16', not {name!r}")


@functools.lru_cache(maxsize=None)
def _torch():
    import torch

    return torch


@functools.lru_cache(maxsize=None)
def _torch_dtype(code: int):
    return _torch().float32 if code == SPECTRE_F32 else _torch().bfloat16


def _check_tensor(name, t, shape, dtype, device):
    """A tensor's shape (a tuple), type and device (``device`` None: any, for host tests)."""
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{name} must be {list(shape)} of {dtype}, not {list(t.shape)} of {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the plan on {device}")


def _check_plain(name, t, shape, dtype, device):
    _check_tensor(name, t, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows_of(name, t) -> Tuple[int, int, int]:
    """[B, L, N] as a gated_scan_rows: any batch and row stride, the N values contiguous."""
    sb, sl, s1 = t.stride()
    if s1 != 1 and t.shape[2] > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return t.data_ptr(), sb, sl


_NO_ROWS = (0, 0, 0)
# struct gated_scan_args, packed in one go: a call's host time counts where its rows are few
_SCAN_ARGS = struct.Struct("@qqPq" + "Pqq" * 6 + "PPPPPPNi4x")


def gated_scan_args(B, L, g, v, y=_NO_ROWS, dy=_NO_ROWS, dg=_NO_ROWS, dv=_NO_ROWS, cu_seqlens=0, nseq=0,
                    h0=0, hT=0, dhT=0, dh0=0, states=0, work=0, work_bytes=0, zero_outside=0) -> bytes:
    """struct gated_scan_args; rows as (data, batch stride, row stride), pointers as
    integers (0: NULL)."""
    return _SCAN_ARGS.pack(B, L, cu_seqlens, nseq, *g, *v, *y, *dy, *dg, *dv, h0, hT, dhT, dh0, states,
                           work, work_bytes, zero_outside)


def _address(t) -> int:
    return 0 if t is None else t.data_ptr()


def _row_stride(name, t) -> int:
    """[..., N] as rows with one stride between them; raises where they have none."""
    if t.is_contiguous():
        return t.shape[-1]
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    stride, extent = None, 1
    for size, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if stride is None:
            stride = st
        elif st != stride * extent:
            raise ValueError(f"the rows of {name} must have one stride between them")
        extent *= size
    return t.shape[-1] if stride is None else stride


def _check_outputs(outputs, inputs):
    """No output may start where an input or another output does."""
    seen = {t.data_ptr(): name for name, t in inputs if t is not None and t.numel()}
    for name, t in outputs:
        if t is None or not t.numel():
            continue
        other = seen.setdefault(t.data_ptr(), name)
        if other != name:
            raise ValueError(f"{name} may not be the same memory as {other}")


def _current_stream(device) -> int:
    return _torch()._C._cuda_getCurrentRawStream(device.index)


def _is_other_stream(stream, device) -> bool:
    if stream is None:
        return False
    return (stream if isinstance(stream, int) else stream.cuda_stream) != _current_stream(device)


def _on_stream(stream, device, call, *tensors):
    """call(*tensors) with ``stream`` as the current one.  What the call makes is that
    stream's memory then: in the caller's stream's own, work enqueued earlier could
    still be writing.  The caller's tensors are marked as in use on ``stream`` and the
    results as in use on the caller's, so that neither are handed out too early."""
    torch = _torch()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    here = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        results = call(*tensors)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    for t in results if isinstance(results, tuple) else (results,):
        if t is not None:
            t.record_stream(here)
    return results


def gated_scan_create_status(H: int, D: int, gate: int, per: int, dtype: int,
                             gate_dtype: int) -> Tuple[int, Optional[int]]:
    h = _vp()
    code = _lib.gated_scan_create(ctypes.byref(h), H, D, gate, per, dtype, gate_dtype)
    return code, h.value


def gated_scan_create(H: int, D: int, gate: int, per: int, dtype: int, gate_dtype: int) -> int:
    code, h = gated_scan_create_status(H, D, gate, per, dtype, gate_dtype)
    _check(code, "gated_scan_create")
    return h


def gated_scan_set_option(h: int, option: int, value: int) -> None:
    _check(_lib.gated_scan_set_option(h, option, value), "gated_scan_set_option")


def gated_scan_workspace_bytes(h: Optional[int], B: int, L: int, backward: bool) -> int:
    return int(_lib.gated_scan_workspace_bytes(h, B, L, int(backward)))


def gated_scan_run(h: int, args: bytes, stream: int) -> None:
    """``args``: gated_scan_args(...)."""
    _check(_lib.gated_scan_run(h, args, stream), "gated_scan_run")


def gated_scan_backward(h: int, args: bytes, stream: int) -> None:
    _check(_lib.gated_scan_backward(h, args, stream), "gated_scan_backward")


def gated_scan_device_status(h: int, stream=None) -> int:
    """Synchronise and return SPECTRE_OK or SPECTRE_ERR_TIMEOUT for earlier scans."""
    return _lib.gated_scan_device_status(h, _stream(stream))


def gated_scan_destroy(h: Optional[int]) -> None:
    _check(_lib.gated_scan_destroy(h), "gated_scan_destroy")


def check_scan_sequences(B, L, cu_seqlens, device=None) -> int:
    """Sequences of a call: B, or those of cu_seqlens (int32 [N + 1], B = 1)."""
    torch = _torch()
    if cu_seqlens is None:
        return B
    if B != 1:
        raise ValueError("packed sequences (cu_seqlens) are rows of one batch entry: B must be 1")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must hold one offset more than sequences")
    _check_plain("cu_seqlens", cu_seqlens, cu_seqlens.shape, torch.int32, device)
    return cu_seqlens.numel() - 1


def check_scan_arguments(H, D, per, dtype_code, gate_code, g, v, device=None, **rows) -> Tuple[int, int]:
    """Shapes and types of g, v and further tensors of rows (y, dy, dv as v; dg as g);
    returns (B, L)."""
    if v.dim() != 3:
        raise ValueError(f"v must be [B, L, C = {H * D}]")
    B, L, _ = v.shape
    of_v, of_g = (B, L, H * D), (B, L, H if per == GATED_SCAN_PER["head"] else H * D)
    type_v, type_g = _torch_dtype(dtype_code), _torch_dtype(gate_code)
    _check_tensor("v", v, of_v, type_v, device)
    _check_tensor("g", g, of_g, type_g, device)
    for name, t in rows.items():
        if t is not None:
            gate = name == "dg"
            _check_tensor(name, t, of_g if gate else of_v, type_g if gate else type_v, device)
    return B, L


class GatedScan:
    """The gated linear recurrence over [B, L, C = H * D]: a causal token mixer,
    trained with :meth:`backward` and served token by token with :meth:`step`.

        h_t = a_t h_{t-1} + b_t,  y_t = h_t

    gate="sigmoid": a = sigmoid(g), b = (1 - a) v;  gate="exp": a = exp(g), b = v with
    log decays g <= 0.  gate_per="channel": g is [B, L, C]; "head": [B, L, H].  v and y
    are of ``dtype``, g of ``gate_dtype`` ("f32" or the plan's); states are fp32.

    ``scan(g, v)`` returns (y, hT), hT [B, C] the state after the last row.  With
    ``cu_seqlens`` (int32, N + 1 offsets on the GPU) the L rows of one batch entry are N
    sequences packed one after another, and states are [N, C]; rows in no sequence are
    left as they are in tensors that the caller gives, and zero in those made here.
    For training pass ``states=scan.new_states(B, L)`` to the call and to
    :meth:`backward`.  g, v and dy may be slices of wider rows; the plan holds nothing
    of a call, so it may be used on several streams and threads, and inside a graph's
    capture.  A call with ``stream=`` runs as if that were the current stream: its inputs
    must be ready there.  No autograd graph is recorded: backward() is called explicitly.
    """

    def __init__(self, H: int, D: int, dtype: str = "bf16", gate: str = "sigmoid",
                 gate_per: str = "channel", gate_dtype: Optional[str] = None):
        torch = _torch()
        self.handle = None
        if gate not in GATED_SCAN_GATE or gate_per not in GATED_SCAN_PER:
            raise ValueError("gate must be 'sigmoid' or 'exp', gate_per 'channel' or 'head'")
        self.H, self.D, self.C = H, D, H * D
        self.dtype_code = _dtype_code(dtype, "dtype")
        self.gate_code = self.dtype_code if gate_dtype is None else _dtype_code(gate_dtype, "gate_dtype")
        self.gate, self.per = GATED_SCAN_GATE[gate], GATED_SCAN_PER[gate_per]
        self.handle = gated_scan_create(H, D, self.gate, self.per, self.dtype_code, self.gate_code)
        self.device = torch.device("cuda", torch.cuda.current_device())

    def new_states(self, B: int, L: int):
        """The tensor that a training forward fills and backward reads: the fp32 state
        before every GATED_SCAN_CHUNK-th row."""
        torch = _torch()
        return torch.empty((B, -(-L // GATED_SCAN_CHUNK), self.C), dtype=torch.float32, device=self.device)

    def _check_states(self, B, L, nseq, states, **ends):
        torch = _torch()
        if states is not None:
            _check_plain("states", states, (B, -(-L // GATED_SCAN_CHUNK), self.C), torch.float32, self.device)
        for name, t in ends.items():
            if t is not None:
                _check_plain(name, t, (nseq, self.C), torch.float32, self.device)

    def _work(self, B, L, backward):
        torch = _torch()
        n = gated_scan_workspace_bytes(self.handle, B, L, backward)
        return (torch.empty(n, dtype=torch.uint8, device=self.device), n) if n else (None, 0)

    def __call__(self, g, v, h0=None, cu_seqlens=None, y=None, hT=None, states=None, stream=None):
        torch = _torch()
        device = self.device
        if _is_other_stream(stream, device):
            return _on_stream(stream, device, self, g, v, h0, cu_seqlens, y, hT, states)
        B, L = check_scan_arguments(self.H, self.D, self.per, self.dtype_code, self.gate_code, g, v, device)
        nseq = B if cu_seqlens is None else check_scan_sequences(B, L, cu_seqlens, device)
        if y is not None:
            _check_tensor("y", y, (B, L, self.C), v.dtype, device)
        if h0 is not None or hT is not None or states is not None:
            self._check_states(B, L, nseq, states, h0=h0, hT=hT)
        if y is not None or hT is not None or states is not None:
            _check_outputs([("y", y), ("hT", hT), ("states", states)], [("g", g), ("v", v), ("h0", h0)])
        made = y is None
        if made:
            y = torch.empty((B, L, self.C), dtype=v.dtype, device=device)
        if hT is None:
            hT = torch.empty((nseq, self.C), dtype=torch.float32, device=device)
        work, n = self._work(B, L, False)
        a = gated_scan_args(B, L, _rows_of("g", g), _rows_of("v", v), _rows_of("y", y),
                            cu_seqlens=_address(cu_seqlens), nseq=nseq, h0=_address(h0), hT=hT.data_ptr(),
                            states=_address(states), work=_address(work), work_bytes=n, zero_outside=made)
        gated_scan_run(self.handle, a, _current_stream(device))
        return y, hT

    def backward(self, dy, g, v, states, h0=None, dhT=None, cu_seqlens=None, dg=None, dv=None,
                 dh0=None, stream=None):
        """(dg, dv, dh0) from dy (and dhT, the gradient of the final states); dh0 is None
        where h0 is None and no dh0 is given.  ``states`` is what the forward call with the
        same g, v, h0 and cu_seqlens filled."""
        torch = _torch()
        device = self.device
        if _is_other_stream(stream, device):
            return _on_stream(stream, device, self.backward, dy, g, v, states, h0, dhT, cu_seqlens, dg, dv, dh0)
        B, L = check_scan_arguments(self.H, self.D, self.per, self.dtype_code, self.gate_code, g, v,
                                    device, dy=dy, dg=dg, dv=dv)
        nseq = B if cu_seqlens is None else check_scan_sequences(B, L, cu_seqlens, device)
        if states is None:
            raise ValueError("backward needs the states that the forward call filled")
        if (dg is None) != (dv is None):
            raise ValueError("dg and dv are given together or not at all")
        self._check_states(B, L, nseq, states, h0=h0, dhT=dhT, dh0=dh0)
        made = dg is None
        if not made or dh0 is not None:
            _check_outputs([("dg", dg), ("dv", dv), ("dh0", dh0)],
                           [("g", g), ("v", v), ("dy", dy), ("h0", h0), ("dhT", dhT), ("states", states)])
        if made:
            dg = torch.empty(g.shape, dtype=g.dtype, device=device)
            dv = torch.empty((B, L, self.C), dtype=v.dtype, device=device)
        if dh0 is None and h0 is not None:
            dh0 = torch.empty((nseq, self.C), dtype=torch.float32, device=device)
        work, n = self._work(B, L, True)
        a = gated_scan_args(B, L, _rows_of("g", g), _rows_of("v", v), dy=_rows_of("dy", dy),
                            dg=_rows_of("dg", dg), dv=_rows_of("dv", dv), cu_seqlens=_address(cu_seqlens),
                            nseq=nseq, h0=_address(h0), dhT=_address(dhT), dh0=_address(dh0),
                            states=states.data_ptr(), work=_address(work), work_bytes=n, zero_outside=made)
        gated_scan_backward(self.handle, a, _current_stream(device))
        return dg, dv, dh0

    def step(self, g, v, state, slots=None, y=None, new_state=None, stream=None):
        """One token of each of B sequences: g [B, C or H], v [B, C], ``state`` the fp32 pool
        [S, C], ``slots`` (int32 [B]) each row's place in it (None: row i has place i).
        Returns (y, new_state); new_state is the pool itself, updated in place, unless
        another tensor is given (its other rows are left as they are).  A row whose slot is
        outside the pool is skipped: its y is left as it is, or zero where y is made here."""
        torch = _torch()
        device, B, C = self.device, v.shape[0], self.C
        if _is_other_stream(stream, device):
            return _on_stream(stream, device, self.step, g, v, state, slots, y, new_state)
        _check_tensor("g", g, (B, self.H if self.per == GATED_SCAN_PER["head"] else C),
                      _torch_dtype(self.gate_code), device)
        _check_tensor("v", v, (B, C), _torch_dtype(self.dtype_code), device)
        S = state.shape[0]
        _check_plain("state", state, (S, C), torch.float32, device)
        if new_state is None:
            new_state = state
        else:
            _check_plain("new_state", new_state, (S, C), torch.float32, device)
        if slots is not None:
            _check_plain("slots", slots, (B,), torch.int32, device)
        elif S < B:
            raise ValueError(f"state holds {S} rows, the step has {B}")
        made = y is None
        if made:
            y = torch.empty((B, C), dtype=v.dtype, device=device)
        else:
            _check_tensor("y", y, (B, C), v.dtype, device)
            _check_outputs([("y", y)], [("g", g), ("v", v), ("state", state), ("new_state", new_state)])
        (gs, g1), (vs, v1), (ys, y1) = g.stride(), v.stride(), y.stride()
        if (g1 != 1 and g.shape[1] > 1) or (C > 1 and not v1 == y1 == 1):
            raise ValueError("the last dimension of g, v and y must be contiguous")
        _check(_lib.gated_scan_step(self.handle, B, g.data_ptr(), gs, v.data_ptr(), vs, state.data_ptr(), S,
                                    None if slots is None else slots.data_ptr(), y.data_ptr(), ys,
                                    new_state.data_ptr(), made, _current_stream(device)), "gated_scan_step")
        return y, new_state

    def close(self) -> None:
        if self.handle is not None:
            h, self.handle = self.handle, None
            gated_scan_destroy(h)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def residual_norm_create_status(C: int, dtype: int, norm: int, eps: float = 1e-5) -> Tuple[int, Optional[int]]:
    h = _vp()
    code = _lib.residual_norm_create(ctypes.byref(h), C, dtype, norm, eps)
    return code, h.value


def residual_norm_create(C: int, dtype: int, norm: int, eps: float = 1e-5) -> int:
    code, h = residual_norm_create_status(C, dtype, norm, eps)
    _check(code, "residual_norm_create")
    return h


def residual_norm_set_option(h: int, option: int, value: int) -> None:
    _check(_lib.residual_norm_set_option(h, option, value), "residual_norm_set_option")


def residual_norm_workspace_bytes(h: Optional[int], T: int) -> int:
    return int(_lib.residual_norm_workspace_bytes(h, T))


def residual_norm_device_status(h: int, stream=None) -> int:
    """Synchronise and return SPECTRE_OK or SPECTRE_ERR_TIMEOUT for earlier norms."""
    return _lib.residual_norm_device_status(h, _stream(stream))


def residual_norm_destroy(h: Optional[int]) -> None:
    _check(_lib.residual_norm_destroy(h), "residual_norm_destroy")


def check_norm_arguments(C, dtype_code, device=None, vectors=(), **rows) -> Tuple[int, ...]:
    """Shapes and types of a residual norm's tensors: rows [..., C] of the plan's type,
    all of one shape, and ``vectors`` ((name, tensor), ...) of C fp32 values.  Returns
    that shape."""
    torch = _torch()
    shape, dtype = None, _torch_dtype(dtype_code)
    for name, t in rows.items():
        if t is None:
            continue
        if shape is None:
            shape = t.shape
            if not shape or shape[-1] != C:
                raise ValueError(f"{name} must be [..., C = {C}]")
        _check_tensor(name, t, shape, dtype, device)
    for name, t in vectors:
        if t is not None:
            _check_plain(name, t, (C,), torch.float32, device)
    return shape


class ResidualNorm:
    """y = N(out + x) (norm="post_ln", "post_rms") or N(out) + x ("pre_ln", "pre_rms"),
    N LayerNorm or RMSNorm over the last dimension: the forms that SpectreMix fuses, as an
    operator of its own with its backward pass.

    ``norm(out, x, gamma, beta)`` takes rows [..., C] and returns y.
    ``norm.backward(dy, out, x, gamma)`` returns (dout, dx, dgamma, dbeta); dx is dout in
    the post forms and dy in the pre forms, the same tensor.  Rows may be slices of wider
    rows.  The plan holds nothing of a call (see GatedScan); no autograd graph is recorded.
    """

    def __init__(self, C: int, dtype: str = "bf16", norm: str = "post_ln", eps: float = 1e-5):
        torch = _torch()
        self.handle = None
        if norm not in SPECTRE_NORM:
            raise ValueError(f"norm must be one of {sorted(SPECTRE_NORM)}, not {norm!r}")
        self.C, self.eps, self.norm = C, eps, norm
        self.post = norm.startswith("post")
        self.dtype_code = _dtype_code(dtype, "dtype")
        self.handle = residual_norm_create(C, self.dtype_code, SPECTRE_NORM[norm], eps)
        self.device = torch.device("cuda", torch.cuda.current_device())

    def __call__(self, out, x, gamma, beta, y=None, stream=None):
        torch = _torch()
        if _is_other_stream(stream, self.device):
            return _on_stream(stream, self.device, self, out, x, gamma, beta, y)
        check_norm_arguments(self.C, self.dtype_code, self.device, (("gamma", gamma), ("beta", beta)),
                             out=out, x=x, y=y)
        C = self.C
        if y is None:
            y, y_stride = torch.empty(x.shape, dtype=x.dtype, device=self.device), C
        else:
            _check_outputs([("y", y)], [("out", out), ("x", x)])
            y_stride = _row_stride("y", y)
        _check(_lib.residual_norm_run(self.handle, x.numel() // C, out.data_ptr(), _row_stride("out", out),
                                      x.data_ptr(), _row_stride("x", x), gamma.data_ptr(), beta.data_ptr(),
                                      y.data_ptr(), y_stride, _current_stream(self.device)), "residual_norm_run")
        return y

    def backward(self, dy, out, x, gamma, dout=None, dgamma=None, dbeta=None, stream=None):
        torch = _torch()
        if _is_other_stream(stream, self.device):
            return _on_stream(stream, self.device, self.backward, dy, out, x, gamma, dout, dgamma, dbeta)
        if self.post and x is None:
            raise ValueError("the post forms' gradient needs x")
        check_norm_arguments(self.C, self.dtype_code, self.device,
                             (("gamma", gamma), ("dgamma", dgamma), ("dbeta", dbeta)),
                             dy=dy, out=out, x=x, dout=dout)
        if dout is not None or dgamma is not None or dbeta is not None:
            _check_outputs([("dout", dout), ("dgamma", dgamma), ("dbeta", dbeta)],
                           [("dy", dy), ("out", out), ("x", x), ("gamma", gamma)])
        if dout is None:
            dout = torch.empty(out.shape, dtype=out.dtype, device=self.device)
        if dgamma is None:
            dgamma = torch.empty(self.C, dtype=torch.float32, device=self.device)
        if dbeta is None:
            dbeta = torch.empty(self.C, dtype=torch.float32, device=self.device)
        T = out.numel() // self.C
        n = residual_norm_workspace_bytes(self.handle, T)
        work = torch.empty(n, dtype=torch.uint8, device=self.device) if n else None
        _check(_lib.residual_norm_backward(
            self.handle, T, dy.data_ptr(), _row_stride("dy", dy), out.data_ptr(), _row_stride("out", out),
            x.data_ptr() if self.post else None, _row_stride("x", x) if self.post else 0, gamma.data_ptr(),
            dout.data_ptr(), _row_stride("dout", dout), dgamma.data_ptr(), dbeta.data_ptr(), _ptr(work), n,
            _current_stream(self.device)), "residual_norm_backward")
        return dout, dout if self.post else dy, dgamma, dbeta

    def close(self) -> None:
        if self.handle is not None:
            h, self.handle = self.handle, None
            residual_norm_destroy(h)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
