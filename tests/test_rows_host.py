"""Host-side checks of the gated recurrence and the residual norm (no GPU needed): refusals,
the structure layouts, the 64-bit reference's gradients against differences."""
import ctypes
import os
import re

import pytest
import torch

import rows_reference as ref
from sub_quadratic_attention_b200 import binding as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("header,prefix", [("gated_scan.h", "gated_scan_"), ("residual_norm.h", "residual_norm_")])
def test_every_declared_function_is_exported_and_bound(header, prefix):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = set(re.findall(r"\b(%s[a-z0-9_]*)\s*\(" % prefix, text))
    assert len(names) >= 5
    lib = ctypes.CDLL(b.LIB_PATH)
    for n in names:
        assert hasattr(lib, n) and n in b.SIGNATURES, n


def test_packed_arguments_have_the_header_layout():
    """The bytes that the binding packs, against the structure as a C compiler lays it out."""
    class Rows(ctypes.Structure):
        _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_longlong), ("row_stride", ctypes.c_longlong)]

    class Args(ctypes.Structure):
        _fields_ = ([("B", ctypes.c_longlong), ("L", ctypes.c_longlong), ("cu_seqlens", ctypes.c_void_p), ("nseq", ctypes.c_longlong)] +
                    [(n, Rows) for n in ("g", "v", "y", "dy", "dg", "dv")] +
                    [(n, ctypes.c_void_p) for n in ("h0", "hT", "dhT", "dh0", "states", "work")] +
                    [("work_bytes", ctypes.c_size_t), ("zero_outside", ctypes.c_int)])

    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "gated_scan.h")).read(), flags=re.S)
    body = re.search(r"typedef struct gated_scan_args \{(.*?)\}", text, re.S).group(1)
    names = [n for line in body.split(";") for n in re.findall(r"\b(\w+)\s*(?=,|$)", line.strip())]
    assert names == [n for n, _ in Args._fields_]
    rows = {n: (100 * i + 1, 100 * i + 2, 100 * i + 3) for i, n in enumerate(("g", "v", "y", "dy", "dg", "dv"))}
    rest = {n: 1000 + i for i, n in enumerate(("cu_seqlens", "nseq", "h0", "hT", "dhT", "dh0", "states", "work", "work_bytes"))}
    packed = b.gated_scan_args(7, 8, **rows, **rest, zero_outside=True)
    assert len(packed) == ctypes.sizeof(Args)
    a = Args.from_buffer_copy(packed)
    assert (a.B, a.L, a.zero_outside) == (7, 8, 1)
    for n, want in rest.items():
        assert getattr(a, n) == want, n
    for n, want in rows.items():
        r = getattr(a, n)
        assert (r.data, r.batch_stride, r.row_stride) == want, n


@pytest.mark.parametrize("args", [(0, 4, 0, 0, 0, 0), (4, 0, 0, 0, 0, 0), (2048, 1024, 0, 0, 0, 0),
                                  (2, 4, 2, 0, 0, 0), (2, 4, -1, 0, 0, 0), (2, 4, 0, 2, 0, 0),
                                  (2, 4, 0, 0, 2, 0), (2, 4, 0, 0, 1, 3), (2, 4, 0, 0, 0, 1)])
def test_scan_create_refuses(args):
    code, h = b.gated_scan_create_status(*args)
    assert code == b.SPECTRE_ERR_ARG and h is None


@pytest.mark.parametrize("args", [(0, 0, 0), (8193, 0, 0), (8, 2, 0), (8, 0, 4), (8, 0, -1),
                                  (8, 0, 0, 0.0), (8, 0, 0, float("nan")), (8, 0, 0, float("inf"))])
def test_norm_create_refuses(args):
    code, h = b.residual_norm_create_status(*args)
    assert code == b.SPECTRE_ERR_ARG and h is None


def test_null_handles():
    a = b.gated_scan_args(1, 1, (0, 0, 0), (0, 0, 0))
    assert b._lib.gated_scan_run(None, a, None) == b.SPECTRE_ERR_ARG
    assert b._lib.gated_scan_backward(None, a, None) == b.SPECTRE_ERR_ARG
    assert b._lib.gated_scan_step(None, 1, None, 0, None, 0, None, 0, None, None, 0, None, 0, None) == b.SPECTRE_ERR_ARG
    assert b._lib.gated_scan_device_status(None, None) == b._lib.residual_norm_device_status(None, None) == b.SPECTRE_ERR_ARG
    assert b.gated_scan_workspace_bytes(None, 1, 1, True) == 0
    assert b._lib.residual_norm_run(None, 1, None, 0, None, 0, None, None, None, 0, None) == b.SPECTRE_ERR_ARG
    assert b._lib.residual_norm_backward(None, 1, None, 0, None, 0, None, 0, None, None, 0, None, None, None, 0,
                                         None) == b.SPECTRE_ERR_ARG
    assert b.residual_norm_workspace_bytes(None, 1) == 0
    b.gated_scan_destroy(None)
    b.residual_norm_destroy(None)


def test_plan_names_are_checked_before_the_device():
    for kw in (dict(gate="tanh"), dict(gate_per="token"), dict(dtype="f16"), dict(gate_dtype="f64")):
        with pytest.raises(ValueError):
            b.GatedScan(2, 4, **kw)
    for kw in (dict(norm="ln"), dict(dtype="f16")):
        with pytest.raises(ValueError):
            b.ResidualNorm(8, **kw)


def _scan_tensors(dtype=torch.bfloat16, B=2, L=5, H=2, D=4, head=False):
    return torch.zeros(B, L, H if head else H * D, dtype=dtype), torch.zeros(B, L, H * D, dtype=dtype)


def test_scan_arguments():
    bf, f32 = b.SPECTRE_BF16, b.SPECTRE_F32
    g, v = _scan_tensors()
    assert b.check_scan_arguments(2, 4, 0, bf, bf, g, v, y=v, dy=None) == (2, 5)
    g, v = _scan_tensors(head=True)
    assert b.check_scan_arguments(2, 4, 1, bf, f32, g.float(), v, dg=g.float(), dv=v) == (2, 5)
    for bad in (dict(g=g[:, :4], v=v), dict(g=g, v=v.float()), dict(g=g.float(), v=v), dict(g=v, v=v),
                dict(g=g, v=v[0]), dict(g=g, v=v, y=v[:1]), dict(g=g, v=v, dg=v)):
        with pytest.raises(ValueError):
            b.check_scan_arguments(2, 4, 1, bf, bf, **bad)


def test_sequences():
    cu = torch.tensor([0, 2, 5], dtype=torch.int32)
    assert b.check_scan_sequences(3, 5, None) == 3
    assert b.check_scan_sequences(1, 5, cu) == 2
    for bad in ((2, 5, cu), (1, 5, cu.long()), (1, 5, cu[:0]), (1, 5, cu[None]), (1, 5, cu.repeat(2)[::2])):
        with pytest.raises(ValueError):
            b.check_scan_sequences(*bad)


def test_rows_and_strides():
    t = torch.zeros(3, 5, 16)
    assert b._rows_of("t", t[:, :, 8:]) == (t.data_ptr() + 32, 80, 16)
    with pytest.raises(ValueError):
        b._rows_of("t", t.transpose(1, 2))
    assert b._row_stride("t", t) == 16 and b._row_stride("t", t[..., :7]) == 16
    assert b._row_stride("t", t[:, 0]) == 80 and b._row_stride("t", t[1:2, 2:3, :4]) == 4
    assert b._row_stride("t", torch.zeros(1, 4).expand(6, 4)) == 0
    with pytest.raises(ValueError):
        b._row_stride("t", t[:, :3])
    with pytest.raises(ValueError):
        b._row_stride("t", t[..., ::2])


def test_outputs_apart():
    t, s = torch.zeros(4), torch.zeros(4)
    b._check_outputs([("y", s)], [("x", t), ("n", None)])
    with pytest.raises(ValueError):
        b._check_outputs([("y", t)], [("x", t)])
    with pytest.raises(ValueError):
        b._check_outputs([("y", s), ("z", s)], [("x", t)])


def test_norm_arguments():
    x = torch.zeros(3, 5, 8)
    w = torch.zeros(8)
    assert b.check_norm_arguments(8, 0, None, (("gamma", w),), out=x, x=x, y=None) == (3, 5, 8)
    for bad in (dict(out=x[..., :7], x=x), dict(out=x, x=x[:2]), dict(out=x, x=x.bfloat16()), dict(out=w[0], x=w[0])):
        with pytest.raises(ValueError):
            b.check_norm_arguments(8, 0, None, (("gamma", w),), **bad)
    for g in (w[:7], w.double(), torch.zeros(16)[::2]):
        with pytest.raises(ValueError):
            b.check_norm_arguments(8, 0, None, (("gamma", g),), out=x, x=x)


@pytest.mark.parametrize("form", ["sigmoid", "exp"])
@pytest.mark.parametrize("head", [False, True])
@pytest.mark.parametrize("cu", [None, [0, 3, 3, 7]])
def test_reference_gradients_against_differences(form, head, cu):
    """d/dp sum(dy y) + sum(dhT hT) by central differences: the difference's own error is
    about step^2 + 2^-52 / step, 1e-9 here; values are of order 1 to 10."""
    gen = torch.Generator().manual_seed(3)
    B, L, H, D = (2, 7, 2, 3) if cu is None else (1, 8, 2, 3)   # packed: the last row is in no sequence
    n = B if cu is None else 3
    mk = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    g = mk(B, L, H if head else H * D)
    g = -g.abs() if form == "exp" else g
    p = {"g": g, "v": mk(B, L, H * D), "h0": mk(n, H * D)}
    dy, dhT = mk(B, L, H * D), mk(n, H * D)

    def loss(q):
        val, _ = ref.scan(q["g"], q["v"], H, D, form, q["h0"], cu)
        return float((dy * val["y"].nan_to_num()).sum() + (dhT * val["hT"]).sum())

    val, _ = ref.scan(p["g"], p["v"], H, D, form, p["h0"], cu, dy, dhT)
    for name, t in p.items():
        for at in range(0, t.numel(), 5):
            d = torch.zeros(t.numel(), dtype=torch.float64)
            d[at] = 1e-5
            d = d.view_as(t)
            diff = (loss({**p, name: t + d}) - loss({**p, name: t - d})) / 2e-5
            assert abs(diff - float(val["d" + name].nan_to_num().reshape(-1)[at])) < 1e-7


@pytest.mark.parametrize("form", ["post_ln", "pre_ln", "post_rms", "pre_rms"])
def test_reference_norm_gradients_against_differences(form):
    gen = torch.Generator().manual_seed(4)
    mk = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    p = {"out": mk(3, 7), "x": mk(3, 7), "gamma": mk(7), "beta": mk(7)}
    dy = mk(3, 7)
    val, _ = ref.norm(*p.values(), form, 1e-5, dy)
    grads = {"out": val["dz"], "x": val["dz"] if form.startswith("post") else dy, "gamma": val["dgamma"],
             "beta": val["dbeta"]}
    for name, t in p.items():
        for at in range(t.numel()):
            d = torch.zeros(t.numel(), dtype=torch.float64)
            d[at] = 1e-5
            d = d.view_as(t)
            lo, hi = (ref.norm(*{**p, name: t + s * d}.values(), form, 1e-5)[0]["y"] for s in (-1, 1))
            assert abs(float((dy * (hi - lo)).sum()) / 2e-5 - float(grads[name].reshape(-1)[at])) < 1e-7
