"""The residual norm on the GPU, forward and backward, against the 64-bit reference with its
derived error bounds (rows_reference.py)."""
import math
import threading

import pytest
import torch

import rows_reference as ref
from sub_quadratic_attention_b200 import binding as b

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
FORMS = ["post_ln", "pre_ln", "post_rms", "pre_rms"]
EPS = 1e-5


def _inputs(T, C, dtype, seed=0, shift=0.0, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    out, x, dy = ((torch.randn(T, C, generator=gen) * scale + s).to(TYPES[dtype]) for s in (shift, 0.0, 0.0))
    gamma, beta = torch.randn(C, generator=gen) * 0.1 + 1, torch.randn(C, generator=gen) * 0.1
    return out, x, dy, gamma, beta


def _check(form, dtype, out, x, dy, gamma, beta, place=lambda t: t):
    o, xx, d = (place(t.cuda()) for t in (out, x, dy))
    with b.ResidualNorm(out.shape[-1], dtype, form, EPS) as n:
        y = n(o, xx, gamma.cuda(), beta.cuda())
        dout, dx, dgamma, dbeta = n.backward(d, o, xx, gamma.cuda())
        again = n.backward(d, o, xx, gamma.cuda())
        torch.cuda.synchronize()
        assert b.residual_norm_device_status(n.handle) == b.SPECTRE_OK
    assert dx is (dout if form.startswith("post") else d)
    for p, q in zip((dout, dgamma, dbeta), (again[0], again[2], again[3])):
        assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))
    val, err = ref.norm(out, x, gamma, beta, form, EPS, dy)
    for name, got in (("y", y), ("dz", dout), ("dgamma", dgamma), ("dbeta", dbeta)):
        ref.check(name, got, val[name], err[name])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,C", [(37, 64), (5, 231), (300, 512), (3, 2048)])
def test_forms_and_types(T, C, dtype, form):
    _check(form, dtype, *_inputs(T, C, dtype))


@pytest.mark.parametrize("C", [1, 2, 3, 4, 7, 8, 16, 24, 31, 33, 63, 65, 72, 100, 127, 129, 255, 256, 257, 264, 511, 513, 520, 1000, 1023,
                               1024, 1025, 2040, 2047, 2049, 2056, 4095, 4096, 4104, 8184, 8191, 8192])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_widths(C, dtype):
    _check("post_ln", dtype, *_inputs(11, C, dtype, seed=C))
    _check("pre_rms", dtype, *_inputs(11, C, dtype, seed=C))


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 295, 296, 297, 1185, 2371, 5003])
@pytest.mark.parametrize("C", [40, 300, 2048])
def test_row_counts(T, C):
    _check("pre_ln", "bf16", *_inputs(T, C, "bf16", seed=T))


def test_many_rows():
    _check("post_rms", "f32", *_inputs(40000, 16, "f32"))


@pytest.mark.parametrize("dtype,shift", [("f32", 1000.0), ("bf16", 100.0)])
@pytest.mark.parametrize("form", ["post_ln", "pre_ln"])
def test_large_mean(form, dtype, shift):
    _check(form, dtype, *_inputs(9, 520, dtype, shift=shift))


def test_outlier_channel():
    out, x, dy, gamma, beta = _inputs(9, 512, "f32")
    out[:, 0] = 3000.0
    _check("post_ln", "f32", out, x, dy, gamma, beta)


@pytest.mark.parametrize("form", FORMS)
def test_constant_and_zero_rows(form):
    """No variance: eps alone under the root.  Values that sum without rounding, so that the mean is exact."""
    out, x, dy, gamma, beta = _inputs(6, 256, "f32")
    out[0], x[0] = 0.0, 0.0
    out[1], x[1] = 2.0, 0.0
    out[2], x[2] = -4.0, 1.0
    _check(form, "f32", out, x, dy, gamma, beta)


@pytest.mark.parametrize("form", FORMS)
def test_nan_and_infinity_stay_in_their_row(form):
    out, x, dy, gamma, beta = _inputs(40, 264, "bf16")
    clean = out.clone()
    out[3, 5], out[17, 263], out[18, 0] = math.nan, math.inf, -math.inf
    with b.ResidualNorm(264, "bf16", form, EPS) as n:
        y = n(out.cuda(), x.cuda(), gamma.cuda(), beta.cuda())
        dz, _, _, dbeta = n.backward(dy.cuda(), out.cuda(), x.cuda(), gamma.cuda())
        torch.cuda.synchronize()
    val, err = ref.norm(clean, x, gamma, beta, form, EPS, dy)
    fine = torch.ones(40, dtype=torch.bool)
    fine[[3, 17, 18]] = False
    ref.check("y", y[fine.cuda()], val["y"][fine], err["y"][fine])
    ref.check("dz", dz[fine.cuda()], val["dz"][fine], err["dz"][fine])
    ref.check("dbeta", dbeta, val["dbeta"], err["dbeta"])
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(y[17, 263])) and bool(torch.isnan(y[18, 0]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("left,right", [(0, 8), (8, 0), (1, 3), (4, 1), (3, 5)])
def test_strided_rows(dtype, left, right):
    def place(t):
        big = torch.full((t.shape[0], t.shape[1] + left + right), float("nan"), dtype=t.dtype, device="cuda")
        big[:, left:left + t.shape[1]] = t
        return big[:, left:left + t.shape[1]]
    for C in (256, 250):
        _check("post_ln", dtype, *_inputs(13, C, dtype), place=place)


def test_output_rows_between_others():
    """Outputs as slices of wider rows leave what lies between."""
    out, x, dy, gamma, beta = _inputs(13, 40, "bf16")
    big = torch.full((13, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    with b.ResidualNorm(40, "bf16", "post_ln", EPS) as n:
        y = n(out.cuda(), x.cuda(), gamma.cuda(), beta.cuda(), y=big[:, 8:48])
        assert torch.equal(y, n(out.cuda(), x.cuda(), gamma.cuda(), beta.cuda()))
    assert bool((big[:, :8] == 7).all()) and bool((big[:, 48:] == 7).all())


def test_leading_dimensions_and_broadcast_rows():
    out, x, dy, gamma, beta = _inputs(24, 64, "f32")
    with b.ResidualNorm(64, "f32", "post_ln", EPS) as n:
        g, be = gamma.cuda(), beta.cuda()
        y = n(out.cuda().view(2, 3, 4, 64), x.cuda().view(2, 3, 4, 64), g, be)
        assert y.shape == (2, 3, 4, 64) and torch.equal(y.view(24, 64), n(out.cuda(), x.cuda(), g, be))
        row = x[:1].cuda().expand(24, 64)
        assert torch.equal(n(out.cuda(), row, g, be), n(out.cuda(), row.contiguous(), g, be))
        one = n(out[0].cuda(), x[0].cuda(), g, be)
        assert one.shape == (64,) and torch.equal(one, y.view(24, 64)[0])
        with pytest.raises(ValueError):
            n(out.cuda().view(2, 12, 64)[:, :5], x.cuda().view(2, 12, 64)[:, :5], g, be)


def test_vectors_at_any_alignment():
    """gamma and beta may start anywhere: the rows then go value by value."""
    out, x, dy, gamma, beta = _inputs(13, 64, "f32")
    g, be = (torch.cat([torch.zeros(1), t]).cuda()[1:] for t in (gamma, beta))
    with b.ResidualNorm(64, "f32", "post_ln", EPS) as n:
        y = n(out.cuda(), x.cuda(), g, be)
        dz, _, dgamma, dbeta = n.backward(dy.cuda(), out.cuda(), x.cuda(), g)
        torch.cuda.synchronize()
    val, err = ref.norm(out, x, gamma, beta, "post_ln", EPS, dy)
    for name, got in (("y", y), ("dz", dz), ("dgamma", dgamma), ("dbeta", dbeta)):
        ref.check(name, got, val[name], err[name])


def test_no_rows():
    with b.ResidualNorm(64, "bf16", "post_ln") as n:
        e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
        w = torch.ones(64, device="cuda")
        assert n(e, e.clone(), w, w).shape == (0, 64)
        dout, _, dgamma, dbeta = n.backward(e, e, e, w)
        assert dout.shape == (0, 64) and not bool(dgamma.any()) and not bool(dbeta.any())


def test_offsets_beyond_32_bits():
    T, C, stride = 300, 64, 1 << 23
    big = torch.empty(T * stride, dtype=torch.bfloat16, device="cuda")
    out, x, dy, gamma, beta = _inputs(T, C, "bf16")
    o = big.as_strided((T, C), (stride, 1))
    o.copy_(out)
    y, dz = big.as_strided((T, C), (stride, 1), 256), big.as_strided((T, C), (stride, 1), 512)
    with b.ResidualNorm(C, "bf16", "post_ln", EPS) as n:
        n(o, x.cuda(), gamma.cuda(), beta.cuda(), y=y)
        n.backward(dy.cuda(), o, x.cuda(), gamma.cuda(), dout=dz)
        torch.cuda.synchronize()
    val, err = ref.norm(out, x, gamma, beta, "post_ln", EPS, dy)
    ref.check("y", y, val["y"], err["y"])
    ref.check("dz", dz, val["dz"], err["dz"])


def test_streams_and_graphs():
    out, x, dy, gamma, beta = (t.cuda() for t in _inputs(3000, 512, "bf16"))
    with b.ResidualNorm(512, "bf16", "post_ln", EPS) as n:
        want = [n(out, x, gamma, beta), *n.backward(dy, out, x, gamma)]
        torch.cuda.synchronize()
        streams, got = [torch.cuda.Stream() for _ in range(2)], []
        for i in range(6):
            q = streams[i % 2]
            got.append([n(out, x, gamma, beta, stream=q), *n.backward(dy, out, x, gamma, stream=q.cuda_stream)])
        torch.cuda.synchronize()
        graphs = []
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                res = [n(out, x, gamma, beta), *n.backward(dy, out, x, gamma)]
            graphs.append(graph)
            got.append(res)
        for q, graph in zip(streams, graphs):
            with torch.cuda.stream(q):
                graph.replay()
        torch.cuda.synchronize()
        for one in got:
            assert all(torch.equal(p, q) for p, q in zip(want, one))


def test_matches_the_spectral_mix_fused_norm():
    """The forms are those that SpectreMix fuses: N(out + x) from its pre-norm output gives its y, both within
    4e-6 of the exact norm here (fp32 rows of 64 channels, |y| under 10)."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    B, L, H, D = 1, 256, 1, 64
    q, k, v, x = (torch.randn(B, L, H * D, generator=gen, device="cuda") for _ in range(4))
    G = torch.rand(H, L // 2 + 1, generator=gen, device="cuda") / L
    gamma, beta = torch.rand(64, generator=gen, device="cuda") + 0.5, torch.rand(64, generator=gen, device="cuda")
    for form in FORMS:
        with b.SpectreMix(B, L, H, D, None, "f32", EPS, norm=form) as mix, b.ResidualNorm(64, "f32", form, EPS) as n:
            out = torch.empty(B, L, 64, device="cuda")
            y = mix(q, k, v, x, G, gamma, beta, out=out)
            mine = n(out, x, gamma, beta)
            torch.cuda.synchronize()
        val, err = ref.norm(out.cpu()[0], x.cpu()[0], gamma.cpu(), beta.cpu(), form, EPS)
        ref.check("y", mine[0], val["y"], err["y"])
        ref.check("fused y", y[0], val["y"], 4 * err["y"] + 1e-5)


def test_refusals():
    out, x, dy, gamma, beta = (t.cuda() for t in _inputs(8, 64, "bf16"))
    with b.ResidualNorm(64, "bf16", "post_ln") as n:
        for bad in ((out.cpu(), x, gamma, beta), (out[:, :63], x, gamma, beta), (out.float(), x, gamma, beta),
                    (out, x, gamma.bfloat16(), beta), (out, x, gamma, beta[:8]), (out, x, gamma, beta, x)):
            with pytest.raises(ValueError):
                n(*bad)
        for bad in ((dy, out, None, gamma), (dy[:4], out, x, gamma), (dy, out, x, gamma, dy)):
            with pytest.raises(ValueError):
                n.backward(*bad)
        with pytest.raises(b.SpectreMixError):
            n(out, x, gamma, beta, y=torch.empty(1, 64, dtype=torch.bfloat16, device="cuda").expand(8, 64))
        p = [t.data_ptr() for t in (out, x, gamma, beta, dy)]
        y = torch.empty_like(out)
        run = b._lib.residual_norm_run
        assert run(n.handle, 8, p[0] + 1, 64, p[1], 64, p[2], p[3], y.data_ptr(), 64, None) == b.SPECTRE_ERR_ALIGN
        assert run(n.handle, 8, p[0], -1, p[1], 64, p[2], p[3], y.data_ptr(), 64, None) == b.SPECTRE_ERR_ARG
        assert run(n.handle, 8, p[0], 64, p[1], 64, None, p[3], y.data_ptr(), 64, None) == b.SPECTRE_ERR_ARG
        need = b.residual_norm_workspace_bytes(n.handle, 8000)
        w = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
        assert need > 0

        def back(work, size):
            return b._lib.residual_norm_backward(n.handle, 8000, p[4], 0, p[0], 0, p[1], 0, p[2], y.data_ptr(), 64, p[2],
                                                 p[3], work, size, None)
        assert back(w.data_ptr(), need - 1) == b.SPECTRE_ERR_ARG and back(None, need) == b.SPECTRE_ERR_ARG
        assert back(w.data_ptr() + 4, need) == b.SPECTRE_ERR_ALIGN


def test_two_threads_with_plans_of_two_widths():
    """Plans whose backward passes are one kernel with rings of two sizes, called from two threads at a time."""
    T, calls = 64, 4000
    widths, codes, made, errors = (1992, 2000), {}, {}, []
    go = threading.Barrier(2)

    def work(C):
        try:
            out, x, dy, gamma, _ = (t.cuda() for t in _inputs(T, C, "bf16", seed=C))
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.current_stream())
            with b.ResidualNorm(C, "bf16", "post_ln", EPS) as n:
                dz, dg, db = torch.empty_like(out), torch.empty_like(gamma), torch.empty_like(gamma)
                size = b.residual_norm_workspace_bytes(n.handle, T)
                w = torch.empty(size, dtype=torch.uint8, device="cuda")
                torch.cuda.synchronize()
                args = (n.handle, T, dy.data_ptr(), C, out.data_ptr(), C, x.data_ptr(), C, gamma.data_ptr(), dz.data_ptr(), C,
                        dg.data_ptr(), db.data_ptr(), w.data_ptr(), size, stream.cuda_stream)
                run = b._lib.residual_norm_backward
                go.wait(timeout=60)
                codes[C] = [run(*args) for _ in range(calls)]
                stream.synchronize()
                made[C] = dz, dg, db
        except Exception as e:      # an assertion in a thread would go unseen
            errors.append(e)

    threads = [threading.Thread(target=work, args=(C,)) for C in widths]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for C in widths:
        assert codes[C] == [b.SPECTRE_OK] * calls
        out, x, dy, gamma, beta = _inputs(T, C, "bf16", seed=C)
        val, err = ref.norm(out, x, gamma, beta, "post_ln", EPS, dy)
        for name, got in zip(("dz", "dgamma", "dbeta"), made[C]):
            ref.check(name, got, val[name], err[name])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("T,C,dtype", [(5, 512, "bf16"), (3000, 2048, "bf16"), (3000, 200, "bf16"), (700, 8192, "bf16"), (2500, 1000, "f32")])
def test_copies_that_do_not_come_leave_nan(T, C, dtype, form):
    """The wait for copies of rows made to give up while they are on their way: they are waited for again, the rows
    and the weights' gradients are NaN, the status is reported once, and the next calls are right."""
    if dtype == "f32" and form.startswith("post"):
        form = form.replace("post", "pre")      # fp32 rows of three inputs are loaded, without a wait
    out, x, dy, gamma, _ = (t.cuda() for t in _inputs(T, C, dtype))
    with b.ResidualNorm(C, dtype, form, EPS) as n:
        want = n.backward(dy, out, x, gamma)
        torch.cuda.synchronize()
        assert b.residual_norm_device_status(n.handle) == b.SPECTRE_OK
        b.residual_norm_set_option(n.handle, b.RESIDUAL_NORM_OPT_TEST_WAIT_TIMEOUT, 1)
        dz, _, dgamma, dbeta = n.backward(dy, out, x, gamma)
        assert b.residual_norm_device_status(n.handle) == b.SPECTRE_ERR_TIMEOUT
        assert b.residual_norm_device_status(n.handle) == b.SPECTRE_OK
        b.residual_norm_set_option(n.handle, b.RESIDUAL_NORM_OPT_TEST_WAIT_TIMEOUT, 0)
        after = n.backward(dy, out, x, gamma)
        torch.cuda.synchronize()
        assert b.residual_norm_device_status(n.handle) == b.SPECTRE_OK
    assert all(bool(torch.isnan(t).all()) for t in (dz, dgamma, dbeta))
    assert all(torch.equal(p, q) for p, q in zip(want, after))


def test_wait_option_is_validated():
    with b.ResidualNorm(512) as n:
        for option, value in ((b.RESIDUAL_NORM_OPT_TEST_WAIT_TIMEOUT, 2), (b.RESIDUAL_NORM_OPT_TEST_WAIT_TIMEOUT, -1), (0, 1), (2, 0)):
            with pytest.raises(b.SpectreMixError):
                b.residual_norm_set_option(n.handle, option, value)
    assert b._lib.residual_norm_set_option(None, b.RESIDUAL_NORM_OPT_TEST_WAIT_TIMEOUT, 0) == b.SPECTRE_ERR_ARG
