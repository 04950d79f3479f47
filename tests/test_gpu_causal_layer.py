"""The operators together, as a layer uses them: y = N(scan(g, v) + x), forward, backward and token by token,
against the 64-bit reference.

Each operator's bound holds for its own inputs; what the second reads is the first's rounded output, so the second
is compared with the reference on that output."""
import pytest
import torch

import rows_reference as ref
from sub_quadratic_attention_b200 import binding as b

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,H,D,form,per,norm", [("bf16", 4, 16, "sigmoid", "channel", "post_ln"),
                                                     ("f32", 3, 20, "exp", "head", "pre_rms"),
                                                     ("bf16", 2, 33, "exp", "head", "post_rms")])
def test_train_and_serve_a_layer(dtype, H, D, form, per, norm):
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    B, L, C = 2, 200, H * D
    gen = torch.Generator().manual_seed(1)
    mk = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    g = mk(B, L, C if per == "channel" else H)
    g = (g + 2 if form == "sigmoid" else -0.1 * torch.nn.functional.softplus(g)).to(t)
    v, x, dy = (mk(B, L, C).to(t) for _ in range(3))
    gamma, beta = mk(C) * 0.1 + 1, mk(C) * 0.1
    gd, vd, xd, dyd, gad, bed = (q.cuda() for q in (g, v, x, dy, gamma, beta))
    with b.GatedScan(H, D, dtype, form, per) as scan, b.ResidualNorm(C, dtype, norm) as n:
        states = scan.new_states(B, L)
        h, hT = scan(gd, vd, states=states)
        y = n(h, xd, gad, bed)
        dh, dx, dgamma, dbeta = n.backward(dyd, h, xd, gad)
        dg, dv, _ = scan.backward(dh, gd, vd, states)
        # the same rows served: a prompt of 130, then one token after another
        h1, state = scan(gd[:, :130], vd[:, :130])
        served = [n(h1, xd[:, :130].contiguous(), gad, bed)]
        for i in range(130, L):
            hi, _ = scan.step(gd[:, i], vd[:, i], state)
            served.append(n(hi, xd[:, i], gad, bed)[:, None])
        torch.cuda.synchronize()
    val, err = ref.scan(g, v, H, D, form, None, None, dh.cpu())
    for name, got in (("y", h), ("hT", hT), ("dg", dg), ("dv", dv)):
        ref.check(name, got, val[name], err[name])
    ref.check("served state", state, val["hT"], err["hT"])
    flat = [q.reshape(-1, C) for q in (h.cpu(), x)]
    nv, ne = ref.norm(*flat, gamma, beta, norm, 1e-5, dy.reshape(-1, C))
    for name, got in (("y", y.view(-1, C)), ("dz", dh.view(-1, C)), ("dgamma", dgamma), ("dbeta", dbeta)):
        ref.check(name, got, nv[name], ne[name])
    # the served rows' h may round to the neighbouring value, step away; through the norm, with the row's mean and
    # deviation moving by at most the row's largest step: |dn| <= r (step + (1 + |n|) max step), to first order
    z = (flat[0].double() + flat[1].double() if norm.startswith("post") else flat[0].double())
    z = z - z.mean(-1, keepdim=True) if norm.endswith("ln") else z
    r = 1 / torch.sqrt((z * z).mean(-1, keepdim=True) + 1e-5)
    step = 2 * ref.HALF[t] * flat[0].double().abs() + 2 * err["y"].reshape(-1, C)
    slack = 1.1 * gamma.double().abs() * r * (step + (1 + (z * r).abs()) * step.amax(-1, keepdim=True))
    ref.check("served y", torch.cat(served, 1), nv["y"].view(B, L, C), (ne["y"] + slack).view(B, L, C))


def test_layer_in_one_graph_with_new_inputs():
    B, L, H, D = 1, 700, 2, 32
    gen = torch.Generator(device="cuda").manual_seed(2)
    mk = lambda: torch.randn(B, L, 64, generator=gen, device="cuda").bfloat16()  # noqa: E731
    w = torch.ones(64, device="cuda")
    with b.GatedScan(H, D) as scan, b.ResidualNorm(64) as n:
        def layer(g, v, x, dy):
            states = scan.new_states(B, L)
            h, _ = scan(g, v, states=states)
            y = n(h, x, w, w)
            dh, _, dgamma, dbeta = n.backward(dy, h, x, w)
            return (y, dgamma, dbeta) + scan.backward(dh, g, v, states)[:2]
        ins = [mk() for _ in range(4)]
        layer(*ins)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = layer(*ins)
        for _ in range(3):
            for old in ins:
                old.copy_(mk())
            graph.replay()
            want = layer(*ins)
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(outs, want))


def test_results_on_another_stream_are_not_in_memory_still_in_use():
    """What a call with ``stream=`` makes may not lie where work enqueued earlier on the caller's stream, still
    waiting to run, is about to write: a tensor of a result's size is filled behind a pause of the caller's stream
    and given back before each call."""
    B, L, C = 1, 16384, 128
    gen = torch.Generator(device="cuda").manual_seed(4)
    g, v, x, dy = (torch.randn(B, L, C, generator=gen, device="cuda").bfloat16() for _ in range(4))
    w = torch.ones(C, device="cuda")
    side = torch.cuda.Stream()
    with b.GatedScan(2, 64) as scan, b.ResidualNorm(C) as n:
        states = scan.new_states(B, L)
        rows = [t[0] for t in (g, v)] + [torch.zeros(L, C, device="cuda")]
        calls = [lambda **k: scan(g, v, states=states, **k), lambda **k: scan.backward(dy, g, v, states, **k),
                 lambda **k: scan.step(rows[0], rows[1], rows[2], new_state=states.new_empty(L, C), **k),
                 lambda **k: (n(v, x, w, w, **k),), lambda **k: n.backward(dy, v, x, w, **k)]
        for call in calls:
            want = [t for t in call() if t is not None]
            torch.cuda.synchronize()
            raw = torch.empty_like(v)
            for stream in (side, side.cuda_stream):
                torch.cuda._sleep(100_000_000)
                raw.fill_(7.0)
                del raw
                got = [t for t in call(stream=stream) if t is not None]
                torch.cuda.synchronize()
                assert all(torch.equal(p, q) for p, q in zip(want, got))
                raw = torch.empty_like(v)
            del raw, want, got
