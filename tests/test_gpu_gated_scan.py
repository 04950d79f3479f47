"""The gated recurrence on the GPU, forward, backward and step, against the 64-bit reference
with its derived error bounds (rows_reference.py)."""
import math

import pytest
import torch

import rows_reference as ref
from sub_quadratic_attention_b200 import binding as b

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _inputs(B, L, H, D, dtype, form, per, gate_dtype=None, seed=0, n=None, slow=False):
    gen = torch.Generator().manual_seed(seed)
    C = H * D
    z = torch.randn(B, L, C if per == "channel" else H, generator=gen)
    if form == "sigmoid":
        g = z * 1.5 + (7.0 if slow else 2.0)
    else:
        g = -torch.nn.functional.softplus(z) * (0.002 if slow else 0.3)
    g = g.to(TYPES[gate_dtype or dtype])
    v, dy = (torch.randn(B, L, C, generator=gen).to(TYPES[dtype]) for _ in range(2))
    h0, dhT = (torch.randn(n or B, C, generator=gen) for _ in range(2))
    return g, v, dy, h0, dhT


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _check(H, D, dtype, form, per, g, v, dy, h0=None, dhT=None, cu=None, gate_dtype=None, place=None):
    """Both directions against the reference; ``place`` lays g, v, dy out on the GPU."""
    B, L, _ = v.shape
    gd, vd, dyd, h0d, dhTd = _cuda(g, v, dy, h0, dhT)
    if place:
        gd, vd, dyd = place(gd, vd, dyd)
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    with b.GatedScan(H, D, dtype, form, per, gate_dtype) as s:
        states = s.new_states(B, L)
        y, hT = s(gd, vd, h0=h0d, cu_seqlens=cud, states=states)
        y2, hT2 = s(gd, vd, h0=h0d, cu_seqlens=cud)
        dg, dv, dh0 = s.backward(dyd, gd, vd, states, h0=h0d, dhT=dhTd, cu_seqlens=cud)
        torch.cuda.synchronize()
    assert torch.equal(y.view(torch.uint8), y2.view(torch.uint8)) and torch.equal(hT.view(torch.uint8), hT2.view(torch.uint8))
    val, err = ref.scan(g, v, H, D, form, h0, cu, dy, dhT)
    inside = torch.ones(L, dtype=torch.bool)
    if cu is not None:
        inside[:cu[0]] = False
        inside[cu[-1]:] = False
    for name, got in (("y", y), ("dg", dg), ("dv", dv)):
        ref.check(name, got[:, inside], val[name][:, inside], err[name][:, inside])
        assert not bool(got[:, ~inside].any())      # made by the call: zero outside every sequence
    ref.check("hT", hT, val["hT"], err["hT"])
    if h0 is None:
        assert dh0 is None
    else:
        ref.check("dh0", dh0, val["dh0"], err["dh0"])
    return y, hT, dg, dv, dh0


@pytest.mark.parametrize("form", ["sigmoid", "exp"])
@pytest.mark.parametrize("per", ["channel", "head"])
@pytest.mark.parametrize("dtype,gate_dtype", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("B,L,H,D", [(2, 37, 2, 16), (1, 300, 3, 20)])
def test_types_gates_and_layouts(B, L, H, D, dtype, gate_dtype, form, per):
    g, v, dy, h0, dhT = _inputs(B, L, H, D, dtype, form, per, gate_dtype)
    _check(H, D, dtype, form, per, g, v, dy, h0, dhT, gate_dtype=gate_dtype)


@pytest.mark.parametrize("L", [1, 2, 7, 8, 9, 15, 16, 17, 127, 128, 129, 255, 256, 257, 1000, 5000])
def test_lengths(L):
    g, v, dy, h0, dhT = _inputs(2, L, 2, 36, "f32", "sigmoid", "channel", seed=L, slow=True)
    _check(2, 36, "f32", "sigmoid", "channel", g, v, dy, h0, dhT)


@pytest.mark.parametrize("H,D", [(1, 1), (5, 1), (3, 2), (1, 3), (2, 4), (1, 5), (3, 8), (2, 12), (7, 33), (1, 60), (1, 64),
                                 (2, 68), (1, 100), (3, 128), (1, 130), (1, 257), (2, 320)])
@pytest.mark.parametrize("per", ["channel", "head"])
def test_heads(H, D, per):
    g, v, dy, h0, dhT = _inputs(1, 150, H, D, "bf16", "exp", per, "f32", seed=D)
    _check(H, D, "bf16", "exp", per, g, v, dy, h0, dhT, gate_dtype="f32")


def test_without_initial_state():
    g, v, dy, _, _ = _inputs(3, 200, 2, 8, "f32", "exp", "head")
    _check(2, 8, "f32", "exp", "head", g, v, dy)


@pytest.mark.parametrize("per", ["channel", "head"])
@pytest.mark.parametrize("form", ["sigmoid", "exp"])
def test_long_memory_over_many_chunks(form, per):
    """Gates near one: the state crosses every chunk border of 9,000 rows."""
    g, v, dy, h0, dhT = _inputs(1, 9000, 2, 20, "bf16", form, per, "f32", slow=True)
    _check(2, 20, "bf16", form, per, g, v, dy, h0, dhT, gate_dtype="f32")


@pytest.mark.parametrize("cu", [[0, 300], [0, 1, 2, 3, 300], [0, 0, 128, 128, 256, 300, 300], [5, 17, 17, 140, 290],
                                [0, 127, 129, 299], [300, 300], [0, 0], list(range(0, 301, 3)), [0]])
@pytest.mark.parametrize("per,dtype", [("channel", "f32"), ("head", "bf16")])
def test_packed_sequences(cu, per, dtype):
    """Empty sequences, borders inside and at chunks, rows before the first and behind the last."""
    g, v, dy, h0, dhT = _inputs(1, 300, 3, 12, dtype, "sigmoid", per, "f32", n=max(1, len(cu) - 1))
    h0, dhT = h0[:len(cu) - 1], dhT[:len(cu) - 1]
    _check(3, 12, dtype, "sigmoid", per, g, v, dy, h0, dhT, cu=cu, gate_dtype="f32")
    _check(3, 12, dtype, "sigmoid", per, g, v, dy, None, None, cu=cu, gate_dtype="f32")


@pytest.mark.parametrize("per", ["channel", "head"])
def test_thousands_of_sequences(per):
    """More sequences than a tile looks through one by one: short ones, empty ones, a long one in the middle."""
    cu = list(range(3, 1200, 1)) + [1200] * 900 + [2000] + list(range(2002, 2790, 2))
    L = 2800
    g, v, dy, h0, dhT = _inputs(1, L, 1, 32, "f32", "exp", per, n=len(cu) - 1)
    _check(1, 32, "f32", "exp", per, g, v, dy, h0, dhT, cu=cu)


def test_rows_outside_the_sequences_are_left_as_they_were():
    cu = [10, 130, 270]
    g, v, dy, h0, _ = _inputs(1, 300, 2, 16, "bf16", "exp", "head", n=2)
    gd, vd, dyd, h0d = _cuda(g, v, dy, h0)
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    out = torch.tensor(cu[:1] + cu[-1:]).tolist()
    with b.GatedScan(2, 16, "bf16", "exp", "head") as s:
        y, dv = (torch.full((1, 300, 32), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        dg = torch.full((1, 300, 2), 7.0, dtype=torch.bfloat16, device="cuda")
        states = s.new_states(1, 300)
        s(gd, vd, h0=h0d, cu_seqlens=cud, y=y, states=states)
        s.backward(dyd, gd, vd, states, h0=h0d, cu_seqlens=cud, dg=dg, dv=dv)
        y2, _ = s(gd, vd, h0=h0d, cu_seqlens=cud)
        torch.cuda.synchronize()
    for t in (y, dg, dv):
        assert bool((t[:, :out[0]] == 7).all()) and bool((t[:, out[1]:] == 7).all())
        assert bool((t[:, out[0]:out[1]] != 7).any())
    assert torch.equal(y[:, 10:270], y2[:, 10:270])


@pytest.mark.parametrize("cu", [[-5, 10, 400], [0, 200, 100, 300], [250, 20], [1000, 2000], [-9, -3]])
def test_bad_offsets_stay_inside_the_tensors(cu):
    """Offsets out of range or order: the results are not defined, the neighbouring memory stays."""
    g, v, dy, h0, _ = _inputs(1, 300, 2, 16, "f32", "exp", "channel", n=len(cu) - 1)
    gd, vd, dyd, h0d = _cuda(g, v, dy, h0)
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    guard = [torch.full((1, 340, 32), 7.0, device="cuda") for _ in range(3)]
    y, dg, dv = (t[:, 20:320] for t in guard)
    with b.GatedScan(2, 16, "f32", "exp") as s:
        states = s.new_states(1, 300)
        states.zero_()
        s(gd, vd, h0=h0d, cu_seqlens=cud, y=y, states=states)
        s.backward(dyd, gd, vd, states, h0=h0d, cu_seqlens=cud, dg=dg, dv=dv)
        torch.cuda.synchronize()
    for t in guard:
        assert bool((t[:, :20] == 7).all()) and bool((t[:, 320:] == 7).all())


def _strided(g, v, dy):
    def wide(t, left, right):
        big = torch.full(t.shape[:2] + (t.shape[2] + left + right,), float("nan"), dtype=t.dtype, device="cuda")
        big[..., left:left + t.shape[2]] = t
        return big[..., left:left + t.shape[2]]
    return wide(g, 4, 8), wide(v, 3, 2), wide(dy, 0, 5)


def _time_major(g, v, dy):
    return tuple(t.transpose(0, 1).contiguous().transpose(0, 1) for t in (g, v, dy))


@pytest.mark.parametrize("place", [_strided, _time_major])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("per", ["channel", "head"])
def test_strides(place, dtype, per):
    g, v, dy, h0, dhT = _inputs(3, 140, 2, 12, dtype, "sigmoid", per)
    _check(2, 12, dtype, "sigmoid", per, g, v, dy, h0, dhT, place=place)


def test_halves_of_one_projection_and_of_its_gradient():
    g, v, dy, h0, _ = _inputs(2, 200, 2, 32, "bf16", "sigmoid", "channel")
    both = torch.cat([g, v], -1).cuda()
    gd, vd, dyd = both[..., :64], both[..., 64:], dy.cuda()
    grad = torch.empty_like(both)
    with b.GatedScan(2, 32, "bf16") as s:
        states = s.new_states(2, 200)
        s(gd, vd, states=states)
        s.backward(dyd, gd, vd, states, dg=grad[..., :64], dv=grad[..., 64:])
        dg, dv, _ = s.backward(dyd, gd.contiguous(), vd.contiguous(), states)
    assert torch.equal(grad, torch.cat([dg, dv], -1))


def test_broadcast_inputs():
    """Stride 0: one gate row for all rows; its gradient comes for every row."""
    g, v, dy, h0, dhT = _inputs(2, 150, 2, 16, "f32", "exp", "channel")
    g = g[:1, :1].expand(2, 150, 32)
    _check(2, 16, "f32", "exp", "channel", g, v, dy, h0, dhT,
           place=lambda gd, vd, dyd: (gd[:1, :1].expand(2, 150, 32), vd, dyd))


@pytest.mark.parametrize("form", ["sigmoid", "exp"])
@pytest.mark.parametrize("per", ["channel", "head"])
@pytest.mark.parametrize("low", [-math.inf, torch.finfo(torch.bfloat16).min])
def test_gates_of_zero_cut(form, per, low):
    """A gate of zero takes out all that lies before it, NaN and infinities included, within a chunk and
    across chunks; its gradient there is zero."""
    g, v, dy, h0, dhT = _inputs(1, 600, 1, 16, "bf16", form, per)
    for t in (3, 130, 256, 399, 400):
        g[:, t] = low
    clean = v.clone()
    for t, bad in ((1, math.nan), (129, math.inf), (255, -math.inf), (398, math.nan)):
        v[:, t] = bad
    with b.GatedScan(1, 16, "bf16", form, per) as s:
        states = s.new_states(1, 600)
        y, hT = s(g.cuda(), v.cuda(), h0=h0.cuda(), states=states)
        dg, dv, dh0 = s.backward(dy.cuda(), g.cuda(), v.cuda(), states, h0=h0.cuda())
        torch.cuda.synchronize()
    val, err = ref.scan(g, clean, 1, 16, form, h0, None, dy)
    fine = torch.ones(600, dtype=torch.bool)
    for lo, hi in ((1, 3), (129, 130), (255, 256), (398, 399)):
        fine[lo:hi] = False
        assert not bool(torch.isfinite(y[:, lo:hi]).any())
    ref.check("y", y[:, fine], val["y"][:, fine], err["y"][:, fine])
    ref.check("hT", hT, val["hT"], err["hT"])
    ref.check("dv", dv, val["dv"], err["dv"])
    ref.check("dh0", dh0, val["dh0"], err["dh0"])
    ref.check("dg", dg[:, fine], val["dg"][:, fine], err["dg"][:, fine])


def test_held_rows():
    """sigmoid, g = infinity: the state is held whatever stands in v."""
    g, v, dy, h0, dhT = _inputs(2, 300, 1, 16, "f32", "sigmoid", "channel")
    held = torch.zeros(300, dtype=torch.bool)
    held[5:20] = held[120:140] = held[290:] = True
    g[:, held] = math.inf
    clean = v.clone()
    clean[:, held] = 0
    v[:, held] = math.nan
    with b.GatedScan(1, 16, "f32") as s:
        states = s.new_states(2, 300)
        y, hT = s(g.cuda(), v.cuda(), h0=h0.cuda(), states=states)
        dg, dv, dh0 = s.backward(dy.cuda(), g.cuda(), v.cuda(), states, h0=h0.cuda(), dhT=dhT.cuda())
        torch.cuda.synchronize()
    val, err = ref.scan(g, clean, 1, 16, "sigmoid", h0, None, dy, dhT)
    for name, got in (("y", y), ("hT", hT), ("dg", dg), ("dv", dv), ("dh0", dh0)):
        ref.check(name, got, val[name], err[name])
    assert not bool(dg[:, held].any()) and not bool(dv[:, held].any())


def test_nan_stays_in_its_channel_sequence_and_future():
    g, v, dy, h0, _ = _inputs(1, 300, 1, 16, "f32", "exp", "channel", n=3, slow=True)
    v[0, 140, 3] = math.nan
    cu = [0, 100, 200, 300]
    with b.GatedScan(1, 16, "f32", "exp") as s:
        cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
        states = s.new_states(1, 300)
        y, hT = s(g.cuda(), v.cuda(), cu_seqlens=cud, states=states)
        dg, dv, _ = s.backward(dy.cuda(), g.cuda(), v.cuda(), states, cu_seqlens=cud)
        torch.cuda.synchronize()
    want = torch.zeros(1, 300, 16, dtype=torch.bool)
    want[0, 140:200, 3] = True
    assert torch.equal(torch.isnan(y).cpu(), want)
    assert torch.isnan(hT).cpu().nonzero().tolist() == [[1, 3]]
    assert not bool(torch.isnan(dv).any())
    want[0, 140, 3] = False     # its own gate's slope is the state before it
    assert torch.equal(torch.isnan(dg).cpu(), want)


def test_rows_that_overlap():
    """Windows of one buffer: a row's values begin inside the row before it."""
    flat_g, flat_v = torch.randn(3000) * 0.5 - 3, torch.randn(3000)
    g, v = (f.as_strided((2, 150, 32), (1600, 8, 1)) for f in (flat_g, flat_v))
    dy = torch.randn(2, 150, 32)
    gd, vd = (f.cuda().as_strided((2, 150, 32), (1600, 8, 1)) for f in (flat_g, flat_v))
    _check(2, 16, "f32", "sigmoid", "channel", g, v, dy, place=lambda *_: (gd, vd, dy.cuda()))


@pytest.mark.parametrize("B,L,H,D,per", [(700, 3, 2, 32, "channel"), (300, 130, 1, 64, "head"), (2, 1, 1, 64, "channel"),
                                         (600, 128, 1, 64, "channel")])
def test_many_short_sequences(B, L, H, D, per):
    """More sequences than blocks: a block takes strip after strip."""
    g, v, dy, h0, dhT = _inputs(B, L, H, D, "bf16", "sigmoid", per)
    gd, vd, dyd, h0d, dhTd = _cuda(g, v, dy, h0, dhT)
    with b.GatedScan(H, D, "bf16", "sigmoid", per) as s:
        st = s.new_states(B, L)
        y, hT = s(gd, vd, h0=h0d, states=st)
        dg, dv, dh0 = s.backward(dyd, gd, vd, st, h0=h0d, dhT=dhTd)
        torch.cuda.synchronize()
    pick = torch.tensor([0, 1, B // 2, B - 2, B - 1])
    val, err = ref.scan(g[pick], v[pick], H, D, "sigmoid", h0[pick], None, dy[pick], dhT[pick])
    for name, got in (("y", y), ("hT", hT), ("dg", dg), ("dv", dv), ("dh0", dh0)):
        ref.check(name, got[pick.cuda()], val[name], err[name])


def test_empty_calls():
    with b.GatedScan(2, 8, "bf16", gate_per="head") as s:
        for B, L in ((0, 5), (2, 0), (0, 0)):
            g = torch.empty(B, L, 2, dtype=torch.bfloat16, device="cuda")
            v = torch.empty(B, L, 16, dtype=torch.bfloat16, device="cuda")
            h0 = torch.randn(B, 16, device="cuda")
            st = s.new_states(B, L)
            y, hT = s(g, v, h0=h0, states=st)
            assert y.shape == v.shape and torch.equal(hT, h0)
            _, hT = s(g, v)
            assert torch.equal(hT, torch.zeros_like(h0))
            dg, dv, dh0 = s.backward(v, g, v, st, h0=h0, dhT=h0 * 2)
            assert dg.shape == g.shape and dv.shape == v.shape and torch.equal(dh0, h0 * 2)
        pool = torch.randn(3, 16, device="cuda")
        keep = pool.clone()
        e = torch.empty(0, 2, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
        y, new = s.step(*e, pool)
        assert y.shape == (0, 16) and torch.equal(new, keep)


@pytest.mark.parametrize("form", ["sigmoid", "exp"])
@pytest.mark.parametrize("per", ["channel", "head"])
@pytest.mark.parametrize("dtype,gate_dtype", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("B,H,D", [(1, 1, 1), (3, 2, 16), (5, 7, 33), (2, 3, 130)])
def test_step(B, H, D, dtype, gate_dtype, form, per):
    """The step is a sequence of one row from the pool's state."""
    g, v, _, _, _ = _inputs(B, 1, H, D, dtype, form, per, gate_dtype)
    pool = torch.randn(B + 3, H * D, generator=torch.Generator().manual_seed(1))
    slots = torch.randperm(B + 3, generator=torch.Generator().manual_seed(2))[:B].int()
    val, err = ref.scan(g, v, H, D, form, pool[slots.long()])
    with b.GatedScan(H, D, dtype, form, per, gate_dtype) as s:
        p = pool.cuda()
        y, new = s.step(g[:, 0].cuda(), v[:, 0].cuda(), p, slots=slots.cuda())
        assert new is p
        kept = pool.cuda()
        other = torch.full_like(kept, 7.0)
        y2, new2 = s.step(g[:, 0].cuda(), v[:, 0].cuda(), kept, slots=slots.cuda(), new_state=other)
        y3, new3 = s.step(g[:, 0].cuda(), v[:, 0].cuda(), pool[slots.long()].cuda())
        torch.cuda.synchronize()
    ref.check("y", y[:, None], val["y"], err["y"])
    ref.check("state", new[slots.long().cuda()], val["hT"], err["hT"])
    rest = torch.ones(B + 3, dtype=torch.bool)
    rest[slots.long()] = False
    assert torch.equal(new[rest.cuda()].cpu(), pool[rest]) and bool((new2[rest.cuda()] == 7).all())
    assert torch.equal(kept.cpu(), pool) and torch.equal(y, y2) and torch.equal(y, y3)
    assert torch.equal(new2[slots.long().cuda()], new3) and torch.equal(new[slots.long().cuda()], new3)


def test_step_slots_out_of_range_and_repeated():
    """Rows without a place are skipped; rows of one place are taken in order, as a sequence."""
    g, v, _, _, _ = _inputs(1, 9, 2, 36, "f32", "sigmoid", "channel")
    slots = torch.tensor([2, -1, 2, 4, 0, 5, 2, 0, 2 ** 31 - 1], dtype=torch.int32)
    pool = torch.randn(5, 72, generator=torch.Generator().manual_seed(1))
    for separate in (False, True):
        with b.GatedScan(2, 36, "f32") as s:
            y = torch.full((9, 72), 7.0, device="cuda")
            p = pool.cuda()
            new = torch.full_like(p, 7.0) if separate else p
            s.step(g[0].cuda(), v[0].cuda(), p, slots=slots.cuda(), y=y, new_state=new)
            made, _ = s.step(g[0].cuda(), v[0].cuda(), pool.cuda(), slots=slots.cuda())
            torch.cuda.synchronize()
        for slot in range(5):
            rows = (slots == slot).nonzero()[:, 0]
            if not len(rows):
                assert torch.equal(new[slot].cpu(), torch.full((72,), 7.0) if separate else pool[slot])
                continue
            val, err = ref.scan(g[:, rows], v[:, rows], 2, 36, "sigmoid", pool[slot:slot + 1])
            ref.check("y", y[rows.cuda()][None], val["y"], err["y"])
            ref.check("state", new[slot:slot + 1], val["hT"], err["hT"])
        skipped = ((slots < 0) | (slots >= 5)).cuda()
        assert bool((y[skipped] == 7).all()) and not bool(made[skipped].any())


def test_prefill_then_steps_is_one_scan():
    g, v, _, h0, _ = _inputs(2, 140, 2, 16, "f32", "exp", "head")
    val, err = ref.scan(g, v, 2, 16, "exp", h0)
    gd, vd, h0d = _cuda(g, v, h0)
    with b.GatedScan(2, 16, "f32", "exp", "head") as s:
        y, state = s(gd[:, :131], vd[:, :131], h0=h0d)
        rest = [s.step(gd[:, t], vd[:, t], state)[0] for t in range(131, 140)]
        torch.cuda.synchronize()
    ref.check("y", torch.cat([y, torch.stack(rest, 1)], 1), val["y"], err["y"])
    ref.check("hT", state, val["hT"], err["hT"])


def test_large_step_batch():
    """More rows than a grid's y extent."""
    B = 70000
    gen = torch.Generator(device="cuda").manual_seed(0)
    g, v = (torch.randn(B, 4, generator=gen, device="cuda") for _ in range(2))
    state = torch.randn(B, 4, generator=gen, device="cuda")
    with b.GatedScan(1, 4, "f32") as s:
        y, new = s.step(g, v, state, new_state=torch.empty_like(state))
    a = torch.sigmoid(g.double())
    want = a * state.double() + (1 - a) * v.double()
    assert bool(((new.double() - want).abs() <= ref.K * ref.U * (state.double().abs() + v.double().abs())).all())
    assert torch.equal(y, new)


def test_offsets_beyond_32_bits():
    """Rows whose element offsets pass 2^31 through their strides."""
    L, C, stride = 260, 8, 1 << 23          # 260 rows of 2^23 elements apart: 2.18e9 elements, bf16
    big = torch.empty(L * stride, dtype=torch.bfloat16, device="cuda")
    g, v, dy, h0, dhT = _inputs(1, L, 1, C, "bf16", "exp", "channel", slow=True)
    vd = big.as_strided((1, L, C), (L * stride, stride, 1))
    yd = big.as_strided((1, L, C), (L * stride, stride, 1), 64)
    vd.copy_(v)
    with b.GatedScan(1, C, "bf16", "exp") as s:
        st = s.new_states(1, L)
        _, hT = s(g.cuda(), vd, h0=h0.cuda(), y=yd, states=st)
        dvd = big.as_strided((1, L, C), (L * stride, stride, 1), 128)
        dg = torch.empty_like(g, device="cuda")
        s.backward(dy.cuda(), g.cuda(), vd, st, h0=h0.cuda(), dhT=dhT.cuda(), dg=dg, dv=dvd)
        torch.cuda.synchronize()
    val, err = ref.scan(g, v, 1, C, "exp", h0, None, dy, dhT)
    ref.check("y", yd, val["y"], err["y"])
    ref.check("dv", dvd, val["dv"], err["dv"])
    ref.check("dg", dg, val["dg"], err["dg"])


def test_equal_inputs_give_equal_bits():
    gen = torch.Generator(device="cuda").manual_seed(0)
    g = torch.randn(1, 40000, 128, generator=gen, device="cuda").add_(5).bfloat16()
    v, dy = (torch.randn(1, 40000, 128, generator=gen, device="cuda").bfloat16() for _ in range(2))
    runs = []
    with b.GatedScan(2, 64, "bf16") as s:
        for _ in range(6):
            st = s.new_states(1, 40000)
            out = s(g, v, states=st)
            runs.append([*out, st, *s.backward(dy, g, v, st)[:2]])
        assert b.gated_scan_device_status(s.handle) == b.SPECTRE_OK
    for other in runs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(runs[0], other))


def test_streams_and_two_calls_at_once():
    """One plan on two streams at a time, each call with its own workspace."""
    g, v, dy, h0, _ = _inputs(1, 3000, 2, 32, "f32", "sigmoid", "channel", slow=True)
    gd, vd, dyd = _cuda(g, v, dy)
    with b.GatedScan(2, 32, "f32") as s:
        st0 = s.new_states(1, 3000)
        want = [*s(gd, vd, states=st0), *s.backward(dyd, gd, vd, st0)[:2]]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(3)]
        got = []
        for i in range(12):
            st = s.new_states(1, 3000)
            q = streams[i % 3]
            q.wait_stream(torch.cuda.current_stream())
            handle = q if i % 2 else q.cuda_stream
            out = s(gd, vd, states=st, stream=handle)
            got.append([*out, *s.backward(dyd, gd, vd, st, stream=handle)[:2]])
        torch.cuda.synchronize()
    for one in got:
        assert all(torch.equal(x, y) for x, y in zip(want, one))


def test_captured_graphs():
    """Two graphs of one plan, replayed on two streams with new inputs."""
    g, v, dy, h0, _ = _inputs(1, 2000, 2, 32, "bf16", "exp", "head", slow=True)
    with b.GatedScan(2, 32, "bf16", "exp", "head") as s:
        graphs, outs, ins = [], [], []
        for i in range(2):
            gd, vd, dyd = _cuda(g, v, dy)
            st = s.new_states(1, 2000)
            s(gd, vd, states=st)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = [*s(gd, vd, states=st)]
                out += s.backward(dyd, gd, vd, st)[:2]
            graphs.append(graph)
            outs.append(out)
            ins.append((gd, vd, dyd))
        for seed in (5, 6):
            sides = [torch.cuda.Stream(), torch.cuda.Stream()]
            new = [_cuda(*_inputs(1, 2000, 2, 32, "bf16", "exp", "head", seed=seed + 10 * i, slow=True)[:3]) for i in range(2)]
            for i in range(2):
                for old, n in zip(ins[i], new[i]):
                    old.copy_(n)
            torch.cuda.synchronize()
            for i in range(2):
                with torch.cuda.stream(sides[i]):
                    graphs[i].replay()
            torch.cuda.synchronize()
            for i in range(2):
                st = s.new_states(1, 2000)
                want = [*s(new[i][0], new[i][1], states=st)]
                want += s.backward(new[i][2], new[i][0], new[i][1], st)[:2]
                assert all(torch.equal(x, y) for x, y in zip(outs[i], want))
        del graphs


def test_gradient_against_differences():
    """The kernels' gradients against central differences of the 64-bit forward pass; the gradients' bound is the
    reference's, the differences' own error about 1e-9."""
    H, D, L = 2, 4, 140
    g, v, dy, h0, dhT = _inputs(1, L, H, D, "f32", "sigmoid", "head")
    val, err = ref.scan(g, v, H, D, "sigmoid", h0, None, dy, dhT)
    with b.GatedScan(H, D, "f32", "sigmoid", "head") as s:
        st = s.new_states(1, L)
        s(g.cuda(), v.cuda(), h0=h0.cuda(), states=st)
        dg, dv, dh0 = s.backward(dy.cuda(), g.cuda(), v.cuda(), st, h0=h0.cuda(), dhT=dhT.cuda())
        torch.cuda.synchronize()

    def loss(p):
        o, _ = ref.scan(p["g"], p["v"], H, D, "sigmoid", p["h0"])
        return float((dy.double() * o["y"]).sum() + (dhT.double() * o["hT"]).sum())

    p = {"g": g.double(), "v": v.double(), "h0": h0.double()}
    for name, got, places in (("g", dg, (0, 5, 130, 270)), ("v", dv, (0, 9, 513, 1100)), ("h0", dh0, (0, 7))):
        for at in places:
            d = torch.zeros(p[name].numel(), dtype=torch.float64)
            d[at] = 1e-5
            d = d.view_as(p[name])
            diff = (loss({**p, name: p[name] + d}) - loss({**p, name: p[name] - d})) / 2e-5
            limit = err["d" + name].reshape(-1)[at].item() + 1e-7
            assert abs(got.reshape(-1)[at].item() - diff) <= limit


def test_refusals():
    g, v, dy, h0, _ = _inputs(2, 20, 2, 8, "bf16", "exp", "channel")
    gd, vd, dyd, h0d = _cuda(g, v, dy, h0)
    with b.GatedScan(2, 8, "bf16", "exp") as s:
        st = s.new_states(2, 20)
        for bad in (dict(g=g, v=vd), dict(g=gd, v=vd, h0=h0d[:1]), dict(g=gd, v=vd, h0=h0d.double()),
                    dict(g=gd, v=vd, y=vd), dict(g=gd, v=vd, y=gd), dict(g=gd, v=vd, states=st[:, :0]),
                    dict(g=gd, v=vd, hT=h0d, h0=h0d), dict(g=gd.transpose(1, 2), v=vd),
                    dict(g=gd, v=vd, cu_seqlens=torch.tensor([0, 20], dtype=torch.int32, device="cuda"))):
            with pytest.raises(ValueError):
                s(**bad)
        for bad in (dict(states=None), dict(states=st, dg=torch.empty_like(gd)), dict(states=st, dg=gd, dv=vd)):
            with pytest.raises(ValueError):
                s.backward(dyd, gd, vd, **bad)
        with pytest.raises(b.SpectreMixError) as e:      # rows that overlap
            s(gd, vd, y=torch.empty(2, 1, 16, dtype=torch.bfloat16, device="cuda").expand(2, 20, 16))
        assert e.value.code == b.SPECTRE_ERR_ARG
        pool = torch.zeros(1, 16, device="cuda")
        with pytest.raises(ValueError):
            s.step(gd[:, 0], vd[:, 0], pool)
        with pytest.raises(ValueError):
            s.step(gd[:, 0], vd[:, 0], pool, slots=torch.zeros(2, device="cuda"))
        with pytest.raises(ValueError):
            s.step(gd[:, 0], vd[:, 0], torch.zeros(2, 16, device="cuda"), y=vd[:, 0])
        # the C entry points: short or misaligned workspaces, misaligned rows
        def run(B=2, L=20, g=(gd.data_ptr(), 320, 16)):
            a = b.gated_scan_args(B, L, g, b._rows_of("v", vd), b._rows_of("y", torch.empty_like(vd)))
            return b._lib.gated_scan_run(s.handle, a, None)
        assert run(g=(gd.data_ptr() + 1, 320, 16)) == b.SPECTRE_ERR_ALIGN
        assert run(g=(gd.data_ptr(), 320, -16)) == b.SPECTRE_ERR_ARG and run(g=(0, 320, 16)) == b.SPECTRE_ERR_ARG
        assert run(B=-1) == b.SPECTRE_ERR_ARG and run(B=1 << 40, L=1 << 40) == b.SPECTRE_ERR_ARG
        assert run(B=1 << 31, L=1 << 40) == b.SPECTRE_ERR_ARG and run(B=1 << 31, L=1) == b.SPECTRE_ERR_ARG
    with b.GatedScan(2, 160, "f32", "exp", "head") as s:
        need = b.gated_scan_workspace_bytes(s.handle, 1, 4, True)
        t = [torch.zeros(1, 4, n, device="cuda") for n in (2, 320, 320, 2, 320)]
        st = s.new_states(1, 4)
        work = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
        r = [b._rows_of("t", x) for x in t]
        def back(w, n):
            a = b.gated_scan_args(1, 4, r[0], r[1], dy=r[2], dg=r[3], dv=r[4], states=st.data_ptr(), work=w, work_bytes=n)
            return b._lib.gated_scan_backward(s.handle, a, None)
        assert back(work.data_ptr(), need - 1) == b.SPECTRE_ERR_ARG
        assert back(work.data_ptr() + 4, need) == b.SPECTRE_ERR_ALIGN


@pytest.mark.parametrize("shared", [False, True])
def test_states_beyond_32_bits(shared):
    """More than 2^31 values of h0, hT, states and their gradients: the last sequences' are found, and those on either
    side of the 2^31st.  ``shared``: inputs of stride 0, which are read value by value."""
    B, C = (1 << 21) + 5, 1024
    gen = torch.Generator(device="cuda").manual_seed(0)
    g = torch.randn(B, 1, 1, generator=gen, device="cuda").bfloat16()
    rows = [torch.randn(1 if shared else B, 1, C, generator=gen, device="cuda", dtype=torch.bfloat16).expand(B, 1, C) for _ in range(2)]
    v, dy = rows
    h0 = torch.randn(B, C, generator=gen, device="cuda")
    pick = torch.tensor([0, 1, B // 2, (1 << 21) - 1, 1 << 21, B - 2, B - 1])
    on = pick.cuda()
    with b.GatedScan(1, C, "bf16", "sigmoid", "head") as s:
        st = s.new_states(B, 1)
        y, hT = s(g, v, h0=h0, states=st)
        assert torch.equal(st[on, 0], h0[on])
        got = [("y", y[on]), ("hT", hT[on])]
        del y, hT
        dg, dv, dh0 = s.backward(dy, g, v, st, h0=h0, dhT=h0)
        got += [("dg", dg[on]), ("dv", dv[on]), ("dh0", dh0[on])]
        del dg, dv, dh0, st
        torch.cuda.synchronize()
    g, v, dy, h0 = (t[on].cpu() for t in (g, v, dy, h0))
    val, err = ref.scan(g, v, 1, C, "sigmoid", h0, None, dy, h0)
    for name, t in got:
        ref.check(name, t, val[name], err[name])
    del rows
    torch.cuda.empty_cache()


@pytest.mark.parametrize("p,bad,c", [(1, 3, 6), (8, 10, 16), (5, 50, 77), (100, 120, 128), (100, 120, 130), (128, 140, 256), (120, 260, 290)])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("form,value", [("sigmoid", math.nan), ("exp", math.nan), ("exp", math.inf)])
@pytest.mark.parametrize("dtype,H,D,per", [("bf16", 1, 64, "channel"), ("bf16", 2, 32, "head"), ("f32", 2, 20, "channel"),
                                           ("f32", 3, 7, "head"), ("bf16", 1, 21, "channel")])
def test_nan_gates_stay_between_the_cuts(dtype, H, D, per, form, value, packed, p, bad, c):
    """A gate of NaN (or an infinite decay) between two gates of zero, or in the second of three sequences: the rows
    before the first border and from the second on are those of the scan without it, in both directions, wherever the
    borders lie among a thread's rows, its groups and the tiles."""
    L, cu = 300, [0, p, c, 300] if packed else None
    g, v, dy, h0, dhT = _inputs(1, L, H, D, dtype, form, per, n=3 if packed else 1)
    if not packed:
        g[:, p] = g[:, c] = -math.inf
    val, err = ref.scan(g, v, H, D, form, h0, cu, dy, dhT)
    g[:, bad] = value
    gd, vd, dyd, h0d, dhTd = _cuda(g, v, dy, h0, dhT)
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda") if packed else None
    with b.GatedScan(H, D, dtype, form, per) as s:
        st = s.new_states(1, L)
        y, hT = s(gd, vd, h0=h0d, cu_seqlens=cud, states=st)
        dg, dv, dh0 = s.backward(dyd, gd, vd, st, h0=h0d, dhT=dhTd, cu_seqlens=cud)
        torch.cuda.synchronize()
    clean = torch.ones(L, dtype=torch.bool)
    clean[p:c] = False
    for name, got in (("y", y), ("dv", dv), ("dg", dg)):
        ref.check(name, got[:, clean.cuda()], val[name][:, clean], err[name][:, clean])
    ends = torch.tensor([0, 2] if packed else [0])
    for name, got in (("hT", hT), ("dh0", dh0)):
        ref.check(name, got[ends.cuda()], val[name][ends], err[name][ends])
    assert not bool(torch.isfinite(y[:, bad]).any()) and not bool(torch.isfinite(dv[:, bad - 1]).any())


@pytest.mark.parametrize("form", ["sigmoid", "exp"])
@pytest.mark.parametrize("dtype,H,D,per", [("bf16", 1, 64, "channel"), ("f32", 3, 7, "head")])
def test_gradient_of_a_gate_of_zero(dtype, H, D, per, form):
    """dg has the gate as a factor: where that is zero, dg is zero, though a NaN behind it has reached dh."""
    L = 300
    g, v, dy, h0, dhT = _inputs(1, L, H, D, dtype, form, per)
    cuts = torch.tensor([0, 5, 127, 128, 140, 290])
    g[:, cuts] = -math.inf
    g[:, [2, 60, 200, 295]] = math.nan
    dy[:, [126, 127, 130, 140]] = math.nan
    gd, vd, dyd, h0d = _cuda(g, v, dy, h0)
    with b.GatedScan(H, D, dtype, form, per) as s:
        st = s.new_states(1, L)
        s(gd, vd, h0=h0d, states=st)
        dg, _, dh0 = s.backward(dyd, gd, vd, st, h0=h0d)
        torch.cuda.synchronize()
    assert not bool(dg[:, cuts.cuda()].any()) and not bool(dh0.any())


@pytest.mark.parametrize("dtype,H,D,per", [("bf16", 1, 64, "channel"), ("f32", 2, 20, "head"), ("f32", 3, 7, "head"), ("bf16", 1, 21, "channel"),
                                           ("f32", 32, 3, "head"), ("bf16", 1, 320, "head"), ("bf16", 2, 128, "head")])
@pytest.mark.parametrize("at", [8, 16, 128])
def test_states_that_overflow_end_at_the_cut(dtype, H, D, per, at):
    """Two rows of the type's lowest value give a state past fp32; a gate of zero behind them takes it out, though
    neither the rows of one thread nor the state ahead of them show it alone.  The same for gradients going back."""
    L, C = 300, H * D
    low = torch.finfo(TYPES[dtype]).min
    g, v, dy, h0, dhT = _inputs(1, L, H, D, dtype, "exp", per)
    v[:, at - 1:at + 1] = low           # h is infinite at row `at`
    g[:, at] = 0.0
    g[:, at + 1] = -math.inf
    dy[:, [at + 63, at + 64]] = low     # dh is infinite at row at + 63
    g[:, at + 64] = 0.0
    g[:, at + 63] = -math.inf
    val, err = ref.scan(g, v, H, D, "exp", h0, None, dy, dhT)
    gd, vd, dyd, h0d, dhTd = _cuda(g, v, dy, h0, dhT)
    with b.GatedScan(H, D, dtype, "exp", per) as s:
        st = s.new_states(1, L)
        y, hT = s(gd, vd, h0=h0d, states=st)
        dg, dv, dh0 = s.backward(dyd, gd, vd, st, h0=h0d, dhT=dhTd)
        torch.cuda.synchronize()
    sure = torch.ones(L, dtype=torch.bool)
    sure[at - 1:at + 1] = sure[at + 63:at + 65] = False
    for name, got in (("y", y), ("dv", dv), ("dg", dg)):
        ref.check(name, got[:, sure.cuda()], val[name][:, sure], err[name][:, sure])
    ref.check("hT", hT, val["hT"], err["hT"])
    ref.check("dh0", dh0, val["dh0"], err["dh0"])
    assert bool((y[:, at] == -math.inf).all()) and not bool(torch.isfinite(dv[:, at + 63]).any())
    assert not bool(dg[:, [at + 1, at + 63]].any())


@pytest.mark.parametrize("dtype,H,D,per", [("bf16", 1, 64, "channel"), ("f32", 2, 20, "head"), ("bf16", 1, 21, "channel"), ("f32", 32, 3, "head"),
                                           ("bf16", 2, 128, "head")])
def test_held_rows_far_from_their_state(dtype, H, D, per):
    """sigmoid, g = infinity, with values of the type's lowest beside states near its largest: the state is held and
    the gates' gradients are zero, though the difference between the two is past fp32."""
    L = 200
    top = torch.finfo(TYPES[dtype]).max
    g, v, dy, h0, _ = _inputs(1, L, H, D, dtype, "sigmoid", per)
    g[:, 2:] = math.inf
    g[:, 1] = -math.inf
    v[:, 1], v[:, 2:] = top, -top
    gd, vd, dyd, h0d = _cuda(g, v, dy, h0)
    with b.GatedScan(H, D, dtype, "sigmoid", per) as s:
        st = s.new_states(1, L)
        y, hT = s(gd, vd, h0=h0d, states=st)
        dg, dv, _ = s.backward(dyd, gd, vd, st, h0=h0d)
        torch.cuda.synchronize()
    assert bool((y[:, 1:] == top).all()) and bool((hT == top).all())
    assert not bool(dg[:, 1:].any()) and not bool(dv[:, 2:].any()) and not bool(torch.isnan(dv).any())


def _both_ways(s, gd, vd, dyd, h0d, dhTd, cud):
    st = s.new_states(*vd.shape[:2])
    y, hT = s(gd, vd, h0=h0d, cu_seqlens=cud, states=st)
    return dict(y=y, hT=hT, st=st, **dict(zip(("dg", "dv", "dh0"), s.backward(dyd, gd, vd, st, h0=h0d, dhT=dhTd, cu_seqlens=cud))))


@pytest.mark.parametrize("B,L,H,D,per,dtype,cu", [(2, 300, 2, 32, "channel", "bf16", None), (1, 9000, 4, 16, "head", "f32", None),
                                                  (300, 130, 1, 64, "channel", "bf16", None), (1, 700, 1, 320, "head", "bf16", None),
                                                  (1, 700, 2, 32, "channel", "f32", [3, 3, 128, 400, 400, 690]),
                                                  (1, 700, 2, 32, "head", "bf16", [0, 129, 129, 600])])
def test_copies_that_do_not_come_leave_nan(B, L, H, D, per, dtype, cu):
    """The wait for the copies of rows made to give up while they are on their way: the blocks wait for them again and
    leave NaN in all that they would have written, the status is reported once, and the next calls are right."""
    g, v, dy, h0, dhT = _inputs(B, L, H, D, dtype, "sigmoid", per, n=B if cu is None else len(cu) - 1)
    on = _cuda(g, v, dy, h0, dhT) + [None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")]
    with b.GatedScan(H, D, dtype, "sigmoid", per) as s:
        want = _both_ways(s, *on)
        torch.cuda.synchronize()
        assert b.gated_scan_device_status(s.handle) == b.SPECTRE_OK
        b.gated_scan_set_option(s.handle, b.GATED_SCAN_OPT_TEST_WAIT_TIMEOUT, 1)
        got = _both_ways(s, *on)
        assert b.gated_scan_device_status(s.handle) == b.SPECTRE_ERR_TIMEOUT
        assert b.gated_scan_device_status(s.handle) == b.SPECTRE_OK
        b.gated_scan_set_option(s.handle, b.GATED_SCAN_OPT_TEST_WAIT_TIMEOUT, 0)
        after = _both_ways(s, *on)
        torch.cuda.synchronize()
        assert b.gated_scan_device_status(s.handle) == b.SPECTRE_OK
    lo, hi = (0, L) if cu is None else (cu[0], cu[-1])
    for name in ("y", "dg", "dv"):
        t = got[name].clone()
        assert bool(torch.isnan(t[:, lo:hi]).all())
        t[:, lo:hi] = 0
        assert not bool(t.any())        # rows in no sequence are zero as ever
    full = torch.ones(h0.shape[0], dtype=torch.bool) if cu is None else torch.tensor([p < q for p, q in zip(cu, cu[1:])])
    for name, through in (("hT", h0), ("dh0", dhT)):
        assert bool(torch.isnan(got[name][full.cuda()]).all()) and torch.equal(got[name].cpu()[~full], through[~full])
    for name in want:
        assert torch.equal(want[name], after[name]), name


@pytest.mark.parametrize("L,H,D,per,dtype", [(1000, 1, 64, "channel", "bf16"), (20000, 1, 64, "channel", "bf16"), (20000, 1, 32, "head", "f32"),
                                             (1000, 1, 21, "channel", "f32"), (12000, 3, 7, "head", "f32")])
def test_states_that_do_not_come_leave_nan(L, H, D, per, dtype):
    """The wait for the state ahead of a block of rows made to give up at once, on either way of looking back: the
    rows are NaN where it did and right elsewhere, and the status says whether there are any."""
    g, v, dy, h0, dhT = _inputs(1, L, H, D, dtype, "exp", per, slow=True)
    on = _cuda(g, v, dy, h0, dhT) + [None]
    with b.GatedScan(H, D, dtype, "exp", per) as s:
        want = _both_ways(s, *on)
        b.gated_scan_set_option(s.handle, b.GATED_SCAN_OPT_TEST_WAIT_TIMEOUT, 2)
        st = s.new_states(1, L)
        y, _ = s(*on[:2], h0=on[3], states=st)
        forward = b.gated_scan_device_status(s.handle)
        dg, dv, _ = s.backward(on[2], on[0], on[1], want["st"], h0=on[3], dhT=on[4])
        backward = b.gated_scan_device_status(s.handle)
        b.gated_scan_set_option(s.handle, b.GATED_SCAN_OPT_TEST_WAIT_TIMEOUT, 0)
        after = _both_ways(s, *on)
        torch.cuda.synchronize()
        assert b.gated_scan_device_status(s.handle) == b.SPECTRE_OK
    for status, names, sure in ((forward, dict(y=y), slice(0, 128)), (backward, dict(dg=dg, dv=dv), slice((L - 1) // 128 * 128, L))):
        for name, t in names.items():
            bad = torch.isnan(t)
            assert torch.equal(t[~bad], want[name][~bad]) and not bool(bad[:, sure].any())
            assert bool(bad.any()) == (status == b.SPECTRE_ERR_TIMEOUT)
        if L <= 1000:       # one thread a channel does not look before it gives up
            assert status == b.SPECTRE_ERR_TIMEOUT
    for name in want:
        assert torch.equal(want[name], after[name]), name


def test_wait_option_is_validated():
    with b.GatedScan(1, 8, "f32") as s:
        for option, value in ((b.GATED_SCAN_OPT_TEST_WAIT_TIMEOUT, 3), (b.GATED_SCAN_OPT_TEST_WAIT_TIMEOUT, -1), (0, 1), (2, 0)):
            with pytest.raises(b.SpectreMixError):
                b.gated_scan_set_option(s.handle, option, value)
    assert b._lib.gated_scan_set_option(None, b.GATED_SCAN_OPT_TEST_WAIT_TIMEOUT, 0) == b.SPECTRE_ERR_ARG


@pytest.mark.parametrize("per", ["channel", "head"])
def test_millions_of_sequences(per):
    """Sequences by the million, most of them of one row and some empty: the blocks that others wait for do not walk
    them all (that took half a second here; a wait lasts four)."""
    n, C = 12_000_000, 32
    gen = torch.Generator(device="cuda").manual_seed(0)
    lengths = (torch.rand(n, generator=gen, device="cuda") < 0.9).int()
    lengths[n // 2] = 300
    cu = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    cu[1:] = lengths.cumsum(0)
    L = int(cu[-1])
    g = torch.randn(1, 1, C if per == "channel" else 1, generator=gen, device="cuda").expand(1, L, -1)
    v, h0 = torch.randn(1, L, C, generator=gen, device="cuda"), torch.randn(n, C, generator=gen, device="cuda")
    with b.GatedScan(1, C, "f32", "sigmoid", per) as s:
        st = s.new_states(1, L)
        calls = [lambda: s(g, v, h0=h0, cu_seqlens=cu, states=st)[1],
                 lambda: s.backward(v, g, v, st, h0=h0, dhT=h0, cu_seqlens=cu)[2]]
        ends = []
        for call in calls:
            e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            call()
            e[0].record()
            ends.append(call())
            e[1].record()
            torch.cuda.synchronize()
            took = e[0].elapsed_time(e[1])
            assert took < 200.0, took
        assert b.gated_scan_device_status(s.handle) == b.SPECTRE_OK
    a = torch.sigmoid(g[0, 0].double())
    for k in range(0, n, 3_000_000):        # in parts, for their 64-bit copies
        on = slice(k, k + 3_000_000)
        empty, one, at = lengths[on] == 0, lengths[on] == 1, cu[on].long()
        for name, got in zip(("hT", "dh0"), ends):
            assert torch.equal(got[on][empty], h0[on][empty])
            row, h = v[0][at[one]].double(), h0[on][one].double()
            want = a * h + (1 - a) * row if name == "hT" else a * (h + row)
            off = (got[on][one].double() - want).abs()
            assert bool((off <= ref.K * ref.U * (h.abs() + row.abs())).all())
    del v, h0, st, ends
    torch.cuda.empty_cache()


def _some_channels(H, D, per):
    """Channels (or whole heads) of the first strip, the middle and the last strip, as (H, D) of their own."""
    if per == "channel":
        c = torch.cat([torch.arange(8), torch.arange(8) + H * D // 2, torch.arange(H * D - 40, H * D)])
        return c, c, len(c), 1
    heads = torch.tensor([0, H - 1])
    return heads, (heads[:, None] * D + torch.arange(D)).reshape(-1), 2, D


@pytest.mark.parametrize("B,L,H,D,dtype,form,per,cu", [
    (3, 6001, 10, 64, "bf16", "sigmoid", "channel", None),
    (3, 6001, 10, 64, "f32", "exp", "head", None),
    (3, 6001, 16, 128, "bf16", "exp", "head", None),
    (3, 6001, 10, 64, "f32", "sigmoid", "channel", None),
    (3, 9001, 7, 33, "bf16", "sigmoid", "channel", None),
    (2, 12001, 7, 33, "f32", "exp", "head", None),
    (1, 20003, 10, 64, "bf16", "sigmoid", "channel", [0, 7000, 7000, 7001, 13000, 20003]),
    (1, 20003, 10, 64, "f32", "exp", "head", [100, 128, 9000, 19999]),
    (1, 30001, 7, 33, "bf16", "exp", "channel", [0, 15000, 29000]),
])
def test_blocks_that_take_tile_after_tile(B, L, H, D, dtype, form, per, cu):
    """Three tiles a block and more, joined by looking back, over strips, batch entries and chunks: the strips' order,
    buffers used again and the copies' phases.  Some channels of the first, a middle and the last strip are compared."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    C, t, n = H * D, TYPES[dtype], B if cu is None else len(cu) - 1
    mk = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    z = mk(B, L, C if per == "channel" else H)
    g = (z * 1.5 + 6 if form == "sigmoid" else -0.003 * torch.nn.functional.softplus(z)).to(t)
    v, dy = mk(B, L, C).to(t), mk(B, L, C).to(t)
    h0, dhT = mk(n, C), mk(n, C)
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    with b.GatedScan(H, D, dtype, form, per) as s:
        got = _both_ways(s, g, v, dy, h0, dhT, cud)
        torch.cuda.synchronize()
        assert b.gated_scan_device_status(s.handle) == b.SPECTRE_OK
    cg, cc, h, d = _some_channels(H, D, per)

    def rows(x, c):     # batch entries beside one another: [1, L, B c]
        return x.cpu()[:, :, c].transpose(0, 1).reshape(1, L, -1)

    def ends(x):
        return x.cpu()[:, cc].reshape(1, -1) if cu is None else x.cpu()[:, cc]
    val, err = ref.scan(rows(g, cg), rows(v, cc), h * B, d, form, ends(h0), cu, rows(dy, cc), ends(dhT))
    inside = slice(0, L) if cu is None else slice(cu[0], cu[-1])
    for name, c in (("y", cc), ("dv", cc), ("dg", cg)):
        ref.check(name, rows(got[name], c)[:, inside], val[name][:, inside], err[name][:, inside])
    for name in ("hT", "dh0"):
        ref.check(name, ends(got[name]), val[name], err[name])


@pytest.mark.parametrize("C,gate_dtype", [(64, "bf16"), (64, "f32"), (21, "bf16")])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_far_gates_of_bf16_rows(C, gate_dtype, sign):
    """|g| from 20 to 80, where the hardware's exp2 gets an exponent of up to 115.  Its rounding (u of it) and that of
    log2(e) (0.23 u) are 1.23 |g| u of the factor; exp2 (4 u), 1 + e (u), the reciprocal (2 u) and a product (u) come to
    16 u at most.  The fp32 states show it: sums of small factors times values (sign 1, the other factor being one), or
    the product of one with the state ahead (sign -1, no values)."""
    L, u = (24, ref.U) if sign > 0 else (1, ref.U)
    gen = torch.Generator().manual_seed(3)
    g = (sign * (20 + 60 * torch.rand(1, L, C, generator=gen))).to(TYPES[gate_dtype])
    v, h0 = torch.randn(1, L, C, generator=gen).bfloat16(), torch.randn(1, C, generator=gen)
    if sign > 0:
        h0 = torch.zeros_like(h0)
    else:
        v = torch.zeros_like(v)
    with b.GatedScan(1, C, "bf16", "sigmoid", "channel", gate_dtype) as s:
        _, hT = s(g.cuda(), v.cuda(), h0=h0.cuda())
        torch.cuda.synchronize()
    x = g.double()
    terms = torch.sigmoid(-x) * v.double() if sign > 0 else torch.sigmoid(x) * h0.double()
    # 2 L u: a row's addition, and its larger factor, taken as one
    bound = (terms.abs() * (1.25 * x.abs() + 16 + 2 * L) * u).sum(1)
    assert bool(((hT.cpu().double() - terms.sum(1)).abs() <= bound).all())
