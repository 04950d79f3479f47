"""The operators' measured cases: the gated linear recurrence (forward, forward with backward, and its step for
single tokens) and the residual norm (forward and backward).

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU, ``run`` is one pass, in plain torch where
``own`` is false and by the library's kernels where it is true.  ``exact`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

EPS = 1e-5
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def _scan(name, op, B, L, H, D, dtype, gate, per, gate_dtype=None, seqs=0, h0=False, fused=False, resets=False):
    return {"name": name, "op": op, "B": B, "L": L, "H": H, "D": D, "dtype": dtype, "gate": gate, "per": per,
            "gate_dtype": gate_dtype or dtype, "seqs": seqs, "h0": h0, "fused": fused, "resets": resets}


def _step(name, B, H, D, dtype, gate, per, slots=0):
    return {"name": name, "op": "step", "B": B, "H": H, "D": D, "dtype": dtype, "gate": gate, "per": per,
            "gate_dtype": dtype, "slots": slots}


def _norm(name, op, T, C, dtype, norm):
    return {"name": name, "op": op, "T": T, "C": C, "dtype": dtype, "norm": norm}


def listed():
    return [
        # the shortest prompt of a small model: two chunks of rows, launch latency alone
        _scan("scan_tiny", "scan", 1, 256, 1, 16, "f32", "sigmoid", "channel"),
        # prefill of a serving batch: prompts of ragged lengths packed one after another, each from a cached state
        _scan("scan_prefill_packed", "scan", 1, 6007, 8, 64, "bf16", "exp", "head", "f32", seqs=11, h0=True, resets=True),
        # one very long document, read once
        _scan("scan_very_long", "scan", 1, 1048576, 8, 64, "bf16", "sigmoid", "channel"),
        # training on one long document; gate and value are halves of one projection
        _scan("scan_train_long", "train", 1, 65536, 8, 64, "bf16", "sigmoid", "channel", fused=True),
        # training on a batch at the widest configuration, one decay per head
        _scan("scan_train_heads", "train", 4, 12288, 16, 128, "bf16", "exp", "head", "f32"),
        # training on packed documents with odd head sizes, in fp32
        _scan("scan_train_odd", "train", 1, 5003, 7, 33, "f32", "sigmoid", "channel", seqs=9, h0=True),
        # one new token of one sequence
        _step("step_one", 1, 8, 64, "bf16", "sigmoid", "channel"),
        # one new token of each sequence of a serving batch, states in a pool
        _step("step_batch", 256, 16, 128, "bf16", "exp", "head", slots=1024),
        # the norm after a step: a few rows
        _norm("norm_decode", "norm", 8, 2048, "bf16", "pre_rms"),
        # the norm over one long document
        _norm("norm_long", "norm", 65536, 512, "bf16", "post_ln"),
        # training: the widest configuration's batch
        _norm("norm_grad_wide", "norm_grad", 49152, 2048, "bf16", "post_ln"),
        # training: odd rows and channels, fp32
        _norm("norm_grad_odd", "norm_grad", 5003, 231, "f32", "pre_rms"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "train", "step", "norm", "norm_grad"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("norm", "norm_grad"):
        C = _log(rng, 16, 4096)
        T = _log(rng, 1, min(200000, 2 ** 27 // C))
        return {"op": op, "T": T, "C": C, "dtype": dtype, "norm": rng.choice(["post_ln", "pre_ln", "post_rms", "pre_rms"])}
    H, D = _log(rng, 1, 16), _log(rng, 4, 160)
    gate, per = rng.choice(["sigmoid", "exp"]), rng.choice(["channel", "head"])
    if op == "step":
        B = _log(rng, 1, 1024)
        return {"op": op, "B": B, "H": H, "D": D, "dtype": dtype, "gate": gate, "per": per, "gate_dtype": dtype,
                "slots": rng.choice([0, B + rng.randrange(0, 512)])}
    B = rng.choice([1, 1, 2, 3, 4, 8])
    L = _log(rng, 1, max(1, min(131072, 2 ** 26 // (B * H * D))))
    seqs = rng.randrange(1, 1 + min(L, 24)) if rng.random() < 0.4 else 0
    gate_dtype = rng.choice([dtype, "f32"])
    return {"op": op, "B": 1 if seqs else B, "L": L, "H": H, "D": D, "dtype": dtype, "gate": gate, "per": per,
            "gate_dtype": gate_dtype, "seqs": seqs, "h0": rng.random() < 0.5,
            "fused": per == "channel" and gate_dtype == dtype and rng.random() < 0.5,
            "resets": gate == "exp" and rng.random() < 0.5}


def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] in ("norm", "norm_grad"):
        n, grad = case["T"] * case["C"], case["op"] == "norm_grad"
        # forward: out, x read, y written; backward: dy, out (and x where it is inside the norm) read, the gradient written
        tensors = 3 if not grad else 4 if case["norm"].startswith("post") else 3
        return {"bytes": tensors * n * es + case["C"] * (12 if grad else 8), "flops": n * (18 if grad else 8)}
    C, gs = case["H"] * case["D"], 4 if case["gate_dtype"] == "f32" else 2
    gc = C if case["per"] == "channel" else case["H"]
    if case["op"] == "step":
        n = case["B"]
        return {"bytes": n * (gc * gs + 2 * C * es + 8 * C) + (4 * n if case["slots"] else 0), "flops": 4 * n * C}
    rows, seqs = case["B"] * case["L"], case["seqs"] or case["B"]
    ends = 4 * seqs * C * (2 if case["h0"] else 1)
    if case["op"] == "scan":
        return {"bytes": rows * (gc * gs + 2 * C * es) + ends, "flops": 4 * rows * C}
    # g, v, dy read; y, dg, dv written
    return {"bytes": rows * (2 * gc * gs + 4 * C * es) + ends + (4 * seqs * C if case["h0"] else 0), "flops": 14 * rows * C}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _gates(case, gen, shape):
    """Gate logits (sigmoid: a mean of 0.9, tails to 0.1 and 0.999) or log decays (exp: from a few tokens to hundreds)."""
    z = torch.randn(shape, generator=gen, device="cuda")
    if case["gate"] == "sigmoid":
        return z.mul_(1.5).add_(2.5)
    n = shape[-1]
    rate = torch.exp(torch.linspace(math.log(0.5), math.log(0.004), n, device="cuda")) if n > 1 else torch.full((1,), 0.05, device="cuda")
    g = torch.nn.functional.softplus(z).mul_(-rate)
    if case.get("resets"):   # document borders inside a row of tokens: the state starts again
        g = g.masked_fill(torch.rand(shape[:-1] + (1,), generator=gen, device="cuda") < 1 / 512, -math.inf)
    return g


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] in ("norm", "norm_grad"):
        shape = (case["T"], case["C"])
        s["out"] = torch.randn(shape, generator=gen, device="cuda").to(t)
        s["x"] = torch.randn(shape, generator=gen, device="cuda").to(t)
        s["gamma"] = torch.randn(case["C"], generator=gen, device="cuda") * 0.1 + 1.0
        s["beta"] = torch.randn(case["C"], generator=gen, device="cuda") * 0.1
        if case["op"] == "norm_grad":
            s["dy"] = torch.randn(shape, generator=gen, device="cuda").to(t)
        if own:
            from sub_quadratic_attention_b200.binding import ResidualNorm
            s["plan"] = ResidualNorm(case["C"], case["dtype"], norm=case["norm"], eps=EPS)
        return s
    H, D = case["H"], case["D"]
    C, gt = H * D, TYPES[case["gate_dtype"]]
    gc = C if case["per"] == "channel" else H
    if own:
        from sub_quadratic_attention_b200.binding import GatedScan
        s["plan"] = GatedScan(H, D, case["dtype"], gate=case["gate"], gate_per=case["per"], gate_dtype=case["gate_dtype"])
    if case["op"] == "step":
        B, S = case["B"], case["slots"] or case["B"]
        s["g"] = _gates(case, gen, (B, gc)).to(gt)
        s["v"] = torch.randn((B, C), generator=gen, device="cuda").to(t)
        s["state"] = torch.randn((S, C), generator=gen, device="cuda")
        s["next"] = s["state"].clone()
        s["slots"] = torch.randperm(S, generator=gen, device="cuda")[:B].int() if case["slots"] else None
        return s
    B, L = case["B"], case["L"]
    g = _gates(case, gen, (B, L, gc)).to(gt)
    v = torch.randn((B, L, C), generator=gen, device="cuda").to(t)
    if case["fused"]:   # both are halves of one projection's rows
        both = torch.cat([g, v], dim=-1)
        g, v = both[..., :C], both[..., C:]
    s["g"], s["v"] = g, v
    s["cu"] = None
    if case["seqs"]:
        cuts = sorted(random.Random(seed).choices(range(L + 1), k=case["seqs"] - 1))   # a sequence may be empty
        s["cu"] = torch.tensor([0] + cuts + [L], dtype=torch.int32, device="cuda")
    s["h0"] = torch.randn((case["seqs"] or B, C), generator=gen, device="cuda") if case["h0"] else None
    if case["op"] == "train":
        s["dy"] = torch.randn((B, L, C), generator=gen, device="cuda").to(t)
    return s


# ---------------------------------------------------------------------------------------------------------------
# the passes
# ---------------------------------------------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if op == "scan":
        return _own_scan(s) if own else _plain_scan(s)[:2]
    if op == "train":
        return _own_train(s) if own else _plain_train(s)
    if op == "step":
        return _own_step(s) if own else _plain_step(s)
    if op == "norm":
        return _own_norm(s) if own else _plain_norm(s)
    return _own_norm_grad(s) if own else _plain_norm_grad(s)


def _own_scan(s):
    return s["plan"](s["g"], s["v"], h0=s["h0"], cu_seqlens=s["cu"])


def _own_train(s):
    plan, B, L = s["plan"], s["case"]["B"], s["case"]["L"]
    states = plan.new_states(B, L)
    y, hT = plan(s["g"], s["v"], h0=s["h0"], cu_seqlens=s["cu"], states=states)
    dg, dv, dh0 = plan.backward(s["dy"], s["g"], s["v"], states, h0=s["h0"], cu_seqlens=s["cu"])
    return (y, hT, dg, dv) if s["h0"] is None else (y, hT, dg, dv, dh0)


def _own_step(s):
    return s["plan"].step(s["g"], s["v"], s["state"], slots=s["slots"], new_state=s["next"])


def _own_norm(s):
    return s["plan"](s["out"], s["x"], s["gamma"], s["beta"])


def _own_norm_grad(s):
    dout, dx, dgamma, dbeta = s["plan"].backward(s["dy"], s["out"], s["x"], s["gamma"])
    return dout, dgamma, dbeta


def _recurrence(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from h_{-1} = 0, by pairs: the odd rows are a recurrence of half the length."""
    L = a.shape[1]
    if L == 1:
        return b
    n, m = L // 2 * 2, (L - 1) // 2
    odd = _recurrence(a[:, 1:n:2] * a[:, 0:n:2], a[:, 1:n:2] * b[:, 0:n:2] + b[:, 1:n:2])
    h = torch.empty_like(b)
    h[:, 0] = b[:, 0]
    h[:, 1::2] = odd
    h[:, 2::2] = a[:, 2::2] * odd[:, :m] + b[:, 2::2]
    return h


def _gate_forms(case, g):
    """a_t and the value's factor, in 32 bits."""
    if case["gate"] == "sigmoid":
        return torch.sigmoid(g), torch.sigmoid(-g)
    return torch.exp(g), None


def _rows(s):
    """Gate [B, L, H, D or 1] and value [B, L, H, D] in 32 bits."""
    case = s["case"]
    B, L, H, D = case["B"], case["L"], case["H"], case["D"]
    g = s["g"].float().reshape(B, L, H, D if case["per"] == "channel" else 1)
    return g, s["v"].float().reshape(B, L, H, D)


def _start_states(s, like):
    """Which rows are a sequence's first, the state before each of those, and which packed sequences have rows."""
    case = s["case"]
    B, L, H, D = like.shape
    first = torch.zeros(B, L, dtype=torch.bool, device="cuda")
    before = torch.zeros_like(like) if s["h0"] is not None else None
    if s["cu"] is None:
        first[:, 0] = True
        if before is not None:
            before[:, 0] = s["h0"].view(B, H, D)
        return first, before, None
    cu = s["cu"].long()
    full = cu[1:] > cu[:-1]
    rows = torch.where(full, cu[:-1], L)          # an empty sequence points behind the rows
    pad = torch.zeros(B, L + 1, dtype=torch.bool, device="cuda")
    pad[0, rows] = True
    first = pad[:, :L]
    if before is not None:
        wide = torch.zeros((1, L + 1, H, D), device="cuda")
        wide[0, rows] = s["h0"].view(-1, H, D)
        before = wide[:, :L]
    return first, before, full


def _plain_scan(s):
    case = s["case"]
    g, v = _rows(s)
    a, c = _gate_forms(case, g)
    b = v if c is None else c * v
    first, before, full = _start_states(s, b)
    cut = torch.where(first[..., None, None], 0.0, a)
    if before is not None:
        b = b + a * before
    h = _recurrence(cut, b)
    B, L, H, D = h.shape
    if s["cu"] is None:
        hT = h[:, -1].reshape(B, H * D)
    else:
        last = h[0, (s["cu"][1:].long() - 1).clamp_min(0)].reshape(-1, H * D)
        empty = s["h0"] if s["h0"] is not None else torch.zeros_like(last)
        hT = torch.where(full[:, None], last, empty)
    return h.reshape(B, L, H * D).to(s["v"].dtype), hT.clone(), (g, v, a, c, h, cut, first, before, full)


def _plain_train(s):
    y, hT, (g, v, a, c, h, cut, first, before, full) = _plain_scan(s)
    B, L, H, D = h.shape
    dy = s["dy"].float().view(B, L, H, D)
    # dh_t = dy_t + a_{t+1} dh_{t+1}, a recurrence over the rows in reverse, cut where t + 1 starts a sequence
    after = torch.cat([cut[:, 1:], torch.zeros_like(cut[:, :1])], dim=1)
    dh = _recurrence(after.flip(1), dy.flip(1)).flip(1)
    prev = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], dim=1)
    prev = torch.where(first[..., None, None], 0.0 if before is None else before, prev)
    if c is None:
        dv, dg = dh, dh * prev * a
    else:
        dv, dg = dh * c, dh * (prev - v) * (a * c)
    if _per_head(s):
        dg = dg.sum(-1)
    out = (y, hT, dg.reshape(B, L, -1).to(s["g"].dtype), dv.reshape(B, L, H * D).to(s["v"].dtype))
    if s["h0"] is None:
        return out
    if s["cu"] is None:
        dh0 = (a[:, 0] * dh[:, 0]).reshape(B, H * D)
    else:
        start = s["cu"][:-1].long().clamp_max(L - 1)
        dh0 = torch.where(full[:, None], (a[0, start] * dh[0, start]).reshape(-1, H * D), 0.0)
    return out + (dh0,)


def _per_head(s):
    return s["case"]["per"] == "head"


def _plain_step(s):
    case = s["case"]
    B, H, D = case["B"], case["H"], case["D"]
    g = s["g"].float().view(B, H, -1)
    v = s["v"].float().view(B, H, D)
    before = (s["state"] if s["slots"] is None else s["state"][s["slots"].long()]).view(B, H, D)
    a, c = _gate_forms(case, g)
    h = (a * before + (v if c is None else c * v)).view(B, H * D)
    if s["slots"] is None:
        return h.to(s["v"].dtype), h
    s["next"][s["slots"].long()] = h
    return h.to(s["v"].dtype), s["next"]


def _plain_norm(s):
    form = s["case"]["norm"]
    out, x = s["out"].float(), s["x"].float()
    z = out + x if form.startswith("post") else out
    if form.endswith("ln"):
        z = z - z.mean(-1, keepdim=True)
    y = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS) * s["gamma"] + s["beta"]
    return (y if form.startswith("post") else y + x).to(s["x"].dtype)


def _plain_norm_grad(s):
    form = s["case"]["norm"]
    dy, z = s["dy"].float(), s["out"].float()
    if form.startswith("post"):
        z = z + s["x"].float()
    if form.endswith("ln"):
        z = z - z.mean(-1, keepdim=True)
    r = torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS)
    n = z * r
    dn = dy * s["gamma"]
    dz = dn - n * (dn * n).mean(-1, keepdim=True)
    if form.endswith("ln"):
        dz = dz - dn.mean(-1, keepdim=True)
    return (dz * r).to(s["x"].dtype), (dy * n).sum(0), dy.sum(0)


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] in ("norm", "norm_grad"):
        return _exact_norm(prepare(case, seed))
    if case["op"] == "step":
        return _exact_step(prepare(case, seed))
    if case["L"] > 131072:
        return None     # one row after another: about 20 us a row
    return _exact_scan(prepare(case, seed))


def _wide(s, name):
    """A gate input in 64 bits with one value for each channel."""
    g = s[name].double()
    return g if s["case"]["per"] == "channel" else g.repeat_interleave(s["case"]["D"], dim=-1)


def _exact_scan(s):
    """Row after row, sequence after sequence, as the recurrence is written."""
    case = s["case"]
    B, L, C = case["B"], case["L"], case["H"] * case["D"]
    g, v = _wide(s, "g"), s["v"].double()
    sig = case["gate"] == "sigmoid"
    a = 1 / (1 + torch.exp(-g)) if sig else torch.exp(g)
    b = v / (1 + torch.exp(g)) if sig else v
    h = torch.empty_like(b)
    prev = torch.empty_like(b)
    spans = [(0, L, None)] if s["cu"] is None else [(p, q, n) for n, (p, q) in enumerate(zip(s["cu"].tolist(), s["cu"].tolist()[1:]))]
    zero = torch.zeros((B, C), dtype=torch.float64, device="cuda")
    ends = []
    for p, q, n in spans:
        state = zero if s["h0"] is None else s["h0"].double() if n is None else s["h0"][n:n + 1].double()
        for t in range(p, q):
            prev[:, t] = state
            torch.addcmul(b[:, t], a[:, t], state, out=h[:, t])
            state = h[:, t]
        ends.append(state)
    hT = torch.cat(ends, dim=0)
    if case["op"] == "scan":
        return h, hT
    dy = s["dy"].double()
    dh = torch.empty_like(dy)
    starts = []
    for p, q, n in spans:
        carry = zero          # what reaches h_t from the rows behind it
        for t in range(q - 1, p - 1, -1):
            torch.add(dy[:, t], carry, out=dh[:, t])
            carry = a[:, t] * dh[:, t]
        starts.append(carry)
    if sig:
        dv = dh / (1 + torch.exp(g))
        dg = dh * (prev - v) * a / (1 + torch.exp(g))
    else:
        dv, dg = dh, dh * prev * a
    if case["per"] == "head":
        dg = dg.view(B, L, case["H"], case["D"]).sum(-1)
    return (h, hT, dg, dv) + ((torch.cat(starts, dim=0),) if s["h0"] is not None else ())


def _exact_step(s):
    case = s["case"]
    g, v = _wide(s, "g"), s["v"].double()
    pool = s["state"].double()
    at = torch.arange(case["B"], device="cuda") if s["slots"] is None else s["slots"].long()
    if case["gate"] == "sigmoid":
        h = (pool[at] * torch.exp(g) + v) / (1 + torch.exp(g))
    else:
        h = torch.exp(g) * pool[at] + v
    return h, pool.index_copy(0, at, h)


def _exact_norm(s):
    form = s["case"]["norm"]
    C = s["case"]["C"]
    out, x = s["out"].double(), s["x"].double()
    gamma, beta = s["gamma"].double(), s["beta"].double()
    z = out + x if form in ("post_ln", "post_rms") else out
    mean = z.sum(-1, keepdim=True) / C if form in ("post_ln", "pre_ln") else torch.zeros_like(z[:, :1])
    std = torch.sqrt(((z - mean) ** 2).sum(-1, keepdim=True) / C + EPS)
    n = (z - mean) / std
    if s["case"]["op"] == "norm":
        y = n * gamma + beta
        return y if form in ("post_ln", "post_rms") else y + x
    dy = s["dy"].double()
    dn = dy * gamma
    along = (dn * n).sum(-1, keepdim=True) / C
    level = dn.sum(-1, keepdim=True) / C if form in ("post_ln", "pre_ln") else 0.0
    return (dn - level - n * along) / std, (dy * n).sum(0), dy.sum(0)
