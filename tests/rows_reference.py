"""The gated linear recurrence and the residual norm in 64 bits, each with a bound on the
error of an fp32 computation in any order of association, and the bounds' derivation.

u = 2^-24 is fp32's largest relative rounding.  Outputs in bf16 add half a step,
``torch.finfo(torch.bfloat16).eps / 2`` = 2^-8, of the value (HALF).
"""
import torch

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: torch.finfo(torch.bfloat16).eps / 2}

# Roundings of one factor of the recurrence: exp 2 ulp (4 u), 1 + e (u), the reciprocal (u), e * r (u) for the
# gate or its complement, e's error entering both factors of e * r (4 u more); the product with the state or the
# value and the addition (2 u): 13 in all.  A bound of 16 u for each product covers them.
K = 16


def gate(g, form):
    """a and the value's factor c in 64 bits (c = 1 for exp)."""
    g = g.double()
    if form == "exp":
        return torch.exp(g), torch.ones_like(g)
    return torch.sigmoid(g), torch.sigmoid(-g)


def drop0(f, x):
    """f * x where a factor of zero takes x out."""
    return torch.where(f == 0, torch.zeros((), dtype=torch.float64), f * x)


def _widen(t, H, D):
    """[.., H] or [.., C] to [.., C]."""
    return t if t.shape[-1] == H * D and not (D > 1 and t.shape[-1] == H) else t.repeat_interleave(D, dim=-1)


def scan(g, v, H, D, form, h0=None, cu=None, dy=None, dhT=None):
    """The recurrence over [B, L, C] row by row, and with dy its gradients.  Returns dicts of values and of error
    bounds: y, hT, and dg (summed over each head's channels where g is per head), dv, dh0.

    Bound: h is a sum of products of gates and one input.  M is the same sum of magnitudes; each of a term's
    products adds at most K u of the term, so E_t = a E_{t-1} + K u (a M_{t-1} + |b_t|) bounds |h - h_fp32| whatever
    the order in which terms are joined.  The reverse recurrence of dh has the same form with |dy|.
    """
    B, L, C = v.shape
    per_head = g.shape[-1] != C or (D > 1 and g.shape[-1] == H)
    a, c = gate(_widen(g, H, D) if per_head else g, form)
    v = v.double()
    b = v if form == "exp" else drop0(c, v)
    spans = [(i, 0, L, i) for i in range(B)] if cu is None else [(0, p, q, n) for n, (p, q) in enumerate(zip(cu, cu[1:]))]
    val = {"y": torch.full((B, L, C), float("nan"), dtype=torch.float64), "hT": torch.zeros(len(spans), C, dtype=torch.float64)}
    err = {"y": torch.zeros(B, L, C, dtype=torch.float64), "hT": torch.zeros(len(spans), C, dtype=torch.float64)}
    prev, mag, eprev = (torch.zeros(B, L, C, dtype=torch.float64) for _ in range(3))
    for i, p, q, n in spans:
        h = torch.zeros(C, dtype=torch.float64) if h0 is None else h0[n].double()
        m, e = h.abs(), torch.zeros(C, dtype=torch.float64)
        for t in range(p, q):
            prev[i, t], mag[i, t], eprev[i, t] = h, m, e
            at = a[i, t]
            h = drop0(at, h) + b[i, t]
            e = drop0(at, e) + K * U * (drop0(at, m) + b[i, t].abs())
            m = drop0(at, m) + b[i, t].abs()
            val["y"][i, t], err["y"][i, t] = h, e
        val["hT"][n], err["hT"][n] = h, e
    if dy is None:
        return val, err
    dy = dy.double()
    for k in ("dg", "dv"):
        val[k], err[k] = torch.full((B, L, C), float("nan"), dtype=torch.float64), torch.zeros(B, L, C, dtype=torch.float64)
    val["dh0"], err["dh0"] = torch.zeros(len(spans), C, dtype=torch.float64), torch.zeros(len(spans), C, dtype=torch.float64)
    for i, p, q, n in spans:
        carry = torch.zeros(C, dtype=torch.float64) if dhT is None else dhT[n].double()
        mc, ec = carry.abs(), torch.zeros(C, dtype=torch.float64)
        for t in range(q - 1, p - 1, -1):
            dh, m = carry + dy[i, t], mc + dy[i, t].abs()
            e = ec + K * U * m
            at, ct = a[i, t], c[i, t]
            w = at if form == "exp" else at * ct
            x = prev[i, t] if form == "exp" else prev[i, t] - v[i, t]
            xm = mag[i, t] if form == "exp" else mag[i, t] + v[i, t].abs()
            val["dg"][i, t] = drop0(w, x) * dh
            # the factors' own errors, and K u for each of the products and the two gates
            err["dg"][i, t] = drop0(w, e * xm + m * eprev[i, t] + 2 * K * U * m * xm)
            val["dv"][i, t] = dh if form == "exp" else drop0(ct, dh)
            err["dv"][i, t] = e if form == "exp" else drop0(ct, e + K * U * m)
            carry, mc, ec = drop0(at, dh), drop0(at, m), drop0(at, e) + K * U * drop0(at, m)
        val["dh0"][n], err["dh0"][n] = carry, ec
    if per_head:
        # a sum of D values, D u of their magnitudes at most
        mag_dg = val["dg"].abs().view(B, L, H, D).sum(-1)
        val["dg"], err["dg"] = val["dg"].view(B, L, H, D).sum(-1), err["dg"].view(B, L, H, D).sum(-1) + D * U * mag_dg
    return val, err


# Roundings of a sum over a row: at most 16 values in turn in a thread, 5 exchanges in a warp, 16 warps, the product
# with 1 / C and that quotient's own: under 40.
KN = 40


def norm(out, x, gamma, beta, form, eps, dy=None):
    """y = N(out + x) or N(out) + x over rows [T, C] and with dy its gradients dz, dgamma, dbeta; values and bounds.

    With z's own rounding (u |z|) and the mean's (KN u mean|z|) in units of the deviation, n = (z - mean) r is off by
    at most (1 + |n|) r KN u (|z| + mean|z| + rms z) + KN u |n|: the variance is a mean of squares of z - mean, so its
    relative error is twice that of the deviations, and r's once.
    """
    out, x, gamma, beta = out.double(), x.double(), gamma.double(), beta.double()
    post, ln = form.startswith("post"), form.endswith("ln")
    z = out + x if post else out
    T, C = z.shape
    mean = z.mean(-1, keepdim=True) if ln else torch.zeros(T, 1, dtype=torch.float64)
    r = 1 / torch.sqrt(((z - mean) ** 2).mean(-1, keepdim=True) + eps)
    n = (z - mean) * r
    size = z.abs() + z.abs().mean(-1, keepdim=True) + (z * z).mean(-1, keepdim=True).sqrt()
    en = (1 + n.abs()) * r * KN * U * size + KN * U * n.abs()
    y = n * gamma + beta + (0 if post else x)
    val = {"y": y}
    err = {"y": gamma.abs() * en + 4 * U * ((n * gamma).abs() + beta.abs() + (0 if post else x.abs()))}
    if dy is None:
        return val, err
    dy = dy.double()
    dn = dy * gamma
    level = dn.mean(-1, keepdim=True) if ln else torch.zeros(T, 1, dtype=torch.float64)
    along = (dn * n).mean(-1, keepdim=True)
    val["dz"] = r * (dn - level - n * along)
    total = dn.abs() + dn.abs().mean(-1, keepdim=True) + n.abs() * (dn * n).abs().mean(-1, keepdim=True)
    er = r * KN * U * size.mean(-1, keepdim=True) + KN * U
    err["dz"] = r * (2 * KN * U * total + en * (dn * n).abs().mean(-1, keepdim=True) +
                     n.abs() * (dn.abs() * en).mean(-1, keepdim=True) + er * total)
    # at most T additions, in any order
    val["dgamma"], val["dbeta"] = (dy * n).sum(0), dy.sum(0)
    err["dgamma"] = (dy.abs() * en).sum(0) + (T + KN) * U * (dy * n).abs().sum(0)
    err["dbeta"] = (T + KN) * U * dy.abs().sum(0)
    return val, err


def check(name, got, want, bound):
    """|got - want| <= bound + half a step of got's type, element by element."""
    got64 = got.detach().cpu().double()
    limit = bound + HALF[got.dtype] * want.abs()
    if got.dtype == torch.bfloat16:
        limit = limit + HALF[got.dtype] * bound
    off = (got64 - want).abs() - limit
    bad = ~(off <= 1e-37)       # below the smallest normal number nothing is promised
    same = torch.isinf(want) & (got64 == want)
    bad &= ~same
    assert not bool(bad.any()), (f"{name}: {int(bad.sum())} of {bad.numel()} outside the bound; first at "
                                 f"{bad.nonzero()[0].tolist()}: {got64[bad][0].item()} for {want[bad][0].item()}, "
                                 f"bound {limit[bad][0].item():.3e}")
