"""The norm, the short convolution and the selective scan in 64 bits on the CPU,
token by token, and the rounding bounds that their results are held to.
Independent of the kernels: values come from the definitions, gradients from
automatic differentiation of them.

A bound is a sum of magnitudes (the definition with |.| of every term) times a
number of roundings of 2^-24, beside the rounding of the stored type."""

from __future__ import annotations

import torch

BF16 = torch.finfo(torch.bfloat16).eps / 2  # largest relative error of one rounding
U = torch.finfo(torch.float32).eps / 2


def starts_of(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32)


def worst(got, want, bound, rounding):
    """max |got - want| / (bound + rounding |want|): at most 1 passes.  `rounding`: of the stored type.  The last term
    keeps exact zeros comparable (nothing below 2^-120 matters)."""
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (got.shape, want.shape)
    if not got.numel():
        return 0.0
    ok = torch.isfinite(got)
    assert bool(ok.all()), f"{int((~ok).sum())} of {ok.numel()} values are not finite"
    return float(((got - want).abs() / (bound + rounding * want.abs() + 2.0 ** -120)).max())


# ---------------------------------------------------------------- norm

# A row's sum: at most 64 terms a thread one after another, 10 levels of a tree
# and 16 wavefronts; mean, eps, root, reciprocal and two products: 6 more.  The
# sum enters through a root, so half of it counts.
NORM = (90 / 2 + 8) * U


def norm(x, residual, weight, eps):
    """y and r in fp64, r rounded to the residual's type as the stream is held."""
    r = x.double()
    if residual is not None:
        r = (r + residual.double()).to(residual.dtype).double()
    return r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps) * weight.double(), r


def norm_gradients(r, weight, d_y, d_r, eps):
    r, w, dy = r.double().requires_grad_(), weight.double().requires_grad_(), d_y.double()
    y = r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps) * w
    loss = (y * dy).sum()
    if d_r is not None:
        loss = loss + (r * d_r.double()).sum()
    dr, dw = torch.autograd.grad(loss, (r, w))
    with torch.no_grad():
        s = 1 / torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
        u = (w * dy).abs()
        m = s * u + s ** 3 * r.abs() * (u * r.abs()).mean(-1, keepdim=True)
        if d_r is not None:
            m = m + d_r.double().abs()
        # dr: two sums over the row and three powers of s; dw: a sum over the rows beside them
        return dr, m * 6 * NORM, dw, (s * r.abs() * dy.abs()).sum(0) * (2 * NORM + r.shape[0] * U)


# ---------------------------------------------------------------- convolution

# taps and bias, then silu: its exponent is rounded twice (|p| 2^-23, and p
# silu'(p) grows no faster than silu itself plus 1), exponential, sum,
# reciprocal, product
CONV = 24 * U


def conv_one(line, w, bias, silu):
    """line [width - 1 + n, D], the inputs ahead first -> y [n, D]"""
    n, W = line.shape[0] - (w.shape[1] - 1), w.shape[1]
    p = sum(line[j:j + n] * w[:, j] for j in range(W))
    if bias is not None:
        p = p + bias
    return p * torch.sigmoid(p) if silu else p


def conv(x, weight, bias, lens, initial, silu):
    """y [T, D], final states [B, width - 1, D] and the magnitudes of y, in fp64."""
    w, b, D, back = weight.double(), None if bias is None else bias.double(), x.shape[1], weight.shape[1] - 1
    ys, ms, finals, at = [], [], [], 0
    for i, n in enumerate(lens):
        ahead = initial[i].double() if initial is not None else torch.zeros(back, D, dtype=torch.float64)
        line = torch.cat([ahead, x[at:at + n].double()])
        ys.append(conv_one(line, w, b, silu))
        with torch.no_grad():
            ms.append(conv_one(line.abs(), w.abs(), None if b is None else b.abs(), False))
        finals.append(line[n:])
        at += n
    return torch.cat(ys), torch.stack(finals), torch.cat(ms)


def conv_gradients(x, weight, bias, lens, initial, d_y, d_final, silu):
    """(gradient, bound) of x, weight, bias, initial states."""
    T = sum(lens)
    xs, w = x[:T].double().requires_grad_(), weight.double().requires_grad_()
    b = torch.zeros(x.shape[1], dtype=torch.float64) if bias is None else bias.double()
    b.requires_grad_()
    i0 = (torch.zeros(len(lens), weight.shape[1] - 1, x.shape[1], dtype=torch.float64) if initial is None
          else initial.double()).requires_grad_()
    y, f, m = conv(xs, w, b, lens, i0, silu)
    dy = d_y[:T].double()
    loss = (y * dy).sum()
    if d_final is not None:
        loss = loss + (f * d_final.double()).sum()
    grads = torch.autograd.grad(loss, (xs, w, b, i0), allow_unused=True, materialize_grads=True)
    # magnitudes: the same with |.|, where silu' moves by at most 1/2 for each unit of p's own error, and is
    # itself known to the roundings of CONV of a number below 2
    ax, aw, ai = (t.detach().abs().requires_grad_() for t in (xs, w, i0))
    ab = b.detach().abs().requires_grad_()
    ya, fa, _ = conv(ax, aw, ab, lens, ai, False)
    loss = (ya * dy.abs() * (2 + m)).sum()
    if d_final is not None:
        loss = loss + (fa * d_final.double().abs()).sum()
    sizes = torch.autograd.grad(loss, (ax, aw, ab, ai), allow_unused=True, materialize_grads=True)
    steps = (CONV, CONV + T * U, CONV + T * U, CONV)
    return [(g, s * e) for g, s, e in zip(grads, sizes, steps)]


# ---------------------------------------------------------------- selective scan

def scan_roundings(lens):
    """Of a state, relative to its magnitude: a token's decay is an exponential of a product rounded twice (2 U |x|
    of it, and |x| e^-|x| < 1/2), good to 2 U itself, and the sum is rounded once: under 4 U a token.  The time step
    (softplus: an exponential, a logarithm, a quotient and three roundings) shifts the exponents of all of them by as
    much, which counts |x| e^-|x| again: 16 U.  Sums over states (64 at most), D x and the gate: 64 U."""
    return (4 * max(lens, default=0) + 80) * U


def scan_inputs(lens, D, G, N, seed, *, slots=0, tail=0, decay=1.0):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens) + tail

    def normal(*shape):
        return torch.randn(*shape, generator=g)

    d = dict(x=normal(T, D).bfloat16(), dt=(0.5 * normal(T, D)).bfloat16(), z=normal(T, D).bfloat16(),
             B=normal(T, G, N).bfloat16(), C=normal(T, G, N).bfloat16(), d_y=normal(T, D).bfloat16(),
             A=-decay * torch.arange(1, N + 1).float() * torch.exp(0.3 * normal(D, N)),
             D=1 + 0.1 * normal(D), dt_bias=-2 + normal(D), query_start_loc=starts_of(lens),
             initial=normal(len(lens), D, N), d_final=normal(len(lens), D, N))
    if slots:
        d["pool"] = normal(slots, D, N)
        d["cache_indices"] = torch.randperm(slots, generator=g)[:len(lens)].to(torch.int32)
    return d


def _scan(x, raw, A, B, C, D, z, lens, initial, softplus, size):
    """y, final states; `size`: the same with magnitudes."""
    n, G = B.shape[2], B.shape[1]
    group = torch.arange(x.shape[1]) // (x.shape[1] // G)
    dts = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
    ab = (lambda t: t.abs()) if size else (lambda t: t)
    ys, finals, at = [], [], 0
    for b, n in enumerate(lens):
        h = ab(initial[b])
        for t in range(at, at + n):
            h = torch.exp(dts[t][:, None] * A) * h + ab(dts[t] * x[t])[:, None] * ab(B[t][group])
            ys.append((ab(C[t][group]) * h).sum(-1))
        finals.append(h)
        at += n
    y = torch.stack(ys) if ys else torch.zeros(0, x.shape[1], dtype=torch.float64)
    y = y + ab(D) * ab(x[:at])
    return (y if z is None else y * ab(z[:at] * torch.sigmoid(z[:at]))), torch.stack(finals)


def _doubles(d, lens, initial, use):
    """x, raw time steps, A, B, C, D, z, initial states in fp64; what `use` leaves out is zero (z: None)."""
    T = sum(lens)
    x, A = d["x"][:T].double(), d["A"].double()
    zero = torch.zeros(x.shape[1], dtype=torch.float64)
    h0 = torch.zeros(len(lens), *A.shape, dtype=torch.float64) if initial is None else initial.double()
    return [x, d["dt"][:T].double(), A, d["B"][:T].double(), d["C"][:T].double(),
            d["D"].double() if "D" in use else zero, d["z"][:T].double() if "z" in use else None,
            d["dt_bias"].double() if "dt_bias" in use else zero, h0]


ALL = ("D", "z", "dt_bias")


def scan(d, lens, initial=None, softplus=True, use=ALL):
    """y, its bound, final states, their bound."""
    x, dt, A, B, C, D, z, bias, h0 = _doubles(d, lens, initial, use)
    y, f = _scan(x, dt + bias, A, B, C, D, z, lens, h0, softplus, False)
    my, mf = _scan(x, dt + bias, A, B, C, D, z, lens, h0, softplus, True)
    e = scan_roundings(lens)
    return y, my * e, f, mf * e


def scan_gradients(d, lens, initial=None, d_final=None, softplus=True, use=ALL):
    """{name: (gradient, bound)} of x, dt, A, B, C, D, z, dt_bias, initial."""
    names = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "initial")
    v = _doubles(d, lens, initial, use)
    leaves = [t.clone().requires_grad_() if t is not None else None for t in v]
    x, dt, A, B, C, D, z, bias, h0 = leaves
    y, f = _scan(x, dt + bias, A, B, C, D, z, lens, h0, softplus, False)
    T = sum(lens)
    dy = d["d_y"][:T].double()
    loss = (y * dy).sum()
    if d_final is not None:
        loss = loss + (f * d_final.double()).sum()
    live = [t for t in leaves if t is not None]
    got = iter(torch.autograd.grad(loss, live, allow_unused=True, materialize_grads=True))
    grads = {n: next(got) for n, t in zip(names, leaves) if t is not None}
    sizes = _sizes(v, lens, dy, d_final, softplus)
    # two chains of decays and the sums over channels and tokens (each by parts: 8 tokens, segments, 64 channels)
    e = 2 * scan_roundings(lens) + (64 + T / 8) * U
    return {n: (g, sizes[n] * e) for n, g in grads.items()}


def _sizes(v, lens, dy, d_final, softplus):
    """The gradients' formulas with the magnitude of every term."""
    x, dt, A, B, C, D, z, bias, h0 = v
    T, G = x.shape[0], B.shape[1]
    group = torch.arange(x.shape[1]) // (x.shape[1] // G)
    raw = dt + bias
    dts = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
    slope = torch.sigmoid(raw) if softplus else torch.ones_like(raw)
    e = dy.abs() if z is None else (dy * z * torch.sigmoid(z)).abs()
    out = {n: torch.zeros_like(t) for n, t in zip(("x", "dt", "A", "B", "C", "D"), (x, dt, A, B, C, D))}
    out["initial"] = torch.zeros_like(h0)
    sy = torch.zeros_like(x)
    a = torch.exp(dts[..., None] * A)
    ax, at = x.abs(), 0
    for b, n in enumerate(lens):
        h = [h0[b].abs()]
        for t in range(at, at + n):
            h.append(a[t] * h[-1] + (dts[t].abs() * ax[t])[:, None] * B[t][group].abs())
            sy[t] = (C[t][group].abs() * h[-1]).sum(-1)
        u = d_final[b].double().abs() if d_final is not None else torch.zeros_like(h0[b])
        for t in reversed(range(at, at + n)):
            u = u + C[t][group].abs() * e[t][:, None]
            out["C"][t] = (e[t][:, None] * h[t - at + 1]).unflatten(0, (G, -1)).sum(1)
            out["B"][t] = (u * (dts[t].abs() * ax[t])[:, None]).unflatten(0, (G, -1)).sum(1)
            uB = (u * B[t][group].abs()).sum(-1)
            u = u * a[t]
            q = u * h[t - at]
            out["A"] += dts[t].abs()[:, None] * q
            out["x"][t] = dts[t].abs() * uB + D.abs() * e[t]
            out["dt"][t] = ((q * A.abs()).sum(-1) + ax[t] * uB) * slope[t]
        out["initial"][b] = u
        at += n
    out["D"] = (e * ax).sum(0)
    out["dt_bias"] = out["dt"].sum(0)
    if z is not None:
        p = torch.sigmoid(z)
        out["z"] = dy.abs() * (sy + D.abs() * ax) * p * (1 + z.abs() * (1 - p))
    return out
