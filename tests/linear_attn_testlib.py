"""Linear attention with a fixed decay per head in 64 bits on the CPU, token by
token, and the rounding bounds its results are held to.  Independent of the
kernels: values come from the recurrence (and its automatic gradient)."""

from __future__ import annotations

import torch

BF16 = torch.finfo(torch.bfloat16).eps / 2  # largest relative error of one rounding
# fp32 sums and decays of a chunk, relative to the sum of the terms' magnitudes:
# 64 additions per product chain, the three parts of the weighted v, the decay
# (its exponent n log2 lambda is rounded twice: n |log2 lambda| 2^-23 w, and
# w x <= 0.54 for w = 2^-x), and the chain's own products: under 128 units of
# 2^-24.
FP32 = 2.0 ** -17


def chunk_of(rows, batch, K, V, backward=False):
    """Tokens of a chunk, which decide what reaches an output through rounded scores and what through the rounded
    state: 32 where more than 128 channels are summed over for at most 64 value channels or short sequences, else
    64 (a backward launch goes by the wider of K and V)."""
    k, v = (max(K, V), max(K, V)) if backward else (K, V)
    return 32 if k > 128 and (v <= 64 or -(-rows // batch) <= 256) else 64


def draw(lens, H, G, K, V, seed, *, slots=0, tail=0):
    """Inputs on the CPU: bf16 q, k, v, d_o of sum(lens) + tail rows, slopes, fp32 states."""
    g = torch.Generator().manual_seed(seed)
    T = sum(lens) + tail

    def normal(*shape):
        return torch.randn(*shape, generator=g)

    d = dict(q=normal(T, G, K).bfloat16(), k=normal(T, G, K).bfloat16(), v=normal(T, H, V).bfloat16(),
             d_o=normal(T, H, V).bfloat16(),
             log_decay=-torch.exp2(-8.0 * (torch.arange(H, dtype=torch.float32) + 0.5) / H),
             initial=normal(len(lens), H, V, K), d_final=normal(len(lens), H, V, K))
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    d["query_start_loc"] = torch.tensor(starts, dtype=torch.int32)
    if slots:
        d["pool"] = normal(slots, H, V, K)
        d["cache_indices"] = torch.randperm(slots, generator=g)[:len(lens)].to(torch.int32)
    return d


def recur(q, k, v, lam, scale, S):
    """One sequence: q, k [n, H, K] (already per head), v [n, H, V], lam [H], S [H, V, K] -> o [n, H, V], final."""
    out = []
    for t in range(q.shape[0]):
        S = lam[:, None, None] * S + v[t][:, :, None] * k[t][:, None, :]
        out.append(scale * (S * q[t][:, None, :]).sum(-1))
    return (torch.stack(out) if out else v.new_zeros(v.shape)), S


def spread(x, H):
    return x.repeat_interleave(H // x.shape[1], 1)


def reference(d, lens, scale, initial=None):
    """Forward in fp64 over the ragged batch: o [T, H, V], final [B, H, V, K]."""
    H, V, K = d["v"].shape[1], d["v"].shape[2], d["q"].shape[2]
    lam = torch.exp(d["log_decay"].double())
    o = torch.zeros(sum(lens), H, V, dtype=torch.float64)
    finals, at = [], 0
    for b, n in enumerate(lens):
        S = initial[b].double() if initial is not None else torch.zeros(H, V, K, dtype=torch.float64)
        s = slice(at, at + n)
        o[s], S = recur(spread(d["q"][s].double(), H), spread(d["k"][s].double(), H), d["v"][s].double(), lam, scale, S)
        finals.append(S)
        at += n
    return o, torch.stack(finals)


def gradients(d, lens, scale, initial=None, d_final=None):
    """dq, dk, dv, d_initial in fp64 by automatic differentiation of the recurrence."""
    T, H = sum(lens), d["v"].shape[1]
    q, k, v = (d[n][:T].double().requires_grad_() for n in "qkv")
    S0 = (initial.double() if initial is not None
          else torch.zeros(len(lens), H, v.shape[2], q.shape[2], dtype=torch.float64)).requires_grad_()
    o, f = reference(dict(d, q=q, k=k, v=v), lens, scale, S0)
    loss = (o * d["d_o"][:T].double()).sum()
    if d_final is not None:
        loss = loss + (f * d_final.double()).sum()
    return torch.autograd.grad(loss, (q, k, v, S0), allow_unused=True, materialize_grads=True)


def magnitudes(q, k, v, lam, c_pair, c_state, c_update, S, reverse=False, chunk=64):
    """The chunked sum of one sequence with magnitudes in place of its rounded operands: for each output the sum of
    |rounded operand| |exact operand| (scores and the state are rounded to bf16, once each), and the sum of the
    magnitudes of all the final state's terms.  The scalar c's multiply pairs, state reads and state updates."""
    if reverse:
        q, k, v = q.flip(0), k.flip(0), v.flip(0)
    n, shift = q.shape[0], 1 if reverse else 0
    out = torch.zeros(n, *v.shape[1:], dtype=torch.float64)
    S, A = S.clone(), S.abs()
    qh, kh, vh = (x.transpose(0, 1) for x in (q, k, v))  # [H, n, .]
    for c in range(0, n, chunk):
        s = slice(c, min(c + chunk, n))
        m = s.stop - s.start
        i = torch.arange(m, dtype=torch.float64)
        gap = i[:, None] - i[None, :]
        D = torch.where(gap >= 0, lam[:, None, None] ** gap.clamp(min=0), 0.0)
        P = (qh[:, s] @ kh[:, s].transpose(1, 2)) * D * c_pair
        part = P.abs() @ vh[:, s].abs()
        lead = lam[:, None] ** (i + 1 - shift)
        part = part + c_state * lead[:, :, None] * (qh[:, s].abs() @ S.abs().transpose(1, 2))
        out[s] = part.transpose(0, 1)
        w = c_update * lam[:, None] ** (m - 1 - i + shift)
        keep = lam[:, None, None] ** m
        S = keep * S + (vh[:, s] * w[..., None]).transpose(1, 2) @ kh[:, s]
        A = keep * A + (vh[:, s].abs() * w[..., None]).transpose(1, 2) @ kh[:, s].abs()
    return (out.flip(0) if reverse else out), A


def forward_bounds(d, lens, scale, initial=None):
    """Largest error of o before its own rounding, and of the final states in fp32."""
    H, V, K = d["v"].shape[1], d["v"].shape[2], d["q"].shape[2]
    lam = torch.exp(d["log_decay"].double())
    o, f, at = [], [], 0
    for b, n in enumerate(lens):
        S = initial[b].double() if initial is not None else torch.zeros(H, V, K, dtype=torch.float64)
        s = slice(at, at + n)
        m, A = magnitudes(spread(d["q"][s].double(), H), spread(d["k"][s].double(), H), d["v"][s].double(), lam,
                          scale, scale, 1.0, S, chunk=chunk_of(d["v"].shape[0], len(lens), K, V))
        o.append(m)
        f.append(A)
        at += n
    return torch.cat(o) * (BF16 + 2 * FP32), torch.stack(f) * FP32


def backward_bounds(d, lens, scale, initial=None, d_final=None):
    """The same for dq, dk, dv (the heads of a group summed) and d_initial."""
    H, V, K = d["v"].shape[1], d["v"].shape[2], d["q"].shape[2]
    G = d["q"].shape[1]
    lam = torch.exp(d["log_decay"].double())
    zero = torch.zeros(H, V, K, dtype=torch.float64)
    dq, dk, dv, di, at, chunk = [], [], [], [], 0, chunk_of(d["v"].shape[0], len(lens), K, V, True)
    for b, n in enumerate(lens):
        s = slice(at, at + n)
        q, k, v, g = (spread(d[x][s].double(), H) for x in ("q", "k", "v", "d_o"))
        S = initial[b].double() if initial is not None else zero
        R = d_final[b].double() if d_final is not None else zero
        dq.append(magnitudes(g, v, k, lam, scale, scale, 1.0, S.transpose(1, 2), chunk=chunk)[0])
        dk.append(magnitudes(v, g, q, lam, scale, 1.0, scale, R.transpose(1, 2), reverse=True, chunk=chunk)[0])
        m, A = magnitudes(k, q, g, lam, scale, 1.0, scale, R, reverse=True, chunk=chunk)
        dv.append(m)
        di.append(A)
        at += n

    def groups(x):
        return x.reshape(x.shape[0], G, H // G, K).sum(2)

    e = BF16 + 2 * FP32
    return groups(torch.cat(dq)) * e, groups(torch.cat(dk)) * e, torch.cat(dv) * e, torch.stack(di) * FP32


def worst(got, want, bound, rounding):
    """max |got - want| / (bound + rounding |want|): at most 1 passes.  `rounding`: of the stored type.  The last term
    keeps exact zeros comparable (nothing below 2^-120 matters)."""
    got = got.detach().cpu().double()
    assert got.shape == want.shape
    if not got.numel():
        return 0.0
    ok = torch.isfinite(got)
    assert bool(ok.all()), f"{int((~ok).sum())} of {ok.numel()} values are not finite"
    return float(((got - want).abs() / (bound + rounding * want.abs() + 2.0 ** -120)).max())
