"""The operators of a selective state space layer, as they are measured.

Three operators, in the forms that serving and training call them in:

``norm``        root-mean-square norm with the residual's addition, the output
                in bf16 or in 8 bits with one scale a row;
``norm_train``  its backward pass;
``conv``        the short causal depthwise convolution over a ragged batch of
                prompts, with a pool of the last inputs updated in place;
``conv_step``   the same for one token per sequence;
``conv_train``  its backward pass;
``scan``        the selective scan (a decay per channel and state, a time step
                per channel) over a ragged batch of prompts, pool in place;
``scan_step``   its recurrence for one token per sequence;
``scan_train``  its backward pass.

Norm, of x and the residual stream res, which is held in its own type:

    r = res + x     y = r / sqrt(mean(r^2) + eps) * w

In 8 bits a row of y becomes e4m3 codes under the least power of two that brings
max|y| / scale to 448 or less.

Convolution of channel d with `width` taps and silu:

    y_t = silu(bias + sum_j w[j] x_{t - (width - 1) + j})

Scan of channel d in group g = d // (channels / ngroups), with dts =
softplus(dt + dt_bias):

    h_t[n] = exp(dts A[n]) h_{t-1}[n] + dts x_t B_t[g,n]
    y_t = (sum_n C_t[g,n] h_t[n] + D x_t) silu(z_t)

``run`` computes these with elementary torch operations in fp32 unless ``own``
is true; ``exact`` computes them in fp64, the scan token by token.
"""

import math
import random

import torch

own = False

EPS = 1e-5


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a decode loop ahead of an 8-bit projection: latency
        dict(name="norm_1", op="norm", rows=1, width=4096, residual="bf16", out="e4m3"),
        # a batch of prompts, the residual stream in fp32
        dict(name="norm_16384", op="norm", rows=16384, width=4096, residual="f32", out="bf16"),
        # packed documents of a training step, an odd number of tokens
        dict(name="norm_train_5001", op="norm_train", rows=5001, width=2560, residual="bf16"),
        # ragged prompts of a busy server, some resuming: x, B and C of 128 heads of 64 with 8 groups of 128, a part
        # of the layer's projection
        dict(name="conv_ragged_32", op="conv", lens="ragged 32 17 8192 3", channels=10240, width=4, stride=18560,
             init="half"),
        # a full decode batch of the same layer, over a 1024-slot pool
        dict(name="conv_step_512", op="conv_step", lens="512x1", channels=10240, width=4, stride=18560, init="all"),
        # a training batch of fixed length: 16 heads of 64, one group of 256
        dict(name="conv_train_4x4096", op="conv_train", lens="4x4096", channels=1536, width=4, stride=2576,
             init="none"),
        # a few tokens of prompt at low load: latency
        dict(name="scan_17", op="scan", lens="17", channels=1024, ngroups=1, dstate=16, states="f32", init="none"),
        # ragged prompts of a busy server, some resuming
        dict(name="scan_ragged_32", op="scan", lens="ragged 32 17 8192 3", channels=4096, ngroups=1, dstate=16,
             states="bf16", init="half"),
        # one long document: few rows, the work lies along the sequence
        dict(name="scan_65536", op="scan", lens="65536", channels=2048, ngroups=1, dstate=16, states="f32", init="all"),
        # a full decode batch over a 1024-slot pool
        dict(name="scan_step_512", op="scan_step", lens="512x1", channels=4096, ngroups=1, dstate=16, states="f32",
             init="all"),
        # a fine-tuning step on short samples, grouped B and C of uneven width
        dict(name="scan_train_3x100", op="scan_train", lens="3x100", channels=400, ngroups=2, dstate=12, states="f32",
             init="all"),
        # a training batch of fixed length
        dict(name="scan_train_8x2048", op="scan_train", lens="8x2048", channels=4096, ngroups=1, dstate=16,
             states="f32", init="none"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _some_lens(rng, most):
    if rng.random() < 0.4:
        n = _log_int(rng, 1, 8)
        return "%dx%d" % (n, _log_int(rng, 2, max(3, most // n)))
    n = _log_int(rng, 2, 40)
    return "ragged %d 1 %d %d" % (n, max(2, most // n), rng.randrange(1000))


def draw(rng):
    op = rng.choice(["norm", "norm_train", "conv", "conv_step", "conv_train", "scan", "scan", "scan", "scan_step",
                     "scan_train", "scan_train"])
    if op in ("norm", "norm_train"):
        width = rng.choice([8, 64, 200, 512, 1000, 2048, 2560, 4096, 5120, 8192, 16384])
        case = dict(op=op, rows=_log_int(rng, 1, 64_000_000 // max(width, 1000)), width=width,
                    residual=rng.choice(["none", "bf16", "f32"]))
        if op == "norm":
            case["out"] = rng.choice(["bf16", "e4m3"])
        return case
    init = rng.choice(["none", "half", "all"])
    if op.startswith("conv"):
        channels = rng.choice([8, 72, 256, 600, 1536, 2048, 2304, 4096, 8448, 10240])
        case = dict(op=op, channels=channels, width=rng.choice([2, 3, 4, 4, 4]),
                    stride=channels + 8 * rng.randrange(1, 500), init=init)
        if op == "conv_step":
            return dict(case, lens="%dx1" % _log_int(rng, 1, 600))
        most = (300_000_000 if op == "conv" else 60_000_000) // max(channels, 600)
        return dict(case, lens=_some_lens(rng, max(64, min(most, 60_000))))
    dstate = rng.choice([4, 8, 12, 16, 16, 16, 24, 32, 64])
    ngroups = rng.choice([1, 1, 1, 2, 4])
    channels = ngroups * rng.choice([8, 40, 96, 200, 512, 640, 1024, 2048, 2560])
    case = dict(op=op, channels=channels, ngroups=ngroups, dstate=dstate,
                states="f32" if op == "scan_train" else rng.choice(["f32", "bf16"]), init=init)
    if op == "scan_step":
        return dict(case, lens="%dx1" % _log_int(rng, 1, max(2, min(600, 30_000_000 // (channels * dstate)))))
    most = (2_000_000_000 if op == "scan" else 500_000_000) // (channels * dstate)
    return dict(case, lens=_some_lens(rng, max(64, min(most, 60_000))))


def _lens(case):
    """The sequence lengths a case names: "17", "4x4096", or "ragged n lo hi seed" (their logarithms spread evenly)."""
    text = case["lens"]
    if text.startswith("ragged"):
        n, lo, hi, seed = (int(w) for w in text.split()[1:])
        r = random.Random(seed)
        return [_log_int(r, lo, hi) for _ in range(n)]
    if "x" in text:
        n, length = (int(w) for w in text.split("x"))
        return [length] * n
    return [int(text)]


def _resumes(case, batch):
    return [case["init"] == "all" or (case["init"] == "half" and b % 2 == 0) for b in range(batch)]


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    op, f32 = case["op"], torch.float32
    s = dict(case=case)
    if op in ("norm", "norm_train"):
        T, D = case["rows"], case["width"]
        kind = f32 if case["residual"] == "f32" else torch.bfloat16
        s["weight"] = 1 + normal(D, std=0.2, dtype=f32)
        # rows of different size, with some channels larger than the rest
        size = torch.exp(0.5 * normal(T, 1, dtype=f32)) * torch.exp(0.5 * normal(D, dtype=f32))
        if op == "norm":
            s["x"] = (normal(T, D, dtype=f32) * size).bfloat16()
            s["residual"] = None if case["residual"] == "none" else (3 * normal(T, D, dtype=f32) * size).to(kind)
        else:
            s["r"] = (3 * normal(T, D, dtype=f32) * size).to(kind)
            s["d_y"] = normal(T, D)
            s["d_r"] = None if case["residual"] == "none" else normal(T, D, dtype=kind)
        return s

    lens = _lens(case)
    B, T, D = len(lens), sum(lens), case["channels"]
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    s["query_start_loc"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    resumes = torch.tensor(_resumes(case, B), dtype=torch.uint8, device="cuda")
    if op.startswith("conv"):
        W = case["width"]
        at = (case["stride"] - D) // 16 * 8
        s["x"] = normal(T, case["stride"])[:, at:at + D]
        s["weight"] = normal(D, W, std=W ** -0.5, dtype=f32)
        s["bias"] = normal(D, std=0.1, dtype=f32)
        shape, kind = (W - 1, D), torch.bfloat16
    else:
        G, N = case["ngroups"], case["dstate"]
        s["x"], s["dt"] = normal(T, D), normal(T, D, std=0.5)
        s["z"] = normal(T, 2 * D)[:, D:]  # the second half of the layer's projection
        rank = 2 * (-(-D // 32))  # the time step's rank ahead of B and C in theirs
        bc = normal(T, rank + 2 * G * N)
        s["B"] = bc[:, rank:rank + G * N].unflatten(1, (G, N))
        s["C"] = bc[:, rank + G * N:].unflatten(1, (G, N))
        # decays 1 .. N as such layers start with, moved apart by training; steps from 0.001 to 0.1
        s["A"] = -torch.arange(1, N + 1, device="cuda", dtype=f32) * torch.exp(0.3 * normal(D, N, dtype=f32))
        step = torch.exp(math.log(0.001) + uniform(D) * math.log(100))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["D"] = 1 + normal(D, std=0.1, dtype=f32)
        shape, kind = (D, N), f32 if case["states"] == "f32" else torch.bfloat16
    if op.endswith("train"):
        s["d_y"] = normal(T, D)
        given = case["init"] != "none"
        s["initial_states"] = normal(B, *shape, dtype=kind) if given else None
        s["d_final_states"] = normal(B, *shape, dtype=kind) if given else None
        return s
    slots = 2 * B
    s["pool"] = normal(slots, *shape, dtype=kind)
    s["cache_indices"] = torch.randperm(slots, generator=gen, device="cuda")[:B].to(torch.int32)
    s["has_initial_state"] = resumes
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_norm(s):
    from mamba_ssd_chunked_chunk_amd import binding
    x, residual = s["x"], s["residual"]
    r = None if residual is None else torch.empty_like(residual)
    if s["case"]["out"] == "bf16":
        y, scales = torch.empty_like(x), None
    else:
        y = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
        scales = torch.empty(x.shape[0], device=x.device)
    binding.ssd_rms_norm_fwd(y, scales, r, x, residual, s["weight"], eps=EPS)
    return tuple(t for t in (y, scales, r) if t is not None)


def _own_norm_train(s):
    from mamba_ssd_chunked_chunk_amd import binding
    r = s["r"]
    dx = torch.empty(r.shape, dtype=torch.bfloat16, device=r.device)
    d_residual = torch.empty_like(r) if r.dtype == torch.float32 else None
    dw = torch.empty_like(s["weight"])
    binding.ssd_rms_norm_bwd(dx, d_residual, dw, r, s["weight"], s["d_y"], s["d_r"], eps=EPS)
    return tuple(t for t in (dx, d_residual, dw) if t is not None)


def _own_conv(s):
    from mamba_ssd_chunked_chunk_amd import binding
    y = torch.empty(s["x"].shape, dtype=torch.bfloat16, device="cuda")
    binding.ssd_causal_conv_varlen_fwd_inplace(y, s["x"], s["weight"], s["bias"], s["pool"], s["query_start_loc"],
                                               s["has_initial_state"], s["cache_indices"], silu=True)
    return y, s["pool"]


def _own_conv_step(s):
    from mamba_ssd_chunked_chunk_amd import binding
    y = torch.empty(s["x"].shape, dtype=torch.bfloat16, device="cuda")
    binding.ssd_causal_conv_step_inplace(y, s["x"], s["weight"], s["bias"], s["pool"], s["has_initial_state"],
                                         s["cache_indices"], silu=True)
    return y, s["pool"]


def _own_conv_train(s):
    from mamba_ssd_chunked_chunk_amd import binding
    dx = torch.empty(s["x"].shape, dtype=torch.bfloat16, device="cuda")
    dw, db = torch.empty_like(s["weight"]), torch.empty_like(s["bias"])
    init = s["initial_states"]
    d_init = None if init is None else torch.empty_like(init)
    binding.ssd_causal_conv_varlen_bwd(dx, dw, db, d_init, s["x"], s["weight"], s["bias"], s["d_y"], init,
                                       s["d_final_states"], s["query_start_loc"], silu=True)
    return (dx, dw, db) if d_init is None else (dx, dw, db, d_init)


def _own_scan(s):
    from mamba_ssd_chunked_chunk_amd import binding
    y = torch.empty_like(s["x"])
    binding.ssd_selective_scan_varlen_fwd_inplace(y, s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"],
                                                  s["dt_bias"], s["pool"], s["query_start_loc"],
                                                  s["has_initial_state"], s["cache_indices"])
    return y, s["pool"]


def _own_scan_step(s):
    from mamba_ssd_chunked_chunk_amd import binding
    y = torch.empty_like(s["x"])
    binding.ssd_selective_scan_step_inplace(y, s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"],
                                            s["pool"], s["has_initial_state"], s["cache_indices"])
    return y, s["pool"]


def _own_scan_train(s):
    from mamba_ssd_chunked_chunk_amd import binding
    x, B = s["x"], s["B"]
    dx, ddt, dz = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    dB, dC = (torch.empty(B.shape, dtype=B.dtype, device=B.device) for _ in range(2))
    dA, dD, d_bias = torch.empty_like(s["A"]), torch.empty_like(s["D"]), torch.empty_like(s["dt_bias"])
    init = s["initial_states"]
    d_init = None if init is None else torch.empty_like(init)
    binding.ssd_selective_scan_varlen_bwd(dx, ddt, dA, dB, dC, dD, dz, d_bias, d_init, x, s["dt"], s["A"], B, s["C"],
                                          s["D"], s["z"], s["dt_bias"], s["d_y"], init, s["d_final_states"],
                                          s["query_start_loc"])
    r = dx, ddt, dA, dB, dC, dD, dz, d_bias
    return r if d_init is None else r + (d_init,)


_OWN = dict(norm=_own_norm, norm_train=_own_norm_train, conv=_own_conv, conv_step=_own_conv_step,
            conv_train=_own_conv_train, scan=_own_scan, scan_step=_own_scan_step, scan_train=_own_scan_train)


# ------------------------------------------------------------------ the plain form

def _silu(x):
    return x * torch.sigmoid(x)


def _silu_slope(x):
    p = torch.sigmoid(x)
    return p * (1 + x * (1 - p))


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _e4m3(y):
    """Codes (as values) and scales of the rows of y."""
    top = y.abs().amax(-1)
    low, power = torch.frexp(top / 448)  # top / 448 = low 2^power, low in [0.5, 1)
    power = torch.where(low == 0.5, power - 1, power).clamp(min=-126)
    scale = torch.where(top > 0, torch.ldexp(torch.ones_like(top), power), 0.0)
    quotient = y / torch.where(scale > 0, scale, 1.0)[:, None]
    _, e = torch.frexp(quotient)
    step = torch.ldexp(torch.ones_like(quotient), (e - 1).clamp(min=-6) - 3)
    return torch.round(quotient / step) * step, scale


def _plain_norm(s):
    x, residual = s["x"].float(), s["residual"]
    if residual is not None:
        kept = (x + residual.float()).to(residual.dtype)
        x = kept.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["weight"]
    if s["case"]["out"] == "bf16":
        out = (y.bfloat16(),)
    else:
        codes, scale = _e4m3(y)
        out = (codes.to(torch.float8_e4m3fn), scale)
    return out if residual is None else out + (kept,)


def _plain_norm_train(s):
    r, dy, w = s["r"].float(), s["d_y"].float(), s["weight"]
    scale = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
    unit, u = r * scale, dy * w
    dr = scale * (u - unit * (u * unit).mean(-1, keepdim=True))
    if s["d_r"] is not None:
        dr = dr + s["d_r"].float()
    dw = (dy * unit).sum(0)
    return (dr.bfloat16(), dw) if s["r"].dtype != torch.float32 else (dr.bfloat16(), dr, dw)


def _places(s):
    """Of every token: its sequence, and its place in it; and the sequences' lengths."""
    qsl = s["query_start_loc"].long()
    t = torch.arange(s["x"].shape[0], device=qsl.device)
    seq = torch.searchsorted(qsl, t, right=True) - 1
    return seq, t - qsl[seq], qsl[1:] - qsl[:-1]


def _earlier(x, history, seq, place, k):
    """The inputs k tokens before each token: of its own sequence, or of the history [batch, width - 1, channels]."""
    back = history.shape[1]
    t = torch.arange(x.shape[0], device=x.device)
    inside = (place >= k)[:, None]
    return torch.where(inside, x[(t - k).clamp(min=0)], history[seq, (back + place - k).clamp(0, max(back - 1, 0))])


def _history(s):
    """The inputs ahead of each sequence, in fp32, zero where none are given."""
    if "pool" in s:
        h = s["pool"][s["cache_indices"].long()].float()
        return torch.where(s["has_initial_state"].bool()[:, None, None], h, 0.0)
    if s["initial_states"] is not None:
        return s["initial_states"].float()
    B = s["query_start_loc"].numel() - 1
    return torch.zeros(B, s["case"]["width"] - 1, s["x"].shape[1], device=s["x"].device)


def _pre(x, history, seq, place, w, bias):
    W = w.shape[1]
    taps = [_earlier(x, history, seq, place, W - 1 - j) for j in range(W)]
    pre = bias.expand(x.shape)
    for j in range(W):
        pre = pre + w[:, j] * taps[j]
    return pre, taps


def _plain_conv(s):
    seq, place, n = _places(s)
    x, history = s["x"].float(), _history(s)
    pre, _ = _pre(x, history, seq, place, s["weight"], s["bias"])
    # the last width - 1 inputs: those of the sequence, and of the history where it is shorter
    back = history.shape[1]
    r = torch.arange(back, device=x.device)
    at = n[:, None] - back + r
    b = torch.arange(n.numel(), device=x.device)[:, None]
    first = s["query_start_loc"].long()[:-1, None]
    last = x[(first + at).clamp(0, x.shape[0] - 1)]
    last = torch.where((at >= 0)[..., None], last, history[b, (at + back).clamp(0, back - 1)])
    s["pool"][s["cache_indices"].long()] = last.to(s["pool"].dtype)
    return _silu(pre).bfloat16(), s["pool"]


def _plain_conv_step(s):
    x, slots = s["x"], s["cache_indices"].long()
    window = torch.cat([_history(s), x.float()[:, None]], 1)  # [batch, width, channels]
    pre = (window * s["weight"].t()).sum(1) + s["bias"]
    s["pool"][slots] = window[:, 1:].to(s["pool"].dtype)
    return _silu(pre).bfloat16(), s["pool"]


def _plain_conv_train(s):
    seq, place, n = _places(s)
    x, history, w = s["x"].float(), _history(s), s["weight"]
    T, W, back = x.shape[0], w.shape[1], history.shape[1]
    pre, taps = _pre(x, history, seq, place, w, s["bias"])
    d_pre = s["d_y"].float() * _silu_slope(pre)
    t = torch.arange(T, device=x.device)
    left = n[seq] - 1 - place  # tokens of the sequence behind this one
    dx = torch.zeros_like(x)
    d_history = torch.zeros_like(history)
    for k in range(W):
        behind = torch.where((left >= k)[:, None], d_pre[(t + k).clamp(max=T - 1)], 0.0)
        dx = dx + w[:, W - 1 - k] * behind
        for p in range(k):  # the history reaches the tokens 0 .. k - 1 with its tap k
            if s["initial_states"] is not None:
                first = s["query_start_loc"].long()[:-1] + p
                reach = torch.where((n > p)[:, None], d_pre[first.clamp(max=T - 1)], 0.0)
                d_history[:, back + p - k] += w[:, W - 1 - k] * reach
    dw = torch.stack([(d_pre * tap).sum(0) for tap in taps], 1)
    if s["initial_states"] is None:
        return dx.bfloat16(), dw, d_pre.sum(0)
    d_final = s["d_final_states"].float()
    row = (back - 1 - left).clamp(min=0)
    dx = dx + torch.where((left < back)[:, None], d_final[seq, row], 0.0)
    for r in range(back):  # rows of the final states that are still the history's
        short = (n <= back - 1 - r)
        m = (r + n).clamp(max=back - 1)
        b = torch.arange(n.numel(), device=x.device)
        d_history[b, m] += torch.where(short[:, None], d_final[:, r], 0.0)
    return dx.bfloat16(), dw, d_pre.sum(0), d_history.to(s["initial_states"].dtype)


def _chain(a, x, longest):
    """h_t = a_t h_{t-1} + x_t along the first dimension, by doubling: sums over 2, 4, 8, ... steps (a is 0 where a
    sequence of at most `longest` steps begins)."""
    reach = 1
    while reach < longest:
        y, b = x.clone(), a.clone()
        y[reach:].addcmul_(a[reach:], x[:-reach])
        b[reach:].mul_(a[:-reach])
        x, a, reach = y, b, 2 * reach
    return x


def _grouped(s):
    """x, the time steps and their raw values [T, G, D / G], A [G, D / G, N], B and C [T, G, 1, N], in fp32."""
    T, G, N = s["B"].shape
    x = s["x"].float().reshape(T, G, -1)
    raw = (s["dt"].float() + s["dt_bias"]).reshape(T, G, -1)
    return x, _softplus(raw), raw, s["A"].reshape(G, -1, N), s["B"].float()[:, :, None], s["C"].float()[:, :, None]


def _initial(s):
    """The states ahead of each sequence [batch, G, D / G, N] in fp32, or None."""
    G, N = s["B"].shape[1:]
    if "pool" in s:
        h = s["pool"][s["cache_indices"].long()].float()
        h = torch.where(s["has_initial_state"].bool()[:, None, None], h, 0.0)
    elif s["initial_states"] is not None:
        h = s["initial_states"].float()
    else:
        return None
    return h.reshape(h.shape[0], G, -1, N)


def _states(s, x, dts, A, B, initial):
    """The states behind every token, and the decays."""
    first = s["query_start_loc"].long()[:-1]
    longest = max(_lens(s["case"]))
    a = torch.exp(dts[..., None] * A)
    u = (dts * x)[..., None] * B
    if initial is not None:
        u[first] += a[first] * initial
    cut = a.clone()
    cut[first] = 0
    return _chain(cut, u, longest), a


def _plain_scan(s):
    x, dts, _, A, B, C = _grouped(s)
    h, _ = _states(s, x, dts, A, B, _initial(s))
    y = (h * C).sum(-1) + s["D"].reshape(x.shape[1:]) * x
    y = y.reshape(s["x"].shape) * _silu(s["z"].float())
    last = s["query_start_loc"].long()[1:] - 1
    s["pool"][s["cache_indices"].long()] = h[last].reshape(-1, *s["pool"].shape[1:]).to(s["pool"].dtype)
    return y.bfloat16(), s["pool"]


def _plain_scan_step(s):
    x, dts, _, A, B, C = _grouped(s)
    h = torch.exp(dts[..., None] * A) * _initial(s) + (dts * x)[..., None] * B
    y = (h * C).sum(-1) + s["D"].reshape(x.shape[1:]) * x
    s["pool"][s["cache_indices"].long()] = h.reshape(-1, *s["pool"].shape[1:]).to(s["pool"].dtype)
    return (y.reshape(s["x"].shape) * _silu(s["z"].float())).bfloat16(), s["pool"]


def _plain_scan_train(s):
    x, dts, raw, A, B, C = _grouped(s)
    T, D, skip = x.shape[0], s["x"].shape[1], s["D"].reshape(x.shape[1:])
    initial = _initial(s)
    h, a = _states(s, x, dts, A, B, initial)
    z, dy = (s[n].float().reshape(x.shape) for n in ("z", "d_y"))
    ys = (h * C).sum(-1) + skip * x
    dz = dy * ys * _silu_slope(z)
    dys = dy * _silu(z)
    dC = (dys[..., None] * h).sum(2)
    first, last = s["query_start_loc"].long()[:-1], s["query_start_loc"].long()[1:] - 1
    before = torch.cat([h[:1], h[:-1]])
    before[first] = 0 if initial is None else initial
    del h
    # the gradient of each token's state: from the last token of a sequence to its first
    u = dys[..., None] * C
    if s["d_final_states"] is not None:
        u[last] += s["d_final_states"].float().reshape(-1, *u.shape[1:])
    later = torch.cat([a[1:], a[:1]])
    later[last] = 0
    g = _chain(later.flip(0), u.flip(0), max(_lens(s["case"]))).flip(0)
    del u, later
    dB = (g * (dts * x)[..., None]).sum(2)
    gB = (g * B).sum(-1)
    d_init = None if initial is None else (a[first] * g[first]).reshape(-1, D, A.shape[-1])
    q = g * a * before
    del g, a, before
    d_dts = (q * A).sum(-1) + x * gB
    dA = (q * dts[..., None]).sum(0).reshape(D, -1)
    d_raw = d_dts * torch.sigmoid(raw)
    dx = dts * gB + skip * dys
    r = (dx, d_raw, dA, dB, dC, (dys * x).sum(0).reshape(D), dz, d_raw.sum(0).reshape(D))
    r = tuple(t.reshape(T, D).bfloat16() if t.dim() == 3 and i not in (2, 3, 4) else t for i, t in enumerate(r))
    r = r[:3] + (r[3].bfloat16(), r[4].bfloat16()) + r[5:]
    return r if d_init is None else r + (d_init.to(s["initial_states"].dtype),)


_PLAIN = dict(norm=_plain_norm, norm_train=_plain_norm_train, conv=_plain_conv, conv_step=_plain_conv_step,
              conv_train=_plain_conv_train, scan=_plain_scan, scan_step=_plain_scan_step, scan_train=_plain_scan_train)


# ------------------------------------------------------------------ in 64 bits, by the definition

#: the values of e4m3 that are not negative, in order
_E4M3 = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]


def _nearest_e4m3(x):
    """The nearest value of the format by search in its table; a tie goes to the even place."""
    table = torch.tensor(_E4M3, dtype=torch.float64, device=x.device)
    a = x.abs()
    hi = torch.searchsorted(table, a).clamp(max=len(_E4M3) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = table[hi] - a, a - table[lo]
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    return torch.where(take_hi, table[hi], table[lo]) * torch.sign(x)


def _exact_norm(s, case):
    r = s["x"].double() if case["op"] == "norm" else s["r"].double()
    w = s["weight"].double()
    kept = ()
    if case["op"] == "norm":
        if s["residual"] is not None:
            # the stream is held in its own type, and what is normed is what is held
            r = (r + s["residual"].double()).to(s["residual"].dtype).double()
            kept = (r,)
        y = r / torch.sqrt(r.square().mean(1, keepdim=True) + EPS) * w
        if case["out"] == "bf16":
            return (y,) + kept
        top = y.abs().amax(1)
        f = torch.exp2(torch.ceil(torch.log2(top / 448)))
        f = torch.where(top / f > 448, 2 * f, torch.where(2 * top / f <= 448, f / 2, f))
        return (_nearest_e4m3(y / f[:, None]), f) + kept
    dy = s["d_y"].double()
    m = r.square().mean(1, keepdim=True) + EPS
    # d/dr of sum_j dy_j w_j r_j m^(-1/2), with dm/dr = 2 r / width
    dr = dy * w / m.sqrt() - r * (dy * w * r).sum(1, keepdim=True) / (m ** 1.5 * r.shape[1])
    dr = dr if s["d_r"] is None else dr + s["d_r"].double()
    dw = (dy * r / m.sqrt()).sum(0)
    return (dr, dw) if s["r"].dtype != torch.float32 else (dr, dr, dw)


def _exact_conv(s, case):
    """Sequence by sequence, as one window of inputs that slides."""
    lens, W, w, bias = _lens(case), case["width"], s["weight"].double(), s["bias"].double()
    D, train = case["channels"], case["op"] == "conv_train"
    ys, states, at = [], [], 0
    dw, db = torch.zeros_like(w), torch.zeros_like(bias)
    for b, n in enumerate(lens):
        if train:
            ahead = s["initial_states"][b].double() if s["initial_states"] is not None else None
        else:
            ahead = s["pool"][int(s["cache_indices"][b])].double() if int(s["has_initial_state"][b]) else None
        if ahead is None:
            ahead = torch.zeros(W - 1, D, dtype=torch.float64, device=w.device)
        line = torch.cat([ahead, s["x"][at:at + n].double()])
        pre = (line.unfold(0, W, 1) * w).sum(-1) + bias
        p = 1 / (1 + torch.exp(-pre))
        if train:
            d_pre = s["d_y"][at:at + n].double() * (p + pre * p * (1 - p))
            d_line = torch.zeros_like(line)
            for j in range(W):
                d_line[j:j + n] += d_pre * w[:, j]
                dw[:, j] += (d_pre * line[j:j + n]).sum(0)
            db += d_pre.sum(0)
            if s["d_final_states"] is not None:
                d_line[n:] += s["d_final_states"][b].double()
            ys.append(d_line[W - 1:])
            states.append(d_line[:W - 1])
        else:
            ys.append(pre * p)
            states.append(line[n:])
        at += n
    if train:
        r = torch.cat(ys), dw, db
        return r if s["initial_states"] is None else r + (torch.stack(states),)
    pool = s["pool"].double()
    pool[s["cache_indices"].long()] = torch.stack(states)
    return torch.cat(ys), pool


def _padded(x, lens):
    """[T, ...] -> [longest, batch, ...] in fp64, zero behind each sequence."""
    out = torch.zeros(max(lens), len(lens), *x.shape[1:], dtype=torch.float64, device=x.device)
    at = 0
    for b, n in enumerate(lens):
        out[:n, b] = x[at:at + n].double()
        at += n
    return out


def _unpadded(x, lens):
    return torch.cat([x[:n, b] for b, n in enumerate(lens)])


def _exact_scan(s, case):
    lens, D, G, N = _lens(case), case["channels"], case["ngroups"], case["dstate"]
    A, skip, bias = (s[n].double() for n in ("A", "D", "dt_bias"))
    group = torch.arange(D, device=A.device) // (D // G)
    live = torch.arange(max(lens), device=A.device)[:, None] < torch.tensor(lens, device=A.device)
    x, raw, z = (_padded(s[n], lens) for n in ("x", "dt", "z"))
    raw = raw + bias
    dts = torch.logaddexp(raw, torch.zeros_like(raw)) * live[..., None]  # no step behind a sequence's end
    B, C = _padded(s["B"], lens), _padded(s["C"], lens)
    if case["op"] == "scan_train":
        h = s["initial_states"].double() if s["initial_states"] is not None else None
    else:
        h = s["pool"][s["cache_indices"].long()].double() * s["has_initial_state"].double()[:, None, None]
    if h is None:
        h = torch.zeros(len(lens), D, N, dtype=torch.float64, device=A.device)
    sig = 1 / (1 + torch.exp(-z))
    train = case["op"] == "scan_train"
    y = torch.empty_like(x)
    kept = [h]
    for t in range(max(lens)):
        h = torch.exp(dts[t][..., None] * A) * h + (dts[t] * x[t])[..., None] * B[t][:, group]
        y[t] = (h * C[t][:, group]).sum(-1)
        if train:
            kept.append(h)
    y = y + skip * x
    if not train:
        pool = s["pool"].double()
        pool[s["cache_indices"].long()] = h
        return _unpadded(y * z * sig, lens), pool
    dy = _padded(s["d_y"], lens)
    dz = dy * y * (sig + z * sig * (1 - sig))
    dy = dy * z * sig
    g = s["d_final_states"].double() if s["d_final_states"] is not None else torch.zeros_like(h)
    dx, ddt, dB, dC, dA = torch.empty_like(x), torch.empty_like(x), torch.empty_like(B), torch.empty_like(C), 0
    for t in reversed(range(max(lens))):
        g = g + dy[t][..., None] * C[t][:, group]
        dC[t] = (dy[t][..., None] * kept[t + 1]).unflatten(1, (G, -1)).sum(2)
        dB[t] = (g * (dts[t] * x[t])[..., None]).unflatten(1, (G, -1)).sum(2)
        into = (g * B[t][:, group]).sum(-1)
        g = g * torch.exp(dts[t][..., None] * A)
        pull = g * kept[t]
        dA = dA + (pull * dts[t][..., None]).sum(0)
        dx[t] = dts[t] * into + skip * dy[t]
        ddt[t] = (pull * A).sum(-1) + x[t] * into
    ddt = ddt * live[..., None] / (1 + torch.exp(-raw))
    r = (_unpadded(dx, lens), _unpadded(ddt, lens), dA, _unpadded(dB, lens), _unpadded(dC, lens),
         (dy * x).sum((0, 1)), _unpadded(dz, lens), ddt.sum((0, 1)))
    return r if s["initial_states"] is None else r + (g,)


def exact(case, seed):
    if case["op"].startswith("scan"):
        lens = _lens(case)
        state = len(lens) * case["channels"] * case["dstate"] * 8
        train = case["op"] == "scan_train"
        # a token of the loop costs about 100 us, or its states' bytes where those take longer
        if max(lens) * max(1.5e-4, 8 * state / 3e12) * (3 if train else 1) > 20 or train and max(lens) * state > 6e10:
            return None
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(s, case)
    return _exact_conv(s, case) if case["op"].startswith("conv") else _exact_scan(s, case)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op.startswith("norm"):
        n = case["rows"] * case["width"]
        e = dict(none=0, bf16=2, f32=4)[case["residual"]]
        if op == "norm":  # x and the residual in, the output and the residual out
            return dict(bytes=n * (2 + 2 * e + (2 if case["out"] == "bf16" else 1)) + 4 * case["width"], flops=5 * n)
        # r, dy and the residual's gradient in; dx (and its fp32 form) out
        return dict(bytes=n * ((e or 2) + 2 + e + 2 + (4 if e == 4 else 0)) + 8 * case["width"], flops=11 * n)
    lens = _lens(case)
    B, T, D = len(lens), sum(lens), case["channels"]
    moved = sum(_resumes(case, B)) + B
    if op.startswith("conv"):
        W = case["width"]
        rows = 2 * (W - 1) * D
        if op == "conv_train":
            return dict(bytes=6 * T * D + (3 * B * rows if case["init"] != "none" else 0) + 8 * D * (W + 1),
                        flops=T * D * (6 * W + 8))
        return dict(bytes=4 * T * D + moved * rows + 4 * D * (W + 1), flops=T * D * (2 * W + 4))
    G, N = case["ngroups"], case["dstate"]
    state = D * N * (4 if case["states"] == "f32" else 2)
    weights = 4 * D * (N + 2)
    if op == "scan_train":
        # x, dt, z, dy, B, C in; dx, ddt, dz, dB, dC out; the states and their gradients
        return dict(bytes=14 * T * D + 8 * T * G * N + (3 * B * state if case["init"] != "none" else 0) + 2 * weights,
                    flops=T * D * (22 * N + 30))
    return dict(bytes=8 * T * D + 4 * T * G * N + moved * state + weights, flops=T * D * (7 * N + 14))
