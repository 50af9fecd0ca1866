"""The operators of the linear-attention family, as they are measured.

Five operators over one kind of state, a pool [slots, nheads, value_dim, key_dim]:

``prefill``  linear attention with a fixed decay per head over a ragged batch of
             prompts, in its chunked form, with the pool updated in place;
``step``     its recurrent form for one token per sequence;
``train``    its backward pass (dq, dk, dv and the gradient of the initial states);
``park``     states quantised to 8 bits as they leave the pool, then read back
             into other slots (a preempted sequence that resumes);
``restore``  states read back from the 8-bit cache alone (a prefix that is hit).

Head h uses q and k of group g = h // (nheads / ngroups) and decays with
lambda = exp(log_decay[h]):

    S_t = lambda S_{t-1} + v_t k_t^T          o_t = scale S_t q_t

A row (slot, head, value channel) of a state is quantised with one fp32 scale:
int8 codes, scale = absmax / 127 rounded to fp32 (rows whose scale would fall
below the smallest normal number are stored as zeros), code = x / scale to the
nearest integer, ties to even; or e4m3 codes with the least power of two that
brings absmax / scale to 448 or less.

``run`` computes these with elementary torch operations in fp32 unless ``own``
is true; ``exact`` computes them token by token in fp64.
"""

import math
import random

import torch

own = False

CHUNK = 64  # tokens of a block in the plain form
TINY = 1.1754943508222875e-38  # smallest normal fp32 number


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a few tokens of prompt at low load: latency of one call
        dict(name="prefill_17", op="prefill", lens="17", nheads=4, ngroups=4, key_dim=64, value_dim=64,
             states="f32", init="none"),
        # ragged prompts of a busy server, some resuming, grouped q and k (32 sequences, 128 heads in 8 groups)
        dict(name="prefill_ragged_32", op="prefill", lens="ragged 32 17 8192 3", nheads=128, ngroups=8, key_dim=128,
             value_dim=64, states="bf16", init="half"),
        # one long document: few rows, the work lies along the sequence
        dict(name="prefill_65536", op="prefill", lens="65536", nheads=16, ngroups=16, key_dim=128, value_dim=128,
             states="f32", init="all"),
        # one request of a decode loop: latency
        dict(name="step_1", op="step", lens="1", nheads=16, ngroups=16, key_dim=128, value_dim=128, states="f32",
             init="all"),
        # a full decode batch, 512 sequences of 128 heads over a 1024-slot pool
        dict(name="step_512", op="step", lens="512x1", nheads=128, ngroups=8, key_dim=128, value_dim=64, states="f32",
             init="all"),
        # a fine-tuning step on two short samples
        dict(name="train_2x100", op="train", lens="2x100", nheads=4, ngroups=2, key_dim=64, value_dim=64, states="f32",
             init="all"),
        # a training batch of fixed length
        dict(name="train_4x4096", op="train", lens="4x4096", nheads=16, ngroups=16, key_dim=128, value_dim=128,
             states="f32", init="none"),
        # packed documents of odd lengths, grouped heads of uneven width
        dict(name="train_packed_12", op="train", lens="ragged 12 33 5000 5", nheads=12, ngroups=4, key_dim=96,
             value_dim=200, states="f32", init="all"),
        # one preempted sequence (16 heads x 64 x 256), out and back
        dict(name="park_1", op="park", slots=1, nheads=16, key_dim=256, value_dim=64, states="f32", codes="e4m3"),
        # 64 preempted sequences of 128 heads
        dict(name="park_64", op="park", slots=64, nheads=128, key_dim=128, value_dim=64, states="f32", codes="i8"),
        # prefix hits of a small batch
        dict(name="restore_3", op="restore", slots=3, nheads=16, key_dim=128, value_dim=128, states="bf16",
             codes="i8"),
        # prefix hits of a large batch
        dict(name="restore_256", op="restore", slots=256, nheads=64, key_dim=128, value_dim=128, states="f32",
             codes="e4m3"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "step", "train", "train", "park", "restore"])
    key_dim = rng.choice([32, 48, 64, 72, 96, 128, 128, 192, 256])
    value_dim = rng.choice([32, 64, 64, 88, 128, 128, 160, 256])
    ngroups = rng.choice([1, 2, 3, 4, 8, 16])
    nheads = ngroups * rng.choice([1, 1, 2, 4, 5])
    states = rng.choice(["f32", "bf16"])
    init = rng.choice(["none", "half", "all"])
    if op in ("park", "restore"):
        slots = _log_int(rng, 1, max(2, 60_000_000 // (nheads * key_dim * value_dim)))
        return dict(op=op, slots=min(slots, 400), nheads=nheads, key_dim=key_dim, value_dim=value_dim, states=states,
                    codes=rng.choice(["i8", "e4m3"]))
    if op == "step":
        batch = _log_int(rng, 1, max(2, min(600, 400_000_000 // (nheads * key_dim * value_dim))))
        return dict(op=op, lens="%dx1" % batch, nheads=nheads, ngroups=ngroups, key_dim=key_dim, value_dim=value_dim,
                    states=states, init=init)
    most = max(64, (40_000_000 if op == "prefill" else 20_000_000) // (nheads * max(key_dim, value_dim)))
    most = min(most, 30_000)
    if rng.random() < 0.4:
        n = _log_int(rng, 1, 8)
        lens = "%dx%d" % (n, _log_int(rng, 5, max(6, most // n)))
    else:
        n = _log_int(rng, 2, 40)
        lens = "ragged %d 1 %d %d" % (n, max(2, most // n), rng.randrange(1000))
    return dict(op=op, lens=lens, nheads=nheads, ngroups=ngroups, key_dim=key_dim, value_dim=value_dim,
                states="f32" if op == "train" else states, init=init)


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

    H, K, V = case["nheads"], case["key_dim"], case["value_dim"]
    kind = torch.float32 if case["states"] == "f32" else torch.bfloat16
    if case["op"] in ("park", "restore"):
        n = case["slots"]
        # state rows of different sizes, as heads of different decay leave them
        size = torch.exp(torch.randn(2 * n, H, V, 1, generator=gen, device="cuda"))
        pool = (torch.randn(2 * n, H, V, K, generator=gen, device="cuda") * size).to(kind)
        perm = torch.randperm(2 * n, generator=gen, device="cuda").to(torch.int32)
        where = torch.randperm(n, generator=gen, device="cuda").to(torch.int32)
        s = dict(case=case, pool=pool, out_of=perm[:n].clone(), into=perm[n:].clone(), where=where)
        scales = torch.zeros(n, H, V, device="cuda")
        if case["codes"] == "i8":
            codes = torch.zeros(n, H, V, K, dtype=torch.int8, device="cuda")
        else:
            codes = torch.zeros(n, H, V, K, dtype=torch.float8_e4m3fn, device="cuda")
        if case["op"] == "restore":  # the cache is full: codes and scales of what was parked before
            c, f = _quantized(torch.randn(n, H, V, K, generator=gen, device="cuda") * size[:n], case["codes"])
            codes.copy_(c.to(codes.dtype))
            scales.copy_(f)
        s.update(codes=codes, scales=scales)
        return s

    lens = _lens(case)
    B, T, G = len(lens), sum(lens), case["ngroups"]
    # the slopes of such layers: a geometric series from about 0.7 down to 2^-8
    log_decay = -torch.exp2(-8.0 * (torch.arange(H, device="cuda", dtype=torch.float32) + 0.5) / H)
    s = dict(case=case, log_decay=log_decay, scale=K ** -0.5,
             q=normal(T, G, K), k=normal(T, G, K), v=normal(T, H, V))
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    s["query_start_loc"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    resumes = torch.tensor(_resumes(case, B), dtype=torch.uint8, device="cuda")
    if case["op"] == "train":
        s["d_o"] = normal(T, H, V)
        s["initial_states"] = normal(B, H, V, K, dtype=torch.float32) if case["init"] != "none" else None
        s["d_final_states"] = normal(B, H, V, K, dtype=torch.float32) if case["init"] != "none" else None
        return s
    slots = 2 * B
    s["pool"] = normal(slots, H, V, K, dtype=kind)
    s["cache_indices"] = torch.randperm(slots, generator=gen, device="cuda")[:B].to(torch.int32)
    s["has_initial_state"] = resumes
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_prefill(s):
    from mamba_ssd_chunked_chunk_amd import binding
    o = torch.empty_like(s["v"])
    binding.ssd_linear_attn_varlen_fwd_inplace(o, s["q"], s["k"], s["v"], s["log_decay"], s["pool"],
                                               s["query_start_loc"], s["has_initial_state"], s["cache_indices"],
                                               scale=s["scale"])
    return o, s["pool"]


def _own_step(s):
    from mamba_ssd_chunked_chunk_amd import binding
    o = torch.empty_like(s["v"])
    binding.ssd_linear_attn_step_inplace(o, s["q"], s["k"], s["v"], s["log_decay"], s["pool"],
                                         s["has_initial_state"], s["cache_indices"], scale=s["scale"])
    return o, s["pool"]


def _own_train(s):
    from mamba_ssd_chunked_chunk_amd import binding
    dq, dk, dv = torch.empty_like(s["q"]), torch.empty_like(s["k"]), torch.empty_like(s["v"])
    init = s["initial_states"]
    d_init = torch.empty_like(init) if init is not None else None
    binding.ssd_linear_attn_varlen_bwd(dq, dk, dv, d_init, s["q"], s["k"], s["v"], s["d_o"], s["log_decay"], init,
                                       s["d_final_states"], s["query_start_loc"], scale=s["scale"])
    return (dq, dk, dv) if d_init is None else (dq, dk, dv, d_init)


def _own_park(s):
    from mamba_ssd_chunked_chunk_amd import binding
    binding.ssd_state_quantize(s["codes"], s["scales"], s["pool"], s["out_of"], s["where"])
    binding.ssd_state_dequantize(s["pool"], s["codes"], s["scales"], s["into"], s["where"])
    return s["pool"]


def _own_restore(s):
    from mamba_ssd_chunked_chunk_amd import binding
    binding.ssd_state_dequantize(s["pool"], s["codes"], s["scales"], s["into"], s["where"])
    return s["pool"]


_OWN = dict(prefill=_own_prefill, step=_own_step, train=_own_train, park=_own_park, restore=_own_restore)


# ------------------------------------------------------------------ the plain form

def _blocks(s):
    """The sequences cut into blocks of CHUNK tokens: sequence, first token and length of each, and the tokens'
    places (clamped) with a mask of the true ones."""
    qsl = s["query_start_loc"].long()
    T, B = s["q"].shape[0], qsl.numel() - 1
    count = (qsl[1:] - qsl[:-1] + CHUNK - 1) // CHUNK
    ends = torch.cumsum(count, 0)
    c = torch.arange(T // CHUNK + B, device=qsl.device)
    seq = torch.searchsorted(ends, c, right=True).clamp(max=B - 1)
    first = qsl[seq] + (c - (ends - count)[seq]) * CHUNK
    length = (qsl[seq + 1] - first).clamp(0, CHUNK)
    row = torch.arange(CHUNK, device=qsl.device)
    at = (first[:, None] + row).clamp(max=max(T - 1, 0))
    true = row < length[:, None]
    return seq, first, length, at, true


def _cut(x, at, true, heads):
    """[T, n, D] -> [blocks, heads, CHUNK, D] in fp32, zero past a block's end, each of the n repeated for its heads."""
    x = (x[at].float() * true[:, :, None, None]).transpose(1, 2)
    return x.repeat_interleave(heads // x.shape[1], 1)


def _decay(log_decay, distance):
    """exp(log_decay[h] * distance), 0 where the distance is negative: [h, *distance.shape], the exponents in fp64."""
    d = distance.double()
    e = torch.exp(log_decay.double().reshape([-1] + [1] * d.dim()) * d.clamp(min=0))
    return (e * (d >= 0)).float()


def _mix(weights, x):
    """[h, m, blocks] x [blocks, h, V, K] -> [m, h, V, K]"""
    n, h, V, K = x.shape
    y = torch.matmul(weights, x.transpose(0, 1).reshape(h, n, V * K))
    return y.reshape(h, -1, V, K).transpose(0, 1)


def _back(x, at, true, like):
    """[blocks, heads, CHUNK, D] -> the shape [T, n, D] of `like`, summed over the heads that share one of the n."""
    x = x.transpose(1, 2)[true]
    T, n, D = like.shape
    out = torch.empty_like(like)
    out[at[true]] = x.reshape(-1, n, x.shape[1] // n, D).sum(2).to(like.dtype)
    return out


def _chain(s, left, right, first, length, seq, initial):
    """The states that enter each block, and those that leave each sequence, from the blocks' own right-weighted
    products (left: the value side, right: the key side, both [blocks, heads, CHUNK, .])."""
    qsl, ld = s["query_start_loc"].long(), s["log_decay"]
    row = torch.arange(CHUNK, device=qsl.device)
    weight = _decay(ld, length[:, None] - 1 - row).transpose(0, 1)  # [blocks, h, CHUNK]
    own_part = torch.matmul((left * weight[..., None]).transpose(2, 3), right)  # [blocks, h, V, K]
    ends = first + length
    same = seq[:, None] == seq[None, :]
    gap = torch.where(same, first[:, None] - ends[None, :], -1)
    gap = torch.where((length[None, :] > 0) & (length[:, None] > 0), gap, -1)
    into = _mix(_decay(ld, gap), own_part)
    b = torch.arange(qsl.numel() - 1, device=qsl.device)
    tail = torch.where((seq[None, :] == b[:, None]) & (length[None, :] > 0), qsl[1:][:, None] - ends[None, :], -1)
    final = _mix(_decay(ld, tail), own_part)
    if initial is not None:
        into = into + _decay(ld, first - qsl[seq]).transpose(0, 1)[:, :, None, None] * initial[seq]
        final = final + _decay(ld, qsl[1:] - qsl[:-1]).transpose(0, 1)[:, :, None, None] * initial
    return into, final


def _plain_prefill(s):
    seq, first, length, at, true = _blocks(s)
    H = s["v"].shape[1]
    q, k, v = (_cut(s[n], at, true, H) for n in "qkv")
    slots = s["cache_indices"].long()
    resumes = s["has_initial_state"].bool()
    initial = torch.where(resumes[:, None, None, None], s["pool"][slots].float(), 0.0)
    into, final = _chain(s, v, k, first, length, seq, initial)
    row = torch.arange(CHUNK, device=q.device)
    scores = torch.matmul(q, k.transpose(2, 3)) * _decay(s["log_decay"], row[:, None] - row[None, :])
    o = torch.matmul(scores, v)
    o = o + torch.matmul(q, into.transpose(2, 3)) * _decay(s["log_decay"], row + 1)[:, :, None]
    s["pool"][slots] = final.to(s["pool"].dtype)
    return _back(o * s["scale"], at, true, s["v"]), s["pool"]


def _plain_step(s):
    H = s["v"].shape[1]
    q, k = (s[n].float().repeat_interleave(H // s[n].shape[1], 1) for n in "qk")
    slots = s["cache_indices"].long()
    resumes = s["has_initial_state"].bool()
    S = torch.where(resumes[:, None, None, None], s["pool"][slots].float(), 0.0)
    S = S * torch.exp(s["log_decay"])[:, None, None] + s["v"].float()[..., None] * k[:, :, None, :]
    o = (S * q[:, :, None, :]).sum(-1) * s["scale"]
    s["pool"][slots] = S.to(s["pool"].dtype)
    return o.to(s["v"].dtype), s["pool"]


def _plain_train(s):
    seq, first, length, at, true = _blocks(s)
    H, scale, ld = s["v"].shape[1], s["scale"], s["log_decay"]
    q, k, v, g = (_cut(s[n], at, true, H) for n in ("q", "k", "v", "d_o"))
    g = g * scale
    row = torch.arange(CHUNK, device=q.device)
    into, _ = _chain(s, v, k, first, length, seq, s["initial_states"])
    within = _decay(ld, row[:, None] - row[None, :])
    scores = torch.matmul(q, k.transpose(2, 3)) * within
    pull = torch.matmul(g, v.transpose(2, 3)) * within
    dq = torch.matmul(pull, k) + torch.matmul(g, into) * _decay(ld, row + 1)[:, :, None]
    # the gradient of the state that leaves each block, from the blocks behind it and the final states' gradient
    qsl, ends = s["query_start_loc"].long(), first + length
    part = torch.matmul((g * _decay(ld, row)[:, :, None]).transpose(2, 3), q)
    live = (length[:, None] > 0) & (length[None, :] > 0) & (seq[:, None] == seq[None, :])
    gap = torch.where(live, first[None, :] - ends[:, None], -1)
    # a token i of a later block reaches the state behind this one over first + i + 1 - end decays, one of them
    # the state's own step
    out = _mix(_decay(ld, torch.where(gap >= 0, gap + 1, -1)), part)
    b = torch.arange(qsl.numel() - 1, device=q.device)
    head = torch.where((seq[None, :] == b[:, None]) & (length[None, :] > 0), first[None, :] - qsl[:-1][:, None], -1)
    d_init = _mix(_decay(ld, torch.where(head >= 0, head + 1, -1)), part)
    if s["d_final_states"] is not None:
        d = s["d_final_states"]
        out = out + _decay(ld, qsl[seq + 1] - ends).transpose(0, 1)[:, :, None, None] * d[seq]
        d_init = d_init + _decay(ld, qsl[1:] - qsl[:-1]).transpose(0, 1)[:, :, None, None] * d
    reach = _decay(ld, length[:, None] - 1 - row).transpose(0, 1)[..., None]
    dk = torch.matmul(pull.transpose(2, 3), q) + torch.matmul(v, out) * reach
    dv = torch.matmul(scores.transpose(2, 3), g) + torch.matmul(k, out.transpose(2, 3)) * reach
    r = _back(dq, at, true, s["q"]), _back(dk, at, true, s["k"]), _back(dv, at, true, s["v"])
    return r if s["initial_states"] is None else r + (d_init,)


def _quantized(x, codes):
    """Codes (as fp64 values) and fp32 scales of the rows of x."""
    top = x.abs().amax(-1).double()
    if codes == "i8":
        scale = (top / 127).float()
        scale = torch.where(scale < TINY, 0.0, scale)
        quotient = x.double() / torch.where(scale > 0, scale, 1.0).double()[..., None]
        return torch.round(quotient) * (scale > 0)[..., None], scale
    low, power = torch.frexp(top / 448)  # top / 448 = low 2^power, low in [0.5, 1)
    power = torch.where(low == 0.5, power - 1, power).clamp(min=-126)
    scale = torch.where(top > 0, torch.ldexp(torch.ones_like(top), power), 0.0)
    quotient = x.double() / torch.where(scale > 0, scale, 1.0)[..., None]
    _, e = torch.frexp(quotient)
    step = torch.ldexp(torch.ones_like(quotient), (e - 1).clamp(min=-6) - 3)
    return torch.round(quotient / step) * step * (scale > 0)[..., None], scale.float()


def _plain_park(s):
    c, f = _quantized(s["pool"][s["out_of"].long()].float(), s["case"]["codes"])
    where = s["where"].long()
    s["codes"][where] = c.to(s["codes"].dtype)
    s["scales"][where] = f
    return _plain_restore(s)


def _plain_restore(s):
    where = s["where"].long()
    x = s["codes"][where].float() * s["scales"][where][..., None]
    s["pool"][s["into"].long()] = x.to(s["pool"].dtype)
    return s["pool"]


_PLAIN = dict(prefill=_plain_prefill, step=_plain_step, train=_plain_train, park=_plain_park, restore=_plain_restore)


# ------------------------------------------------------------------ in 64 bits, by the definition

def _padded(x, lens):
    """[T, n, D] -> [longest, batch, n, D] in fp64, zero behind each sequence."""
    out = torch.zeros(max(lens), len(lens), *x.shape[1:], dtype=torch.float64, device=x.device)
    at = 0
    for b, length in enumerate(lens):
        out[:length, b] = x[at:at + length].double()
        at += length
    return out


def _unpadded(x, lens):
    return torch.cat([x[:length, b] for b, length in enumerate(lens)])


def _exact_states(s, case):
    lens = _lens(case)
    H, G, scale = case["nheads"], case["ngroups"], s["scale"]
    q, k, v = (_padded(s[n], lens) for n in "qkv")
    lam = torch.exp(s["log_decay"].double())[:, None, None]
    n = torch.tensor(lens, device=q.device)

    def heads(x):  # [batch, groups, D] -> [batch, heads, D]
        return x.repeat_interleave(H // G, 1)

    def groups(x):  # the sum over a group's heads
        return x.reshape(x.shape[0], G, H // G, -1).sum(2)

    def step(t, S):  # sequences that have ended keep their state
        live = (t < n).double()[:, None, None, None]
        return S * (live * lam + (1 - live)) + v[t][..., None] * heads(k[t])[:, :, None, :]

    if case["op"] != "train":
        slots = s["cache_indices"].long()
        S = s["pool"][slots].double() * s["has_initial_state"].double()[:, None, None, None]
        o = torch.empty_like(v)
        for t in range(max(lens)):
            S = step(t, S)
            o[t] = scale * torch.matmul(S, heads(q[t])[..., None])[..., 0]
        pool = s["pool"].double()
        pool[slots] = S
        return _unpadded(o, lens), pool

    g = _padded(s["d_o"], lens) * scale
    shape = (len(lens), H, case["value_dim"], case["key_dim"])
    zero = torch.zeros(shape, dtype=torch.float64, device=q.device)
    S = s["initial_states"].double() if s["initial_states"] is not None else zero
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for t in range(max(lens)):
        S = step(t, S)
        dq[t] = groups((S * g[t][..., None]).sum(2))
    R = s["d_final_states"].double() if s["d_final_states"] is not None else zero
    for t in reversed(range(max(lens))):
        R = R + g[t][..., None] * heads(q[t])[:, :, None, :]
        dk[t] = groups((R * v[t][..., None]).sum(2))
        dv[t] = (R * heads(k[t])[:, :, None, :]).sum(3)
        live = (t < n).double()[:, None, None, None]
        R = R * (live * lam + (1 - live))
    r = _unpadded(dq, lens), _unpadded(dk, lens), _unpadded(dv, lens)
    return r if s["initial_states"] is None else r + (R,)


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


def _exact_cache(s, case):
    pool = s["pool"].double()
    where = s["where"].long()
    if case["op"] == "restore":
        pool[s["into"].long()] = s["codes"][where].double() * s["scales"][where].double()[..., None]
        return pool
    x = pool[s["out_of"].long()]
    top = x.abs().amax(-1, keepdim=True)
    if case["codes"] == "i8":
        f = (top / 127).float().double()  # the scale is kept in fp32
        y = torch.round(x / f) * f
    else:
        f = torch.exp2(torch.ceil(torch.log2(top / 448)))
        f = torch.where(top / f > 448, 2 * f, torch.where(2 * top / f <= 448, f / 2, f))
        y = _nearest_e4m3(x / f) * f
    pool[s["into"].long()] = torch.where(top > 0, y, 0.0)
    return pool


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("park", "restore"):
        return _exact_cache(s, case)
    lens = _lens(case)
    # a token of the loop costs about 50 us, or its states' bytes where those take longer
    each = len(lens) * case["nheads"] * case["key_dim"] * case["value_dim"] * 8 * 8 / 2e12
    if max(lens) * max(1e-4, each) * (2 if case["op"] == "train" else 1) > 20:
        return None
    return _exact_states(s, case)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    H, K, V = case["nheads"], case["key_dim"], case["value_dim"]
    es = 4 if case["states"] == "f32" else 2
    if case["op"] in ("park", "restore"):
        rows = case["slots"] * H * V
        one = rows * (K * (es + 1) + 4) + 8 * case["slots"]
        return dict(bytes=one * (2 if case["op"] == "park" else 1), flops=2 * rows * K)
    lens = _lens(case)
    B, T, G = len(lens), sum(lens), case["ngroups"]
    token = 2 * (2 * G * K + 2 * H * V)
    state = H * V * K * es
    if case["op"] == "train":
        # q, k, v, d_o in; dq, dk, dv out; initial states and the final ones' gradient in, the initial ones' out
        return dict(bytes=T * (token + 2 * (2 * G * K + H * V)) + (3 * B * state if case["init"] != "none" else 0),
                    flops=10 * T * H * K * V)
    moved = sum(_resumes(case, B)) + B
    return dict(bytes=T * token + moved * state, flops=4 * T * H * K * V)
