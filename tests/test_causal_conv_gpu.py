"""The short causal convolution on the GPU: prompts, single tokens and the
backward pass against the definition in 64 bits, within bounds counted from the
roundings (layer_testlib), and the ways of calling them."""

import pytest

torch = pytest.importorskip("torch")
import layer_testlib as L  # noqa: E402
from mamba_ssd_chunked_chunk_amd import binding  # noqa: E402

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def draw(lens, D, W, seed, *, tail=0, slots=0):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens) + tail
    d = dict(x=torch.randn(T, D, generator=g).bfloat16(), d_y=torch.randn(T, D, generator=g).bfloat16(),
             weight=torch.randn(D, W, generator=g) * W ** -0.5, bias=0.3 * torch.randn(D, generator=g),
             initial=torch.randn(len(lens), W - 1, D, generator=g).bfloat16(),
             d_final=torch.randn(len(lens), W - 1, D, generator=g).bfloat16(), query_start_loc=L.starts_of(lens))
    if slots:
        d["pool"] = torch.randn(slots, W - 1, D, generator=g).bfloat16()
        d["cache_indices"] = torch.randperm(slots, generator=g)[:len(lens)].to(torch.int32)
    return d


def cuda(d):
    return {k: v.cuda() for k, v in d.items()}


def check_prompt(lens, D, W, seed, init="half", tail=0, silu=True, bias=True):
    d = draw(lens, D, W, seed, tail=tail, slots=len(lens) + 2)
    c = cuda(d)
    flags = torch.tensor([init == "all" or (init == "half" and b % 2 == 0) for b in range(len(lens))],
                         dtype=torch.uint8)
    # a slot that no flag marks is not read: NaN there stays out
    slots = d["cache_indices"].long()
    before = d["pool"].clone()
    before[slots[flags == 0]] = float("nan")
    pool = before.cuda()
    y = torch.full_like(c["x"], 7.0)
    b = d["bias"] if bias else None
    binding.ssd_causal_conv_varlen_fwd_inplace(y, c["x"], c["weight"], c["bias"] if bias else None, pool,
                                               c["query_start_loc"], flags.cuda() if init != "none" else None,
                                               c["cache_indices"], silu=silu)
    initial = torch.where(flags.bool()[:, None, None], before[slots], torch.zeros((), dtype=BF16))
    want, final, size = L.conv(d["x"], d["weight"], b, lens, initial, silu)
    T = sum(lens)
    assert L.worst(y[:T], want, size * L.CONV, L.BF16) <= 1
    assert bool((y[T:] == 7.0).all())  # rows behind the last sequence
    after = pool.cpu()
    assert torch.equal(after[slots], final.bfloat16())  # the inputs themselves
    rest = [s for s in range(len(lens) + 2) if s not in slots.tolist()]
    assert torch.equal(after[rest], before[rest])


@pytest.mark.parametrize("D", [8, 72, 504, 512, 520, 1536])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_prompt_sizes(D, W):
    check_prompt([70, 1, 0, 133], D, W, D + W)


@pytest.mark.parametrize("n", [0, 1, 2, 3, 4, 7, 8, 9, 31, 32, 33, 34, 35, 63, 64, 65, 200])
def test_prompt_lengths(n):
    check_prompt([n], 64, 4, 100 + n, init="all")
    check_prompt([n, 3, n], 64, 3, 130 + n, init="none", tail=2)


@pytest.mark.parametrize("init", ["none", "half", "all"])
@pytest.mark.parametrize("silu,bias", [(True, False), (False, True), (False, False)])
def test_prompt_forms(init, silu, bias):
    check_prompt([40, 0, 2, 65], 136, 4, 200, init=init, tail=9, silu=silu, bias=bias)


@pytest.mark.parametrize("n", [63, 64, 65, 700, 5000])
def test_prompt_many_sequences(n):
    lens = [int(x) for x in torch.randint(0, 5, (n,), generator=torch.Generator().manual_seed(n))]
    lens[n // 2] = 150
    check_prompt(lens, 8, 4, 300 + n, tail=1)


def test_no_tokens_at_all():
    check_prompt([0, 0, 0], 64, 4, 310)


def test_padding_entries():
    d = draw([40, 37, 5], 72, 4, 320, slots=4)
    c = cuda(d)
    c["cache_indices"][1] = -1
    pool, y = c["pool"].clone(), torch.full_like(c["x"], 7.0)
    binding.ssd_causal_conv_varlen_fwd_inplace(y, c["x"], c["weight"], c["bias"], pool, c["query_start_loc"], None,
                                               c["cache_indices"])
    want, final, size = L.conv(d["x"], d["weight"], d["bias"], [40, 37, 5], None, True)
    keep = torch.ones(82, dtype=torch.bool)
    keep[40:77] = False
    assert L.worst(y.cpu()[keep], want[keep], size[keep] * L.CONV, L.BF16) <= 1
    assert bool((y.cpu()[~keep] == 7.0).all())
    slots = d["cache_indices"].long()[[0, 2]]
    assert torch.equal(pool.cpu()[slots], final[[0, 2]].bfloat16())
    rest = [s for s in range(4) if s not in slots.tolist()]
    assert torch.equal(pool.cpu()[rest], d["pool"][rest])


def test_nan_reaches_the_next_tokens_of_its_channel_only():
    d = draw([50, 30], 64, 4, 330, slots=2)
    d["x"][20, 3], d["x"][49, 5] = float("nan"), float("nan")
    c = cuda(d)
    y = torch.empty_like(c["x"])
    binding.ssd_causal_conv_varlen_fwd_inplace(y, c["x"], c["weight"], c["bias"], c["pool"], c["query_start_loc"],
                                               None, c["cache_indices"])
    bad = torch.zeros(80, 64, dtype=torch.bool)
    bad[20:24, 3] = True
    bad[49, 5] = True
    assert torch.equal(torch.isnan(y.cpu()), bad)


def test_wrong_tables_stay_inside():
    """Boundaries are clamped to the rows there are, whatever the table says."""
    for table in ([0, 500, 40], [-7, 3, 1000000], [30, 20, 10], [0, 0, -5]):
        d = draw([20, 20], 64, 4, 335, slots=2)
        c = cuda(d)
        qsl = torch.tensor(table, dtype=torch.int32, device="cuda")
        guard = torch.full((42, 64), 7.0, dtype=BF16, device="cuda")
        binding.ssd_causal_conv_varlen_fwd_inplace(guard[1:41], c["x"], c["weight"], c["bias"], c["pool"], qsl, None,
                                                   c["cache_indices"])
        torch.cuda.synchronize()
        assert bool((guard[[0, 41]] == 7.0).all())


def test_slices_of_one_projection():
    d = draw([50, 0, 33], 136, 4, 340)
    c = cuda(d)
    wide = torch.randn(83, 300 * 2, device="cuda").bfloat16()
    wide[:, 16:152] = c["x"]
    y0, y1 = torch.empty_like(c["x"]), torch.empty_like(c["x"])
    f0, f1 = torch.empty_like(c["initial"]), torch.empty_like(c["initial"])
    for x, y, f in ((c["x"], y0, f0), (wide[:, 16:152], y1, f1)):
        binding.ssd_causal_conv_varlen_fwd(y, x, c["weight"], c["bias"], c["initial"], f, c["query_start_loc"])
    assert torch.equal(y0, y1) and torch.equal(f0, f1)
    want, final, size = L.conv(d["x"], d["weight"], d["bias"], [50, 0, 33], d["initial"], True)
    assert L.worst(y0, want, size * L.CONV, L.BF16) <= 1 and torch.equal(f0.cpu(), final.bfloat16())
    same = c["initial"].clone()  # initial and final states in one buffer
    binding.ssd_causal_conv_varlen_fwd(y1, c["x"], c["weight"], c["bias"], same, same, c["query_start_loc"])
    assert torch.equal(y0, y1) and torch.equal(f0, same)
    a, b = [torch.empty_like(t) for t in (c["x"], c["weight"], c["bias"], c["initial"])], []
    b = [torch.empty_like(t) for t in a]
    for x, g in ((c["x"], a), (wide[:, 16:152], b)):
        binding.ssd_causal_conv_varlen_bwd(*g, x, c["weight"], c["bias"], c["d_y"], c["initial"], c["d_final"],
                                           c["query_start_loc"])
    assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_slots_behind_2_31_elements():
    D, slots = 8192, (1 << 31) // (3 * 8192) + 4
    d = draw([40], D, 4, 350)
    c = cuda(d)
    pool = torch.zeros(slots, 3, D, dtype=BF16, device="cuda")
    last = slots - 1
    pool[last] = c["initial"][0]
    idx = torch.tensor([last], dtype=torch.int32, device="cuda")
    one = torch.ones(1, dtype=torch.uint8, device="cuda")
    y = torch.empty_like(c["x"])
    binding.ssd_causal_conv_varlen_fwd_inplace(y, c["x"], c["weight"], c["bias"], pool, c["query_start_loc"], one, idx)
    want, final, size = L.conv(d["x"], d["weight"], d["bias"], [40], d["initial"], True)
    assert L.worst(y, want, size * L.CONV, L.BF16) <= 1 and torch.equal(pool[last].cpu(), final[0].bfloat16())
    binding.ssd_causal_conv_step_inplace(y[:1], c["x"][:1], c["weight"], c["bias"], pool, one, idx)
    want, after, size = L.conv(d["x"][:1], d["weight"], d["bias"], [1], final.bfloat16(), True)
    assert L.worst(y[:1], want, size * L.CONV, L.BF16) <= 1 and torch.equal(pool[last].cpu(), after[0].bfloat16())


def test_tokens_behind_2_31_elements():
    D, n = 4096, (1 << 31) // 4096 + 100
    x = torch.empty(n, D, dtype=BF16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(2))
    d = draw([1], D, 4, 360)
    c = cuda(d)
    y, f = torch.empty_like(x), torch.empty(1, 3, D, dtype=BF16, device="cuda")
    qsl = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    binding.ssd_causal_conv_varlen_fwd(y, x, c["weight"], c["bias"], None, f, qsl)
    for at in (n // 2, n - 40):
        want, final, size = L.conv(x[at:at + 40].cpu(), d["weight"], d["bias"], [40], x[None, at - 3:at].cpu(), True)
        assert L.worst(y[at:at + 40], want, size * L.CONV, L.BF16) <= 1
    assert torch.equal(f.cpu(), final.bfloat16())


# ------------------------------------------------------------------ single tokens

@pytest.mark.parametrize("B,D,W", [(1, 8, 4), (3, 72, 2), (17, 520, 3), (130, 1536, 4), (2, 10240, 4)])
@pytest.mark.parametrize("silu", [True, False])
def test_step(B, D, W, silu):
    d = draw([1] * B, D, W, 400 + B, slots=B + 2)
    c = cuda(d)
    flags = (torch.arange(B) % 3 != 1).to(torch.uint8)
    slots = d["cache_indices"].long()
    before = d["pool"].clone()
    before[slots[flags == 0]] = float("nan")
    pool = before.cuda()
    wide = torch.zeros(B, D + 8, dtype=BF16, device="cuda")
    wide[:, 8:] = c["x"]
    y = torch.empty_like(c["x"])
    binding.ssd_causal_conv_step_inplace(y, wide[:, 8:], c["weight"], c["bias"], pool, flags.cuda(),
                                         c["cache_indices"], silu=silu)
    initial = torch.where(flags.bool()[:, None, None], before[slots], torch.zeros((), dtype=BF16))
    want, final, size = L.conv(d["x"], d["weight"], d["bias"], [1] * B, initial, silu)
    assert L.worst(y, want, size * L.CONV, L.BF16) <= 1
    assert torch.equal(pool.cpu()[slots], final.bfloat16())
    rest = [s for s in range(B + 2) if s not in slots.tolist()]
    assert torch.equal(pool.cpu()[rest], before[rest])


def test_step_padding_and_no_flags():
    d = draw([1] * 4, 64, 4, 420, slots=5)
    c = cuda(d)
    c["cache_indices"][2] = 5
    pool, y = c["pool"].clone(), torch.full_like(c["x"], 7.0)
    binding.ssd_causal_conv_step_inplace(y, c["x"], c["weight"], None, pool, None, c["cache_indices"])
    want, final, size = L.conv(d["x"], d["weight"], None, [1] * 4, None, True)
    live = [0, 1, 3]
    assert L.worst(y[live], want[live], size[live] * L.CONV, L.BF16) <= 1 and bool((y[2] == 7.0).all())
    slots = d["cache_indices"].long()
    assert torch.equal(pool.cpu()[slots[live]], final[live].bfloat16())
    rest = [s for s in range(5) if s not in slots[live].tolist()]
    assert torch.equal(pool.cpu()[rest], d["pool"][rest])


def test_steps_continue_a_prompt():
    """A prompt and its next tokens one by one give what the whole gives, bit for bit (the same sums)."""
    d = draw([30], 72, 4, 430, slots=1)
    c = cuda(d)
    f = torch.empty(1, 3, 72, dtype=BF16, device="cuda")
    whole = torch.empty_like(c["x"])
    binding.ssd_causal_conv_varlen_fwd(whole, c["x"], c["weight"], c["bias"], None, f, c["query_start_loc"])
    y, one = torch.empty_like(whole), torch.ones(1, dtype=torch.uint8, device="cuda")
    binding.ssd_causal_conv_varlen_fwd_inplace(y[:22], c["x"][:22], c["weight"], c["bias"], c["pool"],
                                               torch.tensor([0, 22], dtype=torch.int32, device="cuda"), None,
                                               c["cache_indices"])
    for t in range(22, 30):
        binding.ssd_causal_conv_step_inplace(y[t:t + 1], c["x"][t:t + 1], c["weight"], c["bias"], c["pool"], one,
                                             c["cache_indices"])
    assert torch.equal(y, whole) and torch.equal(c["pool"], f)


# ------------------------------------------------------------------ backward

def check_backward(lens, D, W, seed, initial=True, final=True, tail=0, silu=True, bias=True):
    d = draw(lens, D, W, seed, tail=tail)
    c = cuda(d)
    dx = torch.full_like(c["x"], 7.0)
    dw, db = torch.full_like(c["weight"], 7.0), torch.full_like(c["bias"], 7.0)
    d_init = torch.full_like(c["initial"], 7.0)
    binding.ssd_causal_conv_varlen_bwd(dx, dw, db if bias else None, d_init, c["x"], c["weight"],
                                       c["bias"] if bias else None, c["d_y"], c["initial"] if initial else None,
                                       c["d_final"] if final else None, c["query_start_loc"], silu=silu)
    want = L.conv_gradients(d["x"], d["weight"], d["bias"] if bias else None, lens,
                            d["initial"] if initial else None, d["d_y"], d["d_final"] if final else None, silu)
    T = sum(lens)
    assert L.worst(dx[:T], *want[0], L.BF16) <= 1 and bool((dx[T:] == 7.0).all())
    assert L.worst(dw, *want[1], L.U) <= 1
    assert not bias or L.worst(db, *want[2], L.U) <= 1
    assert L.worst(d_init, *want[3], L.BF16) <= 1


@pytest.mark.parametrize("D", [8, 72, 512, 520, 1536])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_backward_sizes(D, W):
    check_backward([70, 1, 0, 133], D, W, 500 + D + W)


@pytest.mark.parametrize("n", [0, 1, 2, 3, 4, 7, 8, 9, 29, 30, 31, 32, 33, 34, 35, 64, 65, 200])
def test_backward_lengths(n):
    check_backward([n], 64, 4, 600 + n)
    check_backward([n, 3, n], 64, 3, 640 + n, tail=2)


@pytest.mark.parametrize("initial,final", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("silu,bias", [(True, True), (True, False), (False, True), (False, False)])
def test_backward_forms(initial, final, silu, bias):
    check_backward([40, 0, 2, 65], 136, 4, 700, initial, final, tail=9, silu=silu, bias=bias)


def test_backward_many_sequences():
    lens = [int(x) for x in torch.randint(0, 40, (300,), generator=torch.Generator().manual_seed(6))]
    check_backward(lens, 24, 4, 710, tail=3)


def test_backward_against_differences():
    """The gradients predict how the forward kernel's sum(y dy) changes along a direction of weights and bias, where
    the step is not rounded away; y's own roundings bound the rest."""
    lens, h = [40, 25], 2.0 ** -5
    d = draw(lens, 64, 4, 720)
    c = cuda(d)
    g = torch.Generator().manual_seed(721)
    way = [torch.randn(t.shape, generator=g) for t in (d["weight"], d["bias"])]
    dx, dw, db = (torch.empty_like(c[n]) for n in ("x", "weight", "bias"))
    binding.ssd_causal_conv_varlen_bwd(dx, dw, db, None, c["x"], c["weight"], c["bias"], c["d_y"], None, None,
                                       c["query_start_loc"])
    predicted = sum(float((a.cpu().double() * b.double()).sum()) for a, b in zip((dw, db), way))
    dy, sums, exact, size = d["d_y"].double(), [], [], 0.0
    for s in (h, -h):
        w, b = d["weight"] + s * way[0], d["bias"] + s * way[1]
        y, f = torch.empty_like(c["x"]), torch.empty_like(c["initial"])
        binding.ssd_causal_conv_varlen_fwd(y, c["x"], w.cuda(), b.cuda(), None, f, c["query_start_loc"])
        sums.append(float((y.cpu().double() * dy).sum()))
        size += float((y.cpu().double() * dy).abs().sum())
        exact.append(float((L.conv(d["x"], w, b, lens, None, True)[0] * dy).sum()))
    assert abs((sums[0] - sums[1]) - (exact[0] - exact[1])) <= size * L.BF16
    assert abs((exact[0] - exact[1]) / (2 * h) - predicted) <= 0.02 * abs(predicted) + 0.5


# ------------------------------------------------------------------ ways of calling

def test_refusals():
    c = cuda(draw([5, 4], 64, 4, 800, slots=3))
    y = torch.empty_like(c["x"])

    def f(y=y, x=c["x"], weight=c["weight"], bias=c["bias"], pool=c["pool"], qsl=c["query_start_loc"], flags=None,
          idx=c["cache_indices"]):
        binding.ssd_causal_conv_varlen_fwd_inplace(y, x, weight, bias, pool, qsl, flags, idx)

    f()
    for kw, error, text in [(dict(x=c["x"].float()), TypeError, "x"), (dict(y=y[:5]), ValueError, "y"),
                            (dict(weight=c["weight"].bfloat16()), TypeError, "weight"),
                            (dict(weight=c["weight"][:, :3]), ValueError, "weight"),
                            (dict(weight=c["weight"][0]), ValueError, "weight"),
                            (dict(bias=c["bias"][:32]), ValueError, "bias"),
                            (dict(pool=c["pool"].float()), TypeError, "pool"),
                            (dict(pool=c["pool"][:, :2]), ValueError, "pool"),
                            (dict(qsl=c["query_start_loc"].long()), TypeError, "query_start_loc"),
                            (dict(idx=c["cache_indices"][:1]), ValueError, "cache_indices"),
                            (dict(idx=c["cache_indices"].long()), TypeError, "cache_indices"),
                            (dict(flags=torch.ones(3, dtype=torch.uint8, device="cuda")), ValueError, "has_initial"),
                            (dict(y=y.cpu()), ValueError, "y is on")]:
        with pytest.raises(error, match=text):
            f(**kw)
    with pytest.raises(binding.SsdError) as e:
        wide = torch.zeros(64, 5, device="cuda")
        f(weight=wide, pool=torch.zeros(3, 4, 64, dtype=BF16, device="cuda"))
    assert e.value.status == 3


def test_streams_and_graphs():
    lens = [100, 0, 33, 270]
    c = cuda(draw(lens, 136, 4, 810, slots=6))
    ones = torch.ones(4, dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(c[n]) for n in ("x", "x", "weight", "bias", "initial", "pool")] + [torch.empty_like(c["x"][:4])]

    def all_calls(stream=None):
        y, dx, dw, db, di, pool, ys = outs
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            pool.copy_(c["pool"])
        binding.ssd_causal_conv_varlen_fwd_inplace(y, c["x"], c["weight"], c["bias"], pool, c["query_start_loc"], ones,
                                                   c["cache_indices"], stream=stream)
        binding.ssd_causal_conv_step_inplace(ys, c["x"][:4], c["weight"], c["bias"], pool, ones, c["cache_indices"],
                                             stream=stream)
        binding.ssd_causal_conv_varlen_bwd(dx, dw, db, di, c["x"], c["weight"], c["bias"], c["d_y"], c["initial"],
                                           c["d_final"], c["query_start_loc"], stream=stream)

    all_calls()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    for t in outs:
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    all_calls(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        all_calls()
    for _ in range(4):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        all_calls()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("use", ["both", "y", "final", "sum"])
def test_autograd(use):
    """Gradients reach a projection whose slice x is, weights, bias and initial states; rows behind the last sequence
    get zeros."""
    from mamba_ssd_chunked_chunk_amd.mixer import causal_conv
    lens, D, tail = [90, 0, 2, 65], 72, 5
    d = draw(lens, D, 4, 820, tail=tail)
    c = cuda(d)
    T = sum(lens)
    wide = torch.cat([torch.zeros(T + tail, 16, dtype=BF16, device="cuda"), c["x"]], 1).requires_grad_()
    leaves = [wide] + [c[n].clone().requires_grad_() for n in ("weight", "bias", "initial")]
    y, final = causal_conv(wide[:, 16:], leaves[1], leaves[2], c["query_start_loc"], leaves[3], padded=True)
    assert bool((y[T:] == 0).all())
    dy, df = d["d_y"], d["d_final"]
    if use == "sum":
        y[:T].float().sum().backward()
        dy, df = torch.ones_like(dy), None
    else:
        given = dict(both=([y, final], [c["d_y"], c["d_final"]]), y=([y], [c["d_y"]]), final=([final], [c["d_final"]]))
        torch.autograd.backward(*given[use])
        dy, df = (torch.zeros_like(dy) if use == "final" else dy), (None if use == "y" else df)
    want = L.conv_gradients(d["x"], d["weight"], d["bias"], lens, d["initial"], dy, df, True)
    assert L.worst(leaves[0].grad[:T, 16:], *want[0], L.BF16) <= 1 and bool((leaves[0].grad[T:] == 0).all())
    for leaf, w, e in zip(leaves[1:], want[1:], (L.U, L.U, L.BF16)):
        assert L.worst(leaf.grad, *w, e) <= 1
