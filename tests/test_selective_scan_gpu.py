"""The selective scan on the GPU: prompts, single tokens and the backward pass
against the recurrence in 64 bits, within bounds counted from the roundings
(layer_testlib), and the ways of calling them."""

import pytest

torch = pytest.importorskip("torch")
import layer_testlib as L  # noqa: E402
from mamba_ssd_chunked_chunk_amd import binding  # noqa: E402

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
NAMES = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")


def cuda(d):
    return {k: v.cuda() for k, v in d.items()}


def rounding(dtype):
    return torch.finfo(dtype).eps / 2


def inputs(c, use=L.ALL):
    return [c[n] if n in use or n not in L.ALL else None for n in NAMES]


def check_prompt(lens, D, G, N, seed, dtype=F32, init="half", tail=0, softplus=True, use=L.ALL, decay=1.0):
    d = L.scan_inputs(lens, D, G, N, seed, slots=len(lens) + 2, tail=tail, decay=decay)
    if not softplus:
        d["dt"], d["dt_bias"] = d["dt"].abs(), d["dt_bias"].abs() * 0.1
    c = cuda(d)
    flags = torch.tensor([init == "all" or (init == "half" and b % 2 == 0) for b in range(len(lens))],
                         dtype=torch.uint8)
    slots = d["cache_indices"].long()
    before = d["pool"].to(dtype)
    before[slots[flags == 0]] = float("nan")  # not read
    pool = before.cuda()
    y = torch.full_like(c["x"], 7.0)
    binding.ssd_selective_scan_varlen_fwd_inplace(y, *inputs(c, use), pool, c["query_start_loc"],
                                                  flags.cuda() if init != "none" else None, c["cache_indices"],
                                                  dt_softplus=softplus)
    initial = torch.where(flags.bool()[:, None, None], before[slots].float(), 0.0)
    want, by, final, bf = L.scan(d, lens, initial, softplus, use)
    T = sum(lens)
    assert L.worst(y[:T], want, by, L.BF16) <= 1
    assert bool((y[T:] == 7.0).all())  # rows behind the last sequence
    after = pool.cpu()
    assert L.worst(after[slots], final, bf, rounding(dtype)) <= 1
    rest = [s for s in range(len(lens) + 2) if s not in slots.tolist()]
    assert torch.equal(after[rest], before[rest])


@pytest.mark.parametrize("N", [4, 8, 12, 16, 20, 24, 28, 32, 36, 48, 64])
@pytest.mark.parametrize("D,G", [(8, 1), (200, 1), (144, 2)])
def test_prompt_sizes(D, G, N):
    check_prompt([35, 1, 0, 50], D, G, N, D + N)


@pytest.mark.parametrize("D,G", [(64, 1), (72, 1), (128, 4), (24, 3), (520, 5)])
def test_prompt_groups(D, G):
    check_prompt([17, 40], D, G, 16, 200 + D)


@pytest.mark.parametrize("n", [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 100])
def test_prompt_lengths(n):
    check_prompt([n], 72, 1, 16, 300 + n, init="all")
    check_prompt([n, 3, n], 8, 1, 8, 330 + n, init="none", tail=2)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("init", ["none", "half", "all"])
def test_prompt_states(dtype, init):
    check_prompt([40, 0, 64, 0, 1], 72, 1, 16, 400, dtype=dtype, init=init, tail=9)


@pytest.mark.parametrize("use", [(), ("D",), ("z",), ("dt_bias",), ("z", "D")])
@pytest.mark.parametrize("softplus", [True, False])
def test_prompt_forms(use, softplus):
    check_prompt([40, 33], 72, 1, 16, 410, softplus=softplus, use=use)


@pytest.mark.parametrize("n", [63, 64, 65, 700, 5000])
def test_prompt_many_sequences(n):
    lens = [int(x) for x in torch.randint(0, 4, (n,), generator=torch.Generator().manual_seed(n))]
    check_prompt(lens, 8, 1, 4, 500 + n, tail=1)


@pytest.mark.parametrize("lens", [[255], [256], [257], [271, 300], [512], [513], [5, 600, 0, 1500, 256, 257], [2100]])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompt_long(lens, dtype):
    """Sequences that are cut into segments, among others that are not, in place."""
    check_prompt(lens, 72, 1, 16, 600 + sum(lens), dtype=dtype, init="all", tail=3)
    check_prompt(lens, 16, 2, 8, 601 + sum(lens), dtype=dtype, init="half", decay=0.01)


def lens_of_many(n, seed):
    """Ragged prompts of 128 tokens and more on average, whole and cut ones of every class of length, some empty."""
    lens = [int(x) for x in torch.randint(0, 260, (n,), generator=torch.Generator().manual_seed(seed))]
    for i, long in enumerate((1500, 700, 391, 385, 384, 383, 0, 0, 1, 1100)):
        lens[i * (n // 10) + (3 if i % 2 else 0)] = long
    return lens


@pytest.mark.parametrize("n", [64, 65, 130, 256])
def test_prompt_many_long_sequences(n):
    lens = lens_of_many(n, 60 + n)
    assert sum(lens) // n >= 128
    check_prompt(lens, 8, 1, 8, 560 + n)


def test_prompt_cut_among_many():
    lens = [int(x) for x in torch.randint(0, 30, (200,), generator=torch.Generator().manual_seed(3))]
    lens[0], lens[100], lens[199] = 700, 1100, 513
    check_prompt(lens, 8, 1, 8, 700, init="half", tail=2)


def test_decays():
    """Almost none, very strong ones (the state is the token alone), and none at all."""
    for decay in (1e-6, 1e4, 0.0):
        check_prompt([90, 300], 16, 1, 16, 710, decay=decay, init="all")


def test_growing_states():
    d = L.scan_inputs([60], 16, 1, 16, 720, decay=-0.05)
    c = cuda(d)
    y, f = torch.empty_like(c["x"]), torch.empty(1, 16, 16, device="cuda")
    binding.ssd_selective_scan_varlen_fwd(y, *inputs(c), c["initial"], f, c["query_start_loc"])
    want, by, final, bf = L.scan(d, [60], d["initial"])
    # a growing power's exponent x counts |x| instead of |x| e^-|x|: sums of them here
    dts = torch.logaddexp(d["dt"].double() + d["dt_bias"].double(), torch.zeros(60, 16, dtype=torch.float64))
    grow = 1 + 4 * float((dts.sum(0)[:, None] * d["A"].double()).max())
    assert L.worst(y, want, by * grow, L.BF16) <= 1 and L.worst(f, final, bf * grow, L.U) <= 1


def test_steps_of_every_size():
    """Time steps from 2^-40 to 80: softplus keeps its relative accuracy at both ends."""
    d = L.scan_inputs([64], 64, 1, 4, 730)
    d["dt"] = torch.linspace(-28, 80, 64)[:, None].expand(64, 64).bfloat16().contiguous()
    d["dt_bias"].zero_()
    d["A"].fill_(-1e-3)
    c = cuda(d)
    y, f = torch.empty_like(c["x"]), torch.empty(1, 64, 4, device="cuda")
    binding.ssd_selective_scan_varlen_fwd(y, *inputs(c, ()), None, f, c["query_start_loc"])
    want, by, final, bf = L.scan(d, [64], None, use=())
    assert L.worst(y, want, by, L.BF16) <= 1 and L.worst(f, final, bf, L.U) <= 1


def test_padding_entries():
    lens = [40, 300, 5]
    d = L.scan_inputs(lens, 72, 1, 16, 740, slots=4)
    c = cuda(d)
    c["cache_indices"][1] = -1
    pool, y = c["pool"].clone(), torch.full_like(c["x"], 7.0)
    binding.ssd_selective_scan_varlen_fwd_inplace(y, *inputs(c), pool, c["query_start_loc"], None, c["cache_indices"])
    want, by, final, bf = L.scan(d, lens)
    keep = torch.ones(345, dtype=torch.bool)
    keep[40:340] = False
    assert L.worst(y.cpu()[keep], want[keep], by[keep], L.BF16) <= 1
    assert bool((y.cpu()[~keep] == 7.0).all())
    slots = d["cache_indices"].long()[[0, 2]]
    assert L.worst(pool.cpu()[slots], final[[0, 2]], bf[[0, 2]], L.U) <= 1
    rest = [s for s in range(4) if s not in slots.tolist()]
    assert torch.equal(pool.cpu()[rest], d["pool"][rest])


def test_nan_stays_in_its_sequence_and_channel():
    lens = [300, 40]
    d = L.scan_inputs(lens, 72, 1, 16, 750, slots=2)
    d["x"][270, 3], d["dt"][20, 5] = float("nan"), float("nan")
    c = cuda(d)
    y = torch.empty_like(c["x"])
    binding.ssd_selective_scan_varlen_fwd_inplace(y, *inputs(c), c["pool"], c["query_start_loc"], None,
                                                  c["cache_indices"])
    bad = torch.zeros(340, 72, dtype=torch.bool)
    bad[270:300, 3] = True
    bad[20:300, 5] = True
    assert torch.equal(torch.isnan(y.cpu()), bad)


def test_wrong_tables_stay_inside():
    """Boundaries are clamped to the rows there are, whatever the table says."""
    for table in ([0, 900, 300], [-7, 3, 1000000], [30, 20, 10], [0, 0, -5], [600, 0, 600]):
        d = L.scan_inputs([300, 300], 64, 1, 16, 755, slots=2)
        c = cuda(d)
        qsl = torch.tensor(table, dtype=torch.int32, device="cuda")
        guard = torch.full((602, 64), 7.0, dtype=BF16, device="cuda")
        binding.ssd_selective_scan_varlen_fwd_inplace(guard[1:601], *inputs(c), c["pool"], qsl, None,
                                                      c["cache_indices"])
        torch.cuda.synchronize()
        assert bool((guard[[0, 601]] == 7.0).all())


def test_slices_of_projections_and_separate_states():
    lens, D, N = [50, 0, 333], 136, 16
    d = L.scan_inputs(lens, D, 1, N, 760)
    c, T = cuda(d), sum(lens)
    xz = torch.cat([c["x"], c["z"]], 1)
    bc = torch.cat([torch.zeros(T, 10, dtype=BF16, device="cuda"), c["B"].view(T, N), c["C"].view(T, N)], 1)
    sliced = dict(c, x=xz[:, :D], z=xz[:, D:], B=bc[:, 10:10 + N].unflatten(1, (1, N)),
                  C=bc[:, 10 + N:].unflatten(1, (1, N)))
    assert sliced["B"].data_ptr() % 8 == 4
    outs = []
    for s in (c, sliced):
        y, f = torch.empty_like(c["x"]), torch.empty_like(c["initial"])
        binding.ssd_selective_scan_varlen_fwd(y, *inputs(s), c["initial"], f, c["query_start_loc"])
        outs.append((y, f))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    want, by, final, bf = L.scan(d, lens, d["initial"])
    assert L.worst(outs[0][0], want, by, L.BF16) <= 1 and L.worst(outs[0][1], final, bf, L.U) <= 1
    same = c["initial"].clone()  # initial and final states in one buffer, a cut sequence among them
    y = torch.empty_like(c["x"])
    binding.ssd_selective_scan_varlen_fwd(y, *inputs(c), same, same, c["query_start_loc"])
    assert torch.equal(y, outs[0][0]) and torch.equal(same, outs[0][1])
    pool, ones = c["initial"].clone(), torch.ones(3, dtype=torch.bool, device="cuda")
    binding.ssd_selective_scan_varlen_fwd_inplace(y, *inputs(c), pool, c["query_start_loc"], ones,
                                                  torch.arange(3, dtype=torch.int32, device="cuda"))
    assert torch.equal(y, outs[0][0]) and torch.equal(pool, outs[0][1])
    a, b = gradients(c, c["initial"], c["d_final"]), gradients(sliced, c["initial"], c["d_final"])
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_slots_behind_2_31_elements():
    D, N = 4096, 16
    slots = (1 << 31) // (D * N) + 4
    d = L.scan_inputs([40], D, 1, N, 770)
    c = cuda(d)
    pool = torch.zeros(slots, D, N, dtype=BF16, device="cuda")
    pool[slots - 1] = c["initial"][0].bfloat16()
    idx, one = torch.tensor([slots - 1], dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.uint8,
                                                                                      device="cuda")
    y = torch.empty_like(c["x"])
    binding.ssd_selective_scan_varlen_fwd_inplace(y, *inputs(c), pool, c["query_start_loc"], one, idx)
    want, by, final, bf = L.scan(d, [40], d["initial"].bfloat16().float())
    assert L.worst(y, want, by, L.BF16) <= 1 and L.worst(pool[-1:], final, bf, L.BF16) <= 1
    before = pool[-1:].float().cpu()
    first = {k: c[k][:1] if k in ("x", "dt", "B", "C", "z") else c[k] for k in NAMES}
    binding.ssd_selective_scan_step_inplace(y[:1], *inputs(first), pool, one, idx)
    want, by, final, bf = L.scan(d, [1], before)
    assert L.worst(y[:1], want, by, L.BF16) <= 1 and L.worst(pool[-1:], final, bf, L.BF16) <= 1


def test_tokens_behind_2_31_elements():
    """Rows past 2^31 elements, cut into segments: the last of two sequences is compared."""
    D, n = 8192, (1 << 31) // 8192 + 50
    gen = torch.Generator("cuda").manual_seed(4)
    d = L.scan_inputs([60], D, 1, 4, 780)
    c = cuda(d)
    big = {k: torch.empty(n + 60, *c[k].shape[1:], dtype=BF16, device="cuda").normal_(generator=gen)
           for k in ("x", "dt", "B", "C", "z")}
    for k, t in big.items():
        t[n:] = c[k]
    s = dict(c, **big)
    y, f = torch.empty_like(big["x"]), torch.empty(2, D, 4, device="cuda")
    qsl = torch.tensor([0, n, n + 60], dtype=torch.int32, device="cuda")
    initial = torch.cat([c["initial"], c["initial"]])
    binding.ssd_selective_scan_varlen_fwd(y, *inputs(s), initial, f, qsl)
    want, by, final, bf = L.scan(d, [60], d["initial"])
    assert L.worst(y[n:], want, by, L.BF16) <= 1 and L.worst(f[1:], final, bf, L.U) <= 1
    # the last 60 tokens of the long one, from the state that 2000 tokens ahead of them leave (older ones have
    # decayed by more than 2^-24 or not, so only what follows is compared: a second call from the state in the middle)
    m = n - 60
    g = torch.empty(2, D, 4, device="cuda")
    part = {k: t[:m] for k, t in big.items()}
    binding.ssd_selective_scan_varlen_fwd(y[:m].clone(), *inputs(dict(c, **part)), c["initial"], g[:1],
                                          torch.tensor([0, m], dtype=torch.int32, device="cuda"))
    e = {k: v.cpu() for k, v in s.items() if k in NAMES}
    e.update({k: big[k][m:n].cpu() for k in big})
    e["d_y"] = d["d_y"]
    want, by, final, bf = L.scan(e, [60], g[:1].cpu())
    assert L.worst(y[m:n], want, 2 * by, L.BF16) <= 1


# ------------------------------------------------------------------ single tokens

@pytest.mark.parametrize("N", [4, 8, 12, 16, 20, 24, 28, 32, 36, 48, 64])
@pytest.mark.parametrize("B", [1, 3, 16, 37])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_step(N, B, dtype):
    D, G = 144, 2
    d = L.scan_inputs([1] * B, D, G, N, 800 + N + B, slots=B + 2)
    c = cuda(d)
    flags = (torch.arange(B) % 3 != 1).to(torch.uint8)
    slots = d["cache_indices"].long()
    before = d["pool"].to(dtype)
    before[slots[flags == 0]] = float("nan")
    pool, y = before.cuda(), torch.empty_like(c["x"])
    binding.ssd_selective_scan_step_inplace(y, *inputs(c), pool, flags.cuda(), c["cache_indices"])
    want, by, final, bf = L.scan(d, [1] * B, torch.where(flags.bool()[:, None, None], before[slots].float(), 0.0))
    assert L.worst(y, want, by, L.BF16) <= 1
    assert L.worst(pool.cpu()[slots], final, bf, rounding(dtype)) <= 1
    rest = [s for s in range(B + 2) if s not in slots.tolist()]
    assert torch.equal(pool.cpu()[rest], before[rest])


@pytest.mark.parametrize("use", [(), ("D",), ("z",)])
@pytest.mark.parametrize("softplus", [True, False])
def test_step_forms_and_padding(use, softplus):
    B, D, N = 18, 72, 16
    d = L.scan_inputs([1] * B, D, 1, N, 830, slots=B)
    d["dt"] = d["dt"].abs()
    c = cuda(d)
    c["cache_indices"][4] = B
    pool, y = c["pool"].clone(), torch.full_like(c["x"], 7.0)
    binding.ssd_selective_scan_step_inplace(y, *inputs(c, use), pool, None, c["cache_indices"], dt_softplus=softplus)
    want, by, final, bf = L.scan(d, [1] * B, None, softplus, use)
    live = [b for b in range(B) if b != 4]
    assert L.worst(y[live], want[live], by[live], L.BF16) <= 1 and bool((y[4] == 7.0).all())
    slots = d["cache_indices"].long()
    assert L.worst(pool.cpu()[slots[live]], final[live], bf[live], L.U) <= 1
    assert torch.equal(pool.cpu()[slots[4]], d["pool"][slots[4]])


@pytest.mark.parametrize("N", [12, 16, 64])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_step_of_slices(N, dtype):
    """Rows of B and C at odd dwords, of x, dt and z inside wider ones: bit for bit the results of dense ones."""
    B, D = 19, 72
    d = L.scan_inputs([1] * B, D, 1, N, 835 + N, slots=B)
    c = cuda(d)
    xdz = torch.cat([c["x"], c["dt"], c["z"]], 1)
    bc = torch.cat([torch.zeros(B, 10, dtype=BF16, device="cuda"), c["B"].view(B, N), c["C"].view(B, N)], 1)
    sliced = dict(c, x=xdz[:, :D], dt=xdz[:, D:2 * D], z=xdz[:, 2 * D:], B=bc[:, 10:10 + N].unflatten(1, (1, N)),
                  C=bc[:, 10 + N:].unflatten(1, (1, N)))
    assert sliced["B"].data_ptr() % 8 == 4 and bc.stride(0) % 4 == 2
    flags, outs = torch.ones(B, dtype=torch.uint8, device="cuda"), []
    for s in (c, sliced):
        pool, y = c["pool"].to(dtype, copy=True), torch.empty_like(c["x"])
        binding.ssd_selective_scan_step_inplace(y, *inputs(s), pool, flags, c["cache_indices"])
        outs.append((y, pool))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_steps_continue_a_prompt():
    D, N = 72, 16
    d = L.scan_inputs([40], D, 1, N, 840, slots=1)
    c = cuda(d)
    pool, y = c["pool"].clone(), torch.empty_like(c["x"])
    one = torch.ones(1, dtype=torch.uint8, device="cuda")

    def rows(a, b):
        return inputs({k: c[k][a:b] if k in ("x", "dt", "B", "C", "z") else c[k] for k in NAMES})

    binding.ssd_selective_scan_varlen_fwd_inplace(y[:30], *rows(0, 30), pool,
                                                  torch.tensor([0, 30], dtype=torch.int32, device="cuda"), one,
                                                  c["cache_indices"])
    for t in range(30, 40):
        binding.ssd_selective_scan_step_inplace(y[t:t + 1], *rows(t, t + 1), pool, one, c["cache_indices"])
    want, by, final, bf = L.scan(d, [40], d["pool"])
    assert L.worst(y, want, by, L.BF16) <= 1 and L.worst(pool, final, bf, L.U) <= 1


# ------------------------------------------------------------------ backward

def gradients(c, initial, d_final, use=L.ALL, softplus=True, d_initial=True, **kw):
    """All gradients of a call on the device tensors `c`, by name."""
    out = {n: torch.full(c[n].shape, 7.0, dtype=c[n].dtype, device="cuda") for n in NAMES}
    for n in L.ALL:
        if n not in use:
            out[n] = None
    kind = F32 if initial is None and d_final is None else (d_final if initial is None else initial).dtype
    out["initial"] = torch.full(c["initial"].shape, 7.0, dtype=kind, device="cuda") if d_initial else None
    binding.ssd_selective_scan_varlen_bwd(*[out[n] for n in NAMES], out["initial"], *inputs(c, use), c["d_y"], initial,
                                          d_final, c["query_start_loc"], dt_softplus=softplus, **kw)
    return {n: t for n, t in out.items() if t is not None}


def check_backward(lens, D, G, N, seed, dtype=F32, initial=True, final=True, tail=0, softplus=True, use=L.ALL,
                   decay=1.0):
    d = L.scan_inputs(lens, D, G, N, seed, tail=tail, decay=decay)
    if not softplus:
        d["dt"], d["dt_bias"] = d["dt"].abs(), d["dt_bias"].abs() * 0.1
    d["initial"], d["d_final"] = d["initial"].to(dtype), d["d_final"].to(dtype)
    c = cuda(d)
    got = gradients(c, c["initial"] if initial else None, c["d_final"] if final else None, use, softplus)
    want = L.scan_gradients(d, lens, d["initial"] if initial else None, d["d_final"] if final else None, softplus, use)
    T = sum(lens)
    for n, t in got.items():
        e = L.BF16 if n in ("x", "dt", "B", "C", "z") else rounding(t.dtype)
        rows = n in ("x", "dt", "B", "C", "z")
        assert L.worst(t[:T] if rows else t, *want[n], e) <= 1, n
        assert not rows or bool((t[T:] == 7.0).all()), n


@pytest.mark.parametrize("N", [4, 8, 12, 16, 20, 24, 28, 32, 36, 48, 64])
@pytest.mark.parametrize("D,G", [(8, 1), (200, 1), (144, 2)])
def test_backward_sizes(D, G, N):
    check_backward([35, 1, 0, 50], D, G, N, 900 + D + N)


@pytest.mark.parametrize("D,G", [(64, 1), (128, 4), (24, 3), (520, 5)])
def test_backward_groups(D, G):
    check_backward([17, 40], D, G, 16, 1000 + D)


@pytest.mark.parametrize("n", [0, 1, 2, 7, 8, 9, 15, 16, 17, 33, 100])
def test_backward_lengths(n):
    check_backward([n], 72, 1, 16, 1100 + n)
    check_backward([n, 3, n], 8, 1, 8, 1130 + n, tail=2)


@pytest.mark.parametrize("initial,final", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_backward_states(initial, final, dtype):
    check_backward([40, 0, 300], 72, 1, 16, 1200, dtype, initial, final, tail=9)


@pytest.mark.parametrize("use", [(), ("D",), ("z",), ("dt_bias",), ("z", "D")])
@pytest.mark.parametrize("softplus", [True, False])
def test_backward_forms(use, softplus):
    check_backward([40, 33], 72, 1, 16, 1210, softplus=softplus, use=use)


@pytest.mark.parametrize("lens", [[256], [257], [271, 300], [5, 600, 0, 900, 256, 257]])
def test_backward_long(lens):
    """Sequences that are cut into segments, among others that are not."""
    check_backward(lens, 72, 1, 16, 1300 + sum(lens), tail=3)
    check_backward(lens, 16, 2, 8, 1301 + sum(lens), decay=0.01)


def test_backward_many_sequences():
    lens = [int(x) for x in torch.randint(0, 12, (300,), generator=torch.Generator().manual_seed(6))]
    lens[150] = 400
    check_backward(lens, 8, 1, 4, 1400, tail=3)


@pytest.mark.parametrize("n", [64, 130, 256])
def test_backward_many_long_sequences(n):
    lens = lens_of_many(n, 80 + n)
    assert sum(lens) // n >= 128
    check_backward(lens, 8, 1, 4, 1420 + n, tail=3)


def test_backward_of_wrong_tables_stays_inside():
    """... and sequences that a wrong table lets overlap have no more workspace than there is."""
    for table in ([0, 600, 0, 600, 0, 600], [600, 0, 600, 0, 600, 0], [-7, 1000000, 3, 400, 20, 599]):
        d = L.scan_inputs([120] * 5, 64, 1, 16, 1406)
        c = cuda(d)
        c["query_start_loc"] = torch.tensor(table, dtype=torch.int32, device="cuda")
        bytes_ = binding.ssd_selective_scan_workspace_size(
            binding.ssd_selective_problem(total_len=600, batch=5, channels=64, ngroups=1, dstate=16, max_slots=5,
                                          dt_softplus=1, state_dtype=binding.STATE_F32), backward=True)
        guard = torch.full((bytes_ + 4096,), 7, dtype=torch.uint8, device="cuda")
        gradients(c, None, None, workspace=guard[:bytes_])
        torch.cuda.synchronize()
        assert bool((guard[bytes_:] == 7).all())


def test_backward_of_padding_that_is_not_finite():
    """Rows behind the last sequence are not read: NaN there stays out of the sums over tokens."""
    lens = [13, 30]
    d = L.scan_inputs(lens, 72, 1, 16, 1410, tail=20)
    for n in ("x", "dt", "B", "C", "z", "d_y"):
        d[n][43:] = float("nan")
    c = cuda(d)
    got = gradients(c, None, None)
    want = L.scan_gradients(d, lens)
    for n in ("A", "D", "dt_bias", "initial"):
        assert L.worst(got[n], *want[n], L.U) <= 1, n
    for n in ("B", "C", "x"):
        assert L.worst(got[n][:43], *want[n], L.BF16) <= 1, n


def test_backward_against_differences():
    """The gradients predict how the final states' sum (fp32) changes along a direction of A, D, dt_bias and the
    initial states."""
    lens, D, N, h = [40, 25], 32, 8, 2.0 ** -6
    d = L.scan_inputs(lens, D, 1, N, 1420)
    c = cuda(d)
    g = torch.Generator().manual_seed(1421)
    names = ("A", "dt_bias", "initial")
    way = {n: torch.randn(d[n].shape, generator=g) for n in names}
    got = gradients(dict(c, d_y=torch.zeros_like(c["d_y"])), c["initial"], c["d_final"])
    predicted = sum(float((got[n].cpu().double() * way[n].double()).sum()) for n in names)
    values = []
    for s in (h, -h):
        e = {n: (c[n] + s * way[n].cuda()) if n in names else c[n] for n in c}
        y, f = torch.empty_like(c["x"]), torch.empty_like(c["initial"])
        binding.ssd_selective_scan_varlen_fwd(y, *inputs(e), e["initial"], f, c["query_start_loc"])
        values.append(float((f.double() * c["d_final"].double()).sum()))
    # beside the third-order part, the states' roundings: 2 h has to stand out of 2^-24 of some hundred numbers
    assert abs((values[0] - values[1]) / (2 * h) - predicted) <= 0.02 * abs(predicted) + 0.05


# ------------------------------------------------------------------ ways of calling

def test_refusals():
    c = cuda(L.scan_inputs([5, 4], 64, 1, 16, 1500, slots=3))
    y = torch.empty_like(c["x"])

    def f(y=y, pool=c["pool"], qsl=c["query_start_loc"], flags=None, idx=c["cache_indices"], **kw):
        binding.ssd_selective_scan_varlen_fwd_inplace(y, *inputs(dict(c, **kw)), pool, qsl, flags, idx)

    f()
    for kw, error, text in [(dict(x=c["x"].float()), TypeError, "x"), (dict(y=y[:5]), ValueError, "y"),
                            (dict(dt=c["dt"].float()), TypeError, "dt"), (dict(dt=c["dt"][:, :32]), ValueError, "dt"),
                            (dict(A=c["A"].bfloat16()), TypeError, "A"), (dict(A=c["A"][:, :8]), ValueError, "A"),
                            (dict(B=c["B"][:8]), ValueError, "B"), (dict(B=c["B"][:, 0]), ValueError, "B"),
                            (dict(C=c["C"].float()), TypeError, "C"), (dict(C=c["C"][:, :, :8]), ValueError, "C"),
                            (dict(D=c["D"][:32]), ValueError, "D"), (dict(z=c["z"].float()), TypeError, "z"),
                            (dict(dt_bias=c["dt_bias"].bfloat16()), TypeError, "dt_bias"),
                            (dict(pool=c["pool"].half()), TypeError, "pool"),
                            (dict(pool=c["pool"][:, :32]), ValueError, "pool"),
                            (dict(qsl=c["query_start_loc"].long()), TypeError, "query_start_loc"),
                            (dict(idx=c["cache_indices"].long()), TypeError, "cache_indices"),
                            (dict(flags=torch.ones(2, device="cuda")), TypeError, "has_initial"),
                            (dict(z=c["z"].cpu()), ValueError, "z is on")]:
        with pytest.raises(error, match=text):
            f(**kw)
    with pytest.raises(ValueError, match="dz goes with z"):
        g = [torch.empty_like(c[n]) for n in NAMES]
        g[6] = None
        binding.ssd_selective_scan_varlen_bwd(*g, None, *inputs(c), c["x"], None, None, c["query_start_loc"])
    with pytest.raises(binding.SsdError) as e:
        six = dict(A=c["A"][:, :6].contiguous(), B=c["B"][..., :6].contiguous(), C=c["C"][..., :6].contiguous())
        f(pool=c["pool"][..., :6].contiguous(), **six)
    assert e.value.status == 3


def _all_calls(c, outs, stream=None):
    y, pool, ys = outs[:3]
    ones = torch.ones(4, dtype=torch.uint8, device="cuda") if stream is None else c["ones"]
    with torch.cuda.stream(stream or torch.cuda.current_stream()):
        pool.copy_(c["pool"])
    binding.ssd_selective_scan_varlen_fwd_inplace(y, *inputs(c), pool, c["query_start_loc"], c["ones"],
                                                  c["cache_indices"], stream=stream)
    few = {k: c[k][:4] if k in ("x", "dt", "B", "C", "z") else c[k] for k in NAMES}
    binding.ssd_selective_scan_step_inplace(ys, *inputs(few), pool, c["ones"], c["cache_indices"], stream=stream)
    binding.ssd_selective_scan_varlen_bwd(*outs[3:12], *inputs(c), c["d_y"], c["initial"], c["d_final"],
                                          c["query_start_loc"], stream=stream)
    return ones


def test_streams_and_graphs():
    lens = [100, 0, 33, 700]
    c = cuda(L.scan_inputs(lens, 136, 1, 16, 1510, slots=6))
    c["ones"] = torch.ones(4, dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(c["x"]), torch.empty_like(c["pool"]), torch.empty_like(c["x"][:4])]
    outs += [torch.empty_like(c[n]) for n in NAMES + ("initial",)]
    _all_calls(c, outs)
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    for t in outs:
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    _all_calls(c, outs, side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _all_calls(c, outs)
    for _ in range(4):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        _all_calls(c, outs)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_two_calls_at_once():
    """Calls on two streams, each with a workspace of its own, give what they give one at a time."""
    problems = [cuda(L.scan_inputs([900, 20], 136, 1, 16, 1520 + i)) for i in range(2)]
    want = [gradients(c, c["initial"], None) for c in problems]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in problems]
    got = []
    for c, s in zip(problems, streams):
        s.wait_stream(torch.cuda.current_stream())
    for c, s in zip(problems, streams):
        with torch.cuda.stream(s):
            got.append(gradients(c, c["initial"], None))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("use", ["both", "y", "final", "sum"])
def test_autograd(use):
    """Gradients reach the projections whose slices x, z, B and C are, the parameters and the initial states; rows
    behind the last sequence get zeros."""
    from mamba_ssd_chunked_chunk_amd.mixer import selective_scan
    lens, D, N, tail = [90, 0, 2, 300], 72, 16, 5
    d = L.scan_inputs(lens, D, 1, N, 1530, tail=tail)
    c, T = cuda(d), sum(lens)
    xz = torch.cat([c["x"], c["z"]], 1).requires_grad_()
    bc = torch.cat([c["B"].view(T + tail, N), c["C"].view(T + tail, N)], 1).requires_grad_()
    leaf = {n: c[n].clone().requires_grad_() for n in ("dt", "A", "D", "dt_bias", "initial")}
    y, final = selective_scan(xz[:, :D], leaf["dt"], leaf["A"], bc[:, :N].unflatten(1, (1, N)),
                              bc[:, N:].unflatten(1, (1, N)), leaf["D"], xz[:, D:], leaf["dt_bias"],
                              c["query_start_loc"], leaf["initial"], padded=True)
    assert bool((y[T:] == 0).all())
    e, df = dict(d), d["d_final"]
    if use == "sum":
        y[:T].float().sum().backward()
        e["d_y"], df = torch.ones_like(d["d_y"]), None
    else:
        given = dict(both=([y, final], [c["d_y"], c["d_final"]]), y=([y], [c["d_y"]]), final=([final], [c["d_final"]]))
        torch.autograd.backward(*given[use])
        if use == "final":
            e["d_y"] = torch.zeros_like(d["d_y"])
        if use == "y":
            df = None
    want = L.scan_gradients(e, lens, d["initial"], df)
    got = dict(x=xz.grad[:, :D], z=xz.grad[:, D:], B=bc.grad[:, :N].unflatten(1, (1, N)),
               C=bc.grad[:, N:].unflatten(1, (1, N)), **{n: t.grad for n, t in leaf.items()})
    for n, t in got.items():
        rows = n in ("x", "z", "B", "C", "dt")
        assert L.worst(t[:T] if rows else t, *want[n], L.BF16 if rows else L.U) <= 1, n
        assert not rows or bool((t[T:] == 0).all()), n


def test_autograd_of_shared_and_optional_inputs():
    """One tensor as two inputs gets the sum of both gradients; inputs that are left out get none; empty initial
    states stand for zero, in their own type."""
    from mamba_ssd_chunked_chunk_amd.mixer import selective_scan
    lens, D, N = [40, 30], 64, 8
    d = L.scan_inputs(lens, D, 1, N, 1540)
    d["C"] = d["B"].clone()
    c = cuda(d)
    bc, x = c["B"].clone().requires_grad_(), c["x"].clone().requires_grad_()
    y, final = selective_scan(x, c["dt"], c["A"], bc, bc, None, None, None, c["query_start_loc"],
                              torch.empty(0, dtype=BF16, device="cuda"))
    assert final.dtype == BF16
    y.backward(c["d_y"])
    want = L.scan_gradients(d, lens, use=())
    both = [a + b for a, b in zip(want["B"], want["C"])]
    # each gradient is rounded to bf16, and so is their sum
    assert L.worst(bc.grad, both[0], both[1] + (want["B"][0].abs() + want["C"][0].abs()) * L.BF16, L.BF16 * 1.01) <= 1
    assert L.worst(x.grad, *want["x"], L.BF16) <= 1
