"""Pool states parked in 8 bits and read back: codes, scales and read-back
values equal the definition's, computed in 64 bits, bit for bit."""

import pytest

torch = pytest.importorskip("torch")
from mamba_ssd_chunked_chunk_amd import binding  # noqa: E402

pytestmark = pytest.mark.gpu
F32, BF16, I8, E4M3 = torch.float32, torch.bfloat16, torch.int8, torch.float8_e4m3fn
TINY = torch.finfo(F32).tiny


def quantized(x, kind):
    """Codes (fp64 values) and scales (fp64) of the rows of x, by the definition."""
    x = x.double()
    top = x.abs().amax(-1)
    lost = ~torch.isfinite(top)  # rows that hold an infinity or NaN: codes 0, and a scale that reads back as NaN
    x, top = torch.where(lost[..., None], 0.0, x), torch.where(lost, 0.0, top)
    codes, scale = _quantized(x, top, kind)
    return codes, torch.where(lost, float("nan"), scale)


def _quantized(x, top, kind):
    if kind == I8:
        scale = (top / 127).float().double()
        scale[scale < TINY] = 0
        return torch.round(x / scale.clamp(min=TINY)[..., None]) * (scale > 0)[..., None], scale
    values = torch.arange(127, dtype=torch.uint8).view(E4M3).double()  # the format's values, none negative, in order
    p = torch.arange(-126, 128, dtype=torch.float64)
    powers = torch.exp2(p)
    scale = powers[torch.searchsorted(448 * powers, top)]  # the least with top <= 448 * it
    a = (x / scale[..., None]).abs()
    hi = torch.searchsorted(values, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = values[hi] - a, a - values[lo]
    near = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), values[hi], values[lo])
    scale[top == 0] = 0
    return near * torch.sign(x) * (scale > 0)[..., None], scale


def same(a, b):
    return a.dtype == b.dtype and a.shape == b.shape and bool(((a == b) | (a.isnan() & b.isnan())).all())


def states(S, H, P, N, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(S, H, P, N, generator=g) * torch.exp(3 * torch.randn(S, H, P, 1, generator=g))
    x[0, 0, 0] = 0                              # a row of zeros
    x[0, 0, 1 % P] *= 1e-42                     # subnormal
    x[0, H - 1, 2 % P] *= 1e36                  # near the top of the range
    # ties: with a largest value of 127 the scale is 1, and halves lie between two codes
    x[-1, 0, 0] = torch.arange(N) % 16 - 7.5
    x[-1, 0, 0, 0] = 127.0
    # the format's ties: between two neighbouring values of every size
    v = torch.arange(127, dtype=torch.uint8).view(E4M3).float()
    t = (v[1:] + v[:-1]) / 2
    x[-1, 0, P - 1] = torch.cat([t] * 3)[:N]
    x[-1, 0, P - 1, 0] = 448.0
    return x


@pytest.mark.parametrize("kind", [I8, E4M3])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H,P,N", [(1, 1, 8), (3, 64, 128), (2, 100, 256), (5, 7, 72), (1, 64, 64), (4, 33, 200)])
def test_codes_scales_and_values(H, P, N, dtype, kind):
    S, E = 5, 4
    pool = states(S, H, P, N, 10 + N).to(dtype)
    dev = pool.cuda()
    codes = torch.full((E, H, P, N), 3.0, device="cuda").to(kind)
    scales = torch.full((E, H, P), 5.0, device="cuda")
    src = torch.tensor([4, 0, 0], dtype=torch.int32, device="cuda")  # one slot twice
    dst = torch.tensor([2, 0, 3], dtype=torch.int32, device="cuda")
    binding.ssd_state_quantize(codes, scales, dev, src, dst)
    assert torch.equal(dev.cpu(), pool)
    want, f = quantized(pool[[4, 0, 0]].float(), kind)
    got = codes.float().cpu().double()[[2, 0, 3]]
    assert torch.equal(got, want)
    assert same(scales.cpu().double()[[2, 0, 3]], f)
    assert bool((codes.float()[1] == 3).all()) and bool((scales[1] == 5).all())  # the entry left alone
    # read back into other slots
    back = torch.full_like(dev, 9.0)
    where = torch.tensor([1, 3], dtype=torch.int32, device="cuda")
    binding.ssd_state_dequantize(back, codes, scales, where, dst[:2])
    values = (want[:2] * f[:2, ..., None]).float().to(dtype)
    assert same(back.cpu()[[1, 3]], values)
    assert bool((back[[0, 2, 4]] == 9).all())
    # the values are off by half a code (i8), or by the format's rounding (2^-4, or half its least step), at most
    x = pool[[4, 0]].double()
    s = f[:2, ..., None]
    half = s / 2 if kind == I8 else torch.maximum(x.abs() * 2.0 ** -4, s * 2.0 ** -10)
    half[s[..., 0] == 0] = TINY * 127  # rows too small for a scale
    stored = torch.finfo(dtype).eps / 2
    near = (back.cpu()[[1, 3]].double() - x).abs() <= half * (1 + 2.0 ** -20) + stored * (x.abs() + half)
    assert bool((near | s.isnan()).all())


@pytest.mark.parametrize("kind", [I8, E4M3])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_rows_that_are_not_finite(kind, bad):
    pool = torch.randn(2, 2, 16, 64, device="cuda")
    pool[0, 1, 3, 17] = bad
    codes = torch.zeros(2, 2, 16, 64, device="cuda").to(kind)
    scales = torch.zeros(2, 2, 16, device="cuda")
    i = torch.arange(2, dtype=torch.int32, device="cuda")
    binding.ssd_state_quantize(codes, scales, pool, i, i)
    back = torch.zeros_like(pool)
    binding.ssd_state_dequantize(back, codes, scales, i, i)
    nan = torch.isnan(back)
    assert bool(nan[0, 1, 3].all()) and int(nan.sum()) == 64


def test_every_quotient_near_a_border():
    """Values half a code above a whole number of scales, and one step of fp32 to either side of it."""
    g = torch.Generator().manual_seed(4)
    top = torch.rand(64, generator=g) * 10 + 0.1
    s = (top.double() / 127).float()
    n = torch.arange(126)
    mid = ((n + 0.5)[None, :] * s.double()[:, None]).float()
    up, down = torch.nextafter(mid, torch.tensor(1e9)), torch.nextafter(mid, torch.tensor(0.0))
    rows = torch.stack([mid, up, down, -mid], 1)  # [64, 4, 126]
    x = torch.zeros(1, 64, 4, 128)
    x[0, :, :, 1:127] = rows
    x[0, :, :, 0] = top[:, None]
    dev = x.cuda()
    codes = torch.zeros(1, 64, 4, 128, dtype=I8, device="cuda")
    scales = torch.zeros(1, 64, 4, device="cuda")
    i = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.ssd_state_quantize(codes, scales, dev, i, i)
    want, f = quantized(x, I8)
    assert torch.equal(scales.cpu().double(), f) and torch.equal(codes.cpu().double(), want)


@pytest.mark.parametrize("count", [0, 1, 37])
def test_counts_and_padding(count):
    pool = torch.randn(40, 2, 24, 96, device="cuda")
    codes = torch.zeros(50, 2, 24, 96, dtype=I8, device="cuda")
    scales = torch.zeros(50, 2, 24, device="cuda")
    src = torch.randperm(40, device="cuda")[:count].to(torch.int32)
    dst = torch.randperm(50, device="cuda")[:count].to(torch.int32)
    if count > 2:
        src[1] = 40
        dst[2] = -1
    binding.ssd_state_quantize(codes, scales, pool, src, dst)
    live = [i for i in range(count) if count <= 2 or i not in (1, 2)]
    e = dst[live].long()
    assert int((scales.flatten(1) != 0).any(1).sum()) == len(live)
    back = torch.zeros_like(pool)
    binding.ssd_state_dequantize(back, codes, scales, src, dst)
    assert int((back.flatten(1) != 0).any(1).sum()) == len(live)
    want = codes[e].float() * scales[e][..., None]
    assert torch.equal(back[src[live].long()], want)


def test_entries_behind_2_31_elements():
    """A cache whose last entry starts behind element 2^31."""
    N, P, H = 256, 64, 16
    E = 2 ** 31 // (N * P * H) + 2
    codes = torch.zeros(E, H, P, N, dtype=I8, device="cuda")
    scales = torch.zeros(E, H, P, device="cuda")
    pool = torch.randn(2, H, P, N, device="cuda")
    src = torch.tensor([0], dtype=torch.int32, device="cuda")
    dst = torch.tensor([E - 1], dtype=torch.int32, device="cuda")
    binding.ssd_state_quantize(codes, scales, pool, src, dst)
    want, f = quantized(pool[:1].cpu(), I8)
    assert torch.equal(codes[E - 1].cpu().double(), want[0]) and torch.equal(scales[E - 1].cpu().double(), f[0])
    assert not bool(scales[:E - 1].any())
    binding.ssd_state_dequantize(pool, codes, scales, src + 1, dst)
    assert torch.equal(pool[1], codes[E - 1].float() * scales[E - 1][..., None])


def test_captured_and_replayed():
    pool = torch.randn(4, 2, 64, 128, device="cuda")
    codes = torch.zeros(2, 2, 64, 128, dtype=I8, device="cuda")
    scales = torch.zeros(2, 2, 64, device="cuda")
    a = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    b = torch.tensor([2, 3], dtype=torch.int32, device="cuda")

    def move():
        binding.ssd_state_quantize(codes, scales, pool, a, a)
        binding.ssd_state_dequantize(pool, codes, scales, b, a)

    move()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        move()
    for n in range(4):
        pool[:2] = torch.randn(2, 2, 64, 128, device="cuda") * (n + 1)
        graph.replay()
        torch.cuda.synchronize()
        got = pool[2:].clone()
        pool[2:] = 0
        move()
        assert torch.equal(got, pool[2:])
