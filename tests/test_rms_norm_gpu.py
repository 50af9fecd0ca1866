"""The root-mean-square norm with the residual's addition on the GPU: outputs in
bf16 and in 8 bits and the backward pass against the definition in 64 bits,
within bounds counted from the roundings (layer_testlib)."""

import pytest

torch = pytest.importorskip("torch")
import layer_testlib as L  # noqa: E402
from mamba_ssd_chunked_chunk_amd import binding  # noqa: E402

pytestmark = pytest.mark.gpu
F32, BF16, I8, E4M3 = torch.float32, torch.bfloat16, torch.int8, torch.float8_e4m3fn
EPS = 1e-5


def draw(rows, width, seed, residual=None):
    g = torch.Generator().manual_seed(seed)
    size = torch.exp(torch.randn(rows, 1, generator=g))
    x = (torch.randn(rows, width, generator=g) * size).bfloat16()
    r = None if residual is None else (3 * torch.randn(rows, width, generator=g) * size).to(residual)
    return x, r, 1 + 0.3 * torch.randn(width, generator=g)


def forward(x, r, w, kind=BF16, eps=EPS, same=False, **kw):
    """y, scales, residual_out on the CPU"""
    xc, wc = x.cuda(), w.cuda()
    rc = None if r is None else r.cuda()
    y = torch.full(x.shape, 7.0, device="cuda").to(kind)
    scales = None if kind == BF16 else torch.full((x.shape[0],), 7.0, device="cuda")
    out = rc if same or r is None else torch.full_like(rc, 7.0)
    binding.ssd_rms_norm_fwd(y, scales, out, xc, rc, wc, eps=eps, **kw)
    return y.cpu(), None if scales is None else scales.cpu(), None if out is None else out.cpu()


def check_codes(codes, scales, want, kind):
    """Codes and scales of the rows `want` [rows, width] in fp64, which the kernel knows to L.NORM."""
    top = want.abs().amax(1)
    s = scales.double()
    live = top > 0
    assert bool((s[~live] == 0).all()) and bool((codes.float()[~live] == 0).all())
    if kind == I8:
        assert bool(((s - top / 127).abs() <= top / 127 * (L.NORM + L.U)).all())
        step = s
    else:
        low, _ = torch.frexp(s[live])
        assert bool((low == 0.5).all())  # powers of two
        ratio = top[live] / s[live]
        assert bool((ratio <= 448 * (1 + L.NORM)).all()) and bool((ratio > 224 * (1 - L.NORM)).all())
        # the distance of e4m3 values around a quotient: 2^-3 of its power of two, 2^-9 at the low end
        _, e = torch.frexp(want / torch.where(live, s, 1.0)[:, None])
        step = torch.exp2((e - 1).clamp(min=-6).double() - 3) * s[:, None]
    step = step if step.dim() == 2 else step[:, None]
    got = codes.double() * s[:, None]
    assert bool(((got - want).abs() <= step / 2 * (1 + 2.0 ** -20) + want.abs() * L.NORM).all())


WIDTHS = [8, 64, 72, 504, 512, 520, 1000, 1024, 1032, 2048, 2056, 2560, 4096, 4104, 8192, 8200, 16384, 16392, 32768]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("residual", [None, BF16, F32])
def test_forward_widths(width, residual):
    x, r, w = draw(5, width, width, residual)
    y, _, out = forward(x, r, w)
    want, kept = L.norm(x, r, w, EPS)
    assert L.worst(y, want, want.abs() * L.NORM, L.BF16) <= 1
    if r is not None:
        assert torch.equal(out, (x.float() + r.float()).to(residual))
        assert out.double().sub(kept).abs().max() <= kept.abs().max() * L.U  # fp32: the sum's own rounding


@pytest.mark.parametrize("rows", [0, 1, 2, 3, 4, 5, 63, 64, 65, 1000, 5003])
def test_forward_rows(rows):
    x, r, w = draw(rows, 136, 900 + rows, BF16)
    y, _, out = forward(x, r, w)
    want, _ = L.norm(x, r, w, EPS)
    assert L.worst(y, want, want.abs() * L.NORM, L.BF16) <= 1
    assert torch.equal(out, (x.float() + r.float()).bfloat16())


@pytest.mark.parametrize("kind", [I8, E4M3])
@pytest.mark.parametrize("width", [8, 72, 1032, 4096, 5120, 16384, 20000])
def test_codes(width, kind):
    x, r, w = draw(6, width, width + 1, F32)
    x[2], r[2] = 0, 0
    y, s, out = forward(x, r, w, kind)
    want, _ = L.norm(x, r, w, EPS)
    check_codes(y, s, want, kind)
    assert torch.equal(out, x.float() + r)


@pytest.mark.parametrize("kind", [I8, E4M3])
def test_codes_of_rows_that_are_not_finite(kind):
    x, _, w = draw(4, 64, 5)
    x[1, 3], x[2, 5] = float("nan"), float("inf")
    y, s, _ = forward(x, None, w, kind)
    assert bool(torch.isnan(s[1:3]).all()) and bool((y[1:3].float() == 0).all())
    want, _ = L.norm(x[[0, 3]], None, w, EPS)
    check_codes(y[[0, 3]], s[[0, 3]], want, kind)


@pytest.mark.parametrize("kind", [I8, E4M3])
def test_codes_equal_the_state_caches(kind):
    """A row of the norm in 8 bits is what ssd_state_quantize makes of the same numbers: with weights of one and rows
    of one magnitude the norm leaves numbers that are known."""
    g = torch.Generator().manual_seed(6)
    signs = torch.where(torch.rand(8, 256, generator=g) < 0.5, -1.0, 1.0)
    w = torch.randn(256, generator=g)
    y, s, _ = forward(signs.bfloat16(), None, w, kind, eps=0.0)
    pool = (signs * w).cuda().view(1, 1, 8, 256)
    codes, scales = torch.empty(1, 1, 8, 256, dtype=kind, device="cuda"), torch.empty(1, 1, 8, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.ssd_state_quantize(codes, scales, pool, zero, zero)
    assert torch.equal(scales.view(8).cpu(), s) and torch.equal(codes.view(8, 256).cpu().float(), y.float())


def test_zero_eps_and_zero_rows():
    x, _, w = draw(3, 64, 7)
    x[1] = 0
    y, _, _ = forward(x, None, w, eps=1e-5)
    assert bool((y[1] == 0).all())
    y, _, _ = forward(x, None, w, eps=0.0)  # 0 / 0 stays in its row
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isfinite(y[[0, 2]]).all())


def test_strided_rows_and_the_residual_in_place():
    wide, r, w = draw(9, 3 * 200, 8, None)[0], draw(9, 200, 9, F32)[1], draw(1, 200, 10)[2]
    part = wide.cuda()[:, 200:400]
    y, out = torch.empty(9, 200, dtype=BF16, device="cuda"), r.cuda()
    binding.ssd_rms_norm_fwd(y, None, out, part, out, w.cuda(), eps=EPS)
    want, _, kept = forward(wide[:, 200:400].contiguous(), r, w)
    assert torch.equal(y.cpu(), want) and torch.equal(out.cpu(), kept)
    for residual in (BF16, F32):
        x, r, w = draw(70, 1032, 11, residual)
        a, b = forward(x, r, w), forward(x, r, w, same=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])


def test_rows_behind_2_31_elements():
    rows, width = (1 << 31) // 2048 + 3, 2048
    x = torch.empty(rows, width, dtype=BF16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    y = torch.empty_like(x)
    w = draw(1, width, 12)[2]
    binding.ssd_rms_norm_fwd(y, None, None, x, None, w.cuda())
    for at in (0, rows // 2, rows - 1):
        want, _ = L.norm(x[at:at + 1].cpu(), None, w, 1e-5)
        assert L.worst(y[at:at + 1], want, want.abs() * L.NORM, L.BF16) <= 1


# ------------------------------------------------------------------ backward

def backward(r, w, dy, dr, eps=EPS, both=False, **kw):
    rc = r.cuda()
    dx = torch.full(r.shape, 7.0, dtype=BF16, device="cuda")
    d_residual = torch.full_like(rc, 7.0) if both else None
    dw = torch.full_like(w, 7.0, device="cuda")
    binding.ssd_rms_norm_bwd(dx, d_residual, dw, rc, w.cuda(), dy.cuda(), None if dr is None else dr.cuda(), eps=eps,
                             **kw)
    return dx.cpu(), None if d_residual is None else d_residual.cpu(), dw.cpu()


def check_backward(rows, width, kind, given, seed):
    g = torch.Generator().manual_seed(seed)
    r, w = draw(rows, width, seed, kind)[1:]
    dy = torch.randn(rows, width, generator=g).bfloat16()
    dr = torch.randn(rows, width, generator=g).to(kind) if given else None
    dx, both, dw = backward(r, w, dy, dr, both=True)
    d, bd, dw64, bw = L.norm_gradients(r, w, dy, dr, EPS)
    assert L.worst(dx, d, bd, L.BF16) <= 1
    assert L.worst(both, d, bd, torch.finfo(kind).eps / 2) <= 1
    assert L.worst(dw, dw64, bw, L.U) <= 1


@pytest.mark.parametrize("width", WIDTHS)
def test_backward_widths(width):
    check_backward(5, width, F32 if width % 16 else BF16, True, 2000 + width)


@pytest.mark.parametrize("rows", [0, 1, 3, 4, 5, 100, 1023, 1024, 1025, 5003])
@pytest.mark.parametrize("width", [200, 2056])
def test_backward_rows(rows, width):
    check_backward(rows, width, BF16, rows % 2 == 1, 3000 + rows)


def test_backward_in_the_gradients_buffer():
    r, w = draw(33, 264, 13, F32)[1:]
    g = torch.Generator().manual_seed(14)
    dy, dr = torch.randn(33, 264, generator=g).bfloat16(), torch.randn(33, 264, generator=g)
    want = backward(r, w, dy, dr, both=True)
    d = dr.cuda()
    dx, dw = torch.empty(33, 264, dtype=BF16, device="cuda"), torch.empty(264, device="cuda")
    binding.ssd_rms_norm_bwd(dx, d, dw, r.cuda(), w.cuda(), dy.cuda(), d, eps=EPS)
    assert torch.equal(dx.cpu(), want[0]) and torch.equal(d.cpu(), want[1]) and torch.equal(dw.cpu(), want[2])


def test_backward_against_differences():
    """The gradients predict how sum(y dy) + sum(r dr) changes along a direction, in the forward kernel's own numbers:
    r in fp32, so that the step is not rounded away; y's roundings (2^-8 of each) bound the rest."""
    rows, width, h = 20, 256, 2.0 ** -4
    g = torch.Generator().manual_seed(15)
    x = torch.zeros(rows, width).bfloat16()
    r, w = draw(rows, width, 16, F32)[1:]
    dy, dr = torch.randn(rows, width, generator=g).bfloat16(), torch.randn(rows, width, generator=g)
    way, way_w = torch.randn(rows, width, generator=g), torch.randn(width, generator=g)
    _, d, dw = backward(r, w, dy, dr, both=True)
    predicted = float((d.double() * way.double()).sum() + (dw.double() * way_w.double()).sum())

    def value(s):
        y, _, out = forward(x, r + s * way, w + s * way_w)
        return float((y.double() * dy.double()).sum() + (out.double() * dr.double()).sum()), y

    (up, y1), (down, y0) = value(h), value(-h)
    exact = []
    for s in (h, -h):  # the same difference of the definition, whose own third-order part is not the kernels'
        y, out = L.norm(x, (r + s * way), w + s * way_w, EPS)
        exact.append(float((y * dy.double()).sum() + (out * dr.double()).sum()))
    rounding = float(((y1.double().abs() + y0.double().abs()) * dy.double().abs()).sum()) * 2.0 ** -8
    assert abs((up - down) - (exact[0] - exact[1])) <= rounding
    third = abs((exact[0] - exact[1]) / (2 * h) - predicted)
    assert third <= 0.02 * abs(predicted) + 1.0, (third, predicted)


# ------------------------------------------------------------------ ways of calling

def test_refusals():
    x, r, w = (t.cuda() for t in draw(4, 64, 17, BF16))
    y = torch.empty_like(x)
    f = binding.ssd_rms_norm_fwd
    with pytest.raises(ValueError, match="scales"):
        f(y, torch.empty(4, device="cuda"), None, x, None, w)
    with pytest.raises(ValueError, match="scales"):
        f(y.to(I8), None, None, x, None, w)
    with pytest.raises(ValueError, match="go together"):
        f(y, None, None, x, r, w)
    with pytest.raises(TypeError, match="y: expected"):
        f(y.float(), None, None, x, None, w)
    with pytest.raises(TypeError, match="residual"):
        f(y, None, r.half(), x, r.half(), w)
    with pytest.raises(TypeError, match="weight"):
        f(y, None, None, x, None, w.bfloat16())
    with pytest.raises(ValueError, match="contiguous"):
        f(y, None, r.expand(4, 64), x, torch.empty(64, 4, dtype=BF16, device="cuda").t(), w)
    with pytest.raises(ValueError, match="multiple of 8"):
        f(y, None, None, torch.empty(4, 68, dtype=BF16, device="cuda")[:, :64], None, w)
    with pytest.raises(binding.SsdError) as e:
        f(torch.empty(4, 60, dtype=BF16, device="cuda"), None, None, x[:, :60].contiguous(), None, w[:60].contiguous())
    assert e.value.status == 3
    with pytest.raises(binding.SsdError) as e:  # from no 16-byte boundary
        f(y, None, None, torch.empty(4 * 64 + 1, dtype=BF16, device="cuda")[1:].view(4, 64), None, w)
    assert e.value.status == 7
    with pytest.raises(ValueError, match="workspace"):
        binding.ssd_rms_norm_bwd(y, None, w.clone(), r, w, x, None,
                                 workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_streams_and_graphs():
    """Deterministic, the same on another stream, and captured into a graph and replayed between eager calls."""
    x, r, w = draw(300, 2056, 18, F32)
    dy = x.flip(0).contiguous()
    xc, rc, wc, dyc = x.cuda(), r.cuda(), w.cuda(), dy.cuda()
    outs = [torch.empty_like(xc), torch.empty_like(rc), torch.empty_like(xc), torch.empty_like(rc),
            torch.empty_like(wc), torch.empty(300, 2056, dtype=E4M3, device="cuda"), torch.empty(300, device="cuda")]

    def all_calls(stream=None):
        y, out, dx, d_res, dw, codes, scales = outs
        binding.ssd_rms_norm_fwd(y, None, out, xc, rc, wc, stream=stream)
        binding.ssd_rms_norm_bwd(dx, d_res, dw, out, wc, dyc, rc, stream=stream)
        binding.ssd_rms_norm_fwd(codes, scales, out, xc, rc, wc, stream=stream)

    all_calls()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in outs:
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    all_calls(side)
    side.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        all_calls()
    for _ in range(4):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(outs, want))
        all_calls()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(outs, want))


# ------------------------------------------------------------------ as a differentiable function

@pytest.mark.parametrize("kind", [None, BF16, F32])
@pytest.mark.parametrize("use", ["both", "y", "stream", "sum"])
def test_autograd(kind, use):
    from mamba_ssd_chunked_chunk_amd.mixer import rms_norm
    x, r, w = draw(2 * 7, 136, 19, kind)
    g = torch.Generator().manual_seed(20)
    dy, dr = torch.randn(14, 136, generator=g).bfloat16(), torch.randn(14, 136, generator=g).to(kind or BF16)
    leaves = [x.cuda().view(2, 7, 136).requires_grad_(), w.cuda().requires_grad_()]
    if kind is not None:
        leaves.append(r.cuda().view(2, 7, 136).requires_grad_())
    out = rms_norm(leaves[0], leaves[1], *leaves[2:])
    if kind is None:
        if use in ("stream",):
            return
        y, stream, dr = out, None, None
    else:
        y, stream = out
    if use == "sum":
        y.sum().backward()
        dy, dr = torch.ones_like(dy), None
    elif use == "y" or stream is None:
        torch.autograd.backward(y, dy.cuda().view(y.shape))
        dr = None
    elif use == "stream":
        torch.autograd.backward(stream, dr.cuda().view(y.shape))
        dy = torch.zeros_like(dy)
    else:
        torch.autograd.backward([y, stream], [dy.cuda().view(y.shape), dr.cuda().view(y.shape)])
    kept = x if kind is None else (x.float() + r.float()).to(kind)
    d, bd, dw, bw = L.norm_gradients(kept, w, dy, dr, 1e-5)
    assert L.worst(leaves[0].grad.view(14, 136), d, bd, L.BF16) <= 1
    assert L.worst(leaves[1].grad, dw, bw, L.U) <= 1
    if kind is not None:
        assert leaves[2].grad.dtype == kind
        assert L.worst(leaves[2].grad.view(14, 136), d, bd, torch.finfo(kind).eps / 2) <= 1
