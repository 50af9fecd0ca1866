"""Further forms of the short convolution on the GPU, against the definition in
64 bits within layer_testlib's bounds: outputs beside their inputs in one buffer,
outputs past the caches, and the backward pass in pieces of many groups."""

import pytest

torch = pytest.importorskip("torch")
import layer_testlib as L  # noqa: E402
from mamba_ssd_chunked_chunk_amd import binding  # noqa: E402

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def draw(lens, D, W, seed):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)

    def normal(*shape):
        return torch.randn(*shape, generator=g)

    return dict(x=normal(T, D).bfloat16(), weight=0.5 * normal(D, W), bias=0.3 * normal(D), d_y=normal(T, D).bfloat16(),
                initial=normal(len(lens), W - 1, D).bfloat16(), d_final=normal(len(lens), W - 1, D).bfloat16(),
                query_start_loc=L.starts_of(lens))


def cuda(d):
    return {k: v.cuda() for k, v in d.items()}


def forward(c, x, y, **kw):
    f = torch.empty_like(c["initial"])
    binding.ssd_causal_conv_varlen_fwd(y, x, c["weight"], c["bias"], c["initial"], f, c["query_start_loc"], **kw)
    return f


def test_outputs_beside_their_inputs():
    """Outputs right ahead of, right behind and between the rows of x; among them they are refused."""
    lens, D = [40, 0, 59], 64
    c = cuda(draw(lens, D, 4, 1))
    T = sum(lens)
    want = torch.empty_like(c["x"])
    last = forward(c, c["x"], want)
    three = torch.empty(3 * T, D, dtype=BF16, device="cuda")
    three[T:2 * T] = c["x"]
    wide = torch.empty(T, (T + 1) * D, dtype=BF16, device="cuda")  # a row of x, and room for all rows of y
    wide[:, :D] = c["x"]
    between = wide.view(-1)[D:(T + 1) * D].view(T, D)
    for x, y in ((three[T:2 * T], three[:T]), (three[T:2 * T], three[2 * T:]), (wide[:, :D], between)):
        y.fill_(7.0)
        assert torch.equal(forward(c, x, y), last) and torch.equal(y, want) and torch.equal(x, c["x"])
    for x, y in ((three[T:2 * T], three[T:2 * T]), (three[T:2 * T], three[T + 1:2 * T + 1]),
                 (wide[:, :D], wide.view(-1)[2 * D:(T + 2) * D].view(T, D))):
        with pytest.raises(binding.SsdError) as e:
            forward(c, x, y)
        assert e.value.status == 3 and torch.equal(x, c["x"])


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("silu", [True, False])
def test_outputs_larger_than_the_caches(W, silu):
    """Above 256 MB outputs pass by the caches: sequences around 32 tokens (a piece), windows of each compared."""
    D = 8192
    lens = [16000, 31, 32, 33, 0, 1, 500]
    T = sum(lens)
    assert T * D * 2 > 256 << 20
    d = draw([1] * len(lens), D, W, 10 + W)
    c = cuda(d)
    c["query_start_loc"] = L.starts_of(lens).cuda()
    x = torch.empty(T, D, dtype=BF16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(W))
    y = torch.full_like(x, 7.0)
    f = forward(c, x, y, silu=silu).cpu()
    at = 0
    for b, n in enumerate(lens):
        for t in {0, n // 2, max(0, n - 40)}:
            m = min(40, n - t)
            rows = x[at + max(0, t - (W - 1)):at + t].cpu()  # ahead of the window: the sequence, then its state
            ahead = torch.cat([d["initial"][b], rows])[-(W - 1):]
            want, _, size = L.conv(x[at + t:at + t + m].cpu(), d["weight"], d["bias"], [m], ahead[None], silu)
            assert L.worst(y[at + t:at + t + m], want, size * L.CONV, L.BF16) <= 1, (b, t)
        rows = torch.cat([d["initial"][b], x[at + max(0, n - (W - 1)):at + n].cpu()])[-(W - 1):]
        assert torch.equal(f[b], rows), b
        at += n


# ------------------------------------------------------------------ backward

AHEAD = {2: 8, 3: 6, 4: 8}  # tokens of a group of the walk


def workspace(T, batch, D, W):
    return binding.ssd_causal_conv_workspace_size(
        binding.ssd_conv_problem(total_len=T, batch=batch, channels=D, width=W, max_slots=1, silu=1))


def around_pieces(W, groups, T):
    """Lengths that end on and around the ends of pieces of that many groups, T in all."""
    piece = groups * AHEAD[W] - (W - 1)
    lens = [piece, 0, piece - 1, 1, piece + 1, 2 * piece, W - 1, 2 * piece + W - 1, AHEAD[W], 2 * piece - W]
    out = []
    for n in lens:
        if sum(out) + n <= T:
            out.append(n)
    return out + [T - sum(out)]


def case_of(W, groups, D):
    """Lengths with which pieces of so many groups are the shortest that fit the card (or, with 0, none up to 16 is
    and 8 are taken); the bytes of the workspace tell."""
    blocks = (D + 255) // 256
    for T in range(50, 6000, 7):
        lens = around_pieces(W, groups or 8, T)

        def places(g):
            return T // (g * AHEAD[W] - (W - 1)) + len(lens)

        fits = [g for g in range(2, 17) if places(g) * blocks <= 2048]
        if (fits[0] if fits else 0) == groups:
            share = (places(groups or 8) + 3) // 4 * (W + 1) * D * 4
            assert workspace(T, len(lens), D, W) == (share + 255) // 256 * 256
            return lens
    raise AssertionError("no such lengths")


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("groups", [3, 4, 7, 16, 0])
@pytest.mark.parametrize("silu", [True, False])
def test_backward_in_pieces_of_many_groups(W, groups, silu):
    """Whole groups between the first and the last of a piece.  Channels are independent: those at the ends of blocks
    of 256 and a stretch in the middle are compared."""
    D = 16384
    lens = case_of(W, groups, D)
    d = draw(lens, D, W, 20 + W + groups)
    c = cuda(d)
    dx, dw, db, d_init = (torch.full_like(c[n], 7.0) for n in ("x", "weight", "bias", "initial"))
    binding.ssd_causal_conv_varlen_bwd(dx, dw, db, d_init, c["x"], c["weight"], c["bias"], c["d_y"], c["initial"],
                                       c["d_final"], c["query_start_loc"], silu=silu)
    ch = torch.tensor([0, 3, 4, 255, 256, *range(8190, 8200), D - 257, D - 256, D - 4, D - 1])
    e = {k: d[k][..., ch] for k in ("x", "d_y", "initial", "d_final")}
    want = L.conv_gradients(e["x"], d["weight"][ch], d["bias"][ch], lens, e["initial"], e["d_y"], e["d_final"], silu)
    assert L.worst(dx.cpu()[:, ch], *want[0], L.BF16) <= 1
    assert L.worst(dw.cpu()[ch], *want[1], L.U) <= 1
    assert L.worst(db.cpu()[ch], *want[2], L.U) <= 1
    assert L.worst(d_init.cpu()[..., ch], *want[3], L.BF16) <= 1
    assert bool(torch.isfinite(dx.float()).all())
