"""Further forms of the short convolution on the GPU, against the definition in
64 bits within layer_testlib's bounds: outputs beside their inputs in one buffer."""

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
