"""The norm's backward pass on the GPU for rows of extreme magnitude and for more
wide rows than there are blocks, against the definition in 64 bits within
layer_testlib's bounds."""

import pytest

torch = pytest.importorskip("torch")
import layer_testlib as L  # noqa: E402
from mamba_ssd_chunked_chunk_amd import binding  # noqa: E402

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def check(r, w, dy, dr, eps):
    rc = r.cuda()
    dx, d_residual = torch.full(r.shape, 7.0, dtype=BF16, device="cuda"), torch.full_like(rc, 7.0)
    dw = torch.full_like(w, 7.0, device="cuda")
    binding.ssd_rms_norm_bwd(dx, d_residual, dw, rc, w.cuda(), dy.cuda(), None if dr is None else dr.cuda(), eps=eps)
    d, bd, dw64, bw = L.norm_gradients(r, w, dy, dr, eps)
    assert L.worst(dx, d, bd, L.BF16) <= 1
    assert L.worst(d_residual, d, bd, torch.finfo(r.dtype).eps / 2) <= 1
    assert L.worst(dw, dw64, bw, L.U) <= 1


def draw(rows, width, kind, given, seed):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g)

    return (normal(rows, width).to(kind), 1 + 0.3 * normal(width), normal(rows, width).bfloat16(),
            normal(rows, width).to(kind) if given else None)


@pytest.mark.parametrize("width", [72, 520, 2560, 8200, 20000])
@pytest.mark.parametrize("kind,given", [(F32, True), (BF16, False)])
@pytest.mark.parametrize("power,eps", [(-55, 0.0), (-45, 0.0), (0, 0.0), (45, 0.0), (45, 1e-5), (55, 1e-5)])
def test_rows_of_every_size(width, kind, given, power, eps):
    """Rows from 2^-55 to 2^55, whose squares fp32 holds; the cube of the scale between them it does not."""
    r, w, dy, dr = draw(5, width, kind, given, 100 + width)
    # the stream's own gradient of the order of the norm's, which goes with 1 / r
    check((r.float() * 2.0 ** power).to(kind), w, dy, None if dr is None else dr * 2.0 ** -power, eps)


@pytest.mark.parametrize("width", [4104, 8200, 16392, 32768])
@pytest.mark.parametrize("rows", [257, 513, 600])
@pytest.mark.parametrize("kind,given", [(F32, False), (F32, True), (BF16, False), (BF16, True)])
def test_wide_rows_in_several_turns(width, rows, kind, given):
    """Above 4096 elements 256 blocks walk over the rows, one at a time: two and three turns, the last not whole."""
    r, w, dy, dr = draw(rows, width, kind, given, 200 + width + rows)
    check(r, w, dy, dr, 1e-5)
