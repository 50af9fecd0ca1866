"""Host-side limits of the norm, the short convolution and the selective scan
that need no GPU: refusals that come before anything is launched."""

import ctypes
import os

import pytest

from mamba_ssd_chunked_chunk_amd import binding

OK, UNSUPPORTED = 0, 3


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return binding.load_library()


@pytest.mark.parametrize("N,waves", [(4, 2), (8, 2), (16, 4), (32, 8), (64, 16)])
def test_scan_threads_fit_32_bits(lib, N, waves):
    """`waves`: the most wavefronts of a workgroup of the backward pass.  With 4 states its gradients take two, the
    walk for states one: sequences that only the latter could launch were refused by the second launch, as a HIP error."""
    def status(batch, backward):
        p = binding.ssd_selective_problem(total_len=0, batch=batch, channels=64, ngroups=1, dstate=N, max_slots=1,
                                          dt_softplus=1, state_dtype=binding.STATE_F32)
        return lib.ssd_selective_scan_workspace_size(ctypes.byref(p), backward, ctypes.byref(ctypes.c_size_t(0)))

    # one workgroup of 64 `waves` threads a sequence without tokens, fewer than 2^32 in all
    most = ((1 << 32) - 1) // (64 * waves)
    assert status(most, 1) == OK and status(most + 1, 1) == UNSUPPORTED
    forward = 1 if N == 4 else waves
    most = ((1 << 32) - 1) // (64 * forward)
    assert status(most, 0) == OK and status(most + 1, 0) == UNSUPPORTED


def conv(**kw):
    p = binding.ssd_conv_problem(total_len=100, batch=2, channels=64, width=4, max_slots=2, silu=1)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


X, FAR = 1 << 20, 1 << 30  # addresses, never dereferenced
ROW = 64 * 2
# y, stride of x in elements: 100 rows of y share memory with as many of x from X on
MEET = [(X, 0), (X + 16, 0), (X - 16, 0), (X + 100 * ROW - 16, 0), (X - 100 * ROW + 16, 0), (X + ROW, 128),
        (X + 99 * 2 * ROW, 128), (X + 2 * ROW + 16, 64 * 102), (X + ROW - 16, 64 * 102), (X - 99 * ROW, 64 * 102),
        (X + 99 * 102 * ROW + ROW - 16, 64 * 102)]


@pytest.mark.parametrize("y,stride", MEET)
def test_convolution_refuses_outputs_among_its_inputs(lib, y, stride):
    """A piece reads up to width - 1 rows of the piece ahead of it (and behind it, in the backward pass)."""
    def at(*args):
        return [ctypes.c_void_p(a) for a in args]

    p, ws = ctypes.byref(conv(x_stride=stride)), (ctypes.c_void_p(FAR), 1 << 40, None)
    assert lib.ssd_causal_conv_varlen_fwd(p, *at(y, X, FAR, FAR, FAR, FAR, FAR), None) == UNSUPPORTED
    assert lib.ssd_causal_conv_varlen_fwd_inplace(p, *at(y, X, FAR, FAR, FAR, FAR, FAR, FAR), None) == UNSUPPORTED
    assert lib.ssd_causal_conv_varlen_bwd(p, *at(y, FAR, FAR, FAR, X, FAR, FAR, FAR, FAR, FAR, FAR), *ws) == UNSUPPORTED
    if stride == 0:  # the gradient of the outputs, which is dense
        assert lib.ssd_causal_conv_varlen_bwd(p, *at(y, FAR, FAR, FAR, FAR, FAR, FAR, X, FAR, FAR, FAR),
                                              *ws) == UNSUPPORTED
