"""Host-side limits of the norm, the short convolution and the selective scan
that need no GPU: refusals that come before anything is launched."""

import ctypes
import os

import pytest

from mamba_ssd_chunked_chunk_amd import binding

OK, UNSUPPORTED, WORKSPACE = 0, 3, 4


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
