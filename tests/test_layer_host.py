"""Host-side checks of the norm, the short convolution and the selective scan
that need no GPU: refusals before anything is launched, and workspace sizes."""

import ctypes
import os

import pytest

from mamba_ssd_chunked_chunk_amd import binding

NULL, SHAPE, UNSUPPORTED, WORKSPACE, MISALIGNED = 1, 2, 3, 4, 7
BASE = 1 << 20  # never dereferenced: every call below fails its host checks


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return binding.load_library()


def make(kind, base, kw):
    p = kind()
    for k, v in dict(base, **kw).items():
        setattr(p, k, v)
    return p


def norm(**kw):
    return make(binding.ssd_norm_problem, dict(rows=100, width=512, residual_dtype=1, out_format=2, eps=1e-5), kw)


def conv(**kw):
    return make(binding.ssd_conv_problem, dict(total_len=100, batch=4, channels=512, width=4, max_slots=8, silu=1), kw)


def scan(**kw):
    return make(binding.ssd_selective_problem, dict(total_len=100, batch=4, channels=512, ngroups=2, dstate=16,
                                                    max_slots=8, dt_softplus=1), kw)


# name, what makes its problem, tensor arguments, whether a workspace and its bytes follow them
ENTRIES = [("ssd_rms_norm_fwd", norm, 6, False), ("ssd_rms_norm_bwd", norm, 7, True),
           ("ssd_causal_conv_varlen_fwd_inplace", conv, 8, False), ("ssd_causal_conv_varlen_fwd", conv, 7, False),
           ("ssd_causal_conv_varlen_bwd", conv, 11, True), ("ssd_causal_conv_step_inplace", conv, 7, False),
           ("ssd_selective_scan_varlen_fwd_inplace", scan, 13, True),
           ("ssd_selective_scan_varlen_fwd", scan, 12, True), ("ssd_selective_scan_varlen_bwd", scan, 21, True),
           ("ssd_selective_scan_step_inplace", scan, 12, False)]


def call(lib, entry, p, args=None, ws=BASE, ws_bytes=1 << 50):
    name, _, n, has_ws = entry
    args = [BASE] * n if args is None else args
    tail = [ctypes.c_void_p(ws) if ws else None, ws_bytes] if has_ws else []
    return getattr(lib, name)(ctypes.byref(p) if p is not None else None,
                              *[ctypes.c_void_p(a) if a else None for a in args], *tail, None)


BAD = [(norm, dict(rows=-1), SHAPE), (norm, dict(width=0), SHAPE), (norm, dict(width=12), UNSUPPORTED),
       (norm, dict(width=32776), UNSUPPORTED), (norm, dict(x_stride=500), SHAPE), (norm, dict(x_stride=516), SHAPE),
       (norm, dict(residual_dtype=2), UNSUPPORTED), (norm, dict(out_format=3), UNSUPPORTED),
       (norm, dict(eps=-1.0), UNSUPPORTED), (norm, dict(eps=float("nan")), UNSUPPORTED),
       (norm, dict(eps=float("inf")), UNSUPPORTED), (norm, dict(rows=1 << 27), UNSUPPORTED),
       (norm, dict(rows=1 << 62), UNSUPPORTED), (norm, dict(x_stride=1 << 23), UNSUPPORTED),
       (conv, dict(total_len=-1), SHAPE), (conv, dict(total_len=1 << 31), SHAPE), (conv, dict(batch=0), SHAPE),
       (conv, dict(channels=0), SHAPE), (conv, dict(max_slots=0), SHAPE), (conv, dict(channels=12), UNSUPPORTED),
       (conv, dict(width=1), UNSUPPORTED), (conv, dict(width=5), UNSUPPORTED), (conv, dict(x_stride=504), SHAPE),
       (conv, dict(x_stride=516), SHAPE), (conv, dict(x_stride=-512), SHAPE),
       (conv, dict(channels=1 << 23), UNSUPPORTED), (conv, dict(total_len=1 << 30), UNSUPPORTED),
       (scan, dict(total_len=-1), SHAPE), (scan, dict(total_len=1 << 31), SHAPE), (scan, dict(batch=0), SHAPE),
       (scan, dict(channels=0), SHAPE), (scan, dict(ngroups=0), SHAPE), (scan, dict(ngroups=3), SHAPE),
       (scan, dict(dstate=0), SHAPE), (scan, dict(max_slots=0), SHAPE), (scan, dict(dstate=6), UNSUPPORTED),
       (scan, dict(dstate=68), UNSUPPORTED), (scan, dict(channels=24), UNSUPPORTED),
       (scan, dict(state_dtype=2), UNSUPPORTED), (scan, dict(x_stride=504), SHAPE), (scan, dict(dt_stride=516), SHAPE),
       (scan, dict(z_stride=-1024), SHAPE), (scan, dict(b_stride=31), SHAPE), (scan, dict(c_stride=33), SHAPE),
       (scan, dict(b_stride=1 << 23), UNSUPPORTED), (scan, dict(channels=1 << 23), UNSUPPORTED),
       (scan, dict(total_len=(1 << 31) - 1, batch=1 << 30), UNSUPPORTED),
       (scan, dict(total_len=1 << 30), UNSUPPORTED)]


@pytest.mark.parametrize("kind,kw,status", BAD)
def test_problems_refused(lib, kind, kw, status):
    p, n = kind(**kw), ctypes.c_size_t(0)
    for entry in ENTRIES:
        step = entry[0].endswith("step_inplace")
        if entry[1] is kind and not (step and kw.get("total_len", 0) > 1 << 30):
            assert call(lib, entry, kind(**dict(dict(total_len=kw.get("batch", 4)) if step else {}, **kw))) == status
    if kind is norm:
        assert lib.ssd_rms_norm_workspace_size(ctypes.byref(p), ctypes.byref(n)) == status
    elif kind is conv:
        assert lib.ssd_causal_conv_workspace_size(ctypes.byref(p), ctypes.byref(n)) == status
    else:
        assert lib.ssd_selective_scan_workspace_size(ctypes.byref(p), 1, ctypes.byref(n)) == status


def test_null_problems_and_sizes(lib):
    for entry in ENTRIES:
        assert call(lib, entry, None) == NULL, entry[0]
    assert lib.ssd_rms_norm_workspace_size(ctypes.byref(norm()), None) == NULL
    assert lib.ssd_causal_conv_workspace_size(ctypes.byref(conv()), None) == NULL
    assert lib.ssd_selective_scan_workspace_size(ctypes.byref(scan()), 0, None) == NULL


# tensors that may be missing, by their places in the argument list
OPTIONAL = {"ssd_rms_norm_fwd": {1}, "ssd_rms_norm_bwd": {1, 6},
            "ssd_causal_conv_varlen_fwd_inplace": {3, 6}, "ssd_causal_conv_varlen_fwd": {3, 4},
            "ssd_causal_conv_varlen_bwd": {2, 3, 6, 8, 9}, "ssd_causal_conv_step_inplace": {3, 5},
            "ssd_selective_scan_varlen_fwd_inplace": {6, 7, 8, 11}, "ssd_selective_scan_varlen_fwd": {6, 7, 8, 9},
            "ssd_selective_scan_varlen_bwd": {5, 7, 8, 14, 16, 18, 19}, "ssd_selective_scan_step_inplace": {6, 7, 8, 10}}


@pytest.mark.parametrize("entry", ENTRIES, ids=lambda e: e[0])
def test_missing_and_misaligned_tensors(lib, entry):
    """Each required pointer alone, each pointer one byte off alone (flags are bytes)."""
    name, kind, n, _ = entry
    p = kind() if kind is norm else kind(total_len=4)
    flags = {"ssd_causal_conv_varlen_fwd_inplace": 6, "ssd_causal_conv_step_inplace": 5,
             "ssd_selective_scan_varlen_fwd_inplace": 11, "ssd_selective_scan_step_inplace": 10}.get(name)
    for i in range(n):
        args = [BASE] * n
        args[i] = 0
        if i not in OPTIONAL[name]:  # (z and dz, the residual and its sum: together or not at all)
            assert call(lib, entry, p, args) == NULL, i
        if i != flags:
            args[i] = BASE + 1
            assert call(lib, entry, p, args) == MISALIGNED, i


@pytest.mark.parametrize("entry", [e for e in ENTRIES if e[3]], ids=lambda e: e[0])
def test_workspaces_refused(lib, entry):
    name, kind, _, _ = entry
    p = kind() if kind is norm else kind(total_len=3000, batch=1)  # (a scan of this length is cut)
    for ws, size in ((0, 1 << 40), (BASE, 16), (BASE + 128, 1 << 40)):
        assert call(lib, entry, p, None, ws, size) == WORKSPACE


def test_rows_of_a_step_are_its_sequences(lib):
    for entry in ENTRIES:
        if entry[0].endswith("step_inplace"):
            assert call(lib, entry, entry[1](total_len=5)) == SHAPE


def test_workspace_sizes(lib):
    """Short sequences need none in the forward pass; the backward pass of the scan keeps a state for every 8 tokens."""
    assert binding.ssd_selective_scan_workspace_size(scan(total_len=128)) == 0
    assert binding.ssd_selective_scan_workspace_size(scan(total_len=0)) == 0
    cut = binding.ssd_selective_scan_workspace_size(scan(total_len=100_000, batch=1))
    assert cut >= 512 * 17 * 4 * 2
    many = binding.ssd_selective_scan_workspace_size(scan(total_len=100_000, batch=100_000))
    # what can be cut decides, not how many sequences there are
    assert many <= 100 * cut
    back = binding.ssd_selective_scan_workspace_size(scan(total_len=100_000, batch=1), backward=True)
    assert back >= 100_000 // 8 * 512 * 16 * 4
    assert binding.ssd_rms_norm_workspace_size(norm(rows=0)) > 0  # the gradient of no rows is written too
    assert binding.ssd_causal_conv_workspace_size(conv(total_len=0)) > 0


def test_tensors_refused_by_the_binding():
    """What the binding refuses without a GPU: host tensors, shapes, a missing one."""
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64)
    with pytest.raises(ValueError, match="HIP device"):
        binding.ssd_rms_norm_fwd(torch.empty_like(x), None, None, x, None, w)
    with pytest.raises(ValueError, match="rows, width"):
        binding.ssd_rms_norm_fwd(torch.empty_like(x), None, None, x[0], None, w)
    qsl = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="HIP device"):
        binding.ssd_causal_conv_varlen_fwd(torch.empty_like(x), x, torch.zeros(64, 4), None, None,
                                           torch.zeros(1, 3, 64, dtype=torch.bfloat16), qsl)
    with pytest.raises(ValueError, match="x is required"):
        binding._hip_device(None, "x", ("T", "channels"))
    with pytest.raises(ValueError, match="HIP device"):
        binding.ssd_selective_scan_varlen_fwd(torch.empty_like(x), x, x, torch.zeros(64, 16),
                                              x.view(4, 4, 16)[:, :1], x.view(4, 4, 16)[:, :1], None, None, None, None,
                                              torch.zeros(1, 64, 16), qsl)


def test_row_strides():
    torch = pytest.importorskip("torch")
    cpu = torch.device("cpu")
    t = torch.zeros(6, 64, dtype=torch.bfloat16)
    if binding.torch is None:
        binding._import_torch()
    f = binding._row_stride
    assert f(t, "t", (6, 64), cpu, 8) == 0
    assert f(t[:, 8:40], "t", (6, 32), cpu, 8) == 64
    assert f(t[::2, :32], "t", (3, 32), cpu, 8) == 128
    assert f(t[:1, 8:40], "t", (1, 32), cpu, 8) == 0  # one row has no stride
    assert f(t[:, :32].unflatten(1, (2, 16)), "t", (6, 2, 16), cpu, 2) == 64
    bad = torch.zeros(6, 68, dtype=torch.bfloat16)[:, :64]
    assert f(bad, "t", (6, 64), cpu, 2) == 68
    for u, shape in ((bad, (6, 64)), (t[:, ::2], (6, 32)), (t[0].expand(6, 64), (6, 64)),
                     (torch.zeros(64, 6, dtype=torch.bfloat16).t(), (6, 64))):
        with pytest.raises(ValueError, match="t:"):
            f(u, "t", shape, cpu, 8)
    for u in (t.float(), t[:5], None):
        with pytest.raises((TypeError, ValueError)):
            f(u, "t", (6, 64), cpu, 8)
