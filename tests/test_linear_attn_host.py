"""Host-side checks of linear attention and of the 8-bit state cache that need
no GPU: refusals before anything is launched, and the workspace sizes."""

import ctypes

import pytest

from mamba_ssd_chunked_chunk_amd import binding

NULL, SHAPE, UNSUPPORTED, WORKSPACE, MISALIGNED = 1, 2, 3, 4, 7
BASE = 1 << 20  # never dereferenced: every call below fails its host checks


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(binding.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return binding.load_library()


def prob(**kw):
    base = dict(total_len=100, batch=4, nheads=8, ngroups=2, key_dim=64, value_dim=128, max_slots=8)
    base.update(kw)
    return binding.make_linear_attn_problem(**base)


BAD = [(dict(total_len=-1), SHAPE), (dict(total_len=1 << 31), SHAPE), (dict(batch=0), SHAPE), (dict(nheads=0), SHAPE),
       (dict(ngroups=3), SHAPE), (dict(ngroups=0), SHAPE), (dict(key_dim=0), SHAPE), (dict(value_dim=-8), SHAPE),
       (dict(max_slots=0), SHAPE), (dict(key_dim=60), UNSUPPORTED), (dict(value_dim=4), UNSUPPORTED),
       (dict(key_dim=264), UNSUPPORTED), (dict(value_dim=512), UNSUPPORTED), (dict(state_dtype=2), UNSUPPORTED),
       (dict(scale=float("nan")), UNSUPPORTED), (dict(scale=float("inf")), UNSUPPORTED),
       (dict(q_stride=120), SHAPE), (dict(k_stride=132), SHAPE), (dict(v_stride=1000), SHAPE),
       (dict(q_stride=-128), SHAPE), (dict(batch=1 << 30, nheads=8), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", BAD)
def test_problems_refused(lib, kw, status):
    n = ctypes.c_size_t(0)
    p = prob(**kw)
    for backward in (0, 1):
        assert lib.ssd_linear_attn_workspace_size(ctypes.byref(p), backward, ctypes.byref(n)) == status
    V = [ctypes.c_void_p(BASE)] * 13
    assert lib.ssd_linear_attn_varlen_fwd_inplace(ctypes.byref(p), *V[:10], 1 << 40, None) == status
    assert lib.ssd_linear_attn_varlen_fwd(ctypes.byref(p), *V[:9], 1 << 40, None) == status
    assert lib.ssd_linear_attn_varlen_bwd(ctypes.byref(p), *V[:13], 1 << 40, None) == status
    assert lib.ssd_linear_attn_step_inplace(ctypes.byref(p), *V[:8], None) == status


@pytest.mark.parametrize("kw", [dict(), dict(key_dim=256, value_dim=8), dict(q_stride=128, k_stride=1000 * 8),
                                dict(total_len=0), dict(scale=0.0), dict(scale=-2.0)])
def test_problems_accepted(lib, kw):
    assert binding.ssd_linear_attn_workspace_size(prob(**kw)) >= 0
    assert binding.ssd_linear_attn_workspace_size(prob(**kw), backward=True) >= 0


def test_more_threads_than_a_launch_holds(lib):
    """A grid's threads fit 32 bits (256 or 512 a workgroup): refused on the host beyond, workspace or not."""
    n = ctypes.c_size_t(0)
    V = [ctypes.c_void_p(BASE)] * 13

    def size(p, backward=0):
        return lib.ssd_linear_attn_workspace_size(ctypes.byref(p), backward, ctypes.byref(n))

    few = dict(nheads=16, ngroups=16, key_dim=8, value_dim=8)
    ok, bad = (prob(total_len=b, batch=b, **few) for b in ((1 << 19), (1 << 20)))
    assert size(ok) == 0
    assert size(bad) == UNSUPPORTED and size(bad, 1) == UNSUPPORTED
    assert lib.ssd_linear_attn_varlen_fwd_inplace(ctypes.byref(bad), *V[:10], 1 << 60, None) == UNSUPPORTED
    assert lib.ssd_linear_attn_varlen_fwd(ctypes.byref(bad), *V[:9], 1 << 60, None) == UNSUPPORTED
    assert lib.ssd_linear_attn_varlen_bwd(ctypes.byref(bad), *V[:13], 1 << 60, None) == UNSUPPORTED
    assert lib.ssd_linear_attn_step_inplace(ctypes.byref(bad), *V[:8], None) == UNSUPPORTED
    # 512 threads, and four blocks of channels, of the widest heads
    wide = dict(nheads=16, ngroups=16, key_dim=256, value_dim=256)
    assert size(prob(total_len=257 << 19, batch=1 << 19, **wide)) == UNSUPPORTED
    # the sums of shared heads: one thread for 8 channels of dq
    long = dict(total_len=(1 << 31) - 1, batch=1, nheads=2, ngroups=1, value_dim=64)
    assert size(prob(key_dim=8, **long), 1) == 0
    assert size(prob(key_dim=16, **long), 1) == UNSUPPORTED and size(prob(key_dim=16, **long)) == 0


def test_more_threads_than_a_state_cache_launch_holds(lib):
    a = [ctypes.c_void_p(BASE)] * 5
    for kw in (dict(count=1 << 18, nheads=1 << 4, head_dim=64, dstate=256),
               dict(count=1 << 18, nheads=1 << 8, head_dim=64, dstate=8)):
        p = cache(max_slots=1 << 30, max_entries=1 << 30, **kw)
        assert lib.ssd_state_quantize(ctypes.byref(p), *a, None) == UNSUPPORTED
        assert lib.ssd_state_dequantize(ctypes.byref(p), *a, None) == UNSUPPORTED


def test_workspace_size_arguments(lib):
    n = ctypes.c_size_t(0)
    assert lib.ssd_linear_attn_workspace_size(None, 0, ctypes.byref(n)) == NULL
    assert lib.ssd_linear_attn_workspace_size(ctypes.byref(prob()), 0, None) == NULL


def _each(call, count, required, aligned16, aligned4):
    """`call` with fake pointers, each required one NULL and each one misaligned in turn."""
    for i in required:
        a = [ctypes.c_void_p(BASE)] * count
        a[i] = None
        assert call(a) == NULL, i
    for i, off in [(i, 8) for i in aligned16] + [(i, 2) for i in aligned4]:
        a = [ctypes.c_void_p(BASE)] * count
        a[i] = ctypes.c_void_p(BASE + off)
        assert call(a) == MISALIGNED, i


def test_forward_in_place_refusals(lib):
    p = prob()
    # o q k v log_decay pool qsl has_init cache_idx workspace
    _each(lambda a: lib.ssd_linear_attn_varlen_fwd_inplace(ctypes.byref(p), *a, 1 << 40, None), 10,
          (0, 1, 2, 3, 4, 5, 6, 8), (0, 1, 2, 3, 5), (4, 6, 8))
    assert lib.ssd_linear_attn_varlen_fwd_inplace(None, *[ctypes.c_void_p(BASE)] * 10, 0, None) == NULL


def test_forward_separate_refusals(lib):
    p = prob()
    # o q k v log_decay initial final qsl workspace
    _each(lambda a: lib.ssd_linear_attn_varlen_fwd(ctypes.byref(p), *a, 1 << 40, None), 9,
          (0, 1, 2, 3, 4, 6, 7), (0, 1, 2, 3, 5, 6), (4, 7))
    assert lib.ssd_linear_attn_varlen_fwd(None, *[ctypes.c_void_p(BASE)] * 9, 0, None) == NULL


def test_backward_refusals(lib):
    p = prob()
    # dq dk dv d_initial q k v d_o log_decay initial d_final qsl workspace
    _each(lambda a: lib.ssd_linear_attn_varlen_bwd(ctypes.byref(p), *a, 1 << 40, None), 13,
          (0, 1, 2, 4, 5, 6, 7, 8, 11), (0, 1, 2, 3, 4, 5, 6, 7, 9, 10), (8, 11))
    assert lib.ssd_linear_attn_varlen_bwd(None, *[ctypes.c_void_p(BASE)] * 13, 0, None) == NULL


def test_backward_refuses_states_it_would_overwrite(lib):
    """dq reads initial_states in the launch in which dv writes d_initial."""
    a = [ctypes.c_void_p(BASE + i * 4096) for i in range(13)]
    a[3] = a[9]  # d_initial, initial_states
    assert lib.ssd_linear_attn_varlen_bwd(ctypes.byref(prob()), *a, 1 << 40, None) == UNSUPPORTED


def test_step_refusals(lib):
    p = prob(total_len=4)
    # o q k v log_decay pool has_init cache_idx
    _each(lambda a: lib.ssd_linear_attn_step_inplace(ctypes.byref(p), *a, None), 8,
          (0, 1, 2, 3, 4, 5, 7), (1, 2, 5), (4, 7))
    a = [ctypes.c_void_p(BASE)] * 8
    assert lib.ssd_linear_attn_step_inplace(ctypes.byref(prob(total_len=5)), *a, None) == SHAPE
    assert lib.ssd_linear_attn_step_inplace(None, *a, None) == NULL


def test_workspace_refusals(lib):
    """Each entry point that needs a workspace refuses none, one too small and one misaligned."""
    seen = 0
    for kw in (dict(), dict(total_len=100_000)):
        p = prob(**kw)
        for backward, name, n in ((0, "ssd_linear_attn_varlen_fwd_inplace", 10), (0, "ssd_linear_attn_varlen_fwd", 9),
                                  (1, "ssd_linear_attn_varlen_bwd", 13)):
            need = binding.ssd_linear_attn_workspace_size(p, backward)
            if need == 0:
                continue
            seen += 1
            a = [ctypes.c_void_p(BASE)] * n
            f = getattr(lib, name)
            assert f(ctypes.byref(p), *a, need - 1, None) == WORKSPACE
            assert f(ctypes.byref(p), *a[:-1], None, need, None) == WORKSPACE
            assert f(ctypes.byref(p), *a[:-1], ctypes.c_void_p(BASE + 16), need, None) == WORKSPACE
    assert seen


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("total,batch,nheads,ngroups,K,V", [
    (4096, 4096, 128, 128, 128, 64), (1536, 512, 128, 128, 128, 64), (4096, 1024, 64, 64, 128, 128),
    (12000, 12000, 16, 16, 256, 16), (100_000, 512, 128, 128, 128, 64), (43898, 32, 128, 128, 128, 64),
    (65536, 1, 16, 16, 128, 128), (1000, 3, 2, 2, 64, 64)])
def test_workspace_is_for_sequences_that_can_be_cut(lib, total, batch, nheads, ngroups, K, V, backward):
    """Only sequences of more than a segment (128 tokens at least) leave states in the workspace: two for each 128
    tokens at most (whole segments', and one more for a sequence's end), however many sequences there are."""
    need = binding.ssd_linear_attn_workspace_size(
        prob(total_len=total, batch=batch, nheads=nheads, ngroups=ngroups, key_dim=K, value_dim=V), backward)

    def pad(d):
        return 64 if d <= 64 else 128 if d <= 128 else 256

    state = nheads * 4 * (pad(max(K, V)) ** 2 * 3 if backward else pad(K) * pad(V))
    assert need <= 2 * (total // 128) * state


def cache(**kw):
    base = dict(count=2, nheads=4, head_dim=64, dstate=128, max_slots=8, max_entries=5, state_dtype=0, code_format=0)
    base.update(kw)
    return binding.ssd_state_cache_problem(*base.values())


@pytest.mark.parametrize("kw,status", [
    (dict(count=-1), SHAPE), (dict(nheads=0), SHAPE), (dict(head_dim=0), SHAPE), (dict(dstate=0), SHAPE),
    (dict(max_slots=0), SHAPE), (dict(max_entries=0), SHAPE), (dict(dstate=100), UNSUPPORTED),
    (dict(dstate=264), UNSUPPORTED), (dict(state_dtype=2), UNSUPPORTED), (dict(code_format=2), UNSUPPORTED),
    (dict(code_format=-1), UNSUPPORTED), (dict(count=1 << 30, nheads=1 << 10), UNSUPPORTED)])
def test_cache_problems_refused(lib, kw, status):
    p = cache(**kw)
    a = [ctypes.c_void_p(BASE)] * 5
    assert lib.ssd_state_quantize(ctypes.byref(p), *a, None) == status
    assert lib.ssd_state_dequantize(ctypes.byref(p), *a, None) == status


def test_cache_pointer_refusals(lib):
    p = cache()
    # codes scales pool pool_idx entry_idx
    _each(lambda a: lib.ssd_state_quantize(ctypes.byref(p), *a, None), 5, range(5), (2,), (1, 3, 4))
    # pool codes scales pool_idx entry_idx
    _each(lambda a: lib.ssd_state_dequantize(ctypes.byref(p), *a, None), 5, range(5), (0,), (2, 3, 4))
    a = [ctypes.c_void_p(BASE)] * 5
    a[0] = ctypes.c_void_p(BASE + 4)  # codes: 8 bytes
    assert lib.ssd_state_quantize(ctypes.byref(p), *a, None) == MISALIGNED
    assert lib.ssd_state_quantize(None, *a, None) == NULL
    # nothing to move: nothing is launched, and no pointer is needed
    assert lib.ssd_state_quantize(ctypes.byref(cache(count=0)), *[None] * 5, None) == 0
    assert lib.ssd_state_dequantize(ctypes.byref(cache(count=0)), *[None] * 5, None) == 0


def test_workspaces_refused_by_the_binding():
    """A workspace has to hold its bytes itself: an expanded byte has their number, not their memory."""
    torch = pytest.importorskip("torch")
    binding._import_torch()
    cpu, byte = torch.device("cpu"), torch.zeros(1, dtype=torch.uint8)

    def call(*_):
        raise AssertionError("launched")

    for bad in (byte.expand(512), byte.expand(512).view(8, 64), torch.zeros(1024, dtype=torch.uint8)[::2],
                torch.zeros(256, dtype=torch.uint8), torch.zeros(512, dtype=torch.int8)):
        with pytest.raises(ValueError, match="workspace"):
            binding._run("x", cpu, None, 512, bad, call)


def test_sizes_that_only_the_backward_pass_refuses():
    """A call of the binding goes by its own limits: single tokens by the step's, prompts by the forward pass's."""
    wide = (12000, 12000, 128, 8, 256, 16, 12000, binding.STATE_BF16, 1.0)
    long = ((1 << 31) - 1, 1, 2, 1, 16, 64, 1, binding.STATE_F32, 1.0)
    for sizes in (wide, long):
        assert binding._linear_attn_sizes(None, *sizes)[1] == 0
        assert binding._linear_attn_sizes(False, *sizes)[1] > 0
        with pytest.raises(binding.SsdError):
            binding._linear_attn_sizes(True, *sizes)


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    bf = torch.bfloat16
    q = torch.zeros(4, 2, 64, dtype=bf)
    v = torch.zeros(4, 4, 64, dtype=bf)
    ld, pool = torch.zeros(4), torch.zeros(4, 4, 64, 64)
    idx = torch.arange(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="HIP device"):
        binding.ssd_linear_attn_step_inplace(v.clone(), q, q, v, ld, pool, None, idx)
    with pytest.raises(ValueError, match="HIP device"):
        binding.ssd_state_quantize(torch.zeros(4, 4, 64, 64, dtype=torch.int8), torch.zeros(4, 4, 64), pool, idx, idx)
    with pytest.raises(TypeError, match="states"):
        binding.ssd_linear_attn_step_inplace(v.clone(), q, q, v, ld, pool.half(), None, idx)
    with pytest.raises(ValueError, match="must be"):
        binding.ssd_linear_attn_step_inplace(v.clone(), q[0], q, v, ld, pool, None, idx)
    check = lambda t: binding._token_stride(t, "q", (4, 2, 64), torch.device("cpu"))  # noqa: E731
    assert check(q) == 0
    wide = torch.zeros(4, 200, dtype=bf)
    assert check(wide[:, 8:136].view(4, 2, 64)) == 200
    for bad in (torch.zeros(4, 2, 65, dtype=bf)[..., :64], torch.zeros(4, 3, 64, dtype=bf)[:, ::2],
                torch.zeros(4, 130, dtype=bf)[:, :128].view(4, 2, 64), torch.zeros(1, 2, 64, dtype=bf).expand(4, 2, 64),
                q[:3]):
        with pytest.raises(ValueError):
            check(bad)
    with pytest.raises(TypeError):
        check(q.float())
