"""The selective scan on the GPU where states live long: almost no decay over
sequences of many segments, so that every segment's results hang on all that lie
ahead of it.  The reference, in 64 bits on the device, takes the recurrence in
closed form: with S_t the sum of the time steps and E_t = exp(A S_t),

    h_t = E_t (h_0 + sum_{s <= t} dts_s x_s B_s / E_s)
    U_t = (E_T d_final + sum_{s >= t} E_s C_s e_s) / E_t.

All inputs but A are positive, so every sum is its own magnitude and the bounds
(layer_testlib: 4 roundings of 2^-24 a token, 1.6% of 65536 tokens) are relative."""

import pytest

torch = pytest.importorskip("torch")
import layer_testlib as L  # noqa: E402
from mamba_ssd_chunked_chunk_amd import binding  # noqa: E402

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
NAMES = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")
ROWS = ("x", "dt", "z", "B", "C")


def draw(lens, D, N, seed, decay, dtype=F32):
    """Inputs on the device; time steps about 0.05, so that A = -decay (1 to 2) forgets 0.05 decay a token."""
    g, T, b = torch.Generator("cuda").manual_seed(seed), sum(lens), len(lens)

    def uniform(lo, hi, *shape):
        return torch.empty(*shape, device="cuda").uniform_(lo, hi, generator=g)

    c = {k: uniform(0.5, 1.5, T, D).bfloat16() for k in ("x", "z", "d_y")}
    c.update({k: uniform(0.5, 1.5, T, 1, N).bfloat16() for k in ("B", "C")})
    c.update(dt=uniform(-0.5, 0.5, T, D).bfloat16(), A=-decay * uniform(1, 2, D, N), D=uniform(0.5, 1.5, D),
             dt_bias=uniform(-3.5, -2.5, D), query_start_loc=L.starts_of(lens).cuda(),
             initial=uniform(0, 1, b, D, N).to(dtype), d_final=uniform(0, 1, b, D, N).to(dtype))
    return c


def worst(got, want, bound, rounding):
    """layer_testlib's, on the device"""
    assert got.shape == want.shape, (got.shape, want.shape)
    if not got.numel():
        return 0.0
    got = got.double()
    assert bool(torch.isfinite(got).all())
    return float(((got - want).abs() / (bound + rounding * want.abs() + 2.0 ** -120)).max())


class Walk:
    """The closed form of the channels `ch` of one sequence, rows at .. at + n - 1."""

    def __init__(self, c, at, n, ch, b):
        self.x, self.z, self.dy = (c[k][at:at + n, ch].double() for k in ("x", "z", "d_y"))
        self.B, self.C = (c[k][at:at + n, :1].double() for k in ("B", "C"))  # [n, 1, N]
        self.A, self.D = c["A"][ch].double(), c["D"][ch].double()
        self.raw = c["dt"][at:at + n, ch].double() + c["dt_bias"][ch].double()
        self.dts = torch.logaddexp(self.raw, torch.zeros_like(self.raw))
        self.E = torch.exp(self.A * self.dts.cumsum(0)[..., None])
        self.h0, self.df = c["initial"][b, ch].double(), c["d_final"][b, ch].double()
        self.dx = (self.dts * self.x)[..., None] * self.B  # what a token adds to its state
        self.h = self.E * (self.h0 + (self.dx / self.E).cumsum(0))
        self.gate = self.z * torch.sigmoid(self.z)
        self.s = (self.C * self.h).sum(-1) + self.D * self.x
        self.y = self.s * self.gate
        self.final = self.h[-1] if n else self.h0

    def gradients(self):
        """{name: (gradient, magnitude)}; dB and dC: the share of these channels."""
        e = self.dy * self.gate
        ahead = (self.E * self.C * e[..., None]).flip(0).cumsum(0).flip(0)
        last = self.E[-1] * self.df if len(self.x) else self.df
        U = (last + ahead) / self.E
        uB, q = (U * self.B).sum(-1), U * (self.h - self.dx)
        qA, p, slope = (q * self.A).sum(-1), torch.sigmoid(self.z), torch.sigmoid(self.raw)
        out = dict(x=self.dts * uB + self.D * e, z=self.dy * self.s * p * (1 + self.z * (1 - p)),
                   B=(U * (self.dts * self.x)[..., None]).sum(1, keepdim=True),
                   C=(e[..., None] * self.h).sum(1, keepdim=True), A=(self.dts[..., None] * q).sum(0),
                   D=(e * self.x).sum(0), initial=self.E[0] * U[0] if len(self.x) else self.df)
        out = {n: (t, t) for n, t in out.items()}
        out["dt"] = (qA + self.x * uB) * slope, (self.x * uB - qA) * slope
        out["dt_bias"] = tuple(t.sum(0) for t in out["dt"])
        return out


def spans(c, lens):
    """(sequence, its first row, its tokens, channels): a closed form of each is at most 2^26 numbers"""
    D, N = c["A"].shape
    at = 0
    for b, n in enumerate(lens):
        width = max(1, min(D, (1 << 26) // (max(n, 1) * N)))
        for k in range(0, D, width):
            yield b, at, n, slice(k, min(D, k + width))
        at += n


def check_forward(c, lens):
    """Forward, twice: the same bits, and the closed form's numbers."""
    outs = []
    for _ in range(2):
        y, f = torch.empty_like(c["x"]), torch.empty_like(c["initial"])
        binding.ssd_selective_scan_varlen_fwd(y, *[c[n] for n in NAMES], c["initial"], f, c["query_start_loc"])
        outs.append((y, f))
    (y, f), again = outs
    for b, at, n, ch in spans(c, lens):
        w, e = Walk(c, at, n, ch, b), L.scan_roundings([n])
        assert worst(y[at:at + n, ch], w.y, w.y * e, L.BF16) <= 1, (b, ch)
        assert worst(f[b, ch], w.final, w.final * e, torch.finfo(f.dtype).eps / 2) <= 1, (b, ch)
    assert torch.equal(y, again[0]) and torch.equal(f, again[1])


def check_backward(c, lens):
    out = {n: torch.full_like(c[n], 7.0) for n in NAMES + ("initial",)}
    binding.ssd_selective_scan_varlen_bwd(*out.values(), *[c[n] for n in NAMES], c["d_y"], c["initial"], c["d_final"],
                                          c["query_start_loc"])
    sums = {n: torch.zeros(2, *c[n].shape, dtype=torch.float64, device="cuda") for n in ("A", "B", "C", "D", "dt_bias")}
    # layer_testlib's count of the gradients' roundings
    e = 2 * L.scan_roundings(lens) + (64 + sum(lens) / 8) * L.U
    for b, at, n, ch in spans(c, lens):
        for name, (t, size) in Walk(c, at, n, ch, b).gradients().items():
            if name in ("B", "C"):
                sums[name][:, at:at + n] += torch.stack([t, size])
            elif name in sums:
                sums[name][:, ch] += torch.stack([t, size])
            else:
                got = out[name][b, ch] if name == "initial" else out[name][at:at + n, ch]
                assert worst(got, t, size * e, torch.finfo(got.dtype).eps / 2) <= 1, (name, b, ch)
    for name, (t, size) in sums.items():
        assert worst(out[name], t, size * e, torch.finfo(out[name].dtype).eps / 2) <= 1, name


def segments(T, batch, D, N):
    """Places of segments of cut sequences, from the bytes of their states and sums of steps (a multiple of 256 each)"""
    p = binding.ssd_selective_problem(total_len=T, batch=batch, channels=D, ngroups=1, dstate=N, max_slots=batch,
                                      dt_softplus=1, state_dtype=binding.STATE_F32)
    assert D % 64 == 0
    return binding.ssd_selective_scan_workspace_size(p) // (D * (N + 1) * 4)


# workgroups of a compute unit, by their LDS (a token's share of 64 channels by wavefronts of 4 states): 26.6 KB with 16
# states, 12.8 KB with 4
@pytest.mark.parametrize("N,resident", [(16, 6 * 256), (4, 12 * 256)])
@pytest.mark.parametrize("decay", [0.0, 2e-4, 2e-3])
def test_more_segments_than_fit_the_card(N, resident, decay):
    """The last segments begin when the first have ended, and chain what those left before."""
    T, D = 65536, 2048
    assert (segments(T, 1, D, N) - 2) * (D // 64) > resident
    check_forward(draw([T], D, N, 100 + N, decay), [T])


def test_more_segments_than_fit_the_card_bf16():
    check_forward(draw([50001], 2048, 8, 120, 2e-4, BF16), [50001])


LISTED = [20 + i for i in range(30)]
LISTED[7], LISTED[21] = 30011, 20000
MANY = [i % 29 for i in range(300)]
MANY[0], MANY[150], MANY[299] = 20001, 30000, 9999


@pytest.mark.parametrize("lens", [LISTED, MANY], ids=["listed", "many"])
@pytest.mark.parametrize("decay", [0.0, 2e-4])
def test_long_sequences_among_others(lens, decay):
    """Numbered without gaps, and by places with gaps."""
    D, N = 1024, 8
    assert segments(sum(lens), len(lens), D, N) > 20
    check_forward(draw(lens, D, N, 130 + len(lens), decay), lens)


@pytest.mark.parametrize("N", [4, 16])
@pytest.mark.parametrize("decay", [0.0, 2e-4])
def test_backward_of_many_segments(N, decay):
    check_backward(draw([65536], 1024, N, 140 + N, decay), [65536])


@pytest.mark.parametrize("lens", [LISTED, MANY], ids=["listed", "many"])
def test_backward_of_long_sequences_among_others(lens):
    check_backward(draw(lens, 256, 8, 150 + len(lens), 2e-4), lens)


def test_two_long_sequences_at_once():
    """Two calls side by side, which share the card's places, give what each gives alone."""
    problems = [draw([30000], 1024, 16, 160 + i, 2e-4) for i in range(2)]
    outs = [[(torch.empty_like(c["x"]), torch.empty_like(c["initial"])) for c in problems] for _ in range(2)]

    def call(c, out):
        binding.ssd_selective_scan_varlen_fwd(out[0], *[c[n] for n in NAMES], c["initial"], out[1],
                                              c["query_start_loc"])

    for c, out in zip(problems, outs[0]):
        call(c, out)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in problems]
    for _ in range(3):
        for c, out, s in zip(problems, outs[1], streams):
            with torch.cuda.stream(s):
                call(c, out)
        torch.cuda.synchronize()
        for a, b in zip(*outs):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("N", [4, 8, 12, 20, 32, 36, 64])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_cut_sequences_of_every_state_size(N, dtype):
    """... whose workgroups have 1 to 16 wavefronts, and one or two groups of states a wavefront backwards."""
    lens, D = [35, 900, 0, 450, 1, 500], 136
    c = draw(lens, D, N, 170 + N, 2e-3, dtype)
    check_forward(c, lens)
    check_backward(c, lens)


@pytest.mark.parametrize("N", [4, 12, 20, 32, 36, 64])
@pytest.mark.parametrize("softplus", [True, False])
def test_cut_sequences_of_groups(N, softplus):
    """The same of two groups, random signs and decays that forget, against the recurrence token by token."""
    from test_selective_scan_gpu import check_backward, check_prompt
    check_prompt([300, 35, 0, 420], 144, 2, N, 180 + N, softplus=softplus)
    check_backward([150, 35, 0, 200], 144, 2, N, 190 + N, softplus=softplus, tail=3)
