"""Token statistics of logits (log-probs, entropy, alternatives) and their
gradient against float64.

Tolerances, fixed before the first run (u = 2^-24, all logarithms natural, D =
sum p |z - m| / T of the row): a weight's exponent carries the rounding of the
difference, of its factor (three: log2(e), 1 / T, the product) and the
exponential 2^-22, so the sum S is off by delta = (4 D + 8 + V / 512 + 20) u
relatively, V / 512 being the additions of one lane of a thread.  L = ln S is off by delta + u
|L|; the log-prob adds three roundings of (z_y - m) / T and two of L.  The
entropy's second term E / S has two sums and a reference up to 8 ln2 away:
(delta + 4 u)(2 + 2 D + 8).  Alternatives and the maximum are exact.
A gradient p (A + B ln p): ln p is off by eps = u (4 |z - m| / T + 3 L + 8) + delta (L
is the forward's), so an element by 2 eps p (|g| + |h| (|ln p| + H + 1)) / T and
what the entropy's error brings, then half a step of its type."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24
LOWEST = {F32: torch.finfo(F32).min, BF16: torch.finfo(BF16).min}


def g():
    from vocab_wide_logprob_gb300 import _native
    return _native


def gen(seed):
    r = torch.Generator(device="cuda")
    r.manual_seed(seed)
    return r


def warmth(T):
    return torch.where(T < 1e-6, torch.ones_like(T), T).double()


class Ref:
    """The statistics of one sequence's rows [n, V] in float64."""

    def __init__(self, z, T=1.0, lanes=512):
        z = z.double()
        self.T = float(T)
        self.m = z.amax(-1, keepdim=True)
        x = (z - self.m) / self.T
        w = x.exp()
        S = w.sum(-1, keepdim=True)
        self.L = S.log()
        self.lp = x - self.L
        self.p = w / S
        px = torch.where(self.p > 0, self.p * x, 0.0)
        self.D = -px.sum(-1, keepdim=True)
        self.H = self.L + self.D
        self.x = x
        self.delta = (4 * self.D + 28 + z.shape[-1] / lanes) * U


def order(z, top):
    return z.double().sort(dim=-1, descending=True, stable=True).indices[..., :top]


def check(z, tokens, out, top=0, lens=None, T=None, lanes=512):
    N, R, V = z.shape
    for i in range(N):
        n = R if lens is None else max(0, min(R, int(lens[i])))
        for k in ("logp", "entropy", "norm") + (("top_logp",) if top else ()):
            assert (out[k][i, n:] == 0).all(), k
        if top:
            assert (out["top_tokens"][i, n:] == -1).all()
        if n == 0:
            continue
        r = Ref(z[i, :n], 1.0 if T is None else warmth(T[i:i + 1]).item(), lanes)
        y = tokens[i, :n].unsqueeze(-1)

        def near(have, lp, at):
            tol = r.delta + U * (3 * r.x.gather(-1, at).abs() + 2 * r.L.abs() + lp.abs())
            same = have.double() == lp  # (-inf of a banned token)
            assert (same | ((have.double() - lp).abs() <= tol)).all(), (have.double() - lp).abs().max()

        near(out["logp"][i, :n].unsqueeze(-1), r.lp.gather(-1, y), y)
        tolH = (r.delta + 4 * U) * (10 + 2 * r.D)
        assert ((out["entropy"][i, :n].unsqueeze(-1).double() - r.H).abs() <= tolH).all()
        assert (out["norm"][i, :n, :1].double() == r.m).all()
        assert ((out["norm"][i, :n, 1:].double() - r.L).abs() <= r.delta + U * r.L.abs()).all()
        if top:
            best = order(z[i, :n], top)
            assert torch.equal(out["top_tokens"][i, :n], best)
            near(out["top_logp"][i, :n], r.lp.gather(-1, best), best)


def draw(N, R, V, dt, seed, spread=3.0):
    r = gen(seed)
    z = (torch.randn(N, R, V, generator=r, device="cuda") * spread).to(dt)
    return z, torch.randint(0, V, (N, R), generator=r, device="cuda")


# (short rows in numbers take a warp each: the last ones, and those below 1 KB)
SHAPES = [(1, 1, 1), (1, 1, 5), (2, 3, 7), (3, 2, 100), (2, 2, 511), (2, 2, 512), (2, 2, 513),
          (1, 3, 1000), (2, 1, 2048), (2, 2, 8191), (3, 1, 8193), (1, 2, 32003), (1, 1, 151936),
          (2, 1, 200001), (5, 7, 4099), (64, 12, 1024), (40, 33, 999),
          (20, 70, 4096), (50, 60, 2047), (31, 100, 8190)]


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("top", [0, 1, 5, 32])
def test_stats(shape, dt, top):
    n = g()
    z, y = draw(*shape, dt, 1)
    k = min(top, shape[2])
    out = n.grpo_token_stats(z, y, top=k)
    assert n.grpo_check_error(out["workspace"]) == 0
    assert ("top_tokens" in out) == (k > 0)
    check(z, y, out, k)


@pytest.mark.parametrize("shape, dt, top", [((8, 510, 16411), F32, 0), ((16, 300, 8191), BF16, 5),
                                            ((5, 900, 31999), BF16, 0), ((9, 150, 8003), F32, 9)],
                         ids=str)
def test_many_rows(shape, dt, top):
    """Rows enough that longer ones take a warp each, whose lanes add V / 64 numbers: every
    97th against float64, and all of them bit for bit with a second call's."""
    n = g()
    z, y = draw(*shape, dt, 3)
    out = n.grpo_token_stats(z, y, top=top)
    assert n.grpo_check_error(out["workspace"]) == 0
    some = torch.arange(0, shape[0] * shape[1], 97, device="cuda")
    flat = {k: v.flatten(0, 1)[some][None] for k, v in out.items() if k != "workspace"}
    check(z.flatten(0, 1)[some][None], y.flatten()[some][None], flat, top, lanes=64)
    again = n.grpo_token_stats(z, y, top=top)
    for k in flat:
        assert torch.equal(out[k], again[k]), k


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_views_of_wider_buffers(dt):
    """Rows of [N, P+C, V] logits, rows of a padded vocabulary, one element off."""
    n = g()
    N, P, C, V = 3, 4, 9, 1003
    r = gen(2)
    for pad, shift in ((0, 0), (5, 0), (13, 1), (1, 3)):
        buf = (torch.randn(N * (P + C) * (V + pad) + shift, generator=r, device="cuda") * 3).to(dt)
        z = buf[shift:].view(N, P + C, V + pad)[:, P - 1:-1, :V]
        ids = torch.randint(0, V, (N, P + C), generator=r, device="cuda")
        lens = torch.tensor([9, 0, 4], dtype=torch.int32, device="cuda")
        out = n.grpo_token_stats(z, ids[:, P:], lens, top=6)
        check(z, ids[:, P:], out, 6, lens)
        # one row per sequence, the last
        out = n.grpo_token_stats(z[:, -1:], ids[:, -1:], top=6)
        check(z[:, -1:], ids[:, -1:], out, 6)


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_time_major_rows(dt):
    """[R, N, V] logits and [R, N] tokens, transposed; the gradient in the same layout."""
    n = g()
    N, R, V = 5, 7, 2001
    z, y = draw(R, N, V, dt, 40)
    z, y = z.transpose(0, 1), y.t()
    lens = torch.tensor([7, 0, 3, 1, 7], dtype=torch.int32, device="cuda")
    out = n.grpo_token_stats(z, y, lens, top=5)
    check(z, y, out, 5, lens)
    gl, gh = (torch.randn(N, R, generator=gen(s), device="cuda") for s in (41, 42))
    dz = torch.empty(R, N, V, dtype=dt, device="cuda").transpose(0, 1)
    n.grpo_token_stats_bwd(z, y, out["norm"], out["entropy"], gl, gh, lens, out=dz)
    check_grad(z, y, gl, gh, dz, lens)
    # one row for all sequences (read only)
    one = z[:1].expand(N, R, V)
    out = n.grpo_token_stats(one, y, lens)
    check(one, y, out, 0, lens)
    with pytest.raises(n.GrpoError):
        n.grpo_token_stats_bwd(z, y, out["norm"], out["entropy"], gl, out=dz[:1].expand(N, R, V))


@pytest.mark.parametrize("V", [100_000_007, 50_331_648])
def test_a_long_row(V):
    """Vectors and batches far beyond a vocabulary's."""
    n = g()
    z, y = draw(1, 2, V, BF16, 43)
    z[0, 1, V - 1] = 30.0
    out = n.grpo_token_stats(z, y, top=11)
    check(z, y, out, 11)
    gl = torch.ones(1, 2, device="cuda")
    dz = n.grpo_token_stats_bwd(z, y, out["norm"], out["entropy"], gl, gl)
    for j in range(2):
        check_grad(z[:, j:j + 1], y[:, j:j + 1], gl[:, :1], gl[:, :1], dz[:, j:j + 1])


def test_lengths_and_what_lies_behind():
    n = g()
    z, y = draw(5, 6, 3001, BF16, 3)
    lens = torch.tensor([0, 1, 6, -2, 9], dtype=torch.int32, device="cuda")
    for i, L in enumerate((0, 1, 6, 0, 6)):
        z[i, L:] = float("nan")
        y[i, L:] = -5
    out = n.grpo_token_stats(z, y, lens, top=3)
    assert n.grpo_check_error(out["workspace"]) == 7  # clamped lengths
    check(z, y, out, 3, lens)
    lens = lens.clamp(0, 6)
    out = n.grpo_token_stats(z, y, lens, top=3, out=out)
    assert n.grpo_check_error(out["workspace"]) == 0
    check(z, y, out, 3, lens)


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_temperatures(dt):
    n = g()
    z, y = draw(9, 2, 5003, dt, 4)
    T = torch.tensor([1.0, 0.0, 1e-7, 0.3, 5.0, 100.0, 1e-5, -0.0, 1e6], device="cuda")
    out = n.grpo_token_stats(z, y, temperature=T, top=20)
    assert n.grpo_check_error(out["workspace"]) == 0
    check(z, y, out, 20, T=T)
    bad = torch.tensor([1.0, -1.0, float("nan"), float("inf"), 1, 1, 1, 1, 1], device="cuda")
    out = n.grpo_token_stats(z, y, temperature=bad, top=20)
    assert n.grpo_check_error(out["workspace"]) == 9
    for k in ("logp", "entropy", "norm", "top_logp"):
        assert out[k][1:4].isnan().all() and out[k][0].isfinite().all(), k
    assert (out["top_tokens"][1:4] == -1).all()


@pytest.mark.parametrize("V", [600, 20000, 151936])
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_masks(dt, V):
    """Banned tokens as -inf or as the type's lowest value, few or one left, ties
    everywhere, rows in order, the largest crowded into few threads."""
    n = g()
    inf, low = float("inf"), LOWEST[dt]
    r = gen(5)
    rows = []
    base = (torch.randn(V, generator=r, device="cuda") * 3).to(dt)
    ban = torch.rand(V, generator=r, device="cuda") < 0.9
    for fill in (-inf, low):
        rows.append(base.masked_fill(ban, fill))
        few = torch.full((V,), fill, device="cuda", dtype=dt)
        few[torch.randint(0, V, (3,), generator=r, device="cuda")] = 1.5
        rows.append(few)
        one = torch.full((V,), fill, device="cuda", dtype=dt)
        one[V - 1] = -7.0
        rows.append(one)
    mixed = torch.full((V,), -inf, device="cuda", dtype=dt)
    mixed[V // 3::7] = low
    rows.append(mixed)
    rows.append(torch.full((V,), low, device="cuda", dtype=dt))
    rows.append(torch.zeros(V, device="cuda", dtype=dt))
    zeros = torch.zeros(V, device="cuda", dtype=dt)
    zeros[::3] = -0.0
    rows.append(zeros)
    rows.append(torch.full((V,), 3.25, device="cuda", dtype=dt))
    rows.append(base.sort().values)
    rows.append(base.sort(descending=True).values)
    # ties at the border: 25 values, and everything else one step below
    ties = torch.full((V,), 1.0, device="cuda", dtype=dt)
    ties[torch.randperm(V, generator=r, device="cuda")[:25]] = 2.0
    rows.append(ties)
    crowd = base.clone()  # the vectors of one thread (and its neighbours') hold all large values
    per = 16 // crowd.element_size()
    for k in range(0, V - 3 * per, 256 * per):
        crowd[k:k + 3 * per] = 20.0 + torch.rand(3 * per, generator=r, device="cuda").to(dt)
    rows.append(crowd)
    rows.append((base.float() * 1e5).to(dt))  # far from one another
    rows.append((base.float() * 1e-6 + 30000.0).to(dt))
    z = torch.stack(rows).unsqueeze(1)
    y = z.float().argmax(-1)
    out = n.grpo_token_stats(z, y, top=32)
    assert n.grpo_check_error(out["workspace"]) == 0
    check(z, y, out, 32)
    # tokens that are banned: -inf
    y = z.float().argmin(-1)
    out = n.grpo_token_stats(z, y, top=7)
    check(z, y, out, 7)


@pytest.mark.parametrize("V, copies", [(33, 1), (250, 1), (250, 400), (2039, 300)])
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_masks_of_short_rows(dt, V, copies):
    """Rows that a warp takes, with more candidates than its list holds and with
    hardly any."""
    n = g()
    inf, low = float("inf"), LOWEST[dt]
    r = gen(40)
    rows = []
    base = (torch.randn(V, generator=r, device="cuda") * 3).to(dt)
    for fill in (-inf, low):
        rows.append(base.masked_fill(torch.rand(V, generator=r, device="cuda") < 0.9, fill))
        few = torch.full((V,), fill, device="cuda", dtype=dt)
        few[torch.randint(0, V, (3,), generator=r, device="cuda")] = 1.5
        rows.append(few)
    one = torch.full((V,), -inf, device="cuda", dtype=dt)
    one[V - 1] = -7.0
    rows.append(one)
    zeros = torch.zeros(V, device="cuda", dtype=dt)
    zeros[::3] = -0.0
    rows += [zeros, torch.full((V,), 3.25, device="cuda", dtype=dt),
             base.sort().values, base.sort(descending=True).values]
    for k in (20, 31, 32, 33, 63, 64, 65):  # equal ones at the border, over and under the list's size
        ties = torch.full((V,), 1.0, device="cuda", dtype=dt)
        ties[torch.randperm(V, generator=r, device="cuda")[:k]] = 2.0
        rows.append(ties)
    crowd = base.clone()  # in the vectors of one lane
    for k in range(0, V - 8, 256):
        crowd[k:k + 8] = 20.0 + torch.rand(8, generator=r, device="cuda").to(dt)
    rows.append(crowd)
    z = torch.stack(rows).unsqueeze(1)
    y = z.float().argmax(-1)
    for top in (1, 8, 9, 32):
        out = n.grpo_token_stats(z.repeat(copies, 1, 1), y.repeat(copies, 1), top=top)
        assert n.grpo_check_error(out["workspace"]) == 0
        N = z.shape[0]
        # (the order of a row's sums follows its address's remainder by 16 bytes: copies 16 apart
        # share it, others agree to the tolerance only)
        for c in range(min(copies, 16)):
            check(z, y, {k: v[c * N:(c + 1) * N] for k, v in out.items() if k != "workspace"}, top,
                  lanes=64)
            for k in ("logp", "entropy", "norm", "top_tokens", "top_logp"):
                v = out[k].view(copies, N, -1)[c::16]
                assert torch.equal(v, v[:1].expand_as(v)), k


@pytest.mark.parametrize("V", [9, 700, 40000])
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_rows_without_a_distribution(dt, V):
    n = g()
    z, y = draw(7, 1, V, dt, 6)
    inf, nan = float("inf"), float("nan")
    z[1] = -inf
    z[2, 0, V // 2] = nan
    z[3, 0, V - 1] = inf
    z[4] = nan
    z[5] = -inf
    z[5, 0, 3] = nan
    out = n.grpo_token_stats(z, y, top=4)
    assert n.grpo_check_error(out["workspace"]) == 9
    for k in ("logp", "entropy", "norm", "top_logp"):
        assert out[k][1:6].isnan().all(), k
    assert (out["top_tokens"][1:6] == -1).all()
    for i in (0, 6):
        check(z[i:i + 1], y[i:i + 1], {k: v[i:i + 1] for k, v in out.items() if k != "workspace"}, 4)
    dz = n.grpo_token_stats_bwd(z, y, out["norm"], out["entropy"], torch.ones_like(out["logp"]),
                                torch.ones_like(out["logp"]))
    assert dz[1:6].isnan().all() and dz[0].isfinite().all() and dz[6].isfinite().all()


def test_tokens_out_of_range():
    n = g()
    z, y = draw(3, 2, 50, F32, 7)
    y[0, 1], y[2, 0] = 50, -1
    out = n.grpo_token_stats(z, y, top=2)
    assert n.grpo_check_error(out["workspace"]) == 6
    bad = torch.zeros(3, 2, dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[2, 0] = True
    assert torch.equal(out["logp"].isnan(), bad) and out["entropy"].isfinite().all()
    one = torch.ones(3, 2, device="cuda")
    dz = n.grpo_token_stats_bwd(z, y, out["norm"], out["entropy"], one, one)
    assert torch.equal(dz.isnan().any(-1), bad) and torch.equal(dz.isnan().all(-1), bad)
    dz = n.grpo_token_stats_bwd(z, y, out["norm"], out["entropy"], None, one)
    assert dz.isfinite().all()


def test_no_rows():
    n = g()
    for N, R in ((0, 4), (3, 0)):
        z = torch.zeros(N, R, 11, device="cuda")
        y = torch.zeros(N, R, dtype=torch.int64, device="cuda")
        out = n.grpo_token_stats(z, y, top=2)
        assert out["top_tokens"].shape == (N, R, 2) and n.grpo_check_error(out["workspace"]) == 0
        dz = n.grpo_token_stats_bwd(z, y, out["norm"], out["entropy"], out["logp"])
        assert dz.shape == (N, R, 11)


def test_results_repeat_bit_for_bit_and_outputs_are_reused():
    n = g()
    z, y = draw(4, 5, 30011, BF16, 8)
    a = n.grpo_token_stats(z, y, top=9)
    b = n.grpo_token_stats(z, y, top=9)
    for k in a:
        if k != "workspace":
            assert torch.equal(a[k], b[k]), k
            a[k].fill_(3)
    version = a["logp"]._version
    c = n.grpo_token_stats(z, y, top=9, out=a)
    assert c is a and a["logp"]._version > version
    for k in a:
        if k != "workspace":
            assert torch.equal(a[k], b[k]), k


# ---------------------------------------------------------------------------
# gradient
# ---------------------------------------------------------------------------


def check_grad(z, y, gl, gh, dz, lens=None, T=None):
    N, R, V = z.shape
    half = torch.finfo(z.dtype).eps / 2
    for i in range(N):
        n = R if lens is None else max(0, min(R, int(lens[i])))
        assert (dz[i, n:] == 0).all()
        if n == 0:
            continue
        r = Ref(z[i, :n], 1.0 if T is None else warmth(T[i:i + 1]).item())
        a = torch.zeros(n, 1, device="cuda").double() if gl is None else gl[i, :n, None].double()
        h = torch.zeros(n, 1, device="cuda").double() if gh is None else gh[i, :n, None].double()
        lnp = r.lp.clamp(min=-800)
        want = -a * r.p - h * r.p * (lnp + r.H)
        hit = torch.zeros_like(want).scatter_(-1, y[i, :n].unsqueeze(-1), 1.0)
        want = (want + a * hit) / r.T
        eps = U * (4 * r.x.clamp(min=-800).abs() + 3 * r.L + 8) + r.delta
        tolH = (r.delta + 4 * U) * (10 + 2 * r.D)
        tol = (2 * eps * r.p * (a.abs() + h.abs() * (lnp.abs() + r.H + 1)) + r.p * h.abs() * tolH +
               hit * a.abs() * 4 * U) / r.T + want.abs() * (4 * U + half * 1.001) + 1e-37
        got = dz[i, :n].double()
        bad = (got - want).abs() > tol
        assert not bad.any(), (bad.nonzero()[:5], got[bad][:5], want[bad][:5], tol[bad][:5])


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("of", ["both", "logp", "entropy"])
def test_gradient(shape, dt, of):
    n = g()
    z, y = draw(*shape, dt, 11)
    r = gen(12)
    gl = torch.randn(shape[:2], generator=r, device="cuda") if of != "entropy" else None
    gh = torch.randn(shape[:2], generator=r, device="cuda") if of != "logp" else None
    out = n.grpo_token_stats(z, y)
    dz = n.grpo_token_stats_bwd(z, None if of == "entropy" else y, out["norm"],
                                None if of == "logp" else out["entropy"], gl, gh)
    assert dz.dtype == dt
    check_grad(z, y, gl, gh, dz)


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_gradient_of_views_into_views(dt):
    """Lengths, temperatures, -inf, rows of wider buffers in every phase; what lies
    between the rows stays."""
    n = g()
    N, R, V = 4, 5, 1501
    r = gen(13)
    for pad_in, pad_out, shift in ((0, 0, 0), (3, 8, 0), (0, 1, 5), (7, 7, 1), (2, 0, 0)):
        buf = (torch.randn(N, R + 1, V + pad_in, generator=r, device="cuda") * 2).to(dt)
        z = buf[:, :R, :V]
        z[:, :, torch.rand(V, generator=r, device="cuda") < 0.4] = -math.inf
        y = torch.randint(0, V, (N, R + 2), generator=r, device="cuda")[:, 2:]
        z[torch.arange(N, device="cuda")[:, None], torch.arange(R, device="cuda"), y] = 1.0
        lens = torch.tensor([5, 0, 3, 1], dtype=torch.int32, device="cuda")
        T = torch.tensor([0.5, 1.0, 0.0, 3.0], device="cuda")
        gl = torch.randn(N, R, generator=r, device="cuda")
        gh = torch.randn(N, R, generator=r, device="cuda")
        gl[0, 1] = gh[0, 1] = 0.0
        z[0, 1] = 4.0  # (not read)
        out = n.grpo_token_stats(z, y, lens, T)
        full = torch.full((N * (R + 2) * (V + pad_out) + shift,), 9.0, dtype=dt, device="cuda")
        rows = full[shift:].view(N, R + 2, V + pad_out)
        dz = rows[:, 1:R + 1, :V]
        got = n.grpo_token_stats_bwd(z, y, out["norm"], out["entropy"], gl, gh, lens, T, out=dz)
        assert got is dz
        check_grad(z, y, gl, gh, dz, lens, T)
        assert (dz[0, 1] == 0).all()
        assert (rows[:, 0] == 9).all() and (rows[:, R + 1] == 9).all() and (full[:shift] == 9).all()
        assert (rows[:, :, V:] == 9).all()


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 3, 40011), (2, 3, 16390), (2, 1, 16385), (3, 7, 65537),
                                   (4, 100, 100), (2, 700, 1001), (2, 800, 2503), (1, 2, 9)], ids=str)
def test_gradient_of_rows_at_another_alignment(shape, dt):
    """Every phase of the input against every phase of the output, in long rows of several
    parts and in short ones; what lies around the rows stays."""
    n = g()
    N, R, V = shape
    r = gen(14)
    gl = torch.randn(N, R, generator=r, device="cuda")
    gh = torch.randn(N, R, generator=r, device="cuda")
    y = torch.randint(0, V, (N, R), generator=r, device="cuda")
    y.view(-1)[0], y.view(-1)[-1] = 0, V - 1
    plain = (torch.randn(N, R, V, generator=r, device="cuda") * 2).to(dt)
    for at in range(16 // plain.element_size()):
        for pad_in, pad_out in ((0, 1), (1, 0), (8, 8)):
            buf = torch.full((N * R * (V + pad_in) + at,), math.inf, dtype=dt, device="cuda")
            z = buf[at:].view(N, R, V + pad_in)[:, :, :V]
            z.copy_(plain)
            out = n.grpo_token_stats(z, y)
            full = torch.full((N * R * (V + pad_out) + 16,), 9.0, dtype=dt, device="cuda")
            rows = full[8:-8].view(N, R, V + pad_out)
            n.grpo_token_stats_bwd(z, y, out["norm"], out["entropy"], gl, gh, out=rows[:, :, :V])
            check_grad(z, y, gl, gh, rows[:, :, :V])
            assert (rows[:, :, V:] == 9).all() and (full[:8] == 9).all() and (full[-8:] == 9).all()


def test_gradient_against_differences():
    """Central differences of the float64 definition, every entry."""
    n = g()
    z, y = draw(2, 2, 23, F32, 14, 1.5)
    T = torch.tensor([0.7, 1.3], device="cuda")
    r = gen(15)
    gl, gh = (torch.randn(2, 2, generator=r, device="cuda") for _ in range(2))

    def value(zz):
        lp = torch.log_softmax(zz / T.double().view(2, 1, 1), -1)
        H = -(lp.exp() * lp).sum(-1)
        return float((gl.double() * lp.gather(-1, y[..., None])[..., 0] + gh.double() * H).sum())

    out = n.grpo_token_stats(z, y, temperature=T)
    dz = n.grpo_token_stats_bwd(z, y, out["norm"], out["entropy"], gl, gh, temperature=T)
    step = 1e-5
    for i in range(2):
        for j in range(2):
            for v in range(23):
                zz = z.double()
                zz[i, j, v] += step
                up = value(zz)
                zz[i, j, v] -= 2 * step
                # differences: step^2 of the third derivative (below 10), 1e-16 / step of rounding
                assert abs((up - value(zz)) / (2 * step) - float(dz[i, j, v])) < 1e-6


def test_a_nearly_certain_token_keeps_its_gradient():
    """1 - p far below float32's step at 1: the token's own entry is not 0."""
    n = g()
    z = torch.zeros(1, 1, 100, device="cuda")
    z[0, 0, 7] = 25.0
    y = torch.full((1, 1), 7, device="cuda")
    out = n.grpo_token_stats(z, y)
    one = torch.ones(1, 1, device="cuda")
    dz = n.grpo_token_stats_bwd(z, y, out["norm"], out["entropy"], one)
    p = torch.softmax(z.double(), -1)[0, 0]
    rest = float(p.sum() - p[7])
    # (ln p is itself a float32 difference: the log-sum, below u, may be lost)
    assert abs(float(dz[0, 0, 7]) - rest) <= 2 * U
    assert abs(float(dz[0, 0, 0]) + float(p[0])) <= 1e-5 * float(p[0])


def test_autograd():
    from vocab_wide_logprob_gb300 import autograd
    z, y = draw(3, 4, 517, F32, 16)
    lens = torch.tensor([4, 2, 0], dtype=torch.int32, device="cuda")
    T = torch.tensor([1.0, 0.6, 2.0], device="cuda")
    keep = torch.arange(4, device="cuda") < lens[:, None]
    z.requires_grad_()
    logp, H = autograd.grpo_logp_entropy(z, y, lens, T)
    loss = (logp * logp).sum() * 0.1 - 0.01 * H.sum()
    loss.backward()
    z64 = z.detach().double().requires_grad_()
    lp = torch.log_softmax(z64 / T.double().view(3, 1, 1), -1)
    want = (torch.where(keep, lp.gather(-1, y[..., None])[..., 0], 0.0) ** 2).sum() * 0.1 \
        - 0.01 * torch.where(keep, -(lp.exp() * lp).sum(-1), 0.0).sum()
    want.backward()
    assert (loss - want).detach().abs() <= 1e-5 * want.detach().abs()
    assert (z.grad.double() - z64.grad).abs().max() <= 1e-5 * z64.grad.abs().max()
    # one output alone; neither; a second derivative
    z.grad = None
    logp, H = autograd.grpo_logp_entropy(z, y, lens, T)
    H.sum().backward()
    assert z.grad.isfinite().all() and z.grad.abs().max() > 0
    logp, H = autograd.grpo_logp_entropy(z, y)
    (dz,) = torch.autograd.grad(logp.sum() + H.sum(), z, create_graph=True)
    with pytest.raises(RuntimeError, match="first-order"):
        dz.sum().backward()


# ---------------------------------------------------------------------------
# how it is called
# ---------------------------------------------------------------------------


def test_another_stream_and_a_graph():
    n = g()
    z, y = draw(6, 3, 9001, BF16, 17)
    want = n.grpo_token_stats(z, y, top=8)
    gl = torch.randn(6, 3, device="cuda")
    dwant = n.grpo_token_stats_bwd(z, y, want["norm"], want["entropy"], gl, gl)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = n.grpo_token_stats(z, y, top=8, stream=side)
    dgot = n.grpo_token_stats_bwd(z, y, got["norm"], got["entropy"], gl, gl, stream=side)
    side.synchronize()
    for k in ("logp", "entropy", "norm", "top_tokens", "top_logp"):
        assert torch.equal(got[k], want[k]), k
    assert torch.equal(dgot, dwant)
    # captured, replayed with other logits in the same memory, twice
    zs, out = z.clone(), {k: v.clone() for k, v in want.items()}
    dout = torch.empty_like(dwant)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        n.grpo_token_stats(zs, y, top=8, out=out)
        n.grpo_token_stats_bwd(zs, y, out["norm"], out["entropy"], gl, gl, out=dout)
    for seed in (18, 19):
        z2, _ = draw(6, 3, 9001, BF16, seed)
        zs.copy_(z2)
        graph.replay()
        want = n.grpo_token_stats(z2, y, top=8)
        dwant = n.grpo_token_stats_bwd(z2, y, want["norm"], want["entropy"], gl, gl)
        torch.cuda.synchronize()
        for k in ("logp", "entropy", "norm", "top_tokens", "top_logp"):
            assert torch.equal(out[k], want[k]), k
        assert torch.equal(dout, dwant)


def test_graphs_that_share_a_workspace_and_streams_side_by_side():
    """Two captured graphs with the same outputs and workspace, replayed in turn; then
    calls of different sizes on two streams at once, each with its own."""
    n = g()
    cases = [(draw(6, 3, 9001, BF16, 30), 8), (draw(3, 2, 40011, F32, 31), 8)]
    names = ("logp", "entropy", "norm", "top_tokens", "top_logp")
    want = [n.grpo_token_stats(z, y, top=top) for (z, y), top in cases]
    ws = torch.empty(n.grpo_token_stats_workspace_size(6, 3), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graphs, outs = [], []
    for k, ((z, y), top) in enumerate(cases):
        outs.append({x: torch.empty_like(want[k][x]) for x in names})
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[k]):
            n.grpo_token_stats(z, y, top=top, out=outs[k], workspace=ws)
    for k in (0, 1, 1, 0, 1, 0):
        for o in outs[k].values():
            if isinstance(o, torch.Tensor) and o is not ws:
                o.zero_()
        graphs[k].replay()
        torch.cuda.synchronize()
        assert n.grpo_check_error(ws) == 0
        for x in names:
            assert torch.equal(outs[k][x], want[k][x]), (k, x)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(8):
        for k, ((z, y), top) in enumerate(cases):
            with torch.cuda.stream(side[k]):
                got[k].append(n.grpo_token_stats(z, y, top=top))
    torch.cuda.synchronize()
    for k in (0, 1):
        for o in got[k]:
            for x in names:
                assert torch.equal(o[x], want[k][x]), (k, x)


def test_rows_beyond_two_to_the_31_elements():
    """The last sequence's rows start past 2^32 elements' bytes."""
    n = g()
    N, R, V = 3, 5000, 151936
    z = torch.empty(N, R, V, dtype=BF16, device="cuda")
    z[:2].zero_()
    z[2].normal_(generator=gen(20)).mul_(3)
    y = torch.randint(0, V, (N, R), generator=gen(21), device="cuda")
    lens = torch.tensor([0, 1, R], dtype=torch.int32, device="cuda")
    out = n.grpo_token_stats(z, y, lens, top=4)
    tail = slice(R - 3, R)
    check(z[2:, tail], y[2:, tail],
          {k: v[2:, tail] for k, v in out.items() if k != "workspace"}, 4)
    gl = torch.zeros(N, R, device="cuda")
    gl[2, tail] = 1.0
    dz = n.grpo_token_stats_bwd(z, y, out["norm"], out["entropy"], gl, gl, lens)
    check_grad(z[2:, tail], y[2:, tail], gl[2:, tail], gl[2:, tail], dz[2:, tail])
    assert not dz[:2].any() and not dz[2, :R - 3].any()


def test_agrees_with_the_loss_calls():
    """The log-probs of grpo_logprobs, and of the verification at T = 1, of the
    same rows."""
    n = g()
    N, P, C, V = 3, 4, 6, 2000
    r = gen(22)
    logits = (torch.randn(N, P + C, V, generator=r, device="cuda") * 2).to(BF16)
    ids = torch.randint(0, V, (N, P + C), generator=r, device="cuda")
    lens = torch.tensor([6, 2, 5], dtype=torch.int32, device="cuda")
    lp, _, _ = n.grpo_logprobs(logits, P, ids, lens)
    out = n.grpo_token_stats(logits[:, P - 1:-1], ids[:, P:], lens)
    assert (lp - out["logp"]).abs().max() <= 1e-5
