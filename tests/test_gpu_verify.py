"""Verification of drafted tokens against the definition in float64 (one
sequence after the other, one drafted token after the other).

Tokens and acceptance counts must be equal.  Log-probs: the float32 sum behind
one is off by at most the roundings of its terms (the exponent's, up to 64
halves of 2^-24, ex2's 2^-22) and of the additions of one thread (V / 1024 of
them and a few for the tree), so by (V / 1024 + 80) * 2^-24, then the value's
own rounding to float32."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def g():
    from vocab_wide_logprob_gb300 import _native
    return _native


def gen(seed):
    r = torch.Generator(device="cuda")
    r.manual_seed(seed)
    return r


def log_probs(row, T):
    x = row.double().cpu().numpy() / T
    m = x.max()
    if not np.isfinite(m) or np.isnan(x).any():
        return None
    x = x - m
    return x - math.log(np.exp(x).sum())


def reference(z, x, u, noise, y=None, lens=None, temp=None):
    N, K, V = z.shape[0], z.shape[1] - 1, z.shape[2]
    tokens = np.full((N, K + 1), -1, np.int64)
    acc = np.zeros(N, np.int64)
    logp = np.zeros((N, K + 1))
    x, u = x.cpu().numpy(), u.double().cpu().numpy()
    np.seterr(over="ignore")  # an improbable draft: the ratio may overflow to infinity
    for i in range(N):
        L = K if lens is None else min(max(int(lens[i]), 0), K)
        T = 1.0 if temp is None else float(temp[i])
        greedy = 0 <= T < 1e-6
        for j in range(L + 1):
            acc[i] = j
            bad = not (T >= 0 and math.isfinite(T))
            lp = None if bad else log_probs(z[i, j], 1.0 if greedy else T)
            use = y is not None and j < L and not greedy and not bad
            lq = log_probs(y[i, j], T) if use else None
            if lp is None or (use and lq is None):
                logp[i, j] = np.nan
                break
            if j < L and 0 <= x[i, j] < V:
                t = x[i, j]
                if greedy:
                    ok = t == int(np.argmax(lp))
                else:
                    ok = lp[t] > -np.inf and u[i, j] * np.exp((lq[t] if use else 0.0) - lp[t]) < 1
                if ok:
                    tokens[i, j], logp[i, j] = t, lp[t]
                    continue
            if greedy:
                t = int(np.argmax(lp))
            else:
                p = np.exp(lp)
                rest = p.copy()
                if use:
                    rest = np.maximum(p - np.exp(lq), 0)
                elif j < L and 0 <= x[i, j] < V:
                    rest[x[i, j]] = 0
                if not (rest > 0).any():
                    rest = p
                t = int(np.argmax(rest / noise[i].double().cpu().numpy()))
            tokens[i, j], logp[i, j] = t, lp[t]
            break
    return tokens, acc, logp


def check(out, want, V):
    tokens, acc, logp = want
    assert np.array_equal(out["n_accepted"].cpu().numpy(), acc)
    assert np.array_equal(out["tokens"].cpu().numpy(), tokens)
    got = out["logp"].double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(logp))
    k = ~np.isnan(logp)
    tol = (V / 1024 + 80) * 2.0 ** -24 + np.abs(logp[k]) * 2.0 ** -23
    assert (np.abs(got[k] - logp[k]) <= tol).all(), np.abs(got[k] - logp[k]).max()


def case(N, K, V, dt, seed, draft=True, err=0.7, std=3.0, temp=False, ragged=False, banned=0.0):
    r = gen(seed)
    z = torch.randn(N, K + 1, V, generator=r, device="cuda") * std
    if banned:
        mask = torch.rand(V, generator=r, device="cuda") < banned
        mask[0] = False
        z[..., mask] = -math.inf
    y = z[:, :K] + torch.randn(N, K, V, generator=r, device="cuda") * err
    race = torch.empty(N, K, V, device="cuda").exponential_(generator=r).log_()
    src = y if draft else z[:, :K]
    x = (src.to(dt).float() - race).argmax(-1) if K else torch.zeros(N, 0, dtype=torch.int64, device="cuda")
    if not draft:  # likely copies
        z[:, :K].scatter_(-1, x.unsqueeze(-1), math.log(V) + 6)
    return dict(z=z.to(dt), x=x, u=torch.rand(N, K, generator=r, device="cuda"),
                noise=torch.empty(N, V, device="cuda").exponential_(generator=r).clamp_(min=1e-20),
                y=y.to(dt) if draft and K else None,
                lens=torch.randint(0, K + 1, (N,), generator=r, device="cuda", dtype=torch.int32)
                if ragged else None,
                temp=(torch.rand(N, generator=r, device="cuda") + 0.5) if temp else None)


def run(c, **kw):
    return g().grpo_verify_drafts(c["z"], c["x"], c["u"], c["noise"], c["y"], c["lens"], c["temp"],
                                  **kw)


def both(c, status=0):
    out = run(c)
    assert g().grpo_check_error(out["workspace"]) == status
    check(out, reference(**c), c["z"].shape[2])
    return out


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("draft", [True, False], ids=["drafted", "copied"])
@pytest.mark.parametrize("N,K,V", [(1, 0, 1), (1, 1, 2), (3, 2, 7), (2, 3, 33), (5, 4, 1000),
                                   (9, 3, 1024), (4, 6, 4099), (2, 5, 32003), (3, 2, 151936),
                                   (700, 2, 100), (1, 8, 65536)])
def test_sizes(N, K, V, dt, draft):
    both(case(N, K, V, dt, 100 + V, draft))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("N", [1, 20, 90, 200, 640, 1300])
def test_cluster_splits(N, dt):
    """Batch sizes around the rule that splits a row over a cluster."""
    both(case(N, 2, 70001, dt, 200 + N, err=0.4) if N <= 200 else case(N, 2, 3001, dt, 7, err=0.4))


@pytest.mark.parametrize("dt", [F32, BF16])
def test_temperatures_lengths_and_bans(dt):
    for draft in (True, False):
        c = case(24, 5, 5003, dt, 300, draft, err=0.5, temp=True, ragged=True, banned=0.3)
        c["temp"][::3] = 0.0
        c["temp"][1] = 1e-7
        c["temp"][4] = 50.0
        c["temp"][7] = 0.02
        top = c["z"][:, :5].float().argmax(-1)
        keep = torch.rand(24, 5, generator=gen(1), device="cuda") < 0.7
        c["x"] = torch.where((c["temp"] < 1e-6).view(-1, 1) & keep, top, c["x"])
        both(c)


def test_greedy_ties_take_the_lowest():
    """bfloat16 logits of few values: every maximum is met many times."""
    r = gen(5)
    for V in (8, 1000, 4099):
        z = torch.randint(-2, 3, (40, 4, V), generator=r, device="cuda").to(BF16)
        z[0, :, 0] = 9
        z[1, :, V - 1] = 9
        c = dict(z=z, x=z[:, :3].float().argmax(-1), u=torch.rand(40, 3, device="cuda"),
                 noise=torch.ones(40, V, device="cuda"), y=None, lens=None,
                 temp=torch.zeros(40, device="cuda"))
        low = torch.where(z == z.amax(-1, keepdim=True), torch.arange(V, device="cuda"), V).amin(-1)
        c["x"] = low[:, :3].clone()
        c["x"][5, 1] += 1
        both(c)


def test_race_ties_take_the_lowest():
    V = 5000
    c = case(6, 0, V, F32, 6)
    c["z"].zero_()
    c["noise"].fill_(1.0)
    c["noise"][:, 777] = 0.25
    c["noise"][:, 3333] = 0.25
    out = both(c)
    assert (out["tokens"] == 777).all()


def test_equal_distributions_accept_everything():
    c = case(16, 4, 2000, BF16, 8)
    c["y"] = c["z"][:, :4].contiguous()
    out = both(c)
    assert (out["n_accepted"] == 4).all()


def test_residual_at_the_level_of_rounding():
    """A draft next to the target: the residual is nothing but rounding, the
    race's bounds separate nothing, and the decision falls in float64."""
    c = case(8, 1, 3000, F32, 9, err=0.0)
    c["y"] = c["z"][:, :1].clone()
    c["y"][..., 5] += 1e-2
    c["x"].fill_(5)
    c["u"].fill_(0.99999994)
    out = both(c)
    assert (out["n_accepted"] == 0).all()


@pytest.mark.parametrize("V,at", [(64, 0), (5003, 17), (40000, 39999), (151936, 100)])
@pytest.mark.parametrize("sign", [1, -1])
def test_winner_with_a_residual_inside_the_bounds(V, at, sign):
    """A token whose p and q differ by 4e-6 of themselves, which float32 bounds
    cannot tell from 0, and whose noise makes it the winner by far (or, with
    q above p, not a candidate at all)."""
    c = case(3, 1, V, F32, 31, err=0.0)
    c["z"].mul_(0.5)
    c["y"] = c["z"][:, :1].clone()
    c["y"][:, 0, at] -= sign * 4e-6
    # the residual's ordinary mass, and the rejected token that pays for it:
    # 2 exp(2) = exp(1) + exp(2.48988), so the sums stay equal
    up, paid = (at + 3) % V, (at + 5) % V
    c["z"][:, 0, up] = c["z"][:, 0, paid] = 2.0
    c["y"][:, 0, up] = 1.0
    c["y"][:, 0, paid] = 2.48988012564475
    c["x"].fill_(paid)
    c["u"].fill_(0.999)
    c["noise"][:, at] = 1e-12
    both(c)


def test_no_residual_falls_back_to_the_target():
    """Copied draft of the only possible token, rejected by a NaN random number."""
    z = torch.full((2, 2, 64), -math.inf, device="cuda")
    z[:, :, 9] = 1.0
    c = dict(z=z, x=torch.full((2, 1), 9, device="cuda"), u=torch.full((2, 1), math.nan, device="cuda"),
             noise=torch.ones(2, 64, device="cuda"), y=None, lens=None, temp=None)
    out = both(c)
    assert (out["tokens"][:, 0] == 9).all() and (out["n_accepted"] == 0).all()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("draft", [False, True], ids=["last", "residual"])
@pytest.mark.parametrize("V", [40000, 40003])
def test_close_scores_far_from_zero(dt, draft, V):
    """Logits thousands away from 0 (a shift that changes no probability): the
    winner's score is 1e-4 of itself above that of a token before it."""
    N, r = 64, gen(18)
    shift = (torch.rand(N, 1, 1, generator=r, device="cuda") * 60000 + 1000).to(dt)
    z = shift.expand(N, 2 if draft else 1, V).clone()
    noise = torch.full((N, V), 4.0, device="cuda")
    noise[:, 7] = 1.0
    noise[torch.arange(N, device="cuda"), 4000 + 500 * torch.arange(N, device="cuda")] = 1 / (1 + 1e-4)
    c = dict(z=z, x=torch.zeros(N, 0, dtype=torch.int64, device="cuda"),
             u=torch.zeros(N, 0, device="cuda"), noise=noise, y=None, lens=None, temp=None)
    if draft:  # the draft has all but a little of its mass on the rejected token 0
        c["x"] = torch.zeros(N, 1, dtype=torch.int64, device="cuda")
        c["u"] = torch.ones(N, 1, device="cuda")
        c["y"] = shift.expand(N, 1, V).clone()
        c["y"][:, :, 0] = (c["y"][:, :, 0].float() * 1.25 + 40).to(dt)
    both(c)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("at", [0, 17, 2501, 5002])
def test_noise_at_the_ends_of_its_range(dt, at):
    """An improbable token (2^-99) whose noise is 2^-60 beats, or not, the rest."""
    V = 5003
    c = case(4, 0, V, dt, 25)
    c["z"].zero_()
    c["z"][:, :, at] = -60.0
    for rest, wins in ((2.0 ** 30, True), (1.0, False)):
        c["noise"] = rest * (1 + torch.rand(4, V, generator=gen(26), device="cuda") / 2)
        c["noise"].clamp_(max=2.0 ** 30)
        c["noise"][:, at] = 2.0 ** -60
        out = both(c)
        assert ((out["tokens"] == at).all()) == wins


def far_case(dt, V, T, rows):
    """One sequence per entry of ``rows`` (float64 [V]), nothing drafted, at temperature T."""
    z = torch.stack([r.to(dt) for r in rows]).unsqueeze(1).cuda()
    N, r = len(rows), gen(19)
    return dict(z=z, x=torch.zeros(N, 0, dtype=torch.int64, device="cuda"),
                u=torch.zeros(N, 0, device="cuda"), y=None, lens=None,
                noise=torch.empty(N, V, device="cuda").exponential_(generator=r).clamp_(min=1e-9),
                temp=torch.full((N,), T, device="cuda"))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("V", [37, 4099, 40000])
def test_every_token_at_one_far_level(dt, V):
    """Masks of any size under every token (and the same above 0): a uniform row."""
    levels = [s * v for s in (-1, 1) for v in (1.1e7, 1.2e7, 1e8, 1e9, 3e9, 1e10, 1e13, 1e20, 9.9e29, 1e30)]
    out = both(far_case(dt, V, 1.0, [torch.full((V,), v, dtype=torch.float64) for v in levels]))
    assert (out["logp"] + math.log(V)).abs().max() < 1e-4


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("level", [3e9, 1e10, -1e10, 1e20])
def test_far_rows_of_different_values(dt, level):
    """Random logits far from zero at temperatures that leave a distribution."""
    V, g0 = 9001, torch.Generator().manual_seed(20)
    rows = [level * (1 + torch.rand(V, generator=g0, dtype=torch.float64)) for _ in range(6)]
    for T in (1.0, abs(level) / 4096, abs(level) / 20):
        both(far_case(dt, V, T, rows))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T", [1.1e-6, 3e-6, 1e-5, 1e-4])
def test_small_temperatures(dt, T):
    V, g0 = 9001, torch.Generator().manual_seed(21)
    base = torch.randn(V, generator=g0, dtype=torch.float64)
    rows = [3 * base, -65504 + torch.zeros(V, dtype=torch.float64), 20 + T * base, 3000 * base,
            torch.where(base > 3, 1.0, -65504.0), torch.where(base > 3, 1.0, -1e9)]
    c = far_case(dt, V, T, rows)
    both(c)
    c["z"] = c["z"].expand(6, 3, V).contiguous()  # with drafts, accepted and not
    c["y"] = c["z"][:, :2].clone()
    c["x"] = c["y"].float().argmax(-1)
    c["x"][::2, 1] = (c["x"][::2, 1] + 1) % V
    c["y"][:, 1].scatter_(1, c["x"][:, 1:], 60000.0)
    c["u"] = torch.full((6, 2), 0.5, device="cuda")
    both(c)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("V", [64, 5001, 151936])
@pytest.mark.parametrize("order", ["up", "down", "mixed"])
def test_parts_on_both_sides_of_the_far_form(sign, V, order):
    """A row whose parts have maxima a few units apart around 2^24 / log2(e),
    where the weights' form changes: the parts' sums are merged exactly."""
    edge = 2 ** 24 / math.log2(math.e)
    step = torch.arange(V, dtype=torch.float64) * (12.0 / V)
    if order == "down":
        step = step.flip(0)
    elif order == "mixed":
        step = step[torch.randperm(V, generator=torch.Generator().manual_seed(22))]
    rows = [torch.floor(sign * edge - 6 + k + step) for k in range(-2, 9, 2)]
    c = far_case(F32, V, 1.0, rows)
    both(c)
    # drafted from a row of the other form (a shift changes nothing): accepted
    c["x"] = torch.full((6, 1), V // 2, device="cuda")
    c["u"] = torch.full((6, 1), 0.999, device="cuda")
    c["y"], c["z"] = c["z"] - math.floor(sign * edge), c["z"].expand(6, 2, V).contiguous()
    assert (both(c)["n_accepted"] == 1).all()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("level", [-1e10, 1e10])
def test_far_residual(dt, level):
    """A rejected draft whose distribution is one token: the residual is the
    rest of a uniform row far from zero."""
    V = 4099
    c = far_case(dt, V, 1.0, [torch.full((V,), level, dtype=torch.float64)] * 4)
    c["z"] = c["z"].expand(4, 2, V).contiguous()
    c["x"] = torch.tensor([[0], [5], [2048], [V - 1]], device="cuda")
    c["u"] = torch.full((4, 1), 0.9, device="cuda")
    c["y"] = torch.full((4, 1, V), 2 * abs(level), device="cuda").neg().to(dt)
    c["y"].scatter_(2, c["x"].unsqueeze(-1), abs(level))
    out = both(c)
    assert (out["n_accepted"] == 0).all()
    c["y"] = None
    both(c)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("V", [40, 4099, 40000])
def test_masks_and_nonfinite_rows(dt, V):
    low = torch.finfo(dt).min
    c = case(12, 2, V, dt, 10, err=0.3)
    z, y = c["z"], c["y"]
    z[0, 0] = -math.inf                      # nothing allowed
    z[1, 0] = low                            # everything at the type's lowest value
    z[2, 1] = low
    z[2, 1, V // 2] = 0.0                    # one token left
    z[3, 0, V - 1] = math.inf
    z[4, 0, 3] = math.nan
    y[5, 0] = -math.inf                      # no draft distribution
    y[6, 0, 0] = math.nan
    z[7, 0] = -math.inf
    z[7, 0, V - 1] = low                     # one token, at the lowest value
    y[8, 0] = low
    z[9, :, ::2] = low
    z[10, :, ::2] = -math.inf
    z[11, 0] = -math.inf
    z[11, 0, 1] = math.nan                   # NaN among nothing else
    both(c, 9)
    c["temp"] = torch.zeros(12, device="cuda")
    both(c, 9)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_large_logits(dt):
    c = case(6, 2, 3001, dt, 11, err=0.3)
    c["z"].mul_(1e4)
    c["y"].mul_(1e4)
    c["temp"] = torch.tensor([1.0, 1e4, 3e3, 2e4, 1e5, 0.0], device="cuda")
    both(c)
    c = case(2, 0, 3001, dt, 12)
    c["z"].fill_(3e38)
    c["z"][:, :, 7] = -3e38
    both(c)


def test_bad_ids_lengths_and_temperatures():
    n = g()
    c = case(6, 3, 500, BF16, 13, err=0.2)
    c["x"][0, 0] = -1
    c["x"][1, 1] = 500
    both(c, 6)
    c["y"] = None
    both(c, 6)
    c = case(6, 3, 500, BF16, 13, err=0.2)
    c["lens"] = torch.tensor([0, 1, 2, 3, -5, 99], dtype=torch.int32, device="cuda")
    both(c, 7)
    c["lens"] = None
    c["temp"] = torch.tensor([1.0, -1.0, math.nan, math.inf, 0.0, -0.0], device="cuda")
    out = both(c, 9)
    # the workspace's next call starts clean
    c["temp"] = None
    out = run(c, out=out)
    assert n.grpo_check_error(out["workspace"]) == 0
    check(out, reference(**c), 500)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_views_of_padded_rows(dt):
    c = case(7, 3, 2003, dt, 14, err=0.4)
    for lo, wide in ((0, 2048), (1, 2005), (8, 2016)):
        big = torch.randn(8, 5, wide, device="cuda").to(dt)
        big[:7, :4, lo:lo + 2003] = c["z"]
        yb = torch.randn(7, 6, wide, device="cuda").to(dt)
        yb[:, 1:4, lo:lo + 2003] = c["y"]
        nb = torch.rand(9, wide, device="cuda")
        nb[:7, lo:lo + 2003] = c["noise"]
        d = dict(c, z=big[:7, :4, lo:lo + 2003], y=yb[:, 1:4, lo:lo + 2003],
                 noise=nb[:7, lo:lo + 2003])
        both(d)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("offs", [(0, 0, 1), (1, 0, 0), (0, 3, 2), (5, 5, 5), (8, 8, 8)])
@pytest.mark.parametrize("N", [3, 160])
def test_alignments(dt, offs, N):
    """Rows that begin anywhere relative to 16 bytes, with NaN around them, in
    one and in several steps of the race."""
    V = 20000
    c = case(N, 2, V, dt, 16, err=0.4)
    parts = {}
    for name, t, o in zip(("z", "y", "noise"), (c["z"], c["y"], c["noise"]), offs):
        big = torch.full((*t.shape[:-1], V + 16), math.nan, device="cuda", dtype=t.dtype)
        parts[name] = big[..., o:o + V]
        parts[name].copy_(t)
    both(dict(c, **parts))
    both(dict(c, y=None, z=parts["z"], noise=parts["noise"]))


@pytest.mark.parametrize("dt,N,V", [(BF16, 80, 151936), (F32, 44, 150001), (BF16, 300, 40001)])
def test_rows_behind_a_rejection(dt, N, V):
    """So many rows that those behind a known rejection are left out."""
    both(case(N, 4, V, dt, 17, err=0.6, ragged=True))


@pytest.mark.parametrize("dt,N,V", [(BF16, 300, 40001), (F32, 120, 60000), (BF16, 80, 151936)])
@pytest.mark.parametrize("draft", [True, False], ids=["drafted", "copied"])
def test_rows_behind_rejections_of_every_kind(dt, N, V, draft):
    """Calls that leave rows out, with all that can stop a sequence: rejections,
    greedy ones, undefined rows and temperatures, ids outside [0, V).  The
    workspace holds ones before, so that a part read early shows."""
    K = 4 if draft else 8
    assert N * V * (2 if dt == BF16 else 4) * (2 * K + 1 if draft else K + 1) > 192 << 20
    c = case(N, K, V, dt, 23, draft, err=0.5, temp=True, ragged=True)
    r = gen(24)
    c["lens"][::2] = K
    c["temp"][torch.rand(N, generator=r, device="cuda") < 0.4] = 0.0
    right = (torch.rand(N, K, generator=r, device="cuda") < 0.8) & (c["temp"] == 0).view(N, 1)
    c["x"] = torch.where(right, c["z"][:, :K].float().argmax(-1), c["x"])
    c["temp"][1::17] = -1.0
    c["temp"][2::19] = math.nan
    at = torch.randint(0, K, (N,), generator=r, device="cuda")
    for i in range(0, N, 7):
        c["x"][i, at[i]] = (-1, V, 1 << 40)[i % 3]
    for i in range(3, N, 11):
        c["z"][i, at[i], V // 3] = math.nan
    for i in range(4, N, 13):
        c["z"][i, at[i]] = -math.inf
    if draft:
        for i in range(5, N, 9):
            c["y"][i, at[i], 7] = math.nan
    need = g().grpo_verify_workspace_size(N, K)
    want = reference(**c)
    for _ in range(3):
        out = run(c, workspace=torch.full((need,), 255, dtype=torch.uint8, device="cuda"))
        assert g().grpo_check_error(out["workspace"]) == 6
        check(out, want, V)


def test_distribution_of_the_emitted_tokens():
    """Over many sequences of one distribution, the first emitted or accepted
    token follows the target: a chi-square bound at 7 sigma."""
    V, N = 12, 20000
    r = gen(15)
    z = torch.randn(V, generator=r, device="cuda") * 1.5
    y = torch.randn(V, generator=r, device="cuda") * 1.5
    race = torch.empty(N, 1, V, device="cuda").exponential_(generator=r).log_()
    c = dict(z=z.expand(N, 2, V).contiguous(), x=(y - race).argmax(-1),
             u=torch.rand(N, 1, generator=r, device="cuda"),
             noise=torch.empty(N, V, device="cuda").exponential_(generator=r),
             y=y.expand(N, 1, V).contiguous(), lens=None, temp=None)
    out = run(c)
    count = torch.bincount(out["tokens"][:, 0], minlength=V).double()
    p = torch.softmax(z.double(), 0) * N
    chi = float(((count - p) ** 2 / p).sum())
    assert chi < (V - 1) + 7 * math.sqrt(2 * (V - 1)), chi


def test_reproducible_stream_and_graph():
    n = g()
    c = case(33, 3, 20001, BF16, 16, temp=True)
    out = run(c)
    want = {k: out[k].clone() for k in ("tokens", "n_accepted", "logp")}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out["workspace"].fill_(255)
        run(c, out=out)
    side.synchronize()
    assert all(torch.equal(out[k], want[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(c, out=out)
    d = case(33, 3, 20001, BF16, 17, temp=True)
    for k in ("z", "x", "u", "noise", "y", "temp"):
        c[k].copy_(d[k])
    graph.replay()
    torch.cuda.synchronize()
    check(out, reference(**c), 20001)


def test_offsets_beyond_32_bits():
    """Sequence offsets past 2^31 elements."""
    V = 151936
    K = 8
    N = 1600
    need = N * (K + 1) * V * 2 + N * V * 4 + (2 << 30)
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip("not enough free device memory")
    z = torch.empty(N, K + 1, V, dtype=BF16, device="cuda")
    r = gen(18)
    for i in range(0, N, 100):
        z[i:i + 100] = torch.randn(100, K + 1, V, generator=r, device="cuda") * 3
    noise = torch.empty(N, V, device="cuda").exponential_(generator=r)
    lens = torch.zeros(N, dtype=torch.int32, device="cuda")
    lens[-3:] = torch.tensor([8, 4, 0])
    x = torch.randint(0, V, (N, K), generator=r, device="cuda")
    for j in range(K):  # certain drafts: the last sequences run to their ends
        z[-3:].scatter_(2, x[-3:, j].view(3, 1, 1).expand(3, 1, 1), 0)
        z[-3:, j].scatter_(1, x[-3:, j].view(3, 1), 40.0)
    out = g().grpo_verify_drafts(z, x, torch.full((N, K), 0.5, device="cuda"), noise, None, lens)
    last = slice(N - 3, N)
    c = dict(z=z[last], x=x[last], u=torch.full((3, K), 0.5, device="cuda"), noise=noise[last],
             y=None, lens=lens[last], temp=None)
    check({k: out[k][last] for k in ("tokens", "n_accepted", "logp")}, reference(**c), V)
    assert out["n_accepted"][last].tolist() == [8, 4, 0]


def test_empty_and_refusals():
    n = g()
    out = n.grpo_verify_drafts(torch.empty(0, 3, 10, device="cuda"),
                               torch.empty(0, 2, dtype=torch.int64, device="cuda"),
                               torch.empty(0, 2, device="cuda"), torch.empty(0, 10, device="cuda"))
    assert out["tokens"].shape == (0, 3) and n.grpo_check_error(out["workspace"]) == 0
    c = case(3, 2, 50, F32, 19)
    with pytest.raises(TypeError):
        run(dict(c, z=c["z"].half()))
    with pytest.raises(TypeError):
        run(dict(c, y=c["y"].to(BF16)))
    with pytest.raises(TypeError):
        run(dict(c, x=c["x"].int()))
    with pytest.raises(ValueError):
        run(dict(c, u=c["u"][:, :1].contiguous()))
    with pytest.raises(ValueError):
        run(dict(c, noise=c["noise"][:, :49]))
    with pytest.raises(ValueError):
        run(dict(c, y=c["y"][:, :1]))
    with pytest.raises(ValueError):
        run(dict(c, z=c["z"].transpose(1, 2)))
    with pytest.raises(ValueError):
        run(dict(c, z=c["z"][:1].expand(3, 3, 50)))
    with pytest.raises(ValueError):
        run(dict(c, lens=torch.zeros(2, dtype=torch.int32, device="cuda")))
