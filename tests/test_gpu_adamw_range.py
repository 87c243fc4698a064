"""AdamW where the squares of gradients leave float32's normal range, against the
formula in float32: moments operation by operation, what follows in float64.

Tolerances, fixed before the first run (u = 2^-24).  The moments of 32-bit states are
the same float32 numbers.  From them the root, its bias correction (two roundings), the sum with
eps, the reciprocal (2 u), the first moment's correction (two) and the quotient are off
by 9 u of the update; lr and its product add 2 u of the update and of the decay, and w' is
rounded once.  States in 8 bits are read as code * scale in float32, and written off by
half a step of e4m3 (2^-4 of the value, 2^-10 of the scale near 0, a whole smallest step
for roots, which never become 0) of a scale that has the roundings of 1 / 448, of its product
and, for roots, of the root itself: 3 u."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
U = 2.0 ** -24
LR, B1, B2, DECAY = 1e-3, 0.9, 0.999, 0.1
MAX_ROOT = float(np.nextafter(np.float32(2.0 ** 64), np.float32(0)))  # of the largest float


def g():
    from vocab_wide_logprob_gb300 import _native
    return _native


def host(t):
    return t.detach().reshape(-1).float().cpu().numpy()


def moments(state, k):
    """m and v of tensor k as the step reads them, float32."""
    m = host(state["exp_avg"][k])
    if "scales" not in state:
        return m, host(state["exp_avg_sq"][k])
    sc = np.repeat(state["scales"][k].cpu().numpy(), 256, axis=0)[:m.size]
    root = host(state["exp_avg_root"][k]) * sc[:, 1]
    return m * sc[:, 0], root * root


def keep(params, state):
    return [p.clone() for p in params], {k: [None if t is None else t.clone() for t in v] for k, v in state.items()}


@np.errstate(over="ignore", under="ignore", invalid="ignore", divide="ignore")
def check(was, params, grads, state, step, eps):
    f = np.float32
    for k, p in enumerate(params):
        gr = host(grads[k])
        m, v = moments(was[1], k)
        m = m * f(B1) + gr * f(1 - B1)
        v = v * f(B2) + gr * gr * f(1 - B2)
        assert m.dtype == v.dtype == f
        root = np.sqrt(v.astype(np.float64))
        up = m.astype(np.float64) / (1 - B1 ** step) / (root / np.sqrt(1 - B2 ** step) + eps)
        master = state.get("master", [None] * len(params))[k]
        w0 = host(was[0][k] if master is None else was[1]["master"][k]).astype(np.float64)
        w = w0 - LR * (up + DECAY * w0)
        tol = LR * (11 * U * np.abs(up) + 4 * U * DECAY * np.abs(w0)) + 1.01 * U * np.abs(w) + 1e-45
        got = host(p if master is None else master).astype(np.float64)
        if master is None and p.dtype == BF16:
            tol = tol + 2.0 ** -8 * 1.0001 * np.abs(w)
        assert np.isfinite(w).all() and (np.abs(got - w) <= tol).all(), np.abs(got - w).max()
        if "scales" not in state:
            assert np.array_equal(host(state["exp_avg"][k]), m) and np.array_equal(host(state["exp_avg_sq"][k]), v)
            continue
        # (an infinite root as one that is finite and not below m')
        stored = np.where(np.isinf(root), np.maximum(MAX_ROOT, np.abs(m)), root)
        pad = lambda x: np.pad(np.abs(x).astype(np.float64), (0, -x.size % 256)).reshape(-1, 256)
        sc = state["scales"][k].cpu().numpy().astype(np.float64)
        each = np.repeat(sc, 256, axis=0)[:m.size]
        for j, want in ((0, m), (1, stored)):
            top = pad(want).max(1)
            assert (np.abs(sc[:, j] - top / 448) <= 3.01 * U * top / 448).all(), j
            code = host(state["exp_avg" if j == 0 else "exp_avg_root"][k]).astype(np.float64)
            near = np.maximum(2.0 ** -4 * np.abs(want), (2.0 ** -10 if j == 0 else 2.0 ** -9) * each[:, j])
            assert (np.abs(code * each[:, j] - want) <= near * 1.0001).all(), j
            assert j == 0 or ((code > 0) == (stored > 0)).all()


def start(n, sizes, kind, gts, bits, seed, exponents):
    """Zeroed states, and gradients of the given decimal exponents."""
    r = torch.Generator(device="cuda")
    r.manual_seed(seed)
    pts, master = {"f32": ([F32], False), "bf16": ([BF16], False), "master": ([BF16, F32], True)}[kind]
    params = [(torch.randn(s, generator=r, device="cuda") * 0.02).to(pts[k % len(pts)]) for k, s in enumerate(sizes)]
    state = n.grpo_adamw_state(params, bits, master=master)

    def gradients():
        out = []
        for k, s in enumerate(sizes):
            lo, hi = exponents
            x = 10.0 ** (torch.rand(s, generator=r, device="cuda", dtype=torch.float64) * (hi - lo) + lo)
            sign = torch.randint(0, 2, (s,), generator=r, device="cuda") * 2 - 1
            out.append((x * sign).to(gts[k % len(gts)]))
        return out

    return params, state, gradients


KINDS, GTS = ["f32", "bf16", "master"], {"g32": [F32], "gmix": [BF16, F32]}
SIZES = [5000, 3, 2048, 257]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gts", GTS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("exponents", [(-20.4, -20), (-19.5, -18.5), (-20.4, -17), (-20.4, -2)], ids=str)
def test_squares_below_the_normal_range(exponents, kind, gts, bits):
    """Without eps a first step moves by lr, however small the gradient is (as far as
    float32 holds v')."""
    n = g()
    params, state, gradients = start(n, SIZES, kind, GTS[gts], bits, 1, exponents)
    for step in (1, 2, 3):
        grads = gradients()
        was = keep(params, state)
        n.grpo_adamw_step(params, grads, state, step, LR, beta1=B1, beta2=B2, eps=0.0, weight_decay=DECAY)
        check(was, params, grads, state, step, 0.0)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gts", GTS)
@pytest.mark.parametrize("kind", KINDS)
def test_squares_that_overflow(kind, gts, bits):
    """A finite gradient with an infinite square: m' / infinity is 0, the weight only
    decays; the rest of its block goes on."""
    n = g()
    params, state, gradients = start(n, SIZES, kind, GTS[gts], bits, 2, (-4, -2))
    for step in (1, 2, 3, 4):
        grads = gradients()
        if step == 2:
            for x, value in ((0, 1e20), (7, -3e25), (8, 1e38), (2500, -2e19), (4999, 1e21)):
                grads[0][x] = value
            grads[1][1] = 1e30
            grads[2][:256] = 1e22
        was = keep(params, state)
        n.grpo_adamw_step(params, grads, state, step, LR, beta1=B1, beta2=B2, eps=1e-8, weight_decay=DECAY)
        check(was, params, grads, state, step, 1e-8)
    assert all(torch.isfinite(t).all() for t in params)
    assert all(torch.isfinite(t.float()).all() for t in state["exp_avg"] + state.get("scales", []))


@pytest.mark.parametrize("bits", [32, 8])
def test_from_both_ends_at_once(bits):
    """Every exponent that a float32 gradient can have in one tensor."""
    n = g()
    params, state, gradients = start(n, [70000], "f32", [F32], bits, 3, (-20.4, 37))
    grads = gradients()
    was = keep(params, state)
    n.grpo_adamw_step(params, grads, state, 1, LR, beta1=B1, beta2=B2, eps=0.0, weight_decay=DECAY)
    check(was, params, grads, state, 1, 0.0)


def test_unused_rows_keep_the_code_zero():
    """What never had a gradient keeps the zero bytes that it began with, alone or beside
    others of its block."""
    n = g()
    r = torch.Generator(device="cuda")
    r.manual_seed(4)
    for pt in (F32, BF16):
        p = [torch.randn(s, generator=r, device="cuda").to(pt) for s in (4096, 100, 2500)]
        state = n.grpo_adamw_state(p, 8)
        grads = [torch.randn(x.shape, generator=r, device="cuda") for x in p]
        used = [torch.rand(x.shape, generator=r, device="cuda") < 0.5 for x in p]
        used[0][1024:2048] = False
        for x, u in zip(grads, used):
            x.mul_(u)
        for step in (1, 2, 3):
            n.grpo_adamw_step(p, grads, state, step, LR, weight_decay=DECAY)
            for key in ("exp_avg", "exp_avg_root"):
                for code, u in zip(state[key], used):
                    assert not code.view(torch.uint8)[~u].any(), key
            assert all((c.view(torch.uint8)[u] > 0).all() for c, u in zip(state["exp_avg_root"], used))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-50, 1e-40, 2.0 ** -127, 2.0 ** -126, 1e-30])
def test_an_eps_below_the_normal_range(eps, bits):
    """Keeps elements that never had a gradient from 0 / 0, as any other does."""
    n = g()
    params, state, gradients = start(n, [3000], "f32", [F32], bits, 5, (-9, -3))
    for step in (1, 2):
        grads = gradients()
        grads[0][::3] = 0.0
        grads[0][512:1024] = 0.0
        was = keep(params, state)
        n.grpo_adamw_step(params, grads, state, step, LR, beta1=B1, beta2=B2, eps=eps, weight_decay=DECAY)
        # (beside roots of 10^-11 and more all of these are nothing)
        check(was, params, grads, state, step, max(eps, 2.0 ** -126))
