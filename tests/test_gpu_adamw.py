"""AdamW over many tensors against float64.

Tolerances, fixed before the first run (u = 2^-24).  The clipping coefficient is
off by 3 u, so g by 4 u; m' = b1 m + (1 - b1) g by 8 u of the sum of its terms' magnitudes
M, v' (positive terms, g twice) by 16 u, its root by 8 u and the root's
instruction (2 u); the bias corrections (given by the host to one rounding, or by
the device to 4 u more) and the quotient (4 u) add to 24 u of the update's own
size and 8 u of M's share.  w' adds the products with lr (4 u of the change), half a
step of float32 and, for a bfloat16 param, half a step of its own.
States in 8 bits: the value that is read has one more rounding (2 u, in all the above).
What is written is off by half a step of e4m3: 2^-4 of the value, 2^-10 of the scale near 0
(a whole smallest step, 2^-9, for roots, which never become 0), and the scale's
rounding."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
U = 2.0 ** -24
HYPER = dict(beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)


def g():
    from vocab_wide_logprob_gb300 import _native
    return _native


def gen(seed):
    r = torch.Generator(device="cuda")
    r.manual_seed(seed)
    return r


def at_phase(x, phase):
    """The values of x in memory that begins `phase` elements behind a boundary."""
    raw = torch.empty(x.numel() + phase, dtype=torch.uint8 if x.dtype == F8 else x.dtype, device="cuda")
    raw = raw[phase:]
    raw.copy_((x.view(torch.uint8) if x.dtype == F8 else x).reshape(-1))
    return (raw.view(F8) if x.dtype == F8 else raw).view(x.shape)


def blocks(x):
    """[blocks of 256, 256] of a flat tensor, zeros behind its end."""
    x = x.reshape(-1)
    return torch.nn.functional.pad(x, (0, -x.numel() % 256)).view(-1, 256)


def make(sizes, pts, gts, bits, master, seed, phases=(0,), spread=1.0):
    r = gen(seed)
    params, grads = [], []
    state = {"exp_avg": [], "exp_avg_sq" if bits == 32 else "exp_avg_root": []}
    if bits == 8:
        state["scales"] = []
    if master:
        state["master"] = []
    rnd = lambda s: torch.randn(s, generator=r, device="cuda")
    for k, s in enumerate(sizes):
        ph, pt = phases[k % len(phases)], pts[k % len(pts)]
        w = rnd(s) * 0.02
        params.append(at_phase(w.to(pt), ph))
        grads.append(at_phase((rnd(s) * 1e-3 * spread).to(gts[k % len(gts)]), ph))
        m, root = rnd(s) * 3e-4 * spread, (rnd(s).abs() + 0.3) * 1e-3 * spread
        if bits == 32:
            state["exp_avg"].append(at_phase(m, ph))
            state["exp_avg_sq"].append(at_phase(root * root, ph))
        else:
            bm, br = blocks(m), blocks(root)
            sm, sr = bm.abs().amax(1) / 448, br.amax(1) / 448
            n = m.numel()
            code = lambda b, sc: at_phase((b / sc.clamp(min=1e-30)[:, None]).view(-1)[:n].view(s).to(F8), ph)
            state["exp_avg"].append(code(bm, sm))
            state["exp_avg_root"].append(code(br, sr))
            state["scales"].append(torch.stack([sm, sr], 1).contiguous())
        if master:
            state["master"].append(at_phase(w, ph) if pt == BF16 else None)
    return params, grads, state


def copies(params, grads, state):
    return ([p.clone() for p in params], [None if t is None else t.clone() for t in grads],
            {k: [None if t is None else t.clone() for t in v] for k, v in state.items()})


def state64(state, k):
    """m and sqrt(v) of tensor k in float64."""
    m = state["exp_avg"][k].reshape(-1)
    if "scales" not in state:
        return m.double(), state["exp_avg_sq"][k].reshape(-1).double().sqrt()
    n = m.numel()
    sc = state["scales"][k].double()
    back = lambda c, j: (blocks(c.float().double()) * sc[:, j:j + 1]).view(-1)[:n]
    return back(m, 0), back(state["exp_avg_root"][k].reshape(-1), 1)


def check(before, after, step, lr, coef=1.0, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1):
    """after = the step of before, tensor by tensor."""
    for k in range(len(before[0])):
        grad = before[1][k]
        if grad is None:
            for a, b in zip((before[0], *before[2].values()), (after[0], *after[2].values())):
                assert a[k] is None or torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8))
            continue
        gr = grad.reshape(-1).double() * coef
        m0, r0 = state64(before[2], k)
        m = beta1 * m0 + (1 - beta1) * gr
        M = beta1 * m0.abs() + (1 - beta1) * gr.abs()
        v = beta2 * r0 * r0 + (1 - beta2) * gr * gr
        c1, c2 = -math.expm1(step * math.log(beta1)) if beta1 else 1.0, \
            -math.expm1(step * math.log(beta2)) if beta2 else 1.0
        den = (v / c2).sqrt() + eps
        up = m / c1 / den
        masters = before[2].get("master")
        master = masters is not None and masters[k] is not None
        w0 = (masters[k] if master else before[0][k]).reshape(-1).double()
        w = w0 - lr * (up + weight_decay * w0)
        err = lr * (24 * U * up.abs() + 10 * U * M / c1 / den + 4 * U * (up.abs() + weight_decay * w0.abs()))
        err = err + 2 * U * w.abs() + 1e-40
        if master:
            got = after[2]["master"][k].reshape(-1).double()
            assert ((got - w).abs() <= err).all()
            # the param is the master, rounded
            assert torch.equal(after[0][k], after[2]["master"][k].to(BF16))
        else:
            half = torch.finfo(before[0][k].dtype).eps / 2 * 1.001 if before[0][k].dtype == BF16 else 0.0
            got = after[0][k].reshape(-1).double()
            bad = (got - w).abs() > err + half * w.abs()
            assert not bad.any(), (k, got[bad][:5], w[bad][:5], err[bad][:5])
        if "scales" not in after[2]:
            assert ((after[2]["exp_avg"][k].reshape(-1).double() - m).abs() <= 8 * U * M + 1e-44).all()
            assert ((after[2]["exp_avg_sq"][k].reshape(-1).double() - v).abs() <= 16 * U * v + 1e-44).all()
            continue
        root = v.sqrt()
        sc = after[2]["scales"][k].double()
        top_m, top_r = blocks(m).abs().amax(1), blocks(root).amax(1)
        most = blocks(M).amax(1)
        assert ((sc[:, 0] - top_m / 448).abs() <= (10 * U * most + 4 * U * top_m) / 448 + 1e-40).all()
        assert ((sc[:, 1] - top_r / 448).abs() <= 16 * U * top_r / 448 + 1e-40).all()
        m1, r1 = state64(after[2], k)
        each = sc.repeat_interleave(256, 0)[:m.numel()]
        # half a step of the code; behind it the rounding of what was encoded
        tol = torch.maximum(2.0 ** -4 * m.abs(), 2.0 ** -10 * each[:, 0]) * 1.0001 + 10 * U * M
        assert ((m1 - m).abs() <= tol).all()
        tol = torch.maximum(2.0 ** -4 * root, 2.0 ** -9 * each[:, 1]) * 1.0001 + 16 * U * root
        assert ((r1 - root).abs() <= tol).all()
        assert ((r1 > 0) | (root < 1e-30)).all()


SIZES = [[1], [3, 0, 7], [255, 256, 257, 2047, 2048, 2049], [100000, 1, 33333], [(17, 31), (5, 3, 64)],
         [17] * 600 + [5000], [1000003]]
KINDS = [("f32", [F32], False), ("bf16", [BF16], False), ("master", [BF16], True), ("mixed", [BF16, F32], True)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gts", [[F32], [BF16], [F32, BF16, BF16]], ids=["g32", "g16", "gmix"])
@pytest.mark.parametrize("kind", KINDS, ids=[k[0] for k in KINDS])
@pytest.mark.parametrize("sizes", SIZES, ids=range(len(SIZES)))
def test_step(sizes, kind, gts, bits):
    n = g()
    was = make(sizes, kind[1], gts, bits, kind[2], 1)
    now = copies(*was)
    assert n.grpo_adamw_step(*now, 7, 1e-3, **HYPER) is None
    check(was, now, 7, 1e-3, **HYPER)
    assert all(torch.equal(a, b) for a, b in zip(was[1], now[1]))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kind", KINDS, ids=[k[0] for k in KINDS])
def test_any_alignment(kind, bits):
    n = g()
    sizes = [5000, 777, 4096, 300, 2500, 9]
    for phases in ((1,), (4, 8, 2), (8,), (16, 3)):
        was = make(sizes, kind[1], [F32, BF16], bits, kind[2], 2, phases)
        now = tuple([at_phase(t, phases[k % len(phases)]) if t is not None else None
                     for k, t in enumerate(x)] if isinstance(x, list) else
                    {key: [t if t is None else t.clone() if key == "scales" else
                           at_phase(t, phases[k % len(phases)]) for k, t in enumerate(v)]
                     for key, v in x.items()} for x in was)
        n.grpo_adamw_step(*now, 3, 1e-2, **HYPER)
        check(was, now, 3, 1e-2, **HYPER)


@pytest.mark.parametrize("bits", [32, 8])
def test_the_first_steps_from_nothing(bits):
    """Zeroed states; five steps, each checked from the state it found."""
    n = g()
    params, _, _ = make([1000, 300, (40, 40)], [BF16, F32], [F32], 32, False, 3)
    state = n.grpo_adamw_state(params, bits, master=True)
    assert [t is None for t in state["master"]] == [False, True, False]
    r = gen(4)
    for step in range(1, 6):
        grads = [torch.randn(p.shape, generator=r, device="cuda") * 10.0 ** -step for p in params]
        grads[0][:400] = 0.0  # rows of an embedding that nobody used
        was = copies(params, grads, state)
        n.grpo_adamw_step(params, grads, state, step, 1e-3, **HYPER)
        check(was, (params, grads, state), step, 1e-3, **HYPER)
    assert all(t.isfinite().all() for t in params)
    m, root = state64(state, 0)
    assert (m[:400] == 0).all() and (root[:400] == 0).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("betas", [(0.0, 0.999), (0.9, 0.0), (0.0, 0.0), (0.99, 0.9999)])
@pytest.mark.parametrize("step", [1, 2, 1000, 10 ** 7])
def test_hyperparameters(betas, step, bits):
    n = g()
    for eps, decay, lr in ((1e-8, 0.0, 1e-6), (1e-3, 0.5, 0.1), (0.0, 0.01, 0.0)):
        was = make([3000], [F32], [F32], bits, False, 5)
        now = copies(*was)
        h = dict(beta1=betas[0], beta2=betas[1], eps=eps, weight_decay=decay)
        n.grpo_adamw_step(*now, step, lr, **h)
        check(was, now, step, lr, **h)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("over", [0.3, 1.0, 5.0, float("inf")])
def test_clipping_on_the_way(over, bits):
    """The same as clipping the gradients first, without writing them."""
    n = g()
    was = make([5000, 77, 2048], [F32, BF16], [F32, BF16], bits, False, 6)
    now = copies(*was)
    stats, _ = n.grpo_grad_norm(now[1])
    norm = float(stats[0])
    limit = over * norm
    n.grpo_adamw_step(*now, 4, 1e-3, norm=stats, max_norm=limit, **HYPER)
    check(was, now, 4, 1e-3, min(1.0, limit / (norm + 1e-6)), **HYPER)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_norm_that_is_not_finite_skips_the_step(bad):
    n = g()
    for bits in (32, 8):
        was = make([5000, 77], [F32, BF16], [F32], bits, True, 7)
        was[1][1][5] = bad
        now = copies(*was)
        stats, ws = n.grpo_grad_norm(now[1])
        assert n.grpo_check_error(ws) == 9
        n.grpo_adamw_step(*now, 4, 1e-3, norm=stats, max_norm=1.0, **HYPER)
        for a, b in zip([was[0], *was[2].values()], [now[0], *now[2].values()]):
            for x, y in zip(a, b):
                assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_values_that_are_not_finite_stay_visible():
    """Without the norm: NaN and infinity reach what they belong to (a block of 8-bit
    states as a whole), and nothing else."""
    n = g()
    for bits in (32, 8):
        for bad in (float("nan"), float("inf")):
            p, gr, st = make([2048], [F32], [F32], bits, False, 8)
            gr[0][700] = bad
            n.grpo_adamw_step(p, gr, st, 4, 1e-3, **HYPER)
            rest = torch.ones(2048, dtype=torch.bool, device="cuda")
            rest[700] = False
            assert p[0][rest].isfinite().all() and not p[0][700].isfinite()
            m, root = state64(st, 0)
            rest[512:768] = False
            assert m[rest].isfinite().all() and root[rest].isfinite().all()
            assert not m[700].isfinite() and not root[700].isfinite()


def test_shapes_that_do_not_fit_are_refused():
    n = g()
    p, gr, st = make([(6, 10), 50], [F32], [F32], 32, False, 20)
    for bad in ([gr[0].t().contiguous(), gr[1]], [gr[0], gr[1][:49].contiguous()], [gr[0].t(), gr[1]]):
        with pytest.raises(ValueError):
            n.grpo_adamw_step(p, bad, st, 1, 1e-3)
    with pytest.raises(ValueError):
        n.grpo_adamw_step([p[0].t(), p[1]], gr, st, 1, 1e-3)
    with pytest.raises(n.GrpoError):
        n.grpo_adamw_step([p[0], p[0]], [gr[0], gr[0]], {k: [v[0], v[0].clone()] for k, v in st.items()}, 1, 1e-3)


def test_params_without_gradients_and_empty_ones():
    n = g()
    for bits in (32, 8):
        was = make([5000, 77, 0, 300], [F32, BF16], [F32], bits, True, 9)
        was[1][1] = None
        was[1][3] = None
        now = copies(*was)
        n.grpo_adamw_step(*now, 4, 1e-3, **HYPER)
        check(was, now, 4, 1e-3, **HYPER)
        n.grpo_adamw_step([], [], {k: [] for k in was[2]}, 1, 1e-3)
        n.grpo_adamw_step(now[0], [None] * 4, now[2], 5, 1e-3)


@pytest.mark.parametrize("spread", [1e-30, 1e-18, 1e-10, 1e10, 1e18])
@pytest.mark.parametrize("bits", [32, 8])
def test_small_and_large_gradients(spread, bits):
    """Squares near the ends of float32's range (v of 1e-36 has a root that is far from
    it; below 1e-38 they lose digits in any float32 sum, and nothing is asked but order)."""
    n = g()
    was = make([3000], [F32], [F32], bits, False, 10, spread=spread)
    now = copies(*was)
    n.grpo_adamw_step(*now, 4, 1e-3, **{**HYPER, "eps": 0.0 if spread > 1e-15 else 1e-8})
    if spread >= 1e-10:
        check(was, now, 4, 1e-3, **{**HYPER, "eps": 0.0})
    assert now[0][0].isfinite().all()
    assert (now[0][0] - was[0][0]).abs().max() <= 1e-3 * 20


def test_blocks_of_very_different_values():
    """8 bits: a block with one value of 2^40 times the rest; roots far below the
    largest stay positive."""
    n = g()
    p, gr, st = make([1024], [F32], [F32], 32, False, 11)
    st = n.grpo_adamw_state(p, 8)
    gr[0][::256] = 1e9
    was = copies(p, gr, st)
    n.grpo_adamw_step(p, gr, st, 1, 1e-3, **HYPER)
    check(was, (p, gr, st), 1, 1e-3, **HYPER)
    was = copies(p, gr, st)
    n.grpo_adamw_step(p, gr, st, 2, 1e-3, **HYPER)
    assert p[0].isfinite().all() and (p[0] - was[0][0]).abs().max() <= 2e-3


def test_results_repeat_and_versions():
    n = g()
    for bits in (32, 8):
        was = make([70000, 333], [BF16, F32], [BF16], bits, True, 12)
        a, b = copies(*was), copies(*was)
        versions = [t._version for t in (a[0][0], a[2]["exp_avg"][0], a[2]["master"][0])]
        n.grpo_adamw_step(*a, 4, 1e-3, **HYPER)
        n.grpo_adamw_step(*b, 4, 1e-3, **HYPER)
        assert [t._version for t in (a[0][0], a[2]["exp_avg"][0], a[2]["master"][0])] == \
            [v + 1 for v in versions]
        for x, y in zip([a[0], *a[2].values()], [b[0], *b[2].values()]):
            assert all(s is None or torch.equal(s.view(torch.uint8), t.view(torch.uint8))
                       for s, t in zip(x, y))


def test_step_and_rate_on_the_device_in_a_graph():
    n = g()
    for bits in (32, 8):
        p, gr, st = make([9000, 333], [BF16, F32], [F32], bits, True, 13)
        step = torch.zeros(1, dtype=torch.int64, device="cuda")
        rate = torch.zeros(1, device="cuda")
        stats = torch.zeros(2, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step += 1
            n.grpo_grad_norm(gr, stats=stats)
            n.grpo_adamw_step(p, gr, st, step, rate, norm=stats, max_norm=0.01, **HYPER)
        r = gen(14)
        for t in range(1, 4):
            for x in gr:
                x.copy_(torch.randn(x.shape, generator=r, device="cuda") * 1e-3 * t)
            rate.fill_(1e-3 / t)
            was = copies(p, gr, st)
            graph.replay()
            torch.cuda.synchronize()
            norm = float(stats[0])
            check(was, (p, gr, st), t, float(rate), min(1.0, 0.01 / (norm + 1e-6)), **HYPER)


def test_another_stream():
    n = g()
    was = make([500000], [BF16], [BF16], 32, True, 15)
    a = copies(*was)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n.grpo_adamw_step(*a, 4, 1e-3, stream=side, **HYPER)
    side.synchronize()
    check(was, a, 4, 1e-3, **HYPER)


def test_a_tensor_beyond_two_to_the_31_elements():
    n = g()
    size = 2 ** 31 + 5000
    p = torch.zeros(size, dtype=BF16, device="cuda")
    gr = torch.zeros(size, dtype=BF16, device="cuda")
    st = n.grpo_adamw_state([p], 8)
    tail = slice(size - 3000, size)
    p[tail].normal_(generator=gen(16))
    gr[tail].normal_(generator=gen(17))
    # (the checked piece begins at a block of its own)
    cut = slice((size - 3000) // 256 * 256, size)
    pick = lambda: ([p[cut].clone()], [gr[cut].clone()],
                    {"exp_avg": [st["exp_avg"][0][cut].clone()],
                     "exp_avg_root": [st["exp_avg_root"][0][cut].clone()],
                     "scales": [st["scales"][0][cut.start // 256:].clone()]})
    was = pick()
    n.grpo_adamw_step([p], [gr], st, 1, 1e-2, **HYPER)
    check(was, pick(), 1, 1e-2, **HYPER)
    assert not p[:1000000].any()


def test_eight_bits_follow_thirty_two():
    """The same gradients for sixty steps: the updates with 8-bit states stay near
    those with 32 (half a step of e4m3, 6%, in each of m and the root, and what the
    roundings of sixty steps leave in the moments)."""
    n = g()
    r = gen(18)
    p32 = [torch.zeros(4096, device="cuda")]
    p8 = [torch.zeros(4096, device="cuda")]
    s32, s8 = n.grpo_adamw_state(p32), n.grpo_adamw_state(p8, 8)
    slope = torch.randn(4096, generator=r, device="cuda")
    for step in range(1, 61):
        grad = [slope + 0.5 * torch.randn(4096, generator=r, device="cuda")]
        n.grpo_adamw_step(p32, grad, s32, step, 1e-3, weight_decay=0.0)
        n.grpo_adamw_step(p8, grad, s8, step, 1e-3, weight_decay=0.0)
    off = (p8[0] - p32[0]).norm() / p32[0].norm()
    assert off < 0.25, off
