"""Embedding lookup and its gradient against the definition in float64.

Tolerances, fixed before the first run: the forward rounds the float32 product
once (2^-24 relative) and the result once to its type (half a step, 2^-8 for
bfloat16); the backward adds the c rows of an id in float32, an error of at
most c * 2^-24 of the sum of their magnitudes, scales (2^-24) and rounds once
(accumulating adds one more float32 rounding of the total)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def g():
    from vocab_wide_logprob_gb300 import _native
    return _native


def half_step(dt):
    return torch.finfo(dt).eps / 2


def gen(seed):
    r = torch.Generator(device="cuda")
    r.manual_seed(seed)
    return r


def draw_ids(n, V, seed, law="zipf"):
    r = gen(seed)
    if law == "uniform":
        return torch.randint(0, V, (n,), generator=r, device="cuda")
    if law == "one":
        return torch.full((n,), V // 2, dtype=torch.int64, device="cuda")
    x = torch.rand(n, generator=r, device="cuda", dtype=torch.float64)
    return (torch.exp(x * float(np.log(V + 1))).long() - 1).clamp_(0, V - 1)


def check_fwd(out, ids, weight, scale):
    V = weight.shape[0]
    ok = (ids >= 0) & (ids < V)
    want = weight.double()[ids.clamp(0, V - 1)] * scale
    got = out.double().view(want.shape)
    assert torch.isnan(got[~ok]).all()
    err = (got - want).abs()[ok]
    assert (err <= want[ok].abs() * (2.0 ** -24 + half_step(out.dtype) * 1.001)).all()


@pytest.mark.parametrize("wdt,odt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("n,V,d", [(1, 1, 1), (3, 7, 8), (5, 100, 130), (17, 257, 901), (64, 1024, 896),
                                   (1000, 300, 64), (9, 50, 4099), (2, 33, 20000)])
def test_forward(n, V, d, wdt, odt):
    w = torch.randn(V, d, generator=gen(1), device="cuda").to(wdt)
    ids = draw_ids(n, V, 2, "uniform")
    check_fwd(g().grpo_embed_fwd(ids, w, 1.0, out_dtype=odt), ids, w, 1.0)
    check_fwd(g().grpo_embed_fwd(ids, w, 11.3125, out_dtype=odt), ids, w, 11.3125)


def test_forward_same_type_is_a_copy():
    w = torch.randn(100, 896, generator=gen(3), device="cuda").to(BF16)
    ids = draw_ids(4096, 100, 4).view(64, 64)
    out = g().grpo_embed_fwd(ids, w)
    assert out.shape == (64, 64, 896) and torch.equal(out, w[ids])


def test_forward_views_of_wider_rows_and_odd_addresses():
    n = g()
    buf = torch.randn(50, 100, generator=gen(5), device="cuda").to(BF16)
    ids = draw_ids(33, 50, 6)
    for lo, hi in ((0, 64), (1, 65), (8, 96), (3, 100)):
        w = buf[:, lo:hi]
        out_buf = torch.full((33, 120), 7.0, device="cuda")
        out = out_buf[:, 5:5 + hi - lo]
        n.grpo_embed_fwd(ids, w, 1.0, out=out)
        assert torch.equal(out, w[ids].float())
        assert (out_buf[:, :5] == 7).all() and (out_buf[:, 5 + hi - lo:] == 7).all()


@pytest.mark.parametrize("wdt,odt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("n,d", [(1, 257), (700, 33), (3001, 160), (3001, 161), (700, 515), (5000, 901),
                                 (40, 8192), (3000, 64)])
@pytest.mark.parametrize("lo", [1, 4, 8])
def test_forward_at_any_alignment(n, d, lo, wdt, odt):
    """Tables with NaN around their rows, ids outside, outputs in wider rows."""
    V = 211
    buf = torch.full((V, d + 16), float("nan"), device="cuda", dtype=wdt)
    w = buf[:, lo:lo + d]
    w.copy_(torch.randn(V, d, generator=gen(7), device="cuda"))
    ids = draw_ids(n, V, 8)
    ids[n // 2] = V
    out_buf = torch.full((n, d + 16), 7.0, device="cuda", dtype=odt)
    out = out_buf[:, lo:lo + d]
    g().grpo_embed_fwd(ids, w, 3.5, out=out)
    check_fwd(out, ids, w, 3.5)
    assert (out_buf[:, :lo] == 7).all() and (out_buf[:, lo + d:] == 7).all()


def test_forward_ids_outside_give_nan_rows():
    w = torch.randn(10, 24, device="cuda")
    ids = torch.tensor([0, -1, 9, 10, 1 << 40, -(1 << 62), 3], device="cuda")
    check_fwd(g().grpo_embed_fwd(ids, w), ids, w, 1.0)


def test_forward_nonfinite_weights_pass_through():
    w = torch.zeros(4, 8, device="cuda", dtype=BF16)
    w[1] = float("inf")
    w[2] = float("nan")
    w[3] = -float("inf")
    out = g().grpo_embed_fwd(torch.arange(4, device="cuda"), w, 2.0)
    assert torch.equal(out[1], w[1]) and torch.isnan(out[2]).all() and torch.equal(out[3], w[3])


def test_forward_empty():
    w = torch.randn(4, 8, device="cuda")
    assert g().grpo_embed_fwd(torch.empty(0, dtype=torch.int64, device="cuda"), w).shape == (0, 8)


# ---------------------------------------------------------------------------


def grad64(ids, dout, V, scale, pad):
    """Sums and sums of magnitudes per id, and the counts, in float64."""
    ids, x = ids.reshape(-1), dout.reshape(-1, dout.shape[-1]).double()
    use = (ids >= 0) & (ids < V)
    if pad is not None:
        use &= ids != pad
    s = torch.zeros(V, x.shape[1], dtype=torch.float64, device="cuda")
    m = torch.zeros_like(s)
    c = torch.zeros(V, dtype=torch.float64, device="cuda")
    s.index_add_(0, ids[use], x[use])
    m.index_add_(0, ids[use], x[use].abs())
    c.index_add_(0, ids[use], torch.ones_like(ids[use], dtype=torch.float64))
    return s * scale, m * abs(scale), c.view(-1, 1)


def check_bwd(dw, ids, dout, scale=1.0, pad=None, base=None):
    s, m, c = grad64(ids, dout, dw.shape[0], scale, pad)
    total = s if base is None else s + base.double()
    tol = (c + 1) * 2.0 ** -24 * m + total.abs() * half_step(dw.dtype) * 1.001
    if base is not None:
        tol = tol + (s.abs() + base.double().abs()) * 2.0 ** -23
    err = (dw.double() - total).abs()
    assert (err <= tol + 1e-300).all(), float((err - tol).max())
    if base is None:
        assert (dw[(c == 0).view(-1)] == 0).all()
    else:
        assert torch.equal(dw[(c == 0).view(-1)], base[(c == 0).view(-1)])


@pytest.mark.parametrize("ddt,wdt", [(F32, F32), (BF16, F32), (F32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("n,V,d,law", [(1, 1, 1, "one"), (2, 5, 8, "uniform"), (31, 7, 16, "zipf"),
                                       (33, 500, 130, "uniform"), (257, 100, 901, "zipf"),
                                       (2049, 1024, 64, "zipf"), (5000, 3000, 8, "zipf"),
                                       (4097, 70000, 24, "uniform"), (700, 300000, 8, "zipf"),
                                       (300, 11, 2056, "zipf"), (260, 9, 2057, "uniform"),
                                       (10000, 3, 40, "one")])
def test_gradient(n, V, d, law, ddt, wdt):
    ids = draw_ids(n, V, 10, law)
    dout = torch.randn(n, d, generator=gen(11), device="cuda").to(ddt)
    dw, ws = g().grpo_embed_bwd(ids, dout, V, out_dtype=wdt)
    assert g().grpo_check_error(ws) == 0
    check_bwd(dw, ids, dout)
    base = torch.randn(V, d, generator=gen(12), device="cuda").to(wdt)
    acc, _ = g().grpo_embed_bwd(ids, dout, V, -2.5, pad_id=int(ids[0]), dweight=base.clone(),
                                accumulate=True, workspace=ws)
    check_bwd(acc, ids, dout, -2.5, int(ids[0]), base)


@pytest.mark.parametrize("n", [2047, 2048, 2049, 4096, 100000, 700001])
def test_gradient_sort_sizes(n):
    """Token counts around the sort's tiles; every id of a two-level range."""
    V, d = 200003, 8
    ids = draw_ids(n, V, 20)
    dout = torch.randn(n, d, generator=gen(21), device="cuda")
    dw, _ = g().grpo_embed_bwd(ids, dout, V)
    check_bwd(dw, ids, dout)


def test_gradient_is_reproducible_and_in_token_order():
    ids = draw_ids(5000, 50, 30)
    dout = torch.randn(5000, 72, generator=gen(31), device="cuda")
    a, ws = g().grpo_embed_bwd(ids, dout, 50)
    for _ in range(3):
        ws.fill_(255)
        b, _ = g().grpo_embed_bwd(ids, dout, 50, workspace=ws)
        assert torch.equal(a, b)
    # few tokens of one id: the plain float32 sum in token order
    ids = torch.tensor([4, 2, 4, 4, 2], device="cuda")
    x = torch.randn(5, 16, generator=gen(32), device="cuda")
    dw, _ = g().grpo_embed_bwd(ids, x, 6)
    assert torch.equal(dw[4], (x[0] + x[2]) + x[3]) and torch.equal(dw[2], x[1] + x[4])


def test_gradient_skips_pads_and_reports_ids_outside():
    n = g()
    ids = torch.tensor([1, 5, 1, -3, 99, 5, 0], device="cuda")
    x = torch.randn(7, 40, generator=gen(40), device="cuda")
    x[1] = float("nan")  # a pad's gradient is not read into any sum
    x[3] = float("inf")
    dw, ws = n.grpo_embed_bwd(ids, x, 10, pad_id=5)
    assert n.grpo_check_error(ws) == 6
    check_bwd(dw, ids, torch.nan_to_num(x, 0.0, 0.0, 0.0), 1.0, 5)
    # the next call on the workspace starts clean; a pad id outside the table is no error
    ids = torch.tensor([1, -100, 2], device="cuda")
    dw, ws = n.grpo_embed_bwd(ids, x[:3].nan_to_num(), 10, workspace=ws)
    assert n.grpo_check_error(ws) == 6
    ids = torch.tensor([1, 10, 2], device="cuda")
    dw, ws = n.grpo_embed_bwd(ids, x[:3].nan_to_num(), 10, pad_id=10, workspace=ws)
    assert n.grpo_check_error(ws) == 0
    check_bwd(dw, ids, x[:3].nan_to_num(), 1.0, 10)
    # nothing but pads
    dw, _ = n.grpo_embed_bwd(torch.full((500,), 7, device="cuda"), torch.ones(500, 40, device="cuda"),
                             10, pad_id=7)
    assert (dw == 0).all()


def test_gradient_nonfinite_rows_reach_their_id_only():
    ids = torch.tensor([0, 1, 2, 1], device="cuda")
    x = torch.ones(4, 16, device="cuda")
    x[1, 3] = float("inf")
    x[2, 5] = float("nan")
    dw, _ = g().grpo_embed_bwd(ids, x, 4)
    assert torch.isinf(dw[1, 3]) and torch.isnan(dw[2, 5]) and torch.isfinite(dw[0]).all()
    assert torch.isfinite(dw).sum() == dw.numel() - 2


def test_gradient_into_views_and_from_views():
    n = g()
    ids = draw_ids(100, 20, 50)
    buf = torch.randn(100, 64, generator=gen(51), device="cuda").to(BF16)
    for lo, hi in ((0, 32), (1, 33), (5, 64)):
        out_buf = torch.full((20, 80), 3.0, device="cuda")
        view = out_buf[:, 7:7 + hi - lo]
        n.grpo_embed_bwd(ids, buf[:, lo:hi], 20, dweight=view)
        check_bwd(view, ids, buf[:, lo:hi])
        assert (out_buf[:, :7] == 3).all() and (out_buf[:, 7 + hi - lo:] == 3).all()


@pytest.mark.parametrize("ddt,wdt", [(F32, F32), (BF16, F32), (F32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("n,d", [(1, 257), (900, 33), (3001, 160), (700, 515), (6000, 901), (40, 8192),
                                 (3000, 64)])
@pytest.mark.parametrize("lo", [1, 4])
def test_gradient_at_any_alignment(n, d, lo, ddt, wdt):
    """Gradients with NaN around their rows, results in wider rows."""
    V = 97
    buf = torch.full((n, d + 16), float("nan"), device="cuda", dtype=ddt)
    x = buf[:, lo:lo + d]
    x.copy_(torch.randn(n, d, generator=gen(52), device="cuda"))
    ids = draw_ids(n, V, 53)
    out_buf = torch.full((V, d + 16), 3.0, device="cuda", dtype=wdt)
    view = out_buf[:, lo:lo + d]
    g().grpo_embed_bwd(ids, x, V, dweight=view)
    check_bwd(view, ids, x)
    base = torch.randn(V, d, generator=gen(54), device="cuda").to(wdt)
    view.copy_(base)
    g().grpo_embed_bwd(ids, x, V, 0.5, dweight=view, accumulate=True)
    check_bwd(view, ids, x, 0.5, None, base)
    assert (out_buf[:, :lo] == 3).all() and (out_buf[:, lo + d:] == 3).all()


@pytest.mark.parametrize("n", [1, 512, 1023, 1024, 1025, 3000])
@pytest.mark.parametrize("V", [2, 70, 600, 300000])
def test_gradient_of_few_tokens(n, V):
    """Tokens sorted by one block, two to eight of them per thread."""
    ids = draw_ids(n, V, 55)
    ids[::7] = V + 3
    x = torch.randn(n, 24, generator=gen(56), device="cuda")
    dw, ws = g().grpo_embed_bwd(ids, x, V)
    assert g().grpo_check_error(ws) == 6
    check_bwd(dw, ids, x)


def test_gradient_empty():
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    x = torch.empty(0, 12, device="cuda")
    dw, ws = g().grpo_embed_bwd(ids, x, 5, out_dtype=BF16)
    assert (dw == 0).all() and g().grpo_check_error(ws) == 0
    base = torch.ones(5, 12, device="cuda")
    g().grpo_embed_bwd(ids, x, 5, dweight=base, accumulate=True)
    assert (base == 1).all()


def test_refusals():
    n = g()
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    w = torch.zeros(8, 16, device="cuda")
    with pytest.raises(TypeError):
        n.grpo_embed_fwd(ids.int(), w)
    with pytest.raises(TypeError):
        n.grpo_embed_fwd(ids, w.half())
    with pytest.raises(ValueError):
        n.grpo_embed_fwd(ids, w.t())
    with pytest.raises(ValueError):
        n.grpo_embed_fwd(ids, w, out=torch.empty(4, 15, device="cuda"))
    with pytest.raises(ValueError):
        n.grpo_embed_fwd(ids, w[:1].expand(8, 16))
    with pytest.raises(ValueError):
        n.grpo_embed_bwd(ids, torch.zeros(3, 16, device="cuda"), 8)
    with pytest.raises(ValueError):
        n.grpo_embed_bwd(ids, torch.zeros(4, 16, device="cuda"), 8, accumulate=True)
    with pytest.raises(ValueError):
        n.grpo_embed_bwd(ids, torch.zeros(1, 16, device="cuda").expand(4, 16), 8)
    with pytest.raises(n.GrpoError):
        n.grpo_embed_fwd(ids, w, float("nan"))


def test_other_stream_and_graph():
    n = g()
    V, d = 300, 96
    w = torch.randn(V, d, generator=gen(60), device="cuda")
    ids = draw_ids(3000, V, 61)
    dout = torch.randn(3000, d, generator=gen(62), device="cuda")
    want, want_g = n.grpo_embed_fwd(ids, w, 2.0), n.grpo_embed_bwd(ids, dout, V, 2.0)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, (dw, ws) = n.grpo_embed_fwd(ids, w, 2.0), n.grpo_embed_bwd(ids, dout, V, 2.0)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(dw, want_g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n.grpo_embed_fwd(ids, w, 2.0, out=out)
        n.grpo_embed_bwd(ids, dout, V, 2.0, dweight=dw, workspace=ws)
    ids.copy_(draw_ids(3000, V, 63, "uniform"))
    out.zero_()
    dw.zero_()
    graph.replay()
    torch.cuda.synchronize()
    check_fwd(out, ids, w, 2.0)
    check_bwd(dw, ids, dout, 2.0)


def test_autograd_against_the_formula_and_differences():
    from vocab_wide_logprob_gb300.autograd import grpo_embed
    V, d = 13, 24
    w = torch.randn(V, d, generator=gen(70), device="cuda").requires_grad_()
    ids = draw_ids(40, V, 71).view(5, 8)
    c = torch.randn(5, 8, d, generator=gen(72), device="cuda")
    out = grpo_embed(ids, w, 3.0, pad_id=2)
    (out * c).sum().backward()
    check_bwd(w.grad, ids, c, 3.0, 2)
    # differences of the (linear) forward, exact up to float32's rounding
    with torch.no_grad():
        for v, k in ((0, 0), (5, 11), (12, 23)):
            h = 0.5
            wp, wm = w.clone(), w.clone()
            wp[v, k] += h
            wm[v, k] -= h
            f = lambda x: (g().grpo_embed_fwd(ids, x, 3.0).double() * c.double()).sum()
            diff = float((f(wp) - f(wm)) / (2 * h))
            assert abs(diff - float(w.grad[v, k])) <= 1e-5 * float(c.abs().sum())
    # a broadcast gradient, bfloat16 weights
    wb = torch.randn(V, d, device="cuda").to(BF16).requires_grad_()
    grpo_embed(ids, wb).sum().backward()
    check_bwd(wb.grad, ids, torch.ones(5, 8, d, device="cuda"))
    assert wb.grad.dtype == BF16
