"""Global gradient norm and clipping against float64.

Tolerances, fixed before the first run: a thread adds at most 16 squares to
each of four float32 sums and adds those, so a batch's sum is off by at most
20 roundings (2^-24 each) and the norm by half of that, then one rounding to
float32: 12 * 2^-24 relative.  A clipped element has the coefficient's error,
its own rounding and the product's (15 * 2^-24), then half a step of its
type."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


def g():
    from vocab_wide_logprob_gb300 import _native
    return _native


def gen(seed):
    r = torch.Generator(device="cuda")
    r.manual_seed(seed)
    return r


def norm64(grads, kind=0):
    if kind:
        return max([float(t.double().abs().max()) for t in grads if t.numel()] + [0.0])
    return math.sqrt(math.fsum(float((t.double() ** 2).sum()) for t in grads))


def check(grads, stats, outs, max_norm, kind=0, eps=1e-6):
    n = norm64(grads, kind)
    c = min(1.0, max_norm / (n + eps))
    assert abs(float(stats[0]) - n) <= 12 * U * n
    assert abs(float(stats[1]) - c) <= 14 * U * c
    for t, o in zip(grads, outs):
        want = t.double() * c
        tol = want.abs() * (15 * U + torch.finfo(o.dtype).eps / 2 * 1.001)
        assert ((o.double() - want).abs() <= tol).all()


def make(sizes, dts, seed, spread=1.0):
    r = gen(seed)
    return [(torch.randn(s, generator=r, device="cuda") * spread).to(dts[k % len(dts)])
            for k, s in enumerate(sizes)]


SIZES = [[1], [0, 5, 0], [7, 8, 9, 16383, 16384, 16385, 8193], [100000, 1, 3, 33333],
         [64] * 200, [17] * 1000 + [5000], [3000001]]


@pytest.mark.parametrize("dts", [[F32], [BF16], [F32, BF16]], ids=["f32", "bf16", "mixed"])
@pytest.mark.parametrize("sizes", SIZES, ids=range(len(SIZES)))
@pytest.mark.parametrize("kind", [0, 1], ids=["l2", "max"])
def test_clip(sizes, dts, kind):
    n = g()
    grads = make(sizes, dts, 1)
    before = [t.clone() for t in grads]
    limit = 0.3 * norm64(grads, kind)
    # into other tensors, of the same and of the other type
    for flip in (False, True):
        outs = [torch.empty(t.shape, dtype=t.dtype if not flip else (F32 if t.dtype == BF16 else BF16),
                            device="cuda") for t in grads]
        stats, ws = n.grpo_clip_grad_norm(grads, limit, out=outs, norm_type=kind)
        assert n.grpo_check_error(ws) == 0
        check(grads, stats, outs, limit, kind)
        assert all(torch.equal(a, b) for a, b in zip(grads, before))
    # in place
    stats, _ = n.grpo_clip_grad_norm(grads, limit, norm_type=kind)
    check(before, stats, grads, limit, kind)


def test_under_the_limit():
    n = g()
    grads = make([1000, 77, 50000], [F32, BF16], 2)
    before = [t.clone() for t in grads]
    limit = 3 * norm64(grads)
    stats, _ = n.grpo_clip_grad_norm(grads, limit)
    assert float(stats[1]) == 1.0 and all(torch.equal(a, b) for a, b in zip(grads, before))
    outs = [torch.empty_like(t) for t in grads]
    stats, _ = n.grpo_clip_grad_norm(grads, limit, out=outs)
    assert all(torch.equal(a, b) for a, b in zip(outs, before))
    # some in place, some elsewhere
    mixed = [grads[0], torch.empty_like(grads[1]), grads[2]]
    n.grpo_clip_grad_norm(grads, limit, out=mixed)
    assert torch.equal(mixed[1], before[1]) and torch.equal(grads[0], before[0])
    stats, _ = n.grpo_clip_grad_norm(grads, float("inf"))
    assert float(stats[1]) == 1.0
    stats, _ = n.grpo_grad_norm(grads)
    check(grads, stats, [], float("inf"))
    stats, _ = n.grpo_grad_norm(grads, norm_type=n.GRPO_NORM_MAX)
    check(grads, stats, [], float("inf"), 1)


def test_limit_zero_and_no_tensors():
    n = g()
    grads = make([100, 3], [F32], 3)
    n.grpo_clip_grad_norm(grads, 0.0)
    assert all((t == 0).all() for t in grads)
    stats, ws = n.grpo_clip_grad_norm([], 1.0)
    assert stats.tolist() == [0.0, 1.0] and n.grpo_check_error(ws) == 0
    zero = [torch.zeros(50, device="cuda")]
    stats, _ = n.grpo_clip_grad_norm(zero, 1.0)
    assert stats.tolist() == [0.0, 1.0]


@pytest.mark.parametrize("scale", [1e-42, 1e-30, 1e-20, 1e15, 1e25, 1e37])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_squares_outside_float32(scale, dt):
    """Values whose squares leave float32's range, alone and beside others."""
    n = g()
    r = gen(4)
    t = [(torch.rand(5000, generator=r, device="cuda") + 0.5).double().mul_(scale).to(dt),
         (torch.rand(33, generator=r, device="cuda") + 0.5).to(dt)]
    for grads in (t[:1], t):
        stats, ws = n.grpo_grad_norm(grads)
        want = norm64(grads)
        if want > torch.finfo(F32).max:  # the float32 result is infinite, and said to be
            assert math.isinf(float(stats[0])) and n.grpo_check_error(ws) == 9
            continue
        # a subnormal result is rounded to a step of 2^-149
        assert abs(float(stats[0]) - want) <= 12 * U * want + 2.0 ** -149
        assert n.grpo_check_error(ws) == 0


@pytest.mark.parametrize("at", [0, 3, 12345])
@pytest.mark.parametrize("kind", [0, 1])
def test_nonfinite(at, kind):
    n = g()
    for dt in (F32, BF16):
        a = torch.ones(20000, device="cuda", dtype=dt)
        a[at] = float("inf")
        b = torch.ones(30, device="cuda", dtype=dt)
        stats, ws = n.grpo_clip_grad_norm([b, a], 1.0, norm_type=kind)
        assert n.grpo_check_error(ws) == 9
        assert math.isinf(float(stats[0])) and float(stats[1]) == 0.0
        assert torch.isnan(a[at]) and int((a == 0).sum()) == 19999 and (b == 0).all()
        a.fill_(1)
        a[at] = float("nan")
        stats, ws = n.grpo_clip_grad_norm([a, b.fill_(1)], 1.0, norm_type=kind, workspace=ws)
        assert n.grpo_check_error(ws) == 9 and torch.isnan(stats).all()
        assert torch.isnan(a).all() and torch.isnan(b).all()
        stats, ws = n.grpo_clip_grad_norm([b.fill_(1)], 1.0, norm_type=kind, workspace=ws)
        assert n.grpo_check_error(ws) == 0


@pytest.mark.parametrize("dt", [F32, BF16])
def test_odd_addresses(dt):
    n = g()
    buf = torch.randn(70000, generator=gen(5), device="cuda").to(dt)
    grads = [buf[1:20002], buf[20003:20010], buf[20011:60001]]
    limit = 0.5 * norm64(grads)
    for odt in (F32, BF16):
        dst = torch.full((70000,), 9.0, device="cuda", dtype=odt)
        outs = [dst[3:20004], dst[20005:20012], dst[20013:60003]]
        stats, _ = n.grpo_clip_grad_norm(grads, limit, out=outs)
        check(grads, stats, outs, limit)
        rest = torch.ones(70000, dtype=torch.bool, device="cuda")
        for a, b in ((3, 20004), (20005, 20012), (20013, 60003)):
            rest[a:b] = False
        assert (dst[rest] == 9).all()


@pytest.mark.parametrize("dt", [F32, BF16])
def test_outputs_at_16_bytes(dt):
    """Outputs that begin at a 16-byte boundary that is not one of 32."""
    n = g()
    grads = [torch.randn(50000, generator=gen(8), device="cuda").to(dt) for _ in range(3)]
    limit = 0.5 * norm64(grads)
    dst = [torch.full((50012,), 9.0, device="cuda") for _ in grads]
    outs = [t[4:50004] for t in dst]
    stats, _ = n.grpo_clip_grad_norm(grads, limit, out=outs)
    check(grads, stats, outs, limit)
    assert all((t[:4] == 9).all() and (t[50004:] == 9).all() for t in dst)


def test_reproducible_stream_and_graph():
    n = g()
    grads = make([123457, 1000, 8], [BF16, F32], 6)
    outs = [torch.empty_like(t) for t in grads]
    limit = 0.25 * norm64(grads)
    stats, ws = n.grpo_clip_grad_norm(grads, limit, out=outs)
    want = [stats.clone()] + [o.clone() for o in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ws.fill_(255)
        n.grpo_clip_grad_norm(grads, limit, out=outs, stats=stats, workspace=ws)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip([stats] + outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n.grpo_clip_grad_norm(grads, limit, out=outs, stats=stats, workspace=ws)
    for t in grads:
        t.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    check(grads, stats, outs, limit)


@pytest.mark.parametrize("kind", [0, 1], ids=["l2", "max"])
def test_many_chunks(kind):
    # enough of them that the coefficient is formed once, before the scaling
    n = g()
    grads = make([9000001, 5, 12000000, 3000003], [F32, BF16], 7)
    before = [t.clone() for t in grads]
    limit = 0.4 * norm64(grads, kind)
    outs = [torch.empty_like(t) for t in grads]
    stats, ws = n.grpo_clip_grad_norm(grads, limit, out=outs, norm_type=kind)
    assert n.grpo_check_error(ws) == 0
    check(grads, stats, outs, limit, kind)
    alone, _ = n.grpo_grad_norm(grads, norm_type=kind)
    assert float(alone[0]) == float(stats[0]) and float(alone[1]) == 1.0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n.grpo_clip_grad_norm(grads, limit, stats=stats, workspace=ws, norm_type=kind)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(grads, outs))
    # under the limit in place; with a tensor that goes elsewhere
    for t, b in zip(grads, before):
        t.copy_(b)
    outs = [grads[0], torch.empty_like(grads[1]), grads[2], torch.empty_like(grads[3])]
    n.grpo_clip_grad_norm(grads, 1e9, out=outs, stats=stats, workspace=ws, norm_type=kind)
    assert float(stats[1]) == 1.0 and all(torch.equal(a, b) for a, b in zip(outs, before))
    grads[2][7] = float("nan")
    n.grpo_clip_grad_norm(grads, limit, stats=stats, workspace=ws, norm_type=kind)
    assert n.grpo_check_error(ws) == 9 and torch.isnan(stats).all()
    assert all(torch.isnan(t).all() for t in grads)


def test_refusals():
    n = g()
    t = torch.ones(10, 10, device="cuda")
    with pytest.raises(TypeError):
        n.grpo_clip_grad_norm([t.half()], 1.0)
    with pytest.raises(ValueError):
        n.grpo_clip_grad_norm([t.t()[:5]], 1.0)
    with pytest.raises(ValueError):
        n.grpo_clip_grad_norm([t], 1.0, out=[])
    with pytest.raises(ValueError):
        n.grpo_clip_grad_norm([t], 1.0, out=[torch.ones(5, device="cuda")])
    with pytest.raises(n.GrpoError):
        n.grpo_clip_grad_norm([t], -1.0)
    with pytest.raises(n.GrpoError):
        n.grpo_clip_grad_norm([t.view(-1)[:50]], 1.0, out=[t.view(-1)[10:60]])
