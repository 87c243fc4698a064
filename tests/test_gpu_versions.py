"""Calls that write into a caller's tensor count as in-place operations on it:
a backward pass that saved the old values is refused."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def g():
    from vocab_wide_logprob_gb300 import _native
    return _native


@pytest.mark.parametrize("max_norm", [1e-3, 1e9], ids=["over", "under"])
@pytest.mark.parametrize("out", [False, True], ids=["in place", "elsewhere"])
def test_clipping_a_saved_tensor(max_norm, out):
    w = torch.randn(4000, device="cuda").requires_grad_()
    saved, other = torch.randn(4000, device="cuda"), torch.randn(4000, device="cuda")
    y = (w * saved).sum()  # the product keeps `saved`
    if out:
        g().grpo_clip_grad_norm([other], max_norm, out=[saved])
    else:
        g().grpo_clip_grad_norm([saved], max_norm)
    with pytest.raises(RuntimeError, match="inplace operation"):
        y.backward()
    torch.cuda.synchronize()


def versions(*tensors):
    return [t._version for t in tensors]


def test_what_is_written_and_what_is_not():
    n, dev = g(), dict(device="cuda")
    ids, w, dout = torch.tensor([0, 3, 1], **dev), torch.randn(5, 8, **dev), torch.randn(3, 8, **dev)
    out, dw, stats = torch.empty(3, 8, **dev), torch.zeros(5, 8, **dev), torch.zeros(2, **dev)
    a, b = torch.randn(300, **dev), torch.randn(300, **dev)

    def check(call, writes, reads):
        before_w, before_r = versions(*writes), versions(*reads)
        call()
        assert all(x > y for x, y in zip(versions(*writes), before_w))
        assert versions(*reads) == before_r

    check(lambda: n.grpo_embed_fwd(ids, w, out=out), [out], [ids, w])
    check(lambda: n.grpo_embed_bwd(ids, dout, 5, dweight=dw, accumulate=True), [dw], [ids, dout])
    check(lambda: n.grpo_grad_norm([a, b], stats=stats), [stats], [a, b])
    check(lambda: n.grpo_clip_grad_norm([a], 1.0, out=[b], stats=stats), [b, stats], [a])
    check(lambda: n.grpo_clip_grad_norm([a, b], 1.0), [a, b], [])
    z, x = torch.randn(2, 3, 9, **dev), torch.zeros(2, 2, dtype=torch.int64, **dev)
    u, e = torch.rand(2, 2, **dev), torch.rand(2, 9, **dev) + 0.1
    v = n.grpo_verify_drafts(z, x, u, e)
    check(lambda: n.grpo_verify_drafts(z, x, u, e, out=v),
          [v["tokens"], v["n_accepted"], v["logp"]], [z, x, u, e])
    with torch.inference_mode():  # (its tensors have no versions)
        i = torch.randn(300, **dev)
        n.grpo_clip_grad_norm([i], 1.0)
    n.grpo_clip_grad_norm([i], 1.0)
    torch.cuda.synchronize()
