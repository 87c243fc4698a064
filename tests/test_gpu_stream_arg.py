"""The ``stream`` argument of the operators around the loss: what a call
allocates belongs to the stream that its kernels run on, so that a dropped
workspace is not handed to another stream while they still use it.  No test
writes to memory that a kernel in flight could be using."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def g():
    from vocab_wide_logprob_gb300 import _native
    return _native


def stream_of_memory(t):
    """Handle of the stream whose pool holds the tensor's memory."""
    p = t.untyped_storage().data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= p < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not in the allocator's memory")


def calls():
    n = g()
    dev = dict(device="cuda")
    ids = torch.randint(0, 5000, (3000,), **dev)
    w = torch.randn(5000, 64, **dev)
    dout = torch.randn(3000, 64, **dev)
    grads = [torch.randn(1000, **dev), torch.randn(70000, **dev)]
    z = torch.randn(9, 3, 4000, **dev)
    x = torch.randint(0, 4000, (9, 2), **dev)
    u = torch.rand(9, 2, **dev)
    e = torch.empty(9, 4000, **dev).exponential_().clamp_(min=1e-9)
    dw = torch.zeros(5000, 64, **dev)
    stats = torch.zeros(2, **dev)
    return {
        "embed_fwd": lambda **k: (n.grpo_embed_fwd(ids, w, **k),),
        "embed_bwd": lambda **k: n.grpo_embed_bwd(ids, dout, 5000, **k),
        "embed_bwd_into": lambda **k: n.grpo_embed_bwd(ids, dout, 5000, dweight=dw, **k)[1:],
        "grad_norm": lambda **k: n.grpo_grad_norm(grads, **k),
        "clip": lambda **k: n.grpo_clip_grad_norm(grads, 1e9, **k),
        "clip_stats": lambda **k: n.grpo_clip_grad_norm(grads, 1e9, stats=stats, **k)[1:],
        "verify": lambda **k: tuple(n.grpo_verify_drafts(z, x, u, e, **k).values()),
    }


NAMES = ["embed_fwd", "embed_bwd", "embed_bwd_into", "grad_norm", "clip", "clip_stats", "verify"]


@pytest.mark.parametrize("name", NAMES)
def test_allocations_belong_to_the_given_stream(name):
    call = calls()[name]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, torch.cuda.ExternalStream(side.cuda_stream)):
        for t in call(stream=s):
            assert stream_of_memory(t) == side.cuda_stream
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    for t in call():
        assert stream_of_memory(t) == torch.cuda.default_stream().cuda_stream
    with torch.cuda.stream(side):
        for t in call(stream=torch.cuda.default_stream()):
            assert stream_of_memory(t) == torch.cuda.default_stream().cuda_stream
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", NAMES)
def test_dropped_memory_is_not_handed_to_the_current_stream(name):
    call = calls()[name]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms
    spans = []
    for t in call(stream=side):
        p = t.untyped_storage().data_ptr()
        spans.append((p, p + t.untyped_storage().nbytes()))
        del t
    got = [torch.empty(b - a, dtype=torch.uint8, device="cuda") for a, b in spans for _ in range(2)]
    for t in got:  # (never written)
        assert all(not a <= t.data_ptr() < b for a, b in spans)
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", NAMES)
def test_results_on_a_given_stream(name):
    call = calls()[name]
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(stream=side)
    side.synchronize()
    for a, b in zip(got, want):
        if a.dtype != torch.uint8:  # (not the workspace)
            assert torch.equal(a, b)
