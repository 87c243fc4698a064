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


def loss_calls():
    n = g()
    N, P, C, V, d = 4, 3, 5, 2048, 128
    dev = dict(device="cuda")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    logits = torch.randn(N, P + C, V, generator=gen, **dev)
    ids = torch.randint(0, V, (N, P + C), generator=gen, **dev)
    lens = torch.tensor([5, 0, 3, 1], dtype=torch.int32, **dev)
    adv = torch.randn(N, generator=gen, **dev)
    hidden = torch.randn(N, P + C, d, generator=gen, **dev).bfloat16()
    weight = torch.randn(V, d, generator=gen, **dev).bfloat16()
    host = logits.cpu().pin_memory()
    f = n.grpo_loss_fwd(logits, P, ids, lens, adv)
    torch.cuda.synchronize()

    def cuda(out):
        return tuple(out[k] for k in sorted(out))

    return {
        "mask": lambda **k: n.grpo_mask(ids, P, C, V - 1, **k),
        "advantage": lambda **k: (n.grpo_advantage(adv, 2, **k),),
        "advantage_ex": lambda **k: n.grpo_advantage_ex(adv, 2, count_contrast=True, **k),
        "loss_fwd": lambda **k: cuda(n.grpo_loss_fwd(logits, P, ids, lens, adv, **k)),
        "logprobs": lambda **k: n.grpo_logprobs(logits, P, ids, lens, **k),
        "loss_fwd_static": lambda **k: cuda(n.grpo_loss_fwd_static(logits, P, ids, lens, adv, **k)),
        "loss_bwd": lambda **k: (n.grpo_loss_bwd(logits, P, ids, lens, f["lse"], f["w"], **k),),
        "loss_fwd_bwd": lambda **k: cuda(n.grpo_loss_fwd_bwd(logits, P, ids, lens, adv, **k)),
        "loss_fwd_bwd_host": lambda **k: cuda(n.grpo_loss_fwd_bwd_host(host, P, ids, lens, adv, **k)),
        "lmhead_logprobs": lambda **k: n.grpo_lmhead_logprobs(hidden, weight, P, ids, lens, **k),
        "lmhead_loss_fwd": lambda **k: cuda(n.grpo_lmhead_loss_fwd(hidden, weight, P, ids, lens, adv,
                                                                   **k)),
        "lmhead_loss_bwd": lambda **k: n.grpo_lmhead_loss_bwd(hidden, weight, P, ids, lens, f["lse"],
                                                              f["w"], **k),
    }


LOSS_NAMES = ["mask", "advantage", "advantage_ex", "loss_fwd", "logprobs", "loss_fwd_static",
              "loss_bwd", "loss_fwd_bwd", "loss_fwd_bwd_host", "lmhead_logprobs",
              "lmhead_loss_fwd", "lmhead_loss_bwd"]


@pytest.mark.parametrize("name", LOSS_NAMES)
def test_loss_calls_allocate_on_the_given_stream(name):
    call = loss_calls()[name]
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    handle = type("Handle", (), {"cuda_stream": side.cuda_stream})()
    for s in (side, torch.cuda.ExternalStream(side.cuda_stream), handle):
        out = call(stream=s)
        side.synchronize()
        for t, b in zip(out, want):
            assert stream_of_memory(t) == side.cuda_stream
            if t.dtype != torch.uint8 and name != "loss_fwd_bwd_host":  # (its staging has unread rows)
                assert torch.equal(t, b)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()


def test_a_stream_of_another_device_is_refused():
    n = g()
    other = type("Other", (), {"cuda_stream": 0, "device_index": 7})()
    ids, w = torch.zeros(3, dtype=torch.int64, device="cuda"), torch.zeros(4, 8, device="cuda")
    with pytest.raises(ValueError, match="stream"):
        n.grpo_embed_fwd(ids, w, stream=other)
