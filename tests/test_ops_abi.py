"""Argument checks of the embedding, gradient-clipping and draft-verification
calls, through the C ABI and the Python binding.  CPU only: no call here
reaches a launch."""
import ctypes

import pytest
import torch

OK, INVALID, UNSUPPORTED, WORKSPACE, MISALIGNED = 0, 1, 2, 3, 4
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from vocab_wide_logprob_gb300 import build
    build.build()
    from vocab_wide_logprob_gb300 import _native
    return _native.library()


@pytest.fixture(scope="module")
def n(lib):
    from vocab_wide_logprob_gb300 import _native
    return _native


def A(addr):
    return P(addr)


def _embed(lib, **kw):
    a = dict(ids=A(0x10000), n=8, w=A(0x100000), wdt=1, V=100, d=64, ldw=64, scale=1.0,
             out=A(0x20000), odt=1, ldo=64, stream=None)
    a.update(kw)
    return lib.grpo_embed_fwd(*a.values())


def test_embed_fwd_refusals(lib):
    assert _embed(lib, wdt=3) == UNSUPPORTED
    assert _embed(lib, odt=-1) == UNSUPPORTED
    assert _embed(lib, n=-1) == INVALID
    assert _embed(lib, V=0) == INVALID
    assert _embed(lib, d=0) == INVALID
    assert _embed(lib, ldw=63) == INVALID
    assert _embed(lib, ldo=63) == INVALID
    assert _embed(lib, scale=float("nan")) == INVALID
    assert _embed(lib, scale=float("inf")) == INVALID
    assert _embed(lib, ids=None) == INVALID
    assert _embed(lib, w=None) == INVALID
    assert _embed(lib, out=None) == INVALID
    assert _embed(lib, ids=A(0x10004)) == MISALIGNED
    assert _embed(lib, w=A(0x100001)) == MISALIGNED
    assert _embed(lib, out=A(0x20002), odt=0) == MISALIGNED
    assert _embed(lib, out=A(0x100000 + 100)) == INVALID      # over the weight
    assert _embed(lib, out=A(0x10000 - 16)) == INVALID        # over the ids
    assert _embed(lib, n=1 << 31) == UNSUPPORTED
    assert _embed(lib, d=1 << 25, ldw=1 << 25, ldo=1 << 25) == UNSUPPORTED
    assert _embed(lib, ldw=1 << 62) == UNSUPPORTED
    assert _embed(lib, n=0, ids=None, out=None) == OK          # nothing to do


def _embed_bwd(lib, **kw):
    a = dict(ids=A(0x10000), n=8, dout=A(0x20000), ddt=1, V=100, d=64, ldd=64, scale=1.0, pad=-1,
             dw=A(0x100000), wdt=0, ldw=64, acc=0, ws=A(0x1000000), ws_bytes=1 << 24, stream=None)
    a.update(kw)
    return lib.grpo_embed_bwd(*a.values())


def test_embed_bwd_refusals(lib):
    assert _embed_bwd(lib, ddt=2) == UNSUPPORTED
    assert _embed_bwd(lib, wdt=9) == UNSUPPORTED
    assert _embed_bwd(lib, n=-1) == INVALID
    assert _embed_bwd(lib, ldd=1) == INVALID
    assert _embed_bwd(lib, dw=None) == INVALID
    assert _embed_bwd(lib, ws=None) == INVALID
    assert _embed_bwd(lib, dout=None) == INVALID
    assert _embed_bwd(lib, scale=float("-inf")) == INVALID
    assert _embed_bwd(lib, ws=A(0x1000010)) == MISALIGNED
    assert _embed_bwd(lib, dw=A(0x100002)) == MISALIGNED
    assert _embed_bwd(lib, dout=A(0x20001)) == MISALIGNED
    assert _embed_bwd(lib, ws_bytes=256) == WORKSPACE
    assert _embed_bwd(lib, dw=A(0x20000 + 64)) == INVALID      # over dout
    assert _embed_bwd(lib, dw=A(0x1000000 + 256)) == INVALID   # over the workspace
    out = ctypes.c_size_t(0)
    assert lib.grpo_embed_workspace_size(8, 100, 64, ctypes.byref(out)) == OK and out.value > 256
    assert lib.grpo_embed_workspace_size(8, 100, 64, None) == INVALID
    assert lib.grpo_embed_workspace_size(-1, 100, 64, ctypes.byref(out)) == INVALID
    assert lib.grpo_embed_workspace_size(1 << 31, 100, 64, ctypes.byref(out)) == UNSUPPORTED


def _clip(lib, n, rows=((0x10000, 0, 16, 0, 0),), **kw):
    words = [w for r in rows for w in (r[0], r[1], r[2], r[3] | r[4] << 32)]
    table = (ctypes.c_int64 * max(1, len(words)))(*words)
    a = dict(tensors=table, count=len(rows), type=0, max_norm=1.0, eps=1e-6, stats=A(0x90000),
             ws=A(0x100000), ws_bytes=1 << 20, stream=None)
    a.update(kw)
    return lib.grpo_clip_grad_norm(*a.values())


def test_clip_refusals(lib, n):
    assert _clip(lib, n, type=2) == UNSUPPORTED
    assert _clip(lib, n, count=-1) == INVALID
    assert _clip(lib, n, max_norm=-1.0) == INVALID
    assert _clip(lib, n, max_norm=float("nan")) == INVALID
    assert _clip(lib, n, eps=-1.0) == INVALID
    assert _clip(lib, n, eps=float("inf")) == INVALID
    assert _clip(lib, n, tensors=None) == INVALID
    assert _clip(lib, n, stats=None) == INVALID
    assert _clip(lib, n, ws=None) == INVALID
    assert _clip(lib, n, ws=A(0x100008)) == MISALIGNED
    assert _clip(lib, n, stats=A(0x90002)) == MISALIGNED
    assert _clip(lib, n, ws_bytes=128) == WORKSPACE
    assert _clip(lib, n, rows=[(0x10000, 0, 16, 5, 0)]) == UNSUPPORTED
    assert _clip(lib, n, rows=[(0, 0, 16, 0, 0)]) == INVALID                # no data
    assert _clip(lib, n, rows=[(0x10000, 0, -1, 0, 0)]) == INVALID
    assert _clip(lib, n, rows=[(0x10002, 0, 16, 0, 0)]) == MISALIGNED
    assert _clip(lib, n, rows=[(0x10000, 0, 16, 0, 1)]) == INVALID          # in place, other type
    assert _clip(lib, n, rows=[(0x10000, 0x10010, 16, 0, 0)]) == INVALID    # partly over itself
    assert _clip(lib, n, rows=[(0x10000, 0x100000, 16, 0, 0)]) == INVALID   # over the workspace
    assert _clip(lib, n, rows=[(0x10000, 0, 1 << 62, 0, 0)]) == UNSUPPORTED
    out = ctypes.c_size_t(0)
    assert lib.grpo_grad_norm_workspace_size(0, ctypes.byref(out)) == OK
    assert lib.grpo_grad_norm_workspace_size(-1, ctypes.byref(out)) == INVALID
    assert lib.grpo_grad_norm_workspace_size(3, None) == INVALID


def _verify(lib, **kw):
    a = dict(target=A(0x100000), draft=A(0x800000), dt=1, N=2, K=3, V=100, tseq=400, trow=100,
             dseq=300, drow=100, tokens=A(0x20000), lens=None, u=A(0x30000), noise=A(0x40000),
             nrow=100, temp=None, out=A(0x50000), acc=A(0x60000), logp=A(0x70000),
             ws=A(0x80000), ws_bytes=1 << 16, stream=None)
    a.update(kw)
    return lib.grpo_verify_drafts(*a.values())


def test_verify_refusals(lib):
    assert _verify(lib, dt=2) == UNSUPPORTED
    assert _verify(lib, N=-1) == INVALID
    assert _verify(lib, K=-1) == INVALID
    assert _verify(lib, V=0) == INVALID
    assert _verify(lib, K=(1 << 20) + 1) == UNSUPPORTED
    assert _verify(lib, N=1 << 25) == UNSUPPORTED
    assert _verify(lib, V=1 << 31, trow=1 << 31, tseq=1 << 34, nrow=1 << 31) == UNSUPPORTED
    assert _verify(lib, trow=99) == INVALID
    assert _verify(lib, tseq=399) == INVALID      # sequences overlap
    assert _verify(lib, dseq=299) == INVALID
    assert _verify(lib, drow=99) == INVALID
    assert _verify(lib, nrow=99) == INVALID
    for name in ("target", "tokens", "u", "noise", "out", "acc", "logp", "ws"):
        assert _verify(lib, **{name: None}) == INVALID, name
    for name, bad in (("target", 0x100001), ("draft", 0x800001), ("tokens", 0x20004),
                      ("lens", 0x20002), ("u", 0x30002), ("noise", 0x40002), ("temp", 0x40001),
                      ("out", 0x50004), ("acc", 0x60002), ("logp", 0x70002), ("ws", 0x80010)):
        assert _verify(lib, **{name: A(bad)}) == MISALIGNED, name
    assert _verify(lib, ws_bytes=256) == WORKSPACE
    out = ctypes.c_size_t(0)
    assert lib.grpo_verify_workspace_size(4, 3, ctypes.byref(out)) == OK
    assert lib.grpo_verify_workspace_size(-1, 3, ctypes.byref(out)) == INVALID
    assert lib.grpo_verify_workspace_size(4, 3, None) == INVALID


def test_status_string(lib):
    assert b"norm" in lib.grpo_status_string(9)


def test_binding_refuses_cpu_tensors_and_wrong_types(n):
    ids = torch.zeros(4, dtype=torch.int64)
    w = torch.zeros(8, 16)
    with pytest.raises(ValueError):
        n.grpo_embed_fwd(ids, w)
    with pytest.raises(TypeError):
        n.grpo_embed_fwd([1, 2], w)
    with pytest.raises(ValueError):
        n.grpo_embed_bwd(ids, torch.zeros(4, 16), 8)
    with pytest.raises(ValueError):
        n.grpo_clip_grad_norm([w], 1.0)
    with pytest.raises(TypeError):
        n.grpo_clip_grad_norm([w.tolist()], 1.0)
    with pytest.raises(TypeError):
        n.grpo_clip_grad_norm(7, 1.0)
    with pytest.raises(TypeError):
        n.grpo_clip_grad_norm([], "one")
    with pytest.raises(ValueError):
        n.grpo_verify_drafts(torch.zeros(2, 3), ids, w, w)
    with pytest.raises(ValueError):
        n.grpo_verify_drafts(torch.zeros(2, 1, 8), torch.zeros(2, 0, dtype=torch.int64),
                             torch.zeros(2, 0), torch.zeros(2, 8))


class _Elsewhere(torch.Tensor):
    """A tensor that says it is on a device and has no memory."""

    @staticmethod
    def __new__(cls, device, shape, dtype=torch.float32):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device=device)

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise AssertionError(f"{func} on a tensor without memory")


def _on(device, *shapes, dtype=torch.float32):
    return [_Elsewhere(device, s if isinstance(s, tuple) else (s,), dtype) for s in shapes]


def test_binding_refuses_tensors_of_another_device(n):
    """The library launches on the current device: tensors that agree with one
    another but are on a device that is not current are refused before anything
    is allocated or launched."""
    (ids,), (x,) = _on("cuda:7", 4, dtype=torch.int64), _on("cuda:7", (2, 2), dtype=torch.int64)
    w, dout, z, u, e = _on("cuda:7", (8, 16), (4, 16), (2, 3, 16), (2, 2), (2, 16))
    for call in (lambda: n.grpo_embed_fwd(ids, w), lambda: n.grpo_embed_bwd(ids, dout, 8),
                 lambda: n.grpo_clip_grad_norm([w, dout], 1.0), lambda: n.grpo_grad_norm([w]),
                 lambda: n.grpo_verify_drafts(z, x, u, e)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()


def test_loss_calls_refuse_tensors_of_another_device(n, monkeypatch):
    monkeypatch.setattr(n, "_current_device", lambda: 0)
    i64, i32 = dict(dtype=torch.int64), dict(dtype=torch.int32)
    (ids,), (lens,) = _on("cuda:7", (2, 8), **i64), _on("cuda:7", 2, **i32)
    logits, adv, lse = _on("cuda:7", (2, 8, 100), (2,), (2, 4))
    hidden, weight = _on("cuda:7", (2, 8, 128), (100, 128), dtype=torch.bfloat16)
    for call in (lambda: n.grpo_mask(ids, 4, 4, 9), lambda: n.grpo_advantage(adv, 2),
                 lambda: n.grpo_advantage_ex(adv, 2),
                 lambda: n.grpo_loss_fwd(logits, 4, ids, lens, adv),
                 lambda: n.grpo_loss_fwd_static(logits, 4, ids, lens, adv),
                 lambda: n.grpo_loss_fwd_bwd(logits, 4, ids, lens, adv),
                 lambda: n.grpo_loss_bwd(logits, 4, ids, lens, lse, lse),
                 lambda: n.grpo_logprobs(logits, 4, ids, lens),
                 lambda: n.grpo_lmhead_logprobs(hidden, weight, 4, ids, lens),
                 lambda: n.grpo_lmhead_loss_fwd(hidden, weight, 4, ids, lens, adv),
                 lambda: n.grpo_lmhead_loss_bwd(hidden, weight, 4, ids, lens, lse, lse)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()


def test_binding_hands_on_an_argument_without_a_truth_value(n):
    class Neither:
        def __bool__(self):
            raise ZeroDivisionError("neither")

    ids, = _on("cuda:7", 4, dtype=torch.int64)
    dout, dw = _on("cuda:7", (4, 16), (8, 16))
    with pytest.raises(ZeroDivisionError):
        n.grpo_embed_bwd(ids, dout, 8, dweight=dw, accumulate=Neither())


def test_package_exports():
    import vocab_wide_logprob_gb300 as pkg
    for name in ("grpo_embed_fwd", "grpo_embed_bwd", "grpo_clip_grad_norm", "grpo_grad_norm",
                 "grpo_verify_drafts"):
        assert callable(getattr(pkg, name))
