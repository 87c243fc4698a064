"""Argument checks of the token statistics and AdamW calls, through the C ABI and
the Python binding.  CPU only: no call here reaches a launch."""
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


def _stats(lib, **kw):
    a = dict(z=A(0x100000), dt=1, N=2, R=3, V=100, seq=300, row=100, tokens=A(0x20000), tseq=3, trow=1,
             lens=None, temp=None, top=2, logp=A(0x30000), H=A(0x40000), norm=A(0x50000),
             top_tokens=A(0x60000), top_logp=A(0x70000), ws=A(0x80000), ws_bytes=1 << 16, stream=None)
    a.update(kw)
    return lib.grpo_token_stats(*a.values())


def test_token_stats_refusals(lib):
    assert _stats(lib, dt=2) == UNSUPPORTED
    assert _stats(lib, N=-1) == INVALID
    assert _stats(lib, R=-1) == INVALID
    assert _stats(lib, V=0) == INVALID
    assert _stats(lib, V=1 << 31, row=1 << 31, seq=1 << 33) == UNSUPPORTED
    assert _stats(lib, N=1 << 24, R=1 << 10) == UNSUPPORTED
    assert _stats(lib, row=-1) == INVALID
    assert _stats(lib, seq=-1) == INVALID
    assert _stats(lib, seq=1 << 62) == UNSUPPORTED
    assert _stats(lib, row=1 << 62) == UNSUPPORTED
    assert _stats(lib, tseq=-1) == INVALID
    assert _stats(lib, trow=-1) == INVALID
    assert _stats(lib, tseq=1 << 62) == UNSUPPORTED
    assert _stats(lib, trow=1 << 61) == UNSUPPORTED
    assert _stats(lib, top=-1) == INVALID
    assert _stats(lib, top=33) == UNSUPPORTED
    assert _stats(lib, top=5, V=4) == INVALID
    for name in ("z", "tokens", "logp", "H", "norm", "top_tokens", "top_logp", "ws"):
        assert _stats(lib, **{name: None}) == INVALID, name
    for name, bad in (("z", 0x100001), ("tokens", 0x20004), ("lens", 0x20002), ("temp", 0x20002),
                      ("logp", 0x30002), ("H", 0x40001), ("norm", 0x50002), ("top_tokens", 0x60004),
                      ("top_logp", 0x70002), ("ws", 0x80010)):
        assert _stats(lib, **{name: A(bad)}) == MISALIGNED, name
    assert _stats(lib, ws_bytes=256) == WORKSPACE
    outs = ("logp", "H", "norm", "top_tokens", "top_logp", "ws")
    for name in outs:  # over an input, over another output
        for at in (0x100000, 0x20000):
            assert _stats(lib, **{name: A(at)}) == INVALID, name
        assert _stats(lib, **{name: A(0x90000), "lens": A(0x90004)}) == INVALID, name
        assert _stats(lib, **{name: A(0x90000), "temp": A(0x90004)}) == INVALID, name
        for other in outs:
            if other != name:
                assert _stats(lib, **{name: A(0x90000), other: A(0x90000)}) == INVALID, (name, other)
    out = ctypes.c_size_t(0)
    assert lib.grpo_token_stats_workspace_size(4, 3, ctypes.byref(out)) == OK
    assert out.value >= 256 + 4 * 12
    assert lib.grpo_token_stats_workspace_size(-1, 3, ctypes.byref(out)) == INVALID
    assert lib.grpo_token_stats_workspace_size(4, 3, None) == INVALID
    assert lib.grpo_token_stats_workspace_size(1 << 20, 1 << 20, ctypes.byref(out)) == UNSUPPORTED


def _bwd(lib, **kw):
    a = dict(z=A(0x100000), dt=1, N=2, R=3, V=100, seq=300, row=100, tokens=A(0x20000), tseq=3, trow=1,
             lens=None, temp=None, norm=A(0x30000), H=A(0x40000), gl=A(0x50000), gh=A(0x60000),
             dz=A(0x200000), dseq=300, drow=100, stream=None)
    a.update(kw)
    return lib.grpo_token_stats_bwd(*a.values())


def test_token_stats_bwd_refusals(lib):
    assert _bwd(lib, dt=-1) == UNSUPPORTED
    assert _bwd(lib, N=-1) == INVALID
    assert _bwd(lib, V=0) == INVALID
    assert _bwd(lib, row=-1) == INVALID
    assert _bwd(lib, trow=-1) == INVALID
    assert _bwd(lib, dseq=299) == INVALID          # sequences overlap
    assert _bwd(lib, drow=99) == INVALID           # rows overlap
    assert _bwd(lib, dseq=100, drow=199) == INVALID
    assert _bwd(lib, dseq=99, drow=200) == INVALID
    assert _bwd(lib, dseq=1 << 62) == UNSUPPORTED
    for name in ("z", "norm", "dz", "tokens", "H"):
        assert _bwd(lib, **{name: None}) == INVALID, name
    for name, bad in (("z", 0x100001), ("tokens", 0x20004), ("lens", 0x20002), ("temp", 0x20002),
                      ("norm", 0x30002), ("H", 0x40001), ("gl", 0x50002), ("gh", 0x60001),
                      ("dz", 0x200001)):
        assert _bwd(lib, **{name: A(bad)}) == MISALIGNED, name
    assert _bwd(lib, dz=A(0x100000)) == INVALID           # in place
    assert _bwd(lib, dz=A(0x100000 + 2 * 599)) == INVALID  # over the last element
    for name in ("norm", "H", "gl", "gh", "tokens", "lens", "temp"):
        assert _bwd(lib, **{name: A(0x200000 + 8)}) == INVALID, name
    assert _bwd(lib, N=0) == OK                            # nothing to do


class Tensor(ctypes.Structure):
    _fields_ = [("param", P), ("master", P), ("grad", P), ("avg", P), ("sq", P), ("scales", P),
                ("numel", ctypes.c_int64), ("pdt", ctypes.c_int), ("gdt", ctypes.c_int)]


class Hyper(ctypes.Structure):
    _fields_ = [("step", ctypes.c_int64), ("step_dev", P), ("lr", ctypes.c_double), ("lr_dev", P),
                ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("decay", ctypes.c_double), ("norm", P), ("max_norm", ctypes.c_double),
                ("norm_eps", ctypes.c_double)]


def _adamw(lib, tensors=({},), bits=32, count=None, **kw):
    rows = (Tensor * max(1, len(tensors)))()
    for r, t in zip(rows, tensors):
        e = dict(param=0x100000, master=None, grad=0x200000, avg=0x300000, sq=0x400000,
                 scales=0x500000 if bits == 8 else None, numel=100, pdt=0, gdt=0)
        e.update(t)
        for k, v in e.items():
            setattr(r, k, v)
    h = dict(step=1, step_dev=None, lr=1e-3, lr_dev=None, beta1=0.9, beta2=0.99, eps=1e-8,
             decay=0.1, norm=None, max_norm=1.0, norm_eps=1e-6)
    h.update(kw)
    return lib.grpo_adamw_step(rows, len(tensors) if count is None else count, bits,
                               ctypes.byref(Hyper(**h)), None)


def test_adamw_refusals(lib):
    nan, inf = float("nan"), float("inf")
    assert _adamw(lib, bits=16) == UNSUPPORTED
    assert _adamw(lib, count=-1) == INVALID
    assert _adamw(lib, count=1 << 40) == UNSUPPORTED
    assert lib.grpo_adamw_step(None, 1, 32, ctypes.byref(Hyper(step=1)), None) == INVALID
    assert lib.grpo_adamw_step(None, 0, 32, None, None) == INVALID
    for k, bad in (("beta1", (1.0, -0.1, nan)), ("beta2", (1.0, -0.1, nan)), ("eps", (-1.0, inf, nan)),
                   ("decay", (-1.0, inf, nan)), ("lr", (-1.0, inf, nan)), ("step", (0, -3))):
        for x in bad:
            assert _adamw(lib, **{k: x}) == INVALID, (k, x)
    for k, bad in (("max_norm", (-1.0, nan)), ("norm_eps", (-1.0, inf, nan))):
        for x in bad:
            assert _adamw(lib, norm=0x700000, **{k: x}) == INVALID, (k, x)
    for k, bad in (("norm", 0x700002), ("lr_dev", 0x700001), ("step_dev", 0x700004)):
        assert _adamw(lib, **{k: bad}) == MISALIGNED, k
    one = lambda **t: _adamw(lib, [t])
    assert one(pdt=2) == UNSUPPORTED
    assert one(gdt=-1) == UNSUPPORTED
    assert one(numel=-1) == INVALID
    assert one(numel=1 << 62) == UNSUPPORTED
    for k in ("param", "avg", "sq"):
        assert one(**{k: None}) == INVALID, k
        assert one(**{k: 0x900002}) == MISALIGNED, k
    assert one(grad=0x900002) == MISALIGNED
    assert one(grad=0x900001, gdt=1) == MISALIGNED
    assert one(master=0x900000) == INVALID                    # a float32 param has none
    assert one(master=0x900002, pdt=1) == MISALIGNED
    assert one(scales=0x900000) == INVALID                    # 32-bit states have none
    assert _adamw(lib, [dict(scales=None)], bits=8) == INVALID
    assert _adamw(lib, [dict(scales=0x900002)], bits=8) == MISALIGNED
    for k in ("grad", "avg", "sq"):
        assert one(**{k: 0x100000 + 396}) == INVALID, k       # over the param's last element
    assert one(master=0x300000, pdt=1) == INVALID
    # a param listed twice, or overlapping the one before
    assert _adamw(lib, [{}, dict(grad=0x210000, avg=0x310000, sq=0x410000)]) == INVALID
    assert _adamw(lib, [dict(param=0x100000 + 200), dict(grad=0x210000, avg=0x310000,
                                                         sq=0x410000)]) == INVALID
    # nothing to do: no tensors, empty ones, none with a gradient
    assert _adamw(lib, []) == OK
    assert _adamw(lib, [dict(numel=0, param=None), dict(grad=None)]) == OK


class _Elsewhere(torch.Tensor):
    """A tensor that says it is on a device and has no memory."""

    @staticmethod
    def __new__(cls, device, shape, dtype=torch.float32):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device=device)

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise AssertionError(f"{func} on a tensor without memory")


def test_binding_refuses_tensors_of_another_device(n):
    on = lambda *s, dtype=torch.float32: _Elsewhere("cuda:7", s, dtype)
    z, y, two, x = on(2, 3, 16), on(2, 3, dtype=torch.int64), on(2, 3, 2), on(2, 3)
    for call in (lambda: n.grpo_token_stats(z, y), lambda: n.grpo_token_stats_bwd(z, y, two, x, x),
                 lambda: n.grpo_adamw_step([x], [x], {"exp_avg": [x], "exp_avg_sq": [x]}, 1, 0.1)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()


def test_binding_refuses_cpu_tensors_and_wrong_types(n):
    z, y, x = torch.zeros(2, 3, 16), torch.zeros(2, 3, dtype=torch.int64), torch.zeros(2, 3)
    with pytest.raises(ValueError):
        n.grpo_token_stats(z, y)
    with pytest.raises(TypeError):
        n.grpo_token_stats(z.tolist(), y)
    with pytest.raises(ValueError):
        n.grpo_token_stats_bwd(z, y, x, x)
    with pytest.raises(ValueError):
        n.grpo_adamw_step([x], [x], {"exp_avg": [x], "exp_avg_sq": [x]}, 1, 0.1)
    with pytest.raises(TypeError):
        n.grpo_adamw_step(7, [], {}, 1, 0.1)
    with pytest.raises(TypeError):
        n.grpo_adamw_step([], [], [], 1, 0.1)
    with pytest.raises(ValueError, match="exp_avg"):
        n.grpo_adamw_step([], [], {}, 1, 0.1)
    with pytest.raises(ValueError, match="one tensor per param"):
        n.grpo_adamw_step([], [x], {"exp_avg": [], "exp_avg_sq": []}, 1, 0.1)
    with pytest.raises(TypeError):
        n.grpo_adamw_step([], [], {"exp_avg": [], "exp_avg_sq": []}, 1, "fast")
    with pytest.raises(n.GrpoError):
        n.grpo_adamw_step([], [], {"exp_avg": [], "exp_avg_sq": []}, 0, 0.1)
    with pytest.raises(ValueError):
        n.grpo_adamw_state([x], bits=16)


def test_states(n):
    """The layout of the states (of host tensors, which need no GPU)."""
    params = [torch.zeros(3, 100), torch.ones(257, dtype=torch.bfloat16), torch.zeros(0)]
    s = n.grpo_adamw_state(params)
    assert set(s) == {"exp_avg", "exp_avg_sq"} and s["exp_avg"][1].dtype == torch.float32
    s = n.grpo_adamw_state(params, 8, master=True)
    assert set(s) == {"exp_avg", "exp_avg_root", "scales", "master"}
    assert [tuple(t.shape) for t in s["scales"]] == [(2, 2), (2, 2), (0, 2)]
    assert s["exp_avg"][0].dtype == torch.float8_e4m3fn and s["exp_avg"][0].shape == (3, 100)
    assert (s["exp_avg_root"][1].float() == 0).all()
    assert [t is None for t in s["master"]] == [True, False, True] and (s["master"][1] == 1).all()


def test_package_exports():
    import vocab_wide_logprob_gb300 as pkg
    for name in ("grpo_token_stats", "grpo_token_stats_bwd", "grpo_adamw_state", "grpo_adamw_step",
                 "GRPOTokenStats", "grpo_logp_entropy"):
        assert callable(getattr(pkg, name))


def test_adamw_eps_without_a_reciprocal(lib):
    assert _adamw(lib, [], eps=2.0 ** 126) == OK
    for x in (2.0 ** 126 * 1.01, 3e38):
        assert _adamw(lib, [], eps=x) == INVALID, x


def test_states_of_a_modules_parameters(n):
    """parameters() is a generator: every list of the states has an entry for each."""
    m = torch.nn.Linear(300, 5).bfloat16()
    for bits in (32, 8):
        s = n.grpo_adamw_state(m.parameters(), bits, master=True)
        assert all(len(v) == 2 for v in s.values()), {k: len(v) for k, v in s.items()}
