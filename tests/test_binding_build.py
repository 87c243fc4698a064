"""The binding of the operators around the loss (module _ops) is rebuilt for
another PyTorch or Python, and the loss calls load without it."""
import os
import subprocess
import sys

import pytest

from vocab_wide_logprob_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_another_torch_or_python_makes_it_stale(monkeypatch):
    build.build()
    obj = os.path.join(build.BUILD, "binding.o")
    assert not build._binding_stale(obj)
    target = build.binding_target()
    import torch
    assert torch.__version__ in target and sys.implementation.cache_tag in target
    monkeypatch.setattr(build, "binding_target", lambda: target + " and more")
    assert build._binding_stale(obj)


def _run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


LOSS_ONLY = """
from vocab_wide_logprob_gb300 import _native as n
assert n.grpo_workspace_size(2, 8, 100) > 0
assert n.library().grpo_status_string(0)
import vocab_wide_logprob_gb300.autograd
import torch
for call in (lambda: n.grpo_embed_fwd(torch.zeros(1).long(), torch.zeros(2, 2)),
             lambda: n.grpo_clip_grad_norm([], 1.0)):
    try:
        call()
    except ImportError as e:
        assert "_ops.so" in str(e) and "build" in str(e), e
    else:
        raise AssertionError("no error")
"""


@pytest.mark.parametrize("how", ["missing", "other"])
def test_loss_calls_load_without_it(how):
    build.build()
    stub = "None" if how == "missing" else "types.SimpleNamespace(built_for='torch 1.0')"
    _run("import sys, types\n"
         f"sys.modules['vocab_wide_logprob_gb300._ops'] = {stub}\n" + LOSS_ONLY)


def test_it_loads_where_it_fits():
    build.build()
    _run("from vocab_wide_logprob_gb300 import _native as n, build\n"
         "assert n._ops.built_for == build.binding_target()\n")
