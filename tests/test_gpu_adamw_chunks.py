"""AdamW steps so large that a thread block may take two units of a tensor (where params and
gradients differ in type): tensors that end in either unit, at any alignment, beside a
large one.  Tolerances as for small ones."""
import pytest
import torch

import test_gpu_adamw as small

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
UNIT = 2048  # elements that a thread block takes at once
ENDS = [1, 255, UNIT - 1, UNIT, UNIT + 1, UNIT + 300, 2 * UNIT - 1, 2 * UNIT, 2 * UNIT + 1, 6000, 3 * UNIT + 257]


def sizes():
    """More than 64 chunks of two units per SM in all."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return ENDS[:6] + [64 * 2 * UNIT * (sms + 1) + 77] + ENDS[6:]


@pytest.mark.parametrize("phases", [(0,), (1, 8, 3, 0)], ids=["aligned", "mixed"])
@pytest.mark.parametrize("gts", [[F32], [BF16], [F32, BF16]], ids=["g32", "g16", "gmix"])
@pytest.mark.parametrize("kind", small.KINDS, ids=[k[0] for k in small.KINDS])
def test_large_steps(kind, gts, phases):
    n = small.g()
    was = small.make(sizes(), kind[1], gts, 8, kind[2], 30, phases)
    place = lambda k, t: None if t is None else small.at_phase(t, phases[k % len(phases)])
    now = ([place(k, t) for k, t in enumerate(was[0])], [place(k, t) for k, t in enumerate(was[1])],
           {key: [t.clone() if key == "scales" else place(k, t) for k, t in enumerate(v)]
            for key, v in was[2].items()})
    n.grpo_adamw_step(*now, 7, 1e-3, **small.HYPER)
    small.check(was, now, 7, 1e-3, **small.HYPER)


def test_a_second_unit_with_squares_outside_float32s_range():
    """Each unit's v' that is infinite or tiny is its own affair."""
    n = small.g()
    was = small.make(sizes(), [BF16], [F32], 8, False, 31)
    big = max(range(len(ENDS) + 1), key=lambda k: was[1][k].numel())
    grad = was[1][big]
    grad[UNIT + 5] = 1e25
    grad[10 * UNIT:10 * UNIT + 512] = 1e-19
    now = small.copies(*was)
    n.grpo_adamw_step(*now, 7, 1e-3, **small.HYPER)
    # (an infinite v': the weight only decays)
    w = was[0][big][UNIT + 5].double()
    assert (now[0][big][UNIT + 5].double() - w * (1 - 1e-3 * small.HYPER["weight_decay"])).abs() <= 2.0 ** -8 * 1.001 * w.abs()
    assert now[2]["scales"][big].isfinite().all() and now[0][big].isfinite().all()
    # everything but that element's block as ever
    cut = lambda t, size: torch.cat([t[:UNIT // 256 * size], t[(UNIT // 256 + 1) * size:]])
    pick = lambda x: ([cut(x[0][big], 256)], [cut(x[1][big], 256)],
                      {"scales": [cut(x[2]["scales"][big], 1)], "exp_avg": [cut8(x[2]["exp_avg"][big])],
                       "exp_avg_root": [cut8(x[2]["exp_avg_root"][big])]})
    cut8 = lambda t: cut(t.view(torch.uint8), 256).view(torch.float8_e4m3fn)
    small.check(pick(was), pick(now), 7, 1e-3, **small.HYPER)
