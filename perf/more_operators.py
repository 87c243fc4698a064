"""Timing cases of the per-token statistics of logits (log-probs, entropy, top
alternatives), their gradient, and the AdamW step over many tensors.

Each case describes one call of a rollout or of a policy update.  ``prepare``
draws the inputs from a seed, ``run`` makes one pass (the plain torch form, or
the library's calls when ``own`` is set), ``exact`` gives the results from the
definitions in 64 bits, and ``work`` counts the bytes and operations a pass
cannot do without.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ESIZE = {"f32": 4, "bf16": 2}
VOCAB, HIDDEN, FF = 151936, 896, 4864  # the vocabulary of the loss workloads, the LM head's model
BLOCK = 256  # elements of an 8-bit state that share a scale
F8_MAX, F8_TINY = 448.0, 2.0 ** -9  # e4m3: the largest and the smallest positive value
BETA1, BETA2, EPS, DECAY = 0.9, 0.95, 1e-8, 0.1


def listed():
    return [
        # eight rollouts, one sampled token each: its log-prob and the 20 alternatives a server returns
        {"name": "stats_8_tokens", "op": "stats", "N": 8, "R": 1, "V": VOCAB, "w": "bf16", "top": 20, "tempered": True,
         "banned": 0.0, "ragged": False},
        # the completions of a small update batch, log-probs and entropy, rows behind each end left out
        {"name": "stats_rollout", "op": "stats", "N": 8, "R": 256, "V": VOCAB, "w": "bf16", "top": 0,
         "tempered": False, "banned": 0.0, "ragged": True},
        # scoring a batch with the alternatives of every position
        {"name": "stats_alternatives", "op": "stats", "N": 16, "R": 128, "V": VOCAB, "w": "bf16", "top": 5,
         "tempered": False, "banned": 0.0, "ragged": False},
        # float32 logits of an odd vocabulary, tokens banned by the sampler, temperatures of their own
        {"name": "stats_odd", "op": "stats", "N": 33, "R": 7, "V": 32003, "w": "f32", "top": 32, "tempered": True,
         "banned": 0.3, "ragged": True},
        # every completion of an update batch, entropy watched
        {"name": "stats_batch", "op": "stats", "N": 16, "R": 512, "V": VOCAB, "w": "bf16", "top": 0,
         "tempered": False, "banned": 0.0, "ragged": False},
        # a toy policy's batch: the smallest gradient
        {"name": "grad_tiny", "op": "grad", "N": 8, "R": 32, "V": 1024, "w": "f32", "of": "both", "tempered": False,
         "banned": 0.0, "ragged": True},
        # an entropy bonus alone over an odd vocabulary with banned tokens
        {"name": "grad_odd", "op": "grad", "N": 5, "R": 77, "V": 32003, "w": "bf16", "of": "entropy",
         "tempered": True, "banned": 0.3, "ragged": False},
        # policy gradient with an entropy bonus over an update batch
        {"name": "grad_batch", "op": "grad", "N": 16, "R": 512, "V": VOCAB, "w": "bf16", "of": "both",
         "tempered": False, "banned": 0.0, "ragged": True},
        # a small model, everything in float32
        {"name": "adamw_small", "op": "adamw", "layers": 2, "d": 130, "ff": 351, "kv": 26, "V": 1024, "p": "f32",
         "master": False, "g": "f32", "bits": 32, "over": True},
        # a model with the LM head's vocabulary: bfloat16 weights and gradients, float32 masters and states
        {"name": "adamw_model", "op": "adamw", "layers": 24, "d": HIDDEN, "ff": FF, "kv": 128, "V": VOCAB,
         "p": "bf16", "master": True, "g": "bf16", "bits": 32, "over": True},
        # the same model with states in 8 bits and float32 weights
        {"name": "adamw_model_8bit", "op": "adamw", "layers": 24, "d": HIDDEN, "ff": FF, "kv": 128, "V": VOCAB,
         "p": "f32", "master": False, "g": "bf16", "bits": 8, "over": False},
        # few tensors of odd sizes, bfloat16 weights without masters, states in 8 bits
        {"name": "adamw_odd_8bit", "op": "adamw", "layers": 1, "d": 901, "ff": 2703, "kv": 77, "V": 5001,
         "p": "bf16", "master": False, "g": "f32", "bits": 8, "over": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["stats", "grad", "adamw"])
    if op == "adamw":
        d = rng.choice([64, 130, 256, 510, 768, HIDDEN, 901])
        c = {"op": op, "layers": rng.randint(0, 12), "d": d, "ff": rng.randint(d, 5 * d), "kv": rng.randint(1, d),
             "V": _log(rng, 1000, VOCAB)}
        c["p"], c["master"] = rng.choice([("f32", False), ("bf16", False), ("bf16", True)])
        c["g"], c["bits"], c["over"] = rng.choice(["f32", "bf16"]), rng.choice([8, 32]), rng.random() < 0.5
        return c
    c = {"op": op, "N": _log(rng, 1, 64), "R": _log(rng, 1, 512), "V": _log(rng, 1000, VOCAB),
         "w": rng.choice(["f32", "bf16"]), "tempered": rng.random() < 0.5, "banned": rng.choice([0.0, 0.0, 0.02, 0.5]),
         "ragged": rng.random() < 0.5}
    if op == "stats":
        c["top"] = rng.choice([0, 1, 5, 20, 32])
    else:
        c["of"] = rng.choice(["both", "logp", "entropy"])
    # at most the largest listed batch; with alternatives a quarter of it
    most = 16 * 512 * VOCAB * 2 // (4 if c.get("top") else 1)
    c["R"] = max(1, min(c["R"], most // (c["N"] * c["V"] * ESIZE[c["w"]])))
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _shapes(case):
    d, ff, kv = case["d"], case["ff"], case["kv"]
    layer = [(d, d), (d,), (kv, d), (kv,), (kv, d), (kv,), (d, d), (ff, d), (ff, d), (d, ff), (d,), (d,)]
    return layer * case["layers"] + [(case["V"], d), (d,)]


def _lens(case, g):
    """Completion lengths, evenly spread from 0 to R, in an order of the seed's."""
    N, R = case["N"], case["R"]
    if not case["ragged"]:
        return None
    even = torch.linspace(R if N == 1 else 0, R, N, device="cuda", dtype=torch.float64).round().int()
    return even[torch.randperm(N, generator=g, device="cuda")].contiguous()


def _prepare_rows(case, s, g):
    N, R, V, dt = case["N"], case["R"], case["V"], DTYPES[case["w"]]
    # logits as a model gives them: one row more than is scored (the last token's)
    buf = torch.randn(N, R + 1, V, generator=g, device="cuda", dtype=torch.float32 if N * R * V < 1 << 28 else dt)
    buf = buf.mul_(3.0).to(dt)
    s["logits"] = buf[:, :R]
    s["lens"] = _lens(case, g)
    s["temperature"] = torch.rand(N, generator=g, device="cuda") * 0.9 + 0.6 if case["tempered"] else None
    # tokens as sampled: most of them likely ones
    tokens = torch.randint(0, V, (N, R), generator=g, device="cuda")
    logits = s["logits"]
    for i in range(N):
        race = torch.empty(R, V, device="cuda").exponential_(generator=g).log_()
        T = 1.0 if s["temperature"] is None else s["temperature"][i]
        tokens[i] = (logits[i].float() / T - race).argmax(-1)
    if case["banned"]:
        ban = torch.rand(V, generator=g, device="cuda") < case["banned"]
        for i in range(N):
            logits[i].masked_fill_(ban, -math.inf)
            logits[i].scatter_(1, tokens[i].unsqueeze(1), 6.0)
    s["tokens"] = tokens


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "adamw":
        _prepare_adamw(case, s, g)
        return s
    _prepare_rows(case, s, g)
    if case["op"] == "grad":
        N, R = case["N"], case["R"]
        m = s["logits"].amax(-1).float()
        T = torch.ones(N, device="cuda") if s["temperature"] is None else s["temperature"]
        # what the forward kept: the rows' largest logits, log-sums and entropies
        norm, entropy = torch.zeros(N, R, 2, device="cuda"), torch.zeros(N, R, device="cuda")
        for i in range(N):
            t = (s["logits"][i].float() - m[i].unsqueeze(-1)) / T[i]
            w = t.exp()
            total = w.sum(-1, dtype=torch.float64)
            norm[i, :, 0], norm[i, :, 1] = m[i], total.log()
            t.clamp_(min=-1e30).mul_(w)
            entropy[i] = total.log() - t.sum(-1, dtype=torch.float64) / total
        if s["lens"] is not None:
            left = torch.arange(R, device="cuda") >= s["lens"].unsqueeze(1)
            norm[left], entropy[left] = 0.0, 0.0
        s["norm"], s["entropy"] = norm, entropy
        scale = 1.0 / (N * R)
        s["grad_logp"] = s["grad_entropy"] = None
        if case["of"] != "entropy":
            s["grad_logp"] = torch.randn(N, R, generator=g, device="cuda") * scale
        if case["of"] != "logp":
            s["grad_entropy"] = torch.rand(N, R, generator=g, device="cuda") * (-0.01 * scale)
    return s


def _prepare_adamw(case, s, g):
    shapes = _shapes(case)
    sizes = [math.prod(sh) for sh in shapes]
    # every kind of tensor lies in one buffer, as an optimizer over a flattened model keeps them
    starts, at = [], 0
    for k in sizes:
        starts.append(at)
        at += -(-k // BLOCK) * BLOCK
    used = torch.zeros(at, dtype=torch.bool, device="cuda")
    for a, k in zip(starts, sizes):
        used[a:a + k] = True

    def views(flat):
        return [flat[a:a + k].view(sh) for a, k, sh in zip(starts, sizes, shapes)]

    full = torch.randn(at, generator=g, device="cuda").mul_(0.02).mul_(used)
    s["flat_param"] = full.to(DTYPES[case["p"]])
    s["flat_master"] = full if case["master"] else None
    # gradients of a level of their own for every block, as layers and rows of an embedding have
    level = torch.exp(torch.randn(at // BLOCK, 1, generator=g, device="cuda") - 9.0)
    grad = torch.randn(at // BLOCK, BLOCK, generator=g, device="cuda").mul_(level).view(-1).mul_(used)
    s["norm"] = torch.stack([grad.square().sum(dtype=torch.float64).sqrt().float(), torch.ones((), device="cuda")])
    s["max_norm"] = float(s["norm"][0]) * (0.37 if case["over"] else 2.0)
    s["flat_grad"] = grad.to(DTYPES[case["g"]])
    coef = min(1.0, s["max_norm"] / float(s["norm"][0]))
    avg = torch.randn(at // BLOCK, BLOCK, generator=g, device="cuda").mul_(level * (0.3 * coef)).view(-1).mul_(used)
    spread = torch.rand(at // BLOCK, BLOCK, generator=g, device="cuda").add_(0.5)
    root = spread.mul_(level * coef).view(-1).mul_(used)
    s["flat_scales"] = None
    if case["bits"] == 8:
        s["flat_avg"], s_avg = _to8(avg, False)
        s["flat_sq"], s_root = _to8(root, True)
        s["flat_scales"] = torch.stack([s_avg, s_root], 1)  # [blocks, 2]
    else:
        s["flat_avg"], s["flat_sq"] = avg, root.square_()
    del avg, root, level, used
    s["step"], s["lr"] = 100, 3e-4
    s["params"], s["grads"] = views(s["flat_param"]), views(s["flat_grad"])
    state = {"exp_avg": views(s["flat_avg"])}
    state["exp_avg_sq" if case["bits"] == 32 else "exp_avg_root"] = views(s["flat_sq"])
    if case["master"]:
        state["master"] = views(s["flat_master"])
    if case["bits"] == 8:
        state["scales"] = [s["flat_scales"][a // BLOCK:(a + k + BLOCK - 1) // BLOCK] for a, k in zip(starts, sizes)]
    s["state"] = state


def _to8(x, root):
    """Blocks of 256 values as e4m3 and a scale each: value = code * scale."""
    b = x.view(-1, BLOCK)
    scale = b.abs().amax(-1) / F8_MAX
    code = b / torch.where(scale > 0, scale, 1.0).unsqueeze(-1)
    if root:  # a positive root stays positive
        code = torch.where(b > 0, code.clamp(min=F8_TINY), code)
    return code.view(-1).to(torch.float8_e4m3fn), scale


def _from8(code, scale):
    return (code.float().view(-1, BLOCK) * scale.unsqueeze(-1)).view(-1)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "adamw":
        return _adamw_plain(s)
    if s["op"] == "stats":
        return _stats_plain(s)
    return _grad_plain(s)


def _kept(s):
    """[N, R, 1]: whether a row is inside its sequence."""
    at = torch.arange(s["R"], device="cuda")
    lens = s["lens"] if s["lens"] is not None else torch.full((s["N"],), s["R"], device="cuda")
    return (at < lens.unsqueeze(1)).unsqueeze(-1)


def _warmth(s):
    T = s["temperature"] if s["temperature"] is not None else torch.ones(s["N"], device="cuda")
    return T.view(-1, 1, 1)


def _stats_plain(s):
    z = s["logits"].float()
    m = z.amax(-1, keepdim=True)
    t = (z - m) / _warmth(s)
    w = t.exp()
    total = w.sum(-1, keepdim=True)
    L = total.log()
    logp = t.gather(-1, s["tokens"].unsqueeze(-1)) - L
    entropy = L - torch.where(w > 0, w * t, 0.0).sum(-1, keepdim=True) / total
    keep = _kept(s)
    out = {"logp": torch.where(keep, logp, 0.0).squeeze(-1), "entropy": torch.where(keep, entropy, 0.0).squeeze(-1),
           "norm": torch.where(keep, torch.cat([m, L], -1), 0.0)}
    if s["top"]:
        # unique keys: the value's bits in the order of the values, then the lower id first
        bits = torch.where(z == 0, 0.0, z).view(torch.int32).long()
        order = torch.where(bits < 0, -2147483648 - bits, bits)
        keys = order * 4294967296 + torch.arange(s["V"] - 1, -1, -1, device="cuda")
        best = keys.topk(s["top"], -1).values
        ids = s["V"] - 1 - best.remainder(4294967296)
        out["top_tokens"] = torch.where(keep, ids, -1)
        out["top_logp"] = torch.where(keep, t.gather(-1, ids) - L, 0.0)
    return out


def _grad_plain(s):
    T = _warmth(s)
    logq = (s["logits"].float() - s["norm"][..., :1]) / T - s["norm"][..., 1:]
    p = logq.exp()
    dz = torch.zeros_like(p)
    if s["grad_logp"] is not None:
        dz -= p * s["grad_logp"].unsqueeze(-1)
        dz.scatter_add_(-1, s["tokens"].unsqueeze(-1), s["grad_logp"].unsqueeze(-1))
    if s["grad_entropy"] is not None:
        dz -= torch.where(p > 0, p * (logq + s["entropy"].unsqueeze(-1)), 0.0) * s["grad_entropy"].unsqueeze(-1)
    return torch.where(_kept(s), dz / T, 0.0).to(DTYPES[s["w"]])


def _adamw_plain(s):
    coef = (s["max_norm"] / (s["norm"][0] + 1e-6)).clamp(max=1.0)
    grad = s["flat_grad"].float() * coef
    eight = s["bits"] == 8
    avg = _from8(s["flat_avg"], s["flat_scales"][:, 0]) if eight else s["flat_avg"]
    sq = _from8(s["flat_sq"], s["flat_scales"][:, 1]).square() if eight else s["flat_sq"]
    avg = avg * BETA1 + grad * (1 - BETA1)
    sq = sq * BETA2 + grad * grad * (1 - BETA2)
    root = sq.sqrt()
    up = avg / (1 - BETA1 ** s["step"]) / (root / math.sqrt(1 - BETA2 ** s["step"]) + EPS)
    value = s["flat_master"] if s["master"] else s["flat_param"].float()
    value = value - s["lr"] * (up + DECAY * value)
    if s["master"]:
        s["flat_master"].copy_(value)
    s["flat_param"].copy_(value)
    if eight:
        code, scale = _to8(avg, False)
        s["flat_avg"].copy_(code)
        s["flat_scales"][:, 0] = scale
        code, scale = _to8(root, True)
        s["flat_sq"].copy_(code)
        s["flat_scales"][:, 1] = scale
    else:
        s["flat_avg"].copy_(avg)
        s["flat_sq"].copy_(sq)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    # (8-bit states: the numbers that the codes are, and the blocks' scales)
    return {k: s["flat_" + k] for k in ("param", "master", "avg", "sq", "scales") if s["flat_" + k] is not None}


def _run_own(s):
    import vocab_wide_logprob_gb300 as grpo
    if s["op"] == "stats":
        out = grpo.grpo_token_stats(s["logits"], s["tokens"], s["lens"], s["temperature"], top=s["top"])
        return {k: v for k, v in out.items() if k != "workspace"}
    if s["op"] == "grad":
        return grpo.grpo_token_stats_bwd(s["logits"], s["tokens"], s["norm"], s["entropy"], s["grad_logp"],
                                         s["grad_entropy"], s["lens"], s["temperature"])
    grpo.grpo_adamw_step(s["params"], s["grads"], s["state"], s["step"], s["lr"], beta1=BETA1, beta2=BETA2, eps=EPS,
                         weight_decay=DECAY, norm=s["norm"], max_norm=s["max_norm"])
    return _adamw_outputs(s)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its results in 64 bits
# ---------------------------------------------------------------------------


def work(case):
    if case["op"] == "adamw":
        n = sum(math.prod(sh) for sh in _shapes(case))
        each = 2 * ESIZE[case["p"]] + ESIZE[case["g"]] + (16 if case["bits"] == 32 else 4 + 16 / BLOCK)
        if case["master"]:  # the bfloat16 weight is only written
            each += 8 - ESIZE[case["p"]]
        return {"bytes": n * each, "flops": 16 * n}
    rows = case["N"] * case["R"]
    scored = rows / 2 if case["ragged"] else rows
    row = case["V"] * ESIZE[case["w"]]
    if case["op"] == "stats":
        return {"bytes": scored * (row + 8) + rows * (16 + 12 * case["top"]), "flops": scored * case["V"] * 6}
    return {"bytes": scored * (row + 8 + 12 + 8) + rows * row, "flops": scored * case["V"] * 6}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _adamw_exact(case, s)
    N, R = case["N"], case["R"]
    outs = []
    for i in range(N):  # a sequence at a time: float64 copies of a batch's logits are large
        n = R if s["lens"] is None else int(s["lens"][i])
        T = 1.0 if s["temperature"] is None else s["temperature"][i].double()
        lq = torch.log_softmax(s["logits"][i, :n].double() / T, -1)
        y = s["tokens"][i, :n].unsqueeze(-1)
        neg = torch.special.entr(lq.exp())  # -p ln p, 0 at p = 0
        H = neg.sum(-1, keepdim=True)
        if case["op"] == "stats":
            m = s["logits"][i, :n].double().amax(-1, keepdim=True)
            one = {"logp": _rows(lq.gather(-1, y).squeeze(-1), R), "entropy": _rows(H.squeeze(-1), R),
                   "norm": _rows(torch.cat([m, -lq.amax(-1, keepdim=True)], -1), R)}
            if case["top"]:
                best = s["logits"][i, :n].sort(dim=-1, descending=True, stable=True).indices[:, :case["top"]]
                one["top_tokens"] = _rows(best, R, -1)
                one["top_logp"] = _rows(lq.gather(-1, best), R)
            outs.append(one)
            continue
        d = torch.zeros_like(lq)
        if s["grad_entropy"] is not None:  # dH/dz_v = -p_v ln p_v - p_v H
            d = s["grad_entropy"][i, :n].double().unsqueeze(-1) * (neg - lq.exp() * H)
        if s["grad_logp"] is not None:
            g = s["grad_logp"][i, :n].double().unsqueeze(-1)
            d = d - g * lq.exp()
            d[torch.arange(n, device="cuda"), y.squeeze(-1)] += g.squeeze(-1)
        outs.append(_rows(d / T, R))
    if case["op"] == "grad":
        return torch.stack(outs)
    return {k: torch.stack([o[k] for o in outs]) for k in outs[0]}


def _rows(x, R, fill=0):
    """x with rows of `fill` behind it, R in all."""
    full = x.new_full((R,) + tuple(x.shape[1:]), fill)
    full[:x.shape[0]] = x
    return full


def _adamw_exact(case, s):
    t, lr, norm = s["step"], s["lr"], float(s["norm"][0])
    c = min(1.0, s["max_norm"] / (norm + 1e-6))
    out = {k: [] for k in ("param", "master", "avg", "sq", "scales")}
    n, piece = s["flat_param"].numel(), BLOCK << 18
    for a in range(0, n, piece):
        part = slice(a, min(n, a + piece))
        g = s["flat_grad"][part].double() * c
        m, v = s["flat_avg"][part].double(), s["flat_sq"][part].double()
        if case["bits"] == 8:
            scales = s["flat_scales"][a // BLOCK:(part.stop + BLOCK - 1) // BLOCK].double()
            each = scales.repeat_interleave(BLOCK, 0)
            m, v = m * each[:, 0], (v * each[:, 1]).pow(2)
        m.lerp_(g, 1.0 - BETA1)
        v.lerp_(g * g, 1.0 - BETA2)
        w = (s["flat_master"] if case["master"] else s["flat_param"])[part].double()
        hat = (v / -math.expm1(t * math.log(BETA2))).sqrt()
        w = w * (1.0 - lr * DECAY) - lr * (m / -math.expm1(t * math.log(BETA1))) / (hat + EPS)
        out["param"].append(w)
        out["master"].append(w)
        if case["bits"] == 32:
            out["avg"].append(m)
            out["sq"].append(v)
            continue
        r = v.sqrt()
        top = torch.stack([m.view(-1, BLOCK).abs().amax(-1), r.view(-1, BLOCK).amax(-1)], 1) / F8_MAX
        div = top.clamp(min=1e-300).repeat_interleave(BLOCK, 0)
        out["avg"].append(m / div[:, 0])  # (before their rounding to 8 bits)
        out["sq"].append(r / div[:, 1])
        out["scales"].append(top)
    got = {k: torch.cat(v) for k, v in out.items() if v}
    if not case["master"]:
        got.pop("master")
    return got
