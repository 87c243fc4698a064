"""Timing cases of the operators around the loss: the embedding lookup and its
gradient, the global gradient norm with clipping, and the verification of
drafted tokens.

Each case describes one call of a policy update or of the rollout before it.
``prepare`` draws the inputs from a seed, ``run`` makes one pass (the plain
torch form, or the library's calls when ``own`` is set), ``exact`` gives the
results from the definitions in 64 bits, and ``work`` counts the bytes and
operations a pass cannot do without.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ESIZE = {"f32": 4, "bf16": 2}
VOCAB, HIDDEN = 151936, 896  # the vocabulary of the loss workloads and the LM head's hidden size


def listed():
    return [
        # one new token of each of eight rollouts enters the model
        {"name": "embed_8_tokens", "op": "embed", "n": 8, "V": VOCAB, "d": HIDDEN, "w": "bf16", "out": "bf16",
         "scale": 1.0},
        # prompts and completions of a whole update batch (64 x 1280 tokens)
        {"name": "embed_batch", "op": "embed", "n": 81920, "V": VOCAB, "d": HIDDEN, "w": "bf16", "out": "bf16",
         "scale": 1.0},
        # float32 master weights of an odd vocabulary and hidden size, scaled, cast on the way out
        {"name": "embed_odd_scaled", "op": "embed", "n": 5001, "V": 32003, "d": 901, "w": "f32", "out": "bf16",
         "scale": 30.0},
        # gradient of a small update batch (16 x 768 tokens): the rows nobody used are most of the bytes
        {"name": "embed_grad_small", "op": "embed_grad", "n": 12288, "V": VOCAB, "d": HIDDEN, "w": "bf16",
         "out": "f32", "scale": 1.0, "pads": 0.3},
        # gradient of a whole update batch, float32 gradients, padded with the end token
        {"name": "embed_grad_batch", "op": "embed_grad", "n": 131072, "V": VOCAB, "d": HIDDEN, "w": "f32",
         "out": "f32", "scale": 1.0, "pads": 0.5},
        # a few tokens, small odd table
        {"name": "embed_grad_odd", "op": "embed_grad", "n": 777, "V": 1024, "d": 130, "w": "f32", "out": "bf16",
         "scale": 11.5, "pads": 0.1},
        # a small model's gradients, clipped into the optimizer's buffer
        {"name": "clip_small", "op": "clip", "layers": 2, "d": 130, "ff": 351, "kv": 26, "V": 1024, "w": "f32",
         "out": "f32", "over": True},
        # every gradient of a model with the LM head's vocabulary, bfloat16, over the limit
        {"name": "clip_model", "op": "clip", "layers": 24, "d": HIDDEN, "ff": 4864, "kv": 128, "V": VOCAB,
         "w": "bf16", "out": "bf16", "over": True},
        # float32 gradients under the limit, in place: only the norm is needed
        {"name": "norm_under_limit", "op": "clip", "layers": 5, "d": HIDDEN, "ff": 4864, "kv": 128, "V": VOCAB,
         "w": "f32", "out": "", "over": False},
        # eight rollouts sample one token each, nothing drafted
        {"name": "verify_8_single", "op": "verify", "N": 8, "K": 0, "V": VOCAB, "w": "bf16", "draft": True,
         "spread": 0.7, "greedy": 0.0, "banned": 0.0},
        # a decode batch with a draft model, four tokens drafted
        {"name": "verify_128_by_4", "op": "verify", "N": 128, "K": 4, "V": VOCAB, "w": "bf16", "draft": True,
         "spread": 0.7, "greedy": 0.0, "banned": 0.0},
        # drafts without probabilities (copied from the prompt), ragged, some greedy, some tokens banned
        {"name": "verify_33_copied", "op": "verify", "N": 33, "K": 7, "V": 32003, "w": "f32", "draft": False,
         "spread": 0.0, "greedy": 0.3, "banned": 0.05},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "clip", "verify"])
    pair = rng.choice([("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
    if op in ("embed", "embed_grad"):
        c = {"op": op, "n": _log(rng, 1, 131072), "V": _log(rng, 1000, VOCAB),
             "d": rng.choice([64, 130, 256, 512, 901, HIDDEN, 1024, 2048]), "w": pair[0], "out": pair[1],
             "scale": rng.choice([1.0, rng.uniform(0.1, 30.0)])}
        # at most the largest listed table and batch
        c["n"] = min(c["n"], 131072 * HIDDEN // (2 * c["d"]))
        c["V"] = min(c["V"], VOCAB * HIDDEN // c["d"])
        if op == "embed_grad":
            c["pads"] = rng.choice([0.0, 0.1, 0.5, 0.9])
        return c
    if op == "clip":
        d = rng.choice([64, 130, 256, 510, HIDDEN])
        out = rng.choice([pair[1], pair[1], ""])  # "": in place, and then under the limit (a pass can be repeated)
        return {"op": op, "layers": rng.randint(0, 12 if out else 5), "d": d, "ff": rng.randint(d, 5 * d),
                "kv": rng.randint(1, d), "V": _log(rng, 1000, VOCAB // 2), "w": pair[0], "out": out,
                "over": bool(out) and rng.random() < 0.7}
    c = {"op": op, "N": _log(rng, 1, 128), "K": rng.randint(0, 8), "V": _log(rng, 1000, VOCAB), "w": pair[0],
         "draft": rng.random() < 0.6, "spread": rng.uniform(0.2, 1.5), "greedy": rng.choice([0.0, 0.0, 0.5, 1.0]),
         "banned": rng.choice([0.0, 0.0, 0.02, 0.5])}
    c["N"] = max(1, min(c["N"], 128 * 5 * VOCAB * 2 // ((c["K"] + 1) * c["V"] * ESIZE[c["w"]])))
    if not c["draft"]:
        c["spread"] = 0.0
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _tokens(n, V, g):
    """Token ids with a 1/rank law, the frequent ones spread over the table."""
    rank = torch.exp(torch.rand(n, generator=g, device="cuda", dtype=torch.float64) * math.log(V)).long() - 1
    return rank.clamp_(0, V - 1).mul_(1000003).remainder_(V)


def _shapes(case):
    d, ff, kv = case["d"], case["ff"], case["kv"]
    layer = [(d, d), (d,), (kv, d), (kv,), (kv, d), (kv,), (d, d), (ff, d), (ff, d), (d, ff), (d,), (d,)]
    return layer * case["layers"] + [(case["V"], d), (d,)]


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op = case["op"]
    if op == "embed":
        s["ids"] = _tokens(case["n"], case["V"], g)
        s["weight"] = torch.randn(case["V"], case["d"], generator=g, device="cuda").mul_(0.02).to(DTYPES[case["w"]])
    elif op == "embed_grad":
        n, V = case["n"], case["V"]
        ids = _tokens(n, V, g)
        s["eos"] = V - 1
        ids[torch.rand(n, generator=g, device="cuda") < case["pads"]] = V - 1
        s["ids"] = ids
        s["dout"] = torch.randn(n, case["d"], generator=g, device="cuda").mul_(1e-3).to(DTYPES[case["w"]])
    elif op == "clip":
        shapes = _shapes(case)
        s["grads"] = [torch.randn(sh, generator=g, device="cuda").mul_(1e-3).to(DTYPES[case["w"]]) for sh in shapes]
        sizes = [math.prod(sh) for sh in shapes]
        s["limit"] = (0.37 if case["over"] else 2.0) * 1e-3 * math.sqrt(sum(sizes))
        if case["out"]:
            # the optimizer's flat buffer, each tensor's part on a 16-byte boundary
            step = 16 // ESIZE[case["out"]]
            starts = np.concatenate([[0], np.cumsum([-(-k // step) * step for k in sizes])]).tolist()
            s["flat"] = torch.zeros(starts[-1], dtype=DTYPES[case["out"]], device="cuda")
            s["outs"] = [s["flat"][a:a + k].view(sh) for a, k, sh in zip(starts, sizes, shapes)]
    else:
        N, K, V, dt = case["N"], case["K"], case["V"], DTYPES[case["w"]]
        z = torch.randn(N, K + 1, V, generator=g, device="cuda").mul_(3.0)
        s["temperature"] = torch.rand(N, generator=g, device="cuda") * 0.6 + 0.6
        s["temperature"][torch.rand(N, generator=g, device="cuda") < case["greedy"]] = 0.0
        warm = torch.where(s["temperature"] > 0, s["temperature"], 1.0).view(N, 1, 1)
        if case["banned"]:
            z[(torch.rand(V, generator=g, device="cuda") < case["banned"]).expand_as(z)] = -math.inf
        s["draft_logits"], s["draft_lens"] = None, torch.full((N,), K, dtype=torch.int32, device="cuda")
        right = torch.rand(N, K, generator=g, device="cuda") < 0.7
        if case["draft"]:  # a draft model: the target's logits with an error, and tokens that it sampled
            # (the error scales with the temperature, so that tempering leaves the acceptance as stated)
            y = (z[:, :K] + torch.randn(N, K, V, generator=g, device="cuda") * (case["spread"] * warm)).to(dt)
            race = torch.empty(N, K, V, device="cuda").exponential_(generator=g).log_()
            x = (y.float() / warm - race).argmax(-1)
            # greedy rollouts: mostly right drafts
            x = torch.where((s["temperature"] == 0).view(N, 1) & right, z[:, :K].to(dt).float().argmax(-1), x)
            s["draft_logits"] = y if K else None
        else:  # copied drafts: lengths of their own, most of them what the target expects
            s["draft_lens"] = torch.randint(0, K + 1, (N,), generator=g, device="cuda", dtype=torch.int32)
            x = torch.randint(0, V, (N, K), generator=g, device="cuda")
            # about even odds against all the rest (the log of the sum of V exponentials of N(0, 3^2))
            level = torch.where(right, math.log(V) + 5.5, -3.0).unsqueeze(-1)
            z[:, :K].scatter_(-1, x.unsqueeze(-1), level)
        s["target"], s["draft_tokens"] = z.to(dt), x
        s["u"] = torch.rand(N, K, generator=g, device="cuda")
        s["noise"] = torch.empty(N, V, device="cuda").exponential_(generator=g).clamp_(min=1e-20)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "embed":
        return (s["weight"][s["ids"]].float() * s["scale"]).to(DTYPES[s["out"]])
    if op == "embed_grad":
        dw = torch.zeros(s["V"], s["d"], device="cuda")
        use = s["ids"] != s["eos"]
        # tokens of one id are many: their float32 sum is taken in 64 bits where they add up
        rows, where, count = torch.unique(s["ids"][use], return_inverse=True, return_counts=True)
        part = torch.zeros(rows.numel(), s["d"], device="cuda", dtype=torch.float64)
        part.index_add_(0, where, s["dout"][use].double())
        dw[rows] = (part * s["scale"]).float()
        return dw.to(DTYPES[s["out"]])
    if op == "clip":
        squares = torch.stack([t.float().square().sum(dtype=torch.float64) for t in s["grads"]])
        norm = squares.sum().sqrt()
        coef = (s["limit"] / (norm + 1e-6)).clamp(max=1.0)
        stats = torch.stack([norm, coef]).float()
        if not s["out"]:
            return [stats] + [t.copy_(t.float() * stats[1]) for t in s["grads"]]
        _ = [o.copy_(t.float() * stats[1]) for t, o in zip(s["grads"], s["outs"])]
        return [stats, s["flat"]]
    return _verify_plain(s)


def _softmax64(x):
    x = x - x.amax(-1, keepdim=True)
    x = x.exp()
    return x / x.sum(-1, keepdim=True)


def _first_max(x):
    at = torch.arange(x.shape[-1], device=x.device).expand_as(x)
    return torch.where(x == x.amax(-1, keepdim=True), at, x.shape[-1]).amin(-1)


def _verify_plain(s):
    z, x, N, K = s["target"], s["draft_tokens"], s["N"], s["K"]
    T = s["temperature"].double()
    greedy = T == 0
    T = torch.where(greedy, 1.0, T).view(N, 1, 1)
    p = _softmax64(z.double() / T)  # in 64 bits: the comparisons below are with values next to them
    q = _softmax64(s["draft_logits"].double() / T) if s["draft_logits"] is not None else None
    px = p[:, :K].gather(-1, x.unsqueeze(-1)).squeeze(-1)
    qx = q.gather(-1, x.unsqueeze(-1)).squeeze(-1) if q is not None else torch.ones_like(px)
    top = _first_max(z)
    ok = torch.where(greedy.view(N, 1), x == top[:, :K], s["u"].double() * qx < px)
    step = torch.arange(K, device=x.device)
    ok &= step < s["draft_lens"].view(N, 1)
    n = ok.long().cumprod(-1).sum(-1)
    i = torch.arange(N, device=x.device)
    row = p[i, n]
    rest = row
    if K:
        drafted = n < s["draft_lens"]
        j = n.clamp(max=K - 1)
        other = q[i, j] if q is not None else torch.zeros_like(row).scatter_(1, x[i, j].view(N, 1), 1.0)
        rest = torch.where(drafted.view(N, 1), (row - other).clamp(min=0), row)
        rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, row)
    token = torch.where(greedy, top[i, n], _first_max(rest / s["noise"].double()))
    slot = torch.arange(K + 1, device=x.device)
    every = torch.cat([x, x.new_zeros(N, 1)], 1)
    tokens = torch.where(slot == n.view(N, 1), token.view(N, 1), torch.where(slot < n.view(N, 1), every, -1))
    logp = p.gather(-1, tokens.clamp(min=0).unsqueeze(-1)).squeeze(-1).log()
    logp = torch.where(slot <= n.view(N, 1), logp, 0.0).float()
    return {"tokens": tokens, "n_accepted": n.int(), "logp": logp}


def _run_own(s):
    import vocab_wide_logprob_gb300 as grpo
    op = s["op"]
    if op == "embed":
        return grpo.grpo_embed_fwd(s["ids"], s["weight"], s["scale"], out_dtype=DTYPES[s["out"]])
    if op == "embed_grad":
        return grpo.grpo_embed_bwd(s["ids"], s["dout"], s["V"], s["scale"], pad_id=s["eos"],
                                   out_dtype=DTYPES[s["out"]])[0]
    if op == "clip":
        stats, _ = grpo.grpo_clip_grad_norm(s["grads"], s["limit"], out=s.get("outs"))
        return [stats, s["flat"]] if s["out"] else [stats] + s["grads"]
    out = grpo.grpo_verify_drafts(s["target"], s["draft_tokens"], s["u"], s["noise"], s["draft_logits"],
                                  s["draft_lens"], s["temperature"])
    return {k: out[k] for k in ("tokens", "n_accepted", "logp")}


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its results in 64 bits
# ---------------------------------------------------------------------------


def _distinct(n, V):
    """Expected number of different ids among n draws of the 1/rank law."""
    k = np.arange(1, V + 1, dtype=np.float64)
    p = np.log1p(1.0 / k) / math.log(V + 1)
    return float(-np.expm1(n * np.log1p(-p)).sum())


def work(case):
    op = case["op"]
    if op == "embed":
        n, d = case["n"], case["d"]
        return {"bytes": 8 * n + _distinct(n, case["V"]) * d * ESIZE[case["w"]] + n * d * ESIZE[case["out"]],
                "flops": n * d}
    if op == "embed_grad":
        n, d = case["n"], case["d"]
        used = n * (1 - case["pads"])  # the padding's gradients are not read
        return {"bytes": 8 * n + used * d * ESIZE[case["w"]] + case["V"] * d * ESIZE[case["out"]],
                "flops": used * d}
    if op == "clip":
        total = sum(math.prod(sh) for sh in _shapes(case))
        written = total * ESIZE[case["out"]] if case["out"] else 0  # in place and under the limit: nothing
        return {"bytes": total * ESIZE[case["w"]] + written, "flops": 3 * total}
    # rows up to the first rejection: a drafted token is accepted with the
    # overlap of the two distributions; a copied one in about half the cases
    N, K, row = case["N"], case["K"], case["V"] * ESIZE[case["w"]]
    accept = math.erfc(case["spread"] / (2 * math.sqrt(2))) if case["draft"] else 0.5
    accept = accept * (1 - case["greedy"]) + 0.7 * case["greedy"]
    lens = [K] if case["draft"] else list(range(K + 1))
    target = sum(sum(accept ** j for j in range(L + 1)) for L in lens) / len(lens)
    draft = sum(accept ** j for j in range(K)) if case["draft"] else 0.0
    return {"bytes": N * ((target + draft) * row + case["V"] * 4 * (1 - case["greedy"])),
            "flops": N * (target + draft) * case["V"] * 4}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        w = s["weight"].double()
        return (w.index_select(0, s["ids"]) * case["scale"])
    if op == "embed_grad":
        # rows summed by differences of a running sum over the tokens in id order would cancel:
        # an ordered sum per id on the host instead
        ids = s["ids"].cpu().numpy()
        keep = np.flatnonzero(ids != s["eos"])
        keep = keep[np.argsort(ids[keep], kind="stable")]
        dw = np.zeros((case["V"], case["d"]))
        if keep.size:
            dout = s["dout"].double().cpu().numpy()
            first = np.flatnonzero(np.r_[True, np.diff(ids[keep]) != 0])
            dw[ids[keep][first]] = np.add.reduceat(dout[keep], first, axis=0) * float(case["scale"])
        return torch.from_numpy(dw)
    if op == "clip":
        total = 0.0
        for t in s["grads"]:
            flat = t.reshape(-1).double()
            total += float(torch.dot(flat, flat))
        norm = math.sqrt(total)
        coef = min(1.0, s["limit"] / (norm + 1e-6))
        stats = torch.tensor([norm, coef], dtype=torch.float64)
        if not case["out"]:
            return [stats] + [t.double() * coef for t in s["grads"]]
        flat = torch.zeros(s["flat"].numel(), dtype=torch.float64, device="cuda")
        base = s["flat"].data_ptr()
        for t, o in zip(s["grads"], s["outs"]):
            a = (o.data_ptr() - base) // o.element_size()
            flat[a:a + t.numel()] = t.reshape(-1).double() * coef
        return [stats, flat]
    return _verify_exact(case, s)


def _verify_exact(case, s):
    """One sequence after the other, one drafted token after the other."""
    N, K, V = case["N"], case["K"], case["V"]
    tokens = np.full((N, K + 1), -1, dtype=np.int64)
    accepted = np.zeros(N, dtype=np.int32)
    logp = np.zeros((N, K + 1))
    x, u = s["draft_tokens"].cpu().numpy(), s["u"].double().cpu().numpy()
    lens, temp = s["draft_lens"].cpu().numpy(), s["temperature"].double().cpu().numpy()

    def log_probs(t, T):
        t = t.double().cpu().numpy() / T
        t = t - t.max()
        return t - math.log(math.fsum(np.exp(t)))

    for i in range(N):
        T = temp[i] if temp[i] > 0 else 1.0
        for j in range(int(lens[i]) + 1):
            lp = log_probs(s["target"][i, j], T)
            best = int(np.argmax(lp))
            bonus = j == lens[i]
            lq = None
            if not bonus and s["draft_logits"] is not None:
                lq = log_probs(s["draft_logits"][i, j], T)
            if not bonus:
                t = x[i, j]
                ok = t == best if temp[i] == 0 else (
                    u[i, j] < math.exp(lp[t] - (lq[t] if lq is not None else 0.0)))
                if ok:
                    tokens[i, j], logp[i, j] = t, lp[t]
                    continue
            accepted[i] = j
            if temp[i] == 0:
                pick = best
            else:
                rest = np.exp(lp)
                if lq is not None:
                    rest = np.maximum(rest - np.exp(lq), 0.0)
                elif not bonus:
                    rest = rest.copy()
                    rest[x[i, j]] = 0.0
                if not rest.any():
                    rest = np.exp(lp)
                pick = int(np.argmax(rest / s["noise"][i].double().cpu().numpy()))
            tokens[i, j], logp[i, j] = pick, lp[pick]
            break
    return {"tokens": torch.from_numpy(tokens), "n_accepted": torch.from_numpy(accepted),
            "logp": torch.from_numpy(logp)}
