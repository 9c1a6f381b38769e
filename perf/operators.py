"""Cases of the scoring, loss and adapter operators, with their plain forms.

Four operators that stand next to the sampling path:

  lora        logits of rows that each have their own low-rank adapter beside
              the shared lm_head (``lmhead_logits_local_lora``)
  score       log-probability and entropy of given tokens, and the gradient
              of a function of them (``token_logprobs``,
              ``token_logprobs_backward``)
  policy      clipped policy loss with a KL term, with the gradient of the
              logits (``policy_loss``)
  preference  paired log-ratio loss over ragged sequences, with the gradient
              of the logits (``preference_loss``)

``listed`` gives the cases, ``draw`` more of the same ranges, ``prepare`` a
case's inputs on the GPU, ``run`` one pass (elementary torch operations, or
with ``own`` the framework's calls), ``work`` the bytes and operations that a
pass cannot do without, and ``exact`` the same outputs in float64.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
SCALAR_BYTES = {"fp32": 4, "bf16": 2}


def listed():
    return [
        # Adapters: the smallest call (four requests of a small model), a
        # decode step of 64 requests over 32 adapters, a speculative-decoding
        # step (128 requests x 5 rows, 16 adapters), and a rank's vocabulary
        # slice with a ragged row count and a wide rank.
        {"name": "lora tiny", "op": "lora", "rows": 4, "hidden": 256, "vocab": 4096, "rank": 8,
         "adapters": 3, "per": 1, "pad": 0},
        {"name": "lora decode", "op": "lora", "rows": 64, "hidden": 4096, "vocab": 151936,
         "rank": 16, "adapters": 32, "per": 1, "pad": 0},
        {"name": "lora spec_decode", "op": "lora", "rows": 640, "hidden": 4096, "vocab": 151936,
         "rank": 32, "adapters": 16, "per": 5, "pad": 0},
        {"name": "lora slice ragged", "op": "lora", "rows": 133, "hidden": 2560, "vocab": 31040,
         "rank": 64, "adapters": 9, "per": 7, "pad": 1},
        # Scoring: log-probabilities of four tokens (latency), of a
        # speculative step with entropies, and the gradient of a custom
        # function of both over bf16 logits at a temperature.
        {"name": "score tiny", "op": "score", "rows": 4, "vocab": 4096, "pad": 0, "dtype": "fp32",
         "temperature": 1.0, "backward": False, "masked": False},
        {"name": "score spec_decode", "op": "score", "rows": 640, "vocab": 151936, "pad": 0,
         "dtype": "fp32", "temperature": 1.0, "backward": False, "masked": True},
        {"name": "score backward bf16", "op": "score", "rows": 256, "vocab": 248320, "pad": 0,
         "dtype": "bf16", "temperature": 0.7, "backward": True, "masked": False},
        # Policy loss: evaluation of a short answer, a training step on the
        # projection's fp32 logits, and one on bf16 logits of odd sizes.
        {"name": "policy short", "op": "policy", "rows": 16, "vocab": 151936, "pad": 0,
         "dtype": "fp32", "temperature": 1.0, "backward": False, "masked": False},
        {"name": "policy train", "op": "policy", "rows": 640, "vocab": 151936, "pad": 0,
         "dtype": "fp32", "temperature": 1.0, "backward": True, "masked": False},
        {"name": "policy train odd bf16", "op": "policy", "rows": 1021, "vocab": 100277, "pad": 0,
         "dtype": "bf16", "temperature": 0.9, "backward": True, "masked": True},
        # Preference loss: two short pairs of a small vocabulary, and a batch
        # of eight pairs of ragged answers.
        {"name": "preference tiny", "op": "preference", "rows": 37, "pairs": 2, "vocab": 4096,
         "pad": 0, "dtype": "fp32", "mean": False, "backward": True, "masked": False},
        {"name": "preference batch bf16", "op": "preference", "rows": 1024, "pairs": 8,
         "vocab": 151936, "pad": 0, "dtype": "bf16", "mean": True, "backward": True,
         "masked": False},
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["lora", "score", "policy", "preference"])
    vocab = _log_uniform(rng, 2000, 250000)
    pad = rng.choice([0, 0, 8, 37])
    if op == "lora":
        hidden = 64 * _log_uniform(rng, 4, 96)
        most = 640 * 151936 * 4096 // (hidden * vocab)
        return {"op": op, "rows": _log_uniform(rng, 1, max(1, min(700, most))), "hidden": hidden,
                "vocab": vocab, "rank": rng.choice([8, 16, 32, 64]),
                "adapters": _log_uniform(rng, 1, 40), "per": rng.choice([1, 1, 5]), "pad": pad}
    dtype = rng.choice(["fp32", "bf16"])
    most = 640 * 151936 // (vocab + pad)
    case = {"op": op, "rows": _log_uniform(rng, 1 if op != "preference" else 8,
                                           max(8, min(4000, most))),
            "vocab": vocab, "pad": pad, "dtype": dtype, "masked": rng.random() < 0.5,
            "backward": rng.random() < 0.7}
    if op == "preference":
        case["pairs"] = _log_uniform(rng, 1, max(1, case["rows"] // 8))
        case["mean"] = rng.random() < 0.5
    else:
        case["temperature"] = rng.choice([1.0, round(rng.uniform(0.3, 1.5), 3)])
    return case


def work(case):
    rows, vocab = case["rows"], case["vocab"]
    if case["op"] == "lora":
        hidden, rank = case["hidden"], case["rank"]
        used = min(case["adapters"], -(-rows // case["per"]))
        return {"bytes": 2 * (vocab + rows) * hidden + 4 * rows * vocab
                + 2 * used * rank * (hidden + vocab),
                "flops": 2 * rows * hidden * vocab + 2 * rows * rank * (hidden + vocab)}
    one = rows * vocab * SCALAR_BYTES[case["dtype"]]
    return {"bytes": one * (2 if case["backward"] else 1) + 24 * rows,
            "flops": (9 if case["backward"] else 5) * rows * vocab}


# ------------------------------------------------------------------ inputs
def _lora_inputs(case, gen):
    rows, hidden, vocab, rank, n = (case[k] for k in ("rows", "hidden", "vocab", "rank",
                                                      "adapters"))

    def normal(*shape, std=1.0):
        out = torch.empty(*shape, dtype=torch.bfloat16, device="cuda")
        return out.normal_(0.0, std, generator=gen)

    # Every request has an adapter of its own choice; some have none (-1).
    requests = -(-rows // case["per"])
    ids = torch.randint(-1, n, (requests,), generator=gen, device="cuda", dtype=torch.int32)
    return {
        "hidden": normal(rows, hidden),
        "lm_head": normal(vocab, hidden, std=0.02),
        "lora_a": normal(n, rank, hidden, std=1.0 / math.sqrt(hidden)),
        "lora_b": normal(n, vocab, rank, std=0.05),
        "scales": torch.rand(n, generator=gen, device="cuda") * 2 + 0.5,
        "ids": ids.repeat_interleave(case["per"])[:rows].contiguous(),
        "out": torch.empty(rows, vocab + case["pad"], device="cuda")[:, :vocab],
    }


def _logits(case, gen):
    """Logits as a projection gives them, each row with one likely token;
    with `masked`, every second row allows about half of its tokens."""
    rows, vocab = case["rows"], case["vocab"]
    wide = torch.empty(rows, vocab + case["pad"], dtype=DTYPES[case["dtype"]], device="cuda")
    logits = wide[:, :vocab]
    x = torch.randn(rows, vocab, generator=gen, device="cuda") * 1.28
    likely = torch.randint(0, vocab, (rows, 1), generator=gen, device="cuda")
    x.scatter_add_(1, likely, torch.rand(rows, 1, generator=gen, device="cuda") * 18)
    if case["masked"]:
        shut = torch.rand((rows + 1) // 2, vocab, generator=gen, device="cuda") < 0.5
        x[::2].masked_fill_(shut, -math.inf)
    logits.copy_(x)
    # The tokens are drawn from these logits, as a rollout's are.
    noise = torch.rand(rows, vocab, generator=gen, device="cuda").clamp_min_(1e-30)
    noise.log_().neg_().log_().neg_()
    tokens = (logits.float() / case.get("temperature", 1.0) + noise).argmax(-1)
    return logits, tokens.to(torch.int32)


def _near_logprobs(case, logits, tokens, gen, spread):
    """Log-probabilities of the same tokens under a policy near this one."""
    z = logits.float() / case.get("temperature", 1.0)
    lp = z.gather(1, tokens.long()[:, None])[:, 0] - torch.logsumexp(z, -1)
    return lp + torch.randn(lp.shape, generator=gen, device="cuda") * spread


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    state = {"case": dict(case)}
    if case["op"] == "lora":
        state.update(_lora_inputs(case, gen))
        return state
    rows = case["rows"]
    logits, tokens = _logits(case, gen)
    state["logits"] = logits
    state["reference"] = _near_logprobs(case, logits, tokens, gen, 0.1)
    if case["op"] == "score":
        state["grad_logprobs"] = torch.randn(rows, generator=gen, device="cuda") / rows
        state["grad_entropies"] = torch.randn(rows, generator=gen, device="cuda") * 0.1 / rows
    if case["op"] == "policy":
        state["old"] = _near_logprobs(case, logits, tokens, gen, 0.2)
        state["advantages"] = torch.randn(rows, generator=gen, device="cuda")
        # Padding rows of a rectangular batch have weight 0.
        live = (torch.rand(rows, generator=gen, device="cuda") < 0.95).float()
        live[0] = 1.0
        state["weights"] = live / live.sum()
    if case["op"] == "preference":
        cuts = torch.randint(0, rows + 1, (2 * case["pairs"] - 1,), generator=gen, device="cuda")
        state["offsets"] = torch.cat([torch.zeros(1, dtype=cuts.dtype, device="cuda"),
                                      cuts.sort().values,
                                      torch.full((1,), rows, dtype=cuts.dtype, device="cuda")]
                                     ).to(torch.int32)
    # Prompt tokens inside the rows are left out (token -1).
    prompt = torch.rand(rows, generator=gen, device="cuda") < 0.05
    prompt[0] = False
    state["tokens"] = torch.where(prompt, -1, tokens).to(torch.int32)
    return state


CLIP_LOW, CLIP_HIGH, KL_COEF = 0.2, 0.28, 0.04
BETA, SMOOTHING, MARGIN = 0.1, 0.05, 0.0


# ------------------------------------------------------------- plain forms
def _plain_lora(s):
    c = s["case"]
    x, n, rank = s["hidden"].float(), c["adapters"], c["rank"]
    out = x @ s["lm_head"].float().t()
    at = s["ids"].long()
    has = at >= 0
    down = torch.where(has[:, None], (x @ s["lora_a"].float().reshape(n * rank, -1).t())
                       .reshape(-1, n, rank)[torch.arange(len(at), device=at.device),
                                             at.clamp_min(0)] * s["scales"][at.clamp_min(0)][:, None],
                       0.0)
    spread = torch.zeros(len(at), n, rank, device=at.device)
    spread[torch.arange(len(at), device=at.device), at.clamp_min(0)] = down
    up = s["lora_b"].float().permute(0, 2, 1).reshape(n * rank, -1)
    return {"logits": out + spread.reshape(len(at), -1) @ up}


def _plain_rows(s, left_in):
    """Softmax pieces of the rows; rows that are left out get zeros."""
    c = s["case"]
    t = c.get("temperature", 1.0)
    x = s["logits"].float()
    m = x.amax(-1, keepdim=True)
    e = torch.exp((x - m) / t)
    total = e.sum(-1, keepdim=True)
    at = s["tokens"].long().clamp_min(0)[:, None]
    far = (x.gather(1, at) - m)[:, 0].double() / t
    lp = torch.where(left_in, far - total[:, 0].double().log(), 0.0)
    return t, x, m, e, total, at, lp


def _plain_gradient(s, left_in, rows, g):
    """d/d logits of sum_r g[r] * lp[r], in the logits' type."""
    t, _, _, e, total, at, lp = rows
    g = torch.where(left_in, g, 0.0)
    d = e / total * (-g / t).float()[:, None]
    d.scatter_(1, at, (g * -torch.expm1(lp) / t).float()[:, None])
    return d.to(s["logits"].dtype)


def _plain_score(s):
    left_in = s["tokens"] >= 0
    t, x, m, e, total, at, lp = _plain_rows(s, left_in)
    z = torch.where(e > 0, (x - m) / t, 0.0)
    h = total[:, 0].double().log() - ((e * z).sum(-1, keepdim=True) / total)[:, 0].double()
    h = torch.where(left_in, h, 0.0)
    out = {"logprobs": lp.float(), "entropies": h.float()}
    if s["case"]["backward"]:
        p = e / total
        g = torch.where(left_in, s["grad_logprobs"], 0.0)[:, None]
        k = torch.where(left_in, s["grad_entropies"], 0.0)[:, None]
        d = -p * (g + k * (z - total.log() + h.float()[:, None])) / t
        d.scatter_add_(1, at, g / t)
        out["grad_logits"] = d.to(s["logits"].dtype)
    return out


def _plain_policy(s):
    left_in = (s["tokens"] >= 0) & (s["weights"] != 0)
    rows = _plain_rows(s, left_in)
    lp, w = rows[-1], torch.where(left_in, s["weights"], 0.0).double()
    a = s["advantages"].double()
    ratio = torch.where(left_in, torch.exp(lp - s["old"].double()), 1.0)
    cut = ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH)
    gap = torch.where(left_in, s["reference"].double() - lp, 0.0)
    kl = torch.expm1(gap) - gap
    loss = (w * (KL_COEF * kl - torch.minimum(ratio * a, cut * a))).sum()
    out = {"loss": loss.float(), "logprobs": lp.float(), "ratios": ratio.float(),
           "kl": kl.float()}
    if s["case"]["backward"]:
        g = w * (-torch.expm1(gap) * KL_COEF - torch.where(ratio * a <= cut * a, a * ratio, 0.0))
        out["grad_logits"] = _plain_gradient(s, left_in, rows, g)
    return out


def _plain_preference(s):
    c, offsets = s["case"], s["offsets"].long()
    pairs = c["pairs"]
    left_in = s["tokens"] >= 0
    rows = _plain_rows(s, left_in)
    lp = rows[-1]
    at = torch.arange(c["rows"], device=offsets.device)
    seq = torch.searchsorted(offsets[1:], at, right=True)
    gap = torch.where(left_in, lp - s["reference"].double(), 0.0)
    zero = torch.zeros(1, dtype=torch.float64, device=offsets.device)
    run_gap = torch.cat([zero, gap.cumsum(0)])
    run_n = torch.cat([zero, left_in.double().cumsum(0)])
    total = run_gap[offsets[1:]] - run_gap[offsets[:-1]]
    n = (run_n[offsets[1:]] - run_n[offsets[:-1]]).clamp_min(1.0) if c["mean"] \
        else torch.ones_like(total)
    rho = total / n
    z = BETA * (rho[:pairs] - rho[pairs:]) - MARGIN
    soft = torch.log1p(torch.exp(-z.abs()))
    each = (1 - SMOOTHING) * (soft + (-z).clamp_min(0)) + SMOOTHING * (soft + z.clamp_min(0))
    out = {"loss": each.mean().float(), "pair_losses": each.float(),
           "rewards": (BETA * rho).float(), "logprobs": lp.float()}
    if c["backward"]:
        up = 1 / (1 + torch.exp(-z))
        dz = (SMOOTHING * up - (1 - SMOOTHING) * (1 - up)) * BETA / pairs
        g = (torch.cat([dz, -dz]) / n)[seq]
        out["grad_logits"] = _plain_gradient(s, left_in, rows, g)
    return out


PLAIN = {"lora": _plain_lora, "score": _plain_score, "policy": _plain_policy,
         "preference": _plain_preference}


# ------------------------------------------------------- the framework's calls
def _own(s):
    import top_sampling_amd as ts

    c = s["case"]
    if c["op"] == "lora":
        return {"logits": ts.lmhead_logits_local_lora(
            s["hidden"], s["lm_head"], s["lora_a"], s["lora_b"], s["ids"], s["scales"],
            out=s["out"])}
    if c["op"] == "score":
        o = ts.token_logprobs(s["logits"], s["tokens"], temperature=c["temperature"],
                              entropies=True)
        out = {"logprobs": o.logprobs, "entropies": o.entropies}
        if c["backward"]:
            out["grad_logits"] = ts.token_logprobs_backward(
                s["logits"], s["tokens"], o, s["grad_logprobs"],
                grad_entropies=s["grad_entropies"], temperature=c["temperature"])
        return out
    if c["op"] == "policy":
        o = ts.policy_loss(s["logits"], s["tokens"], s["old"], s["advantages"],
                           ref_logprobs=s["reference"], weights=s["weights"], clip_low=CLIP_LOW,
                           clip_high=CLIP_HIGH, kl_coef=KL_COEF, temperature=c["temperature"],
                           backward=c["backward"])
        out = {"loss": o.loss, "logprobs": o.logprobs, "ratios": o.ratios, "kl": o.kl}
    else:
        o = ts.preference_loss(s["logits"], s["tokens"], s["offsets"],
                               ref_logprobs=s["reference"], beta=BETA,
                               label_smoothing=SMOOTHING, margin=MARGIN, mean=c["mean"],
                               backward=c["backward"])
        out = {"loss": o.loss, "pair_losses": o.pair_losses, "rewards": o.rewards,
               "logprobs": o.logprobs}
    if c["backward"]:
        out["grad_logits"] = o.grad_logits
    return out


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- in float64
def _exact_rows(case, s):
    """Log-probabilities of every token, by the definition of log-softmax."""
    z = s["logits"].double() / case.get("temperature", 1.0)
    return z - torch.logsumexp(z, -1, keepdim=True)


def _exact_gradient(case, s, logp, left_in, g):
    one = torch.zeros_like(logp)
    one.scatter_(1, s["tokens"].long().clamp_min(0)[:, None], 1.0)
    d = (one - logp.exp()) * (torch.where(left_in, g, 0.0) / case.get("temperature", 1.0))[:, None]
    return d


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lora":
        x = s["hidden"].double()
        out = torch.matmul(x, s["lm_head"].double().t())
        for i in range(case["adapters"]):
            mine = (s["ids"] == i).nonzero()[:, 0]
            if len(mine):
                low = torch.matmul(x[mine], s["lora_a"][i].double().t())
                out[mine] += s["scales"][i].double() * torch.matmul(low,
                                                                    s["lora_b"][i].double().t())
        return {"logits": out}
    logp = _exact_rows(case, s)
    tokens = s["tokens"].long()
    left_in = tokens >= 0
    if case["op"] == "policy":
        left_in = left_in & (s["weights"] != 0)
    lp = torch.where(left_in, logp.gather(1, tokens.clamp_min(0)[:, None])[:, 0], 0.0)
    if case["op"] == "score":
        p = logp.exp()
        h = -(p * torch.where(p > 0, logp, 0.0)).sum(-1)
        out = {"logprobs": lp, "entropies": torch.where(left_in, h, 0.0)}
        if case["backward"]:
            g = s["grad_logprobs"].double()
            k = torch.where(left_in, s["grad_entropies"].double(), 0.0)
            d = _exact_gradient(case, s, logp, left_in, g)
            d -= p * torch.where(p > 0, logp + h[:, None], 0.0) * (k / case["temperature"])[:, None]
            out["grad_logits"] = d
        return out
    ref = s["reference"].double()
    if case["op"] == "policy":
        w, a = s["weights"].double(), s["advantages"].double()
        ratio = torch.where(left_in, (lp - s["old"].double()).exp(), 1.0)
        low, high = 1 - CLIP_LOW, 1 + CLIP_HIGH
        inside = torch.where(a >= 0, ratio <= high, ratio >= low)
        gain = torch.where(inside, ratio, torch.where(a >= 0, high, low)) * a
        log_gap = torch.where(left_in, ref - lp, 0.0)
        kl = log_gap.exp() - 1 - log_gap
        loss = torch.where(left_in, w * (KL_COEF * kl - gain), 0.0).sum()
        out = {"loss": loss, "logprobs": lp, "ratios": ratio, "kl": kl}
        g = w * (KL_COEF * (1 - log_gap.exp()) - torch.where(inside, ratio * a, 0.0))
    else:
        pairs = case["pairs"]
        cuts = s["offsets"].tolist()
        rho, counts = [], []
        for i in range(2 * pairs):
            part = slice(cuts[i], cuts[i + 1])
            live = left_in[part]
            counts.append(max(1, int(live.sum())) if case["mean"] else 1)
            rho.append((lp[part] - ref[part])[live].sum() / counts[-1])
        rho = torch.stack(rho)
        z = BETA * (rho[:pairs] - rho[pairs:]) - MARGIN
        each = -(1 - SMOOTHING) * torch.nn.functional.logsigmoid(z) \
            - SMOOTHING * torch.nn.functional.logsigmoid(-z)
        out = {"loss": each.mean(), "pair_losses": each, "rewards": BETA * rho, "logprobs": lp}
        dz = BETA / pairs * (SMOOTHING - (1 - torch.sigmoid(z)))
        g = torch.zeros_like(lp)
        for i in range(2 * pairs):
            side = 1.0 if i < pairs else -1.0
            g[cuts[i]:cuts[i + 1]] = side * dz[i % pairs] / counts[i]
    if case["backward"]:
        out["grad_logits"] = _exact_gradient(case, s, logp, left_in, g)
    return out
