"""The adapter, sampler, scoring and loss calls together, as a fine-tuning step
of adapters makes them: rows of several requests are projected each under its
adapter, a token is sampled for every row, the reference scores it without
adapters, and a loss's gradient comes back for the logits.  Every step is
checked against the float64 oracle on the step's own inputs."""
import numpy as np
import pytest

import workloads
from oracle import losses as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
LSE = 1.2e-5  # of a log-probability, derived in test_gpu_losses.py


def _setup(rows, hidden, vocab, rank, n, seed):
    import torch

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def bf(*shape, std):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(torch.bfloat16)

    x, w = bf(rows, hidden, std=1.0), bf(vocab, hidden, std=0.08)
    a, b = bf(n, rank, hidden, std=hidden ** -0.5), bf(n, vocab, rank, std=0.2)
    ids = torch.randint(-1, n, (rows,), generator=g, device=dev, dtype=torch.int32)
    scales = torch.rand(n, generator=g, device=dev) + 0.5
    return dev, g, x, w, a, b, ids, scales


def _params(rows, dev, temperature):
    import top_sampling_amd as ts

    p = np.zeros(rows, dtype=workloads.PARAMS_DTYPE)
    p["temperature"], p["top_p"] = temperature, 1.0
    p["seed"] = np.arange(rows) + 17
    return ts.params_to_device(p, dev)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("rows,hidden,vocab", [(24, 128, 4097), (200, 192, 33003)])
def test_policy_step(rows, hidden, vocab):
    import torch

    import top_sampling_amd as ts

    dev, g, x, w, a, b, ids, scales = _setup(rows, hidden, vocab, 16, 5, rows)
    temperature = 0.9
    # rollout
    logits = ts.lmhead_logits_local_lora(x, w, a, b, ids, scales)
    drawn = ts.sampler_sample(logits, _params(rows, dev, temperature), processed=True)
    assert (drawn.token_ids >= 0).all() and (drawn.row_status == 0).all()
    # the sampler's log-probabilities of what it drew are those of scoring it:
    # the sampler's own bound is 1e-4
    scored = ts.token_logprobs(logits, drawn.token_ids, temperature)
    assert (scored.logprobs - drawn.token_logprobs).abs().max() < 1e-4 + LSE
    # reference: the same rows without adapters
    base = ts.lmhead_logits_local(x, w)
    none = torch.full_like(ids, -1)
    assert torch.equal(base, ts.lmhead_logits_local_lora(x, w, a, b, none, scales))
    reference = ts.token_logprobs(base, drawn.token_ids, temperature).logprobs
    # the policy has moved since: every adapter a little
    b2 = (b.float() * 1.05).to(torch.bfloat16)
    now = ts.lmhead_logits_local_lora(x, w, a, b2, ids, scales)
    adv = torch.randn(rows, generator=g, device=dev)
    live = (torch.rand(rows, generator=g, device=dev) < 0.9).float()
    weights = live / live.sum()
    kw = dict(clip_low=0.2, clip_high=0.28, kl_coef=0.05, temperature=temperature)
    got = ts.policy_loss(now, drawn.token_ids, drawn.token_logprobs, adv, reference, weights,
                         backward=True, **kw)
    torch.cuda.synchronize()
    tokens = drawn.token_ids.cpu().numpy()
    want = ref.policy(f64(now), tokens, f64(drawn.token_logprobs), f64(adv), f64(reference),
                      f64(weights), **kw)
    lp = want["logprobs"]
    assert (np.abs(f64(got.logprobs) - lp) <= LSE + U * np.abs(lp)).all()
    # rows whose ratio is nearer to a border than its error may take either side
    near = np.minimum(np.abs(want["ratios"] - 0.8), np.abs(want["ratios"] - 1.28)) < 1e-4
    size = f64(weights) * (np.abs(f64(adv)) * want["ratios"] + 0.05 * 4)
    tol = size[:, None] * 3 * LSE / temperature + np.abs(want["grad"]) * 4e-5
    off = np.abs(f64(got.grad_logits) - want["grad"]) - tol
    assert (off[~near] <= 0).all()
    # the loss along a direction, by differences: its fp32 value is off by
    # 2 U |loss| + LSE sum(size), over a step of 2 h; the third derivative
    # adds h^2.
    d = torch.randn(rows, vocab, generator=g, device=dev)
    h = 1e-2
    up, down = (ts.policy_loss(now + s * h * d, drawn.token_ids, drawn.token_logprobs, adv,
                               reference, weights, **{**kw, "clip_low": np.inf,
                                                      "clip_high": np.inf}).loss.item()
                for s in (1, -1))
    free = ts.policy_loss(now, drawn.token_ids, drawn.token_logprobs, adv, reference, weights,
                          backward=True, **{**kw, "clip_low": np.inf, "clip_high": np.inf})
    slope = (free.grad_logits.double() * d.double()).sum().item()
    bound = (2 * U * abs(up) + LSE * size.sum()) / h + 10 * h * h * size.sum()
    assert abs((up - down) / (2 * h) - slope) <= bound


def test_preference_step_in_place():
    import torch

    import top_sampling_amd as ts

    rows, hidden, vocab, pairs = 60, 128, 5001, 3
    dev, g, x, w, a, b, ids, scales = _setup(rows, hidden, vocab, 24, 4, 3)
    logits = ts.lmhead_logits_local_lora(x, w, a, b, ids, scales)
    tokens = torch.randint(0, vocab, (rows,), generator=g, device=dev, dtype=torch.int32)
    tokens[::7] = -1  # prompt rows
    reference = ts.token_logprobs(ts.lmhead_logits_local(x, w), tokens).logprobs
    offsets = torch.tensor([0, 11, 19, 30, 30, 52, 60], dtype=torch.int32, device=dev)
    x64 = f64(logits)
    want = ref.preference(x64, tokens.cpu().numpy(), offsets.tolist(), f64(reference), beta=0.2,
                          mean=True)
    got = ts.preference_loss(logits, tokens, offsets, reference, beta=0.2, mean=True,
                             grad_logits=logits)
    torch.cuda.synchronize()
    assert got.grad_logits is logits
    assert abs(got.loss.item() - want["loss"]) < 0.2 * 2 * LSE + 2 * U * want["loss"]
    tol = np.abs(want["grad"]) * 6e-5 + 0.2 / 3 * 4 * LSE * (want["grad"] != 0) * \
        np.exp(ref.log_softmax(x64, 1.0)).clip(1e-9)
    tol[np.arange(rows), tokens.cpu().numpy().clip(0)] += 0.2 / 3 * 4 * LSE
    assert (np.abs(f64(logits) - want["grad"]) <= tol).all()
    assert not logits[::7].any()


def test_two_streams_at_once():
    """The same calls on two streams beside each other, and on the default
    stream by its number, give the results of one after the other."""
    import torch

    import top_sampling_amd as ts

    dev, g, x, w, a, b, ids, scales = _setup(100, 256, 9001, 24, 6, 8)
    other = torch.randn(100, 256, generator=g, device=dev).to(torch.bfloat16)
    tok = torch.randint(0, 9001, (100,), generator=g, device=dev, dtype=torch.int32)
    old = -torch.rand(100, generator=g, device=dev) - 8
    adv = torch.randn(100, generator=g, device=dev)
    off = torch.tensor([0, 30, 50, 80, 100], dtype=torch.int32, device=dev)

    def step(x, stream):
        logits = ts.lmhead_logits_local_lora(x, w, a, b, ids, scales, stream=stream)
        pol = ts.policy_loss(logits, tok, old, adv, backward=True, stream=stream)
        pref = ts.preference_loss(logits, tok, off, backward=True, stream=stream)
        score = ts.token_logprobs(logits, tok, entropies=True, stream=stream)
        return [logits, pol.loss, pol.grad_logits, pref.loss, pref.grad_logits, score.entropies]

    want = [step(x, None), step(other, None)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [step(x, streams[0]), step(other, streams[1])]
        torch.cuda.synchronize()
        for one, two in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(one, two))
    numbered = step(x, torch.cuda.default_stream().cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(numbered, want[0]))


@pytest.mark.parametrize("rows,hidden,vocab", [(24, 128, 4097), (200, 192, 33003)])
def test_step_gradient_entries(rows, hidden, vocab):
    """The gradients of both losses on projected logits, entry by entry: the
    error of a row's coefficient counts with the entry's own probability, so
    entries taken as 0 would not pass."""
    import torch

    import top_sampling_amd as ts

    dev, g, x, w, a, b, ids, scales = _setup(rows, hidden, vocab, 16, 5, rows)
    logits = ts.lmhead_logits_local_lora(x, w, a, b, ids, scales)
    tok = torch.randint(0, vocab, (rows,), generator=g, device=dev, dtype=torch.int32)
    tok[::9] = -1
    reference = ts.token_logprobs(ts.lmhead_logits_local(x, w), tok).logprobs
    old = reference + 0.05
    adv = torch.randn(rows, generator=g, device=dev)
    free = dict(clip_low=np.inf, clip_high=np.inf, kl_coef=0.05)
    x64, tokens = f64(logits), tok.cpu().numpy()
    p = np.exp(ref.log_softmax(x64, 1.0))
    p[np.arange(rows), tokens.clip(0)] = 1.0
    off = [0, rows // 4, rows // 2, rows // 2, rows]
    want = ref.policy(x64, tokens, f64(old), f64(adv), f64(reference), **free)
    got = ts.policy_loss(logits, tok, old, adv, reference, backward=True, **free)
    # exp(reference - lp) is at most the largest of these
    kl = np.exp(np.abs(f64(reference) - want["logprobs"]))
    coef = (np.abs(f64(adv)) * want["ratios"] + 0.05 * kl) * 2 * LSE
    pair = ref.preference(x64, tokens, off, f64(reference), mean=True)
    pref = ts.preference_loss(logits, tok, torch.tensor(off, dtype=torch.int32, device=dev),
                              reference, mean=True, backward=True)
    size = np.array([0.1 / 2 / max(1, (tokens[lo:hi] >= 0).sum())
                     for lo, hi in zip(off, off[1:])])
    torch.cuda.synchronize()
    for have, expect, c in ((got, want, coef), (pref, pair, np.repeat(size, np.diff(off)) * 3 * LSE)):
        # an entry's own exponential is off by 2 U |z - max z| + 6 U, |..| < 100
        tol = np.abs(expect["grad"]) * (2 * LSE + 206 * U) + c[:, None] * p + 2.0 ** -120
        assert (np.abs(f64(have.grad_logits) - expect["grad"]) <= tol).all()
        other = np.abs(expect["grad"]) > 2.0 ** -100
        other[np.arange(rows), tokens.clip(0)] = False
        assert (tol < np.abs(expect["grad"]))[other].mean() > 0.99


def test_current_stream_both_ways():
    """torch's short way to the current device and stream and the public one."""
    import torch

    import top_sampling_amd as ts

    side = torch.cuda.Stream()
    for stream in (torch.cuda.default_stream(), side):
        with torch.cuda.stream(stream):
            assert ts._current_device() == ts._public_current_device() == 0
            assert ts._current_stream(0) == ts._public_current_stream(0) == stream.cuda_stream
