"""Token scoring, the policy and preference losses and their gradients on the
GPU against the float64 oracle (oracle/losses.py).

Tolerances.  u = 2^-24 is fp32's rounding.  A row's sum is added up per thread
in fp32, at most 128 terms one after the other (relative error at most 128 u;
the kernel adds 32 as a tree), each term exp2 of an argument with two roundings (relative error at most
2 u |z - max z| plus 2 u of exp2 itself), and in double from there on.  So ln S
is off by at most
    LSE = 130 u + 2 u * (the p-weighted mean of |z - max z|, below 30 here)
        < 1.2e-5,
a log-probability by LSE plus its own rounding, and the other outputs follow
by their derivatives.  A gradient entry e_j a has the relative errors of e_j
(2 u |z_j - max z| + 4 u), of S (LSE) and of a (LSE where it holds a ratio),
and is rounded once to its type.
"""
import numpy as np
import pytest

from oracle import losses as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
LSE = 1.2e-5
HALF = {"fp32": U, "bf16": 2.0 ** -8}


def _dev():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda:0")


def say(*a):
    print(*a, flush=True)


def make_logits(rows, vocab, dtype, pad, seed, masks=True):
    """(device logits [rows, vocab] in a buffer pad columns wider, the same
    values in float64).  With masks: rows with -inf entries, with a single
    finite entry, with entries of the type's lowest value, and with one token
    far above the rest."""
    import torch

    g = np.random.default_rng(seed)
    x = g.normal(0, 1.5, (rows, vocab)).astype(np.float32)
    if masks:
        for r in range(rows):
            kind = r % 6
            if kind == 1 and vocab > 1:
                x[r, g.random(vocab) < 0.6] = -np.inf
                x[r, g.integers(vocab)] = 0.5
            elif kind == 2:
                x[r] = -np.inf
                x[r, g.integers(vocab)] = -3.0
            elif kind == 3:
                x[r, g.random(vocab) < 0.5] = -3.3e38
                x[r, g.integers(vocab)] = 2.0
            elif kind == 4:
                x[r, g.integers(vocab)] += 25.0
            elif kind == 5:
                x[r] += 300.0
    wide = torch.full((rows, vocab + pad), 7.0, device=_dev(),
                      dtype=torch.float32 if dtype == "fp32" else torch.bfloat16)
    t = wide[:, :vocab]
    t.copy_(torch.from_numpy(x))
    return t, t.cpu().double().numpy()


def allowed_tokens(x, seed, skip=0.15):
    """A finite token of each row; some rows left out."""
    g = np.random.default_rng(seed)
    tok = np.array([g.choice(np.flatnonzero(np.isfinite(r) & (r > -1e38))) for r in x])
    out = g.random(len(x)) < skip
    out[0] = False
    tok[out] = -1 - g.integers(0, 100, out.sum())
    return tok.astype(np.int32)


def to_dev(a, dtype=None):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).to(_dev(), dtype or torch.float32)


def close(got, want, tol, what):
    got = got.detach().double().cpu().numpy()
    want = np.asarray(want, dtype=np.float64)
    tol = np.broadcast_to(tol, want.shape)
    assert got.shape == want.shape, what
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        off = np.where(same, 0.0, np.abs(got - want) - tol)
    off = np.where(np.isnan(off), np.inf, off)
    i = np.unravel_index(off.argmax(), off.shape) if off.size else None
    assert not off.size or off[i] <= 0, (what, i, got[i], want[i], tol[i])


def grad_tol(want, x, temperature, dtype, slack):
    """Entry by entry: rounding to the type, the entry's own exp2, the row's
    sum and coefficient.  An e_j below 2^-126 may be taken as 0; |a| < 64."""
    with np.errstate(invalid="ignore", over="ignore"):
        top = x.max(-1, keepdims=True)
        far = np.minimum(np.where(np.isfinite(x), (top - x) / temperature, 0.0), 140.0)
    rel = HALF[dtype] + 2 * U * far + 6 * U + slack
    return np.abs(np.where(np.isfinite(want), want, 0.0)) * rel + 2.0 ** -120


SHAPES = [
    # rows, vocab, pad: one and two tokens, odd sizes, below and above a
    # vector, a slab (1,024 vectors) and a chunk, unaligned row starts
    (1, 1, 0), (1, 2, 0), (5, 3, 1), (7, 9, 0), (6, 255, 0), (13, 1000, 24), (12, 4096, 0),
    (6, 4097, 0), (37, 8192, 3), (8, 30011, 0), (3, 151936, 0), (70, 16390, 5), (1100, 257, 0), (200, 40001, 0),
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,vocab,pad", SHAPES)
def test_token_logprobs(rows, vocab, pad, dtype):
    import torch

    import top_sampling_amd as ts

    for temperature in (1.0, 0.37):
        say("token_logprobs", rows, vocab, pad, dtype, temperature)
        logits, x = make_logits(rows, vocab, dtype, pad, rows + vocab)
        tok = allowed_tokens(x, 5)
        lp, ent = ref.score(x, tok, temperature)
        tk = to_dev(tok, torch.int32)
        out = ts.token_logprobs(logits, tk, temperature, entropies=True)
        plain = ts.token_logprobs(logits, tk, temperature)
        torch.cuda.synchronize()
        close(out.logprobs, lp, LSE + U * np.abs(lp), "logprobs")
        # H = ln S - E[z - max]: the mean's error is LSE of its size
        close(out.entropies, ent, LSE * (2 + 30), "entropies")
        assert plain.entropies is None
        close(plain.logprobs, lp, LSE + U * np.abs(lp), "logprobs without entropies")
        assert not out.row_status.any() and not plain.row_status.any()
        # gradients of both
        g = np.random.default_rng(3)
        a, b = g.normal(size=rows).astype(np.float32), g.normal(size=rows).astype(np.float32)
        b[rows // 2:] = 0.0
        if rows > 3:
            a[rows - 2:] = 0.0
        for gh, fwd in ((b, out), (None, plain)):
            want = ref.score_gradient(x, tok, temperature, a.astype(np.float64),
                                      None if gh is None else gh.astype(np.float64))
            wide = torch.full((rows, vocab + 2), 7.0, dtype=logits.dtype, device=logits.device)
            got = ts.token_logprobs_backward(logits, tk, fwd, to_dev(a),
                                             None if gh is None else to_dev(gh), temperature,
                                             grad_logits=wide[:, :vocab])
            torch.cuda.synchronize()
            assert (wide[:, vocab:] == 7.0).all()
            tol = grad_tol(want, x, temperature, dtype, 2 * LSE)
            # a term and an entropy term of opposite sign cancel: LSE of the
            # larger, h p (|ln p| + H) with p (|ln p| + H) <= p (140 + 12)
            p = np.exp(ref.log_softmax(x, temperature))
            size = np.abs(a)[:, None] * p
            if gh is not None:
                with np.errstate(invalid="ignore"):
                    far = np.where(p > 0, np.abs(ref.log_softmax(x, temperature)), 0.0)
                size = size + np.abs(gh)[:, None] * p * (far + np.abs(ent)[:, None] + 32)
            size[np.arange(rows), np.maximum(tok, 0)] += np.abs(a) * LSE
            close(got, want, tol + size * (2 * LSE) / temperature, ("gradient", gh is None))
            out_rows = tok < 0
            assert not got[to_dev(out_rows, torch.bool)].any()


def test_backward_in_place_and_repeatable():
    import torch

    import top_sampling_amd as ts

    for dtype in ("fp32", "bf16"):
        logits, x = make_logits(9, 30011, dtype, 0, 1)
        tk = to_dev(allowed_tokens(x, 2), torch.int32)
        g = torch.randn(9, device=_dev())
        fwd = ts.token_logprobs(logits, tk, 0.8, entropies=True)
        one = ts.token_logprobs_backward(logits, tk, fwd, g, g, 0.8)
        two = ts.token_logprobs_backward(logits, tk, fwd, g, g, 0.8)
        same = logits.clone()
        three = ts.token_logprobs_backward(same, tk, fwd, g, g, 0.8, grad_logits=same)
        assert three.data_ptr() == same.data_ptr()
        assert torch.equal(one, two) and torch.equal(one, three)
        adv = torch.randn(9, device=_dev())
        kw = dict(weights=torch.rand(9, device=_dev()), temperature=0.8)
        a = ts.policy_loss(logits, tk, fwd.logprobs, adv, backward=True, **kw)
        same = logits.clone()
        b = ts.policy_loss(same, tk, fwd.logprobs, adv, grad_logits=same, **kw)
        assert torch.equal(a.grad_logits, same) and torch.equal(a.loss, b.loss)


def policy_inputs(rows, x, tok, temperature, seed):
    g = np.random.default_rng(seed)
    lp, _ = ref.score(x, tok, temperature)
    lp = np.where(np.isfinite(lp), lp, -1.0)
    # Ratios away from the clip borders by far more than their error, so both
    # sides take the same branch: spread them over fixed points.
    steps = np.array([-0.6, -0.1, 0.0, 0.15, 0.55])
    old = (lp - steps[g.integers(0, 5, rows)]).astype(np.float32)
    rf = (lp + g.normal(0, 0.4, rows)).astype(np.float32)
    adv = g.normal(size=rows).astype(np.float32)
    w = g.uniform(0.1, 1.0, rows).astype(np.float32) / rows
    if rows > 4:
        adv[3] = 0.0
        w[4] = 0.0
    return old, rf, adv, w


def check_policy(got, want, x, temperature, dtype, rows, w, adv, kl_coef, scale=1.0):
    r = want["ratios"]
    close(got.logprobs, want["logprobs"], LSE + U * np.abs(want["logprobs"]), "logprobs")
    close(got.ratios, r, r * (LSE + 2 * U), "ratios")
    # dkl/dlp = 1 - exp(gap), at most e^2 here
    k = want["kl"]
    close(got.kl, k, 8 * LSE + U * np.abs(k), "kl")
    each = w * (np.abs(adv) * r + kl_coef * 8)
    close(got.loss, want["loss"], (each * LSE).sum() + 2 * U * abs(want["loss"]), "loss")
    if got.grad_logits is not None:
        # the coefficient's absolute error, beside the entry's relative one
        coef = scale * w * (np.abs(adv) * r + kl_coef * 8) * 2 * LSE / temperature
        p = np.exp(ref.log_softmax(x, temperature))
        tol = grad_tol(want["grad"], x, temperature, dtype, 2 * LSE) + coef[:, None] * \
            np.maximum(p, (want["grad"] != 0))
        close(got.grad_logits, want["grad"], tol, "gradient")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,vocab,pad", SHAPES)
def test_policy_loss(rows, vocab, pad, dtype):
    import torch

    import top_sampling_amd as ts

    for temperature, kl_coef, scale in ((1.0, 0.0, 1.0), (0.7, 0.2, 3.0)):
        say("policy_loss", rows, vocab, pad, dtype, temperature, kl_coef)
        logits, x = make_logits(rows, vocab, dtype, pad, rows * 3 + vocab)
        tok = allowed_tokens(x, 6)
        old, rf, adv, w = policy_inputs(rows, x, tok, temperature, 8)
        kw = dict(clip_low=0.2, clip_high=0.28, kl_coef=kl_coef, temperature=temperature)
        f = lambda a: a.astype(np.float64)  # noqa: E731
        with_ref = kl_coef > 0
        want = ref.policy(x, tok, f(old), f(adv), f(rf) if with_ref else None, f(w),
                          grad_loss=scale, **kw)
        args = (to_dev(tok, torch.int32), to_dev(old), to_dev(adv))
        kws = dict(ref_logprobs=to_dev(rf) if with_ref else None, weights=to_dev(w), **kw)
        gl = torch.full((1,), scale, device=_dev()) if scale != 1.0 else None
        got = ts.policy_loss(logits, *args, backward=True, grad_loss=gl, **kws)
        fwd = ts.policy_loss(logits, *args, **kws)
        torch.cuda.synchronize()
        assert fwd.grad_logits is None and not got.row_status.any()
        for o in (got, fwd):
            check_policy(o, want, x, temperature, dtype, rows, f(w), f(adv), kl_coef, scale)


@pytest.mark.parametrize("dtype,rows,vocab,pad", [
    # rows held on the chip as a whole, with a part that is read again, of
    # more than that twice over, and unaligned
    ("fp32", 96, 33000, 0), ("fp32", 96, 114688, 0), ("fp32", 97, 120001, 0),
    ("bf16", 128, 131077, 3), ("bf16", 130, 262144, 0), ("fp32", 3, 32768, 0),
    # two passes
    ("fp32", 95, 33001, 0), ("bf16", 127, 40000, 1), ("fp32", 2, 300000, 0),
])
def test_policy_loss_long_rows(dtype, rows, vocab, pad):
    import torch

    import top_sampling_amd as ts

    logits, x = make_logits(rows, vocab, dtype, pad, rows + vocab)
    tok = allowed_tokens(x, 6)
    old, rf, adv, w = policy_inputs(rows, x, tok, 0.8, 8)
    kw = dict(clip_low=0.2, clip_high=0.28, kl_coef=0.1, temperature=0.8)
    f = lambda a: a.astype(np.float64)  # noqa: E731
    want = ref.policy(x, tok, f(old), f(adv), f(rf), f(w), **kw)
    args = (to_dev(tok, torch.int32), to_dev(old), to_dev(adv), to_dev(rf), to_dev(w))
    wide = torch.full((rows, vocab + 1), 7.0, dtype=logits.dtype, device=logits.device)
    got = ts.policy_loss(logits, *args, grad_logits=wide[:, :vocab], **kw)
    torch.cuda.synchronize()
    assert (wide[:, vocab:] == 7.0).all()
    check_policy(got, want, x, 0.8, dtype, rows, f(w), f(adv), 0.1)
    first = [t.clone() for t in (got.grad_logits, got.loss)]
    same = ts.policy_loss(logits, *args, grad_logits=wide[:, :vocab], **kw)
    assert torch.equal(same.grad_logits, first[0]) and torch.equal(same.loss, first[1])
    # In this gradient the rows start elsewhere in their cache lines, so the
    # sums run in another order: both are within the bound, not bit for bit one.
    again = ts.policy_loss(logits, *args, backward=True, **kw)
    check_policy(again, want, x, 0.8, dtype, rows, f(w), f(adv), 0.1)
    same = logits.clone()
    beside = ts.policy_loss(same, *args, backward=True, **kw)
    ts.policy_loss(same, *args, grad_logits=same, **kw)
    assert torch.equal(same, beside.grad_logits)


def test_policy_clip_limits_and_no_weights():
    import torch

    import top_sampling_amd as ts

    rows, vocab = 10, 500
    logits, x = make_logits(rows, vocab, "fp32", 0, 4, masks=False)
    tok = allowed_tokens(x, 1, skip=0.0)
    old, rf, adv, _ = policy_inputs(rows, x, tok, 1.0, 2)
    f = lambda a: a.astype(np.float64)  # noqa: E731
    for low, high in ((0.0, 0.0), (np.inf, np.inf), (0.5, np.inf)):
        want = ref.policy(x, tok, f(old), f(adv), clip_low=low, clip_high=high)
        if low == 0.0:
            # the fixed point 0 of the ratios' logarithms is the border itself
            keep = np.abs(want["ratios"] - 1) > 1e-3
        else:
            keep = np.ones(rows, bool)
        got = ts.policy_loss(logits, to_dev(tok, torch.int32), to_dev(old), to_dev(adv),
                             clip_low=low, clip_high=high, backward=True)
        torch.cuda.synchronize()
        tol = grad_tol(want["grad"], x, 1.0, "fp32", 4 * LSE) + \
            (np.abs(adv) * want["ratios"] * 2 * LSE)[:, None] * (want["grad"] != 0)
        close(got.grad_logits[to_dev(keep, torch.bool)], want["grad"][keep], tol[keep],
              (low, high))


def pref_offsets(rows, pairs, seed):
    g = np.random.default_rng(seed)
    cuts = np.sort(g.integers(0, rows + 1, 2 * pairs - 1))
    return np.concatenate([[0], cuts, [rows]]).astype(np.int32)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,vocab,pad,pairs", [
    (1, 1, 0, 1), (2, 2, 0, 1), (5, 3, 1, 2), (13, 1000, 24, 3), (37, 4097, 0, 9),
    (8, 30011, 0, 1), (300, 600, 0, 2), (1100, 257, 0, 40), (20, 70001, 0, 3), (200, 40001, 2, 4),
])
def test_preference_loss(rows, vocab, pad, pairs, dtype):
    import torch

    import top_sampling_amd as ts

    for mean, smoothing, temperature, margin in ((False, 0.0, 1.0, 0.0), (True, 0.1, 0.7, 0.3)):
        say("preference_loss", rows, vocab, pad, pairs, dtype, mean)
        logits, x = make_logits(rows, vocab, dtype, pad, rows * 5 + vocab)
        tok = allowed_tokens(x, 7)
        off = pref_offsets(rows, pairs, 11)
        if rows > 30:  # rows outside the sequences on both sides
            off = np.clip(off, 2, rows - 5)
        g = np.random.default_rng(9)
        lp, _ = ref.score(x, tok, temperature)
        rf = (lp + g.normal(0, 0.5, rows)).astype(np.float32)
        w = g.uniform(0.1, 1, pairs).astype(np.float32)
        if pairs > 2:
            w[1] = 0.0
        beta = 0.3
        kw = dict(beta=beta, label_smoothing=smoothing, margin=margin, mean=mean,
                  temperature=temperature)
        for weights, reference, scale in ((w, rf, 2.0), (None, None, 1.0)):
            f = lambda a: None if a is None else a.astype(np.float64)  # noqa: E731
            d = lambda a: None if a is None else to_dev(a)  # noqa: E731
            want = ref.preference(x, tok, off, f(reference), f(weights), grad_loss=scale, **kw)
            args = (to_dev(tok, torch.int32), to_dev(off, torch.int32), d(reference), d(weights))
            gl = torch.full((), scale, device=_dev()) if scale != 1.0 else None
            got = ts.preference_loss(logits, *args, backward=True, grad_loss=gl, **kw)
            fwd = ts.preference_loss(logits, *args, **kw)
            torch.cuda.synchronize()
            # every row of a sequence may be off by LSE
            live = np.maximum(np.diff(off), 1)
            rho_tol = beta * LSE * (1.0 if mean else live)
            z_tol = (np.broadcast_to(rho_tol, 2 * pairs)[:pairs]
                     + np.broadcast_to(rho_tol, 2 * pairs)[pairs:])
            pw = np.full(pairs, 1 / pairs) if weights is None else f(weights)
            for o in (got, fwd):
                close(o.logprobs, want["logprobs"], LSE + U * np.abs(want["logprobs"]), "lp")
                close(o.rewards, want["rewards"], rho_tol + U * np.abs(want["rewards"]), "rewards")
                close(o.pair_losses, want["pair_losses"],
                      z_tol + 2 * U * np.abs(want["pair_losses"]), "pair losses")
                close(o.loss, want["loss"], (pw * z_tol).sum() + 2 * U * abs(want["loss"]), "loss")
                assert not o.row_status.any()
            assert fwd.grad_logits is None
            # dl/dz changes by at most z_tol / 4
            p = np.exp(ref.log_softmax(x, temperature))
            k = np.zeros(rows)
            for i in range(2 * pairs):
                n = 1 if not mean else max(1, int((tok[off[i]:off[i + 1]] >= 0).sum()))
                k[off[i]:off[i + 1]] = scale * pw[i % pairs] * beta / n * \
                    (z_tol[i % pairs] + 2 * LSE) / temperature
            tol = grad_tol(want["grad"], x, temperature, dtype, 2 * LSE) + k[:, None] * \
                np.maximum(p, want["grad"] != 0)
            close(got.grad_logits, want["grad"], tol, "gradient")


def test_rows_left_out_may_hold_anything():
    """NaN and infinite logits in rows that take no part change nothing; in a
    row that does they are reported and reach the loss."""
    import torch

    import top_sampling_amd as ts

    for dtype in ("fp32", "bf16"):
        logits, x = make_logits(12, 777, dtype, 0, 3, masks=False)
        tok = allowed_tokens(x, 4, skip=0.0)
        tok[5] = -1
        w = np.full(12, 0.25, np.float32)
        w[8] = 0.0
        old, rf, adv, _ = policy_inputs(12, x, tok, 1.0, 2)
        args = (to_dev(tok, torch.int32), to_dev(old), to_dev(adv))
        clean = ts.policy_loss(logits, *args, weights=to_dev(w), backward=True)
        spoilt = logits.clone()
        spoilt[5] = float("nan")
        spoilt[8, 3] = float("inf")
        got = ts.policy_loss(spoilt, *args, weights=to_dev(w), backward=True)
        assert torch.equal(got.loss, clean.loss) and torch.isfinite(got.loss)
        assert torch.equal(got.grad_logits, clean.grad_logits)
        assert not got.grad_logits[5].any() and not got.grad_logits[8].any()
        # preference: rows 10 and 11 lie behind the last sequence
        off = torch.tensor([0, 4, 10], dtype=torch.int32, device=_dev())
        a = ts.preference_loss(logits, args[0], off, backward=True)
        spoilt = logits.clone()
        spoilt[5] = float("nan")
        spoilt[10:] = float("nan")
        b = ts.preference_loss(spoilt, args[0], off, backward=True)
        assert torch.equal(a.loss, b.loss) and torch.equal(a.grad_logits, b.grad_logits)
        assert not b.grad_logits[10:].any() and not b.logprobs[10:].any()


def test_bad_rows_are_reported():
    import torch

    import top_sampling_amd as ts

    vocab = 5000
    for dtype in ("fp32", "bf16"):
        logits, x = make_logits(8, vocab, dtype, 0, 3, masks=False)
        tok = allowed_tokens(x, 4, skip=0.0)
        tok[1] = vocab
        logits[2, 4999] = float("nan")
        logits[3, 17] = float("inf")
        logits[4] = -float("inf")
        logits[6, int(tok[6])] = -float("inf")  # a token of probability 0: not a bad row
        logits[7] = torch.finfo(logits.dtype).min
        tk = to_dev(tok, torch.int32)
        out = ts.token_logprobs(logits, tk, entropies=True)
        assert out.row_status.tolist() == [0, 1, 2, 2, 2, 0, 0, 0]
        for v in (out.logprobs, out.entropies):
            assert torch.isnan(v).tolist() == [False, True, True, True, True, False, False, False]
        assert out.logprobs[6] == -float("inf")
        # a row of nothing but the lowest value is uniform
        assert abs(out.logprobs[7].item() + np.log(vocab)) < LSE + 9 * U
        assert abs(out.entropies[7].item() - np.log(vocab)) < LSE + 9 * U
        ones = torch.ones(8, device=_dev())
        d = ts.token_logprobs_backward(logits, tk, out, ones)
        assert torch.isnan(d[1:5]).all() and torch.isfinite(d[[0, 5, 6, 7]]).all()
        skip = ones.clone()
        skip[1:5] = 0
        d = ts.token_logprobs_backward(logits, tk, out, skip)
        assert torch.isfinite(d).all() and not d[1:5].any()
        got = ts.policy_loss(logits, tk, -ones, ones, backward=True)
        assert torch.isnan(got.loss) and got.row_status.tolist() == [0, 1, 2, 2, 2, 0, 0, 0]
        assert torch.isnan(got.grad_logits[1:5]).all()
        zero = torch.zeros(8, device=_dev())
        assert torch.isnan(ts.policy_loss(logits, tk, -ones, zero).loss)
        keep = ones.clone()
        keep[1:5] = 0
        good = ts.policy_loss(logits, tk, -ones, ones, weights=keep, backward=True)
        assert torch.isfinite(good.loss) and not good.row_status.any()
        off = torch.tensor([0, 1, 5, 6, 8], dtype=torch.int32, device=_dev())
        pref = ts.preference_loss(logits, tk, off, backward=True)
        # pair 0 is rows 0 and 5; pair 1 rows 1-4 (bad) and 6-7
        assert torch.isnan(pref.pair_losses).tolist() == [False, True]
        assert torch.isfinite(pref.grad_logits[[0, 5]]).all()
        one = torch.tensor([1.0, 0.0], device=_dev())
        pref = ts.preference_loss(logits, tk, off, pair_weights=one, backward=True)
        assert torch.isfinite(pref.loss) and not pref.grad_logits[1:5].any()


def test_bad_offsets_stay_in_bounds():
    """Offsets outside the rows are clamped, descending ones give empty
    sequences."""
    import torch

    import top_sampling_amd as ts

    logits, x = make_logits(9, 300, "fp32", 0, 3, masks=False)
    tk = to_dev(allowed_tokens(x, 4, skip=0.0), torch.int32)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=_dev())  # noqa: E731
    a = ts.preference_loss(logits, tk, i32(-5, 4, 2 ** 30), backward=True)
    b = ts.preference_loss(logits, tk, i32(0, 4, 9), backward=True)
    assert torch.equal(a.loss, b.loss) and torch.equal(a.grad_logits, b.grad_logits)
    c = ts.preference_loss(logits, tk, i32(9, 3, 0), backward=True)
    assert abs(c.loss.item() - np.log(2)) < 2 * U and not c.rewards.any()


def test_empty_calls():
    import torch

    import top_sampling_amd as ts

    e = torch.empty(0, 100, device=_dev())
    t = torch.empty(0, dtype=torch.int32, device=_dev())
    f = torch.empty(0, device=_dev())
    assert ts.token_logprobs(e, t).logprobs.numel() == 0
    assert ts.policy_loss(e, t, f, f, backward=True).loss.item() == 0.0
    z = torch.zeros(1, dtype=torch.int32, device=_dev())
    assert ts.preference_loss(e, t, z, backward=True).loss.item() == 0.0
    p = ts.preference_loss(e, t, torch.zeros(5, dtype=torch.int32, device=_dev()), backward=True)
    assert abs(p.loss.item() - np.log(2)) < 2 * U
    # rows but no pairs: a loss of 0 and zero gradients
    x = torch.randn(3, 50, device=_dev())
    p = ts.preference_loss(x, torch.zeros(3, dtype=torch.int32, device=_dev()), z, backward=True)
    assert p.loss.item() == 0.0 and not p.grad_logits.any()


def test_every_row_left_out():
    import torch

    import top_sampling_amd as ts

    x = torch.full((4, 3000), float("nan"), device=_dev())
    t = torch.full((4,), -1, dtype=torch.int32, device=_dev())
    f = torch.zeros(4, device=_dev())
    got = ts.policy_loss(x, t, f, f, backward=True)
    assert got.loss.item() == 0.0 and not got.grad_logits.any() and (got.ratios == 1).all()
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device=_dev())
    for mean in (False, True):
        p = ts.preference_loss(x, t, off, mean=mean, backward=True)
        assert abs(p.loss.item() - np.log(2)) < 2 * U and not p.grad_logits.any()


def test_streams_and_graph():
    """On a stream of its own, and captured once and replayed with new inputs
    between other work."""
    import torch

    import top_sampling_amd as ts

    rows, vocab = 24, 9001
    logits, x = make_logits(rows, vocab, "fp32", 0, 3)
    tok = allowed_tokens(x, 4)
    old, rf, adv, w = policy_inputs(rows, x, tok, 1.0, 2)
    tk, old, rf, adv, w = to_dev(tok, torch.int32), *(to_dev(a) for a in (old, rf, adv, w))
    off = to_dev(pref_offsets(rows, 3, 1), torch.int32)

    def step(x, stream=None):
        p = ts.policy_loss(x, tk, old, adv, rf, w, kl_coef=0.1, backward=True, stream=stream)
        q = ts.preference_loss(x, tk, off, rf, backward=True, stream=stream)
        s = ts.token_logprobs(x, tk, entropies=True, stream=stream)
        d = ts.token_logprobs_backward(x, tk, s, adv, adv, stream=stream)
        return [p.loss, p.kl, p.grad_logits, q.loss, q.grad_logits, s.logprobs, d]

    plain = step(logits)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got = step(logits, stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(plain, got))

    static = logits.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(static)
    for i in range(4):
        static.copy_(logits * (1 + 0.1 * i))
        graph.replay()
        want = step(static)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, captured)), i


def test_long_rows_pass_32_bits():
    """Row offsets past 2^31 elements (fp32: a buffer of 9 GB)."""
    import torch

    import top_sampling_amd as ts

    rows, vocab, ld = 3, 2000, 1_150_000_000
    wide = torch.empty((rows - 1) * ld + vocab, device=_dev())
    big = wide.as_strided((rows, vocab), (ld, 1))
    logits, x = make_logits(rows, vocab, "fp32", 0, 3, masks=False)
    big.copy_(logits)
    tk = to_dev(allowed_tokens(x, 4, skip=0.0), torch.int32)
    a, b = ts.token_logprobs(big, tk), ts.token_logprobs(logits, tk)
    assert torch.equal(a.logprobs, b.logprobs)
    g = torch.ones(rows, device=_dev())
    want = ts.token_logprobs_backward(logits, tk, b, g)
    got = ts.token_logprobs_backward(big, tk, a, g, grad_logits=big)
    assert torch.equal(got, want)


def test_longest_row():
    """One row of 2^31 - 1 entries (4 GB in bf16), the last ones short of a
    vector: the largest accepted size."""
    import torch

    import top_sampling_amd as ts

    vocab = 2 ** 31 - 1
    dev = torch.device("cuda:0")
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB of GPU memory")
    x = torch.zeros(1, vocab, dtype=torch.bfloat16, device=dev)
    x[0, -1], x[0, 5] = 20.0, 18.0
    token = torch.tensor([vocab - 1], dtype=torch.int32, device=dev)
    total = vocab - 2 + np.exp(20.0) + np.exp(18.0)
    lp = 20.0 - np.log(total)
    out = ts.token_logprobs(x, token)
    assert abs(out.logprobs.item() - lp) < LSE + U * abs(lp)
    one = torch.ones(1, device=dev)
    grad = ts.token_logprobs_backward(x, token, out, one)
    # a probability is off by 2 LSE of itself, and then rounded to bf16
    for at, want in ((vocab - 1, 1 - np.exp(lp)), (vocab - 2, -1 / total), (5, -np.exp(18) / total),
                     (0, -1 / total), (2 ** 30 + 1, -1 / total)):
        assert abs(grad[0, at].item() - want) <= abs(want) * (2.0 ** -8 + 4 * LSE), at
    pol = ts.policy_loss(x, token, out.logprobs, one, grad_logits=x)
    torch.cuda.synchronize()
    assert abs(pol.loss.item() + 1) < 4 * LSE
    assert abs(x[0, -1].item() + (1 - np.exp(lp))) <= 2.0 ** -8 + 4 * LSE
    assert abs(x[0, 7].item() * total - 1) <= 2.0 ** -8 + 4 * LSE


def test_graphs_that_share_a_workspace():
    """Two captured calls with one workspace, replayed in turn on one stream:
    nothing is kept in it from call to call."""
    import torch

    import top_sampling_amd as ts

    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(2)
    rows, vocab = 24, 40001
    x = torch.randn(rows, vocab, generator=g, device=dev)
    tokens = torch.randint(0, vocab, (rows,), generator=g, device=dev, dtype=torch.int32)
    old = -torch.rand(rows, generator=g, device=dev) - 10
    adv = torch.randn(rows, generator=g, device=dev)
    offsets = torch.tensor([0, 7, 12, 20, 24], dtype=torch.int32, device=dev)
    ws = torch.empty(ts.preference_loss_workspace_bytes(rows, vocab, 2), dtype=torch.uint8,
                     device=dev)
    calls = (lambda: ts.policy_loss(x, tokens, old, adv, backward=True, workspace=ws),
             lambda: ts.preference_loss(x, tokens, offsets, backward=True, workspace=ws))
    for call in calls:
        call()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for call in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call())
        graphs.append(graph)
    for i in range(3):
        x.mul_(0.9)
        ws.fill_(255)
        for graph in graphs:
            graph.replay()
        got = [(o.loss.clone(), o.grad_logits.clone()) for o in outs]
        want = [call() for call in calls]
        torch.cuda.synchronize()
        for (loss, grad), w in zip(got, want):
            assert torch.equal(loss, w.loss) and torch.equal(grad, w.grad_logits), i


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("vocab", [1, 6, 40, 71, 131, 1000, 33001])
def test_every_alignment(dtype, vocab):
    """Rows that start anywhere in a cache line, the gradient's elsewhere than
    the logits'; what lies between the rows is left alone."""
    import torch

    import top_sampling_amd as ts

    rows = 3
    kind = torch.float32 if dtype == "fp32" else torch.bfloat16
    g = torch.Generator(device="cpu")
    g.manual_seed(vocab)
    x0 = torch.randn(rows, vocab, generator=g).mul(3).to(kind)
    tok = torch.tensor([0, vocab - 1, vocab // 2], dtype=torch.int32, device=_dev())
    x = x0.double().numpy()
    e = np.exp(x - x.max(-1, keepdims=True))
    prob = e / e.sum(-1, keepdims=True)
    lp = np.log(prob[np.arange(rows), tok.cpu().numpy()])
    adv = torch.tensor([1.0, -2.0, 0.5], device=_dev())
    want = prob.copy()
    want[np.arange(rows), tok.cpu().numpy()] -= 1.0
    # 1 - p of a likely token comes from its log-probability
    tol = grad_tol(want, x, 1.0, dtype, 4 * LSE) + 4 * LSE * (want < 0)
    old = to_dev(lp)
    for at, stride, grad_at, grad_stride in ((0, 0, 0, 0), (1, 0, 1, 0), (5, 3, 0, 1), (63, 0, 2, 7),
                                             (32, 64 - vocab % 64, 31, 64 - vocab % 64),
                                             (7, 1, 7, 1)):
        say("alignment", dtype, vocab, at, stride, grad_at, grad_stride)
        ld, ldg = vocab + stride, vocab + grad_stride
        wide = torch.full((at + rows * ld + 70,), 7.0, dtype=kind, device=_dev())
        logits = wide[at:].as_strided((rows, vocab), (ld, 1), at)
        logits.copy_(x0)
        out = ts.token_logprobs(logits, tok)
        close(out.logprobs, lp, LSE + U * np.abs(lp), "logprobs")
        buf = torch.full((grad_at + rows * ldg + 70,), 7.0, dtype=kind, device=_dev())
        grad = buf.as_strided((rows, vocab), (ldg, 1), grad_at)
        ts.token_logprobs_backward(logits, tok, out, -torch.ones_like(adv), grad_logits=grad)
        close(grad, want, tol, "backward")
        grad.fill_(7.0)
        pol = ts.policy_loss(logits, tok, old, adv, clip_low=np.inf, clip_high=np.inf,
                             grad_logits=grad)
        close(pol.logprobs, lp, LSE + U * np.abs(lp), "policy logprobs")
        a = adv.cpu().double().numpy()[:, None]
        close(grad, a * want, np.abs(a) * (tol + np.abs(want) * 2 * LSE), "policy")
        pair = ts.preference_loss(logits, tok, torch.tensor([0, 1, 3], dtype=torch.int32,
                                                            device=_dev()), grad_logits=grad)
        close(pair.logprobs, lp, LSE + U * np.abs(lp), "preference logprobs")
        rho = 0.1 * (lp[0] - lp[1] - lp[2])
        k = 0.1 / (1 + np.exp(rho)) * np.array([[1.0], [-1.0], [-1.0]])
        close(grad, k * want, np.abs(k) * (tol + np.abs(want) * 4 * LSE), "preference")
        grad.fill_(7.0)
        assert (buf == 7.0).all()
        inplace = ts.token_logprobs_backward(logits, tok, out, -torch.ones_like(adv),
                                             grad_logits=logits)
        close(inplace, want, tol, "in place")
        logits.fill_(7.0)
        assert (wide == 7.0).all()


def test_many_rows():
    """More rows than one launch has workgroups for, two logits each: loss
    sums, and rows past 2^22."""
    import torch

    import top_sampling_amd as ts

    rows = (1 << 23) + 1001
    x = torch.zeros(rows, 2, device=_dev())
    g = torch.Generator(device=_dev())
    g.manual_seed(1)
    x[:, 1] = torch.randn(rows, generator=g, device=_dev())
    tok = (torch.arange(rows, device=_dev()) % 2).int()
    lp = torch.log_softmax(x.double(), -1).gather(1, tok.long()[:, None])[:, 0]
    out = ts.token_logprobs(x, tok)
    assert ((out.logprobs.double() - lp).abs() <= LSE + U * lp.abs()).all()
    adv = torch.where(tok == 0, 1.0, -0.5)
    w = torch.full((rows,), 1.0 / rows, device=_dev())
    one = torch.softmax(x.double(), -1)
    one.scatter_add_(1, tok.long()[:, None], torch.full_like(lp, -1.0)[:, None])
    want = one * adv.double()[:, None] * w.double()[:, None]
    for back in (False, True):
        pol = ts.policy_loss(x, tok, lp.float(), adv, weights=w, backward=back)
        # each ratio is off by 2 LSE, and the old log-probabilities' rounding
        assert abs(pol.loss.item() + adv.double().mean().item()) <= 3 * LSE
    assert ((pol.grad_logits.double() - want).abs() <= 8 * LSE / rows).all()
    half = rows // 2
    off = torch.tensor([0, half, rows], dtype=torch.int32, device=_dev())
    pair = ts.preference_loss(x, tok, off, mean=True, backward=True)
    z = 0.1 * (lp[:half].mean() - lp[half:].mean()).item()
    assert abs(pair.loss.item() - np.log1p(np.exp(-z))) <= 0.1 * 2 * LSE + 2 * U
    k = -0.1 / (1 + np.exp(z)) / half
    assert ((pair.grad_logits[:half].double() + k * one[:half]).abs() <= 8 * LSE * -k).all()
    # rows are consecutive entries: a left-out end stays zero
    tok[-3:] = -1
    assert not ts.token_logprobs(x, tok).logprobs[-3:].any()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows", [5, 130])
def test_gradient_beside_the_logits(rows, dtype):
    """Logits and gradient as columns of one buffer, in either order."""
    import torch

    import top_sampling_amd as ts

    vocab = 33003
    logits, x = make_logits(rows, vocab, dtype, 0, 3, masks=False)
    tok = to_dev(allowed_tokens(x, 4), torch.int32)
    old = to_dev(np.full(rows, -9.0))
    adv = to_dev(np.linspace(-1, 1, rows))
    for left, right in ((0, vocab + 2), (vocab + 3, 1)):
        wide = torch.full((rows, 2 * vocab + 5), 7.0, dtype=logits.dtype, device=_dev())
        here, grad = wide[:, left:left + vocab], wide[:, right:right + vocab]
        here.copy_(logits)
        apart = torch.empty_like(wide)[:, right:right + vocab]
        want = ts.policy_loss(here, tok, old, adv, grad_logits=apart)
        got = ts.policy_loss(here, tok, old, adv, grad_logits=grad)
        assert torch.equal(grad, apart) and torch.equal(got.loss, want.loss)
        assert torch.equal(here, logits)
        grad.fill_(7.0)
        here.fill_(7.0)
        assert (wide == 7.0).all()


def entry_tol(want, x, tok, coef, temperature, dtype):
    """Of a loss's gradient: grad_tol's relative part, and the error `coef` of
    each row's coefficient times what multiplies it, the entry's own
    probability, or 1 - p_t <= 1 at the token."""
    scale = np.exp(ref.log_softmax(x, temperature))
    scale[np.arange(len(x)), np.maximum(tok, 0)] = 1.0
    return grad_tol(want, x, temperature, dtype, 2 * LSE) + coef[:, None] * scale


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("smoothing", [0.0, 0.1, 1.0])
@pytest.mark.parametrize("mean", [False, True])
def test_preference_answers_with_a_masked_token(dtype, smoothing, mean):
    """A token of probability 0 in the rejected answer of a pair and in the
    chosen one: z is +-inf, and a term of factor 0 stays 0."""
    import torch

    import top_sampling_amd as ts

    for vocab in (700, 40001):  # whole rows, and in chunks
        say("masked token", dtype, smoothing, mean, vocab)
        rows, pairs, beta = 12, 3, 0.3
        logits, x = make_logits(rows, vocab, dtype, 0, 21, masks=False)
        tok = allowed_tokens(x, 7, skip=0.0)
        off = np.arange(0, 13, 2, dtype=np.int32)
        for r in (2, 9):  # the chosen and the rejected answer of pair 1
            logits[r, int(tok[r])] = -float("inf")
        x = logits.cpu().double().numpy()
        for masked, left_out in ((9, 2), (2, 9)):
            t = tok.copy()
            t[left_out] = -1
            kw = dict(beta=beta, label_smoothing=smoothing, mean=mean)
            want = ref.preference(x, t, off, **kw)
            got = ts.preference_loss(logits, to_dev(t, torch.int32), to_dev(off, torch.int32),
                                     backward=True, **kw)
            fwd = ts.preference_loss(logits, to_dev(t, torch.int32), to_dev(off, torch.int32),
                                     **kw)
            torch.cuda.synchronize()
            # by hand: z = +inf, then -inf
            lost = (smoothing if masked == 9 else 1 - smoothing) > 0
            assert want["pair_losses"][1] == (np.inf if lost else 0.0)
            # at most four rows in a z, and values below 16
            z_tol = 4 * beta * LSE
            for o in (got, fwd):
                close(o.pair_losses, want["pair_losses"], z_tol + 16 * U, "pair losses")
                close(o.loss, want["loss"], z_tol + 16 * U, "loss")
                close(o.rewards, want["rewards"], z_tol + 16 * U, "rewards")
                assert not o.row_status.any()
            k = np.full(rows, beta / pairs * (z_tol + 2 * LSE))
            close(got.grad_logits, want["grad"], entry_tol(want["grad"], x, t, k, 1.0, dtype),
                  "gradient")
            assert torch.isfinite(got.grad_logits).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(6, 700), (6, 40001), (130, 33001)])
def test_policy_token_masked_since_it_was_drawn(rows, vocab, dtype):
    """A token of probability 0 with a finite reference: the ratio is 0 and the
    KL term infinite, and nothing of it reaches another row."""
    import torch

    import top_sampling_amd as ts

    logits, x = make_logits(rows, vocab, dtype, 0, 22, masks=False)
    tok = allowed_tokens(x, 7, skip=0.0)
    old, rf, adv, _ = policy_inputs(rows, x, tok, 1.0, 3)
    w = np.full(rows, 1.0 / rows, np.float32)
    logits[4, int(tok[4])] = -float("inf")
    x = logits.cpu().double().numpy()
    f = lambda a: a.astype(np.float64)  # noqa: E731
    args = (to_dev(tok, torch.int32), to_dev(old), to_dev(adv), to_dev(rf), to_dev(w))
    others = np.arange(rows) != 4
    for kl_coef in (0.0, 0.2):
        say("masked token", dtype, rows, vocab, kl_coef)
        kw = dict(clip_low=0.2, clip_high=0.28, kl_coef=kl_coef)
        with np.errstate(invalid="ignore"):
            want = ref.policy(x, tok, f(old), f(adv), f(rf), f(w), **kw)
        coef = f(w) * (np.abs(f(adv)) * want["ratios"] + kl_coef * 8) * 2 * LSE
        for back in (False, True):
            got = ts.policy_loss(logits, *args, backward=back, **kw)
            torch.cuda.synchronize()
            assert not got.row_status.any()
            assert got.logprobs[4] == -float("inf") and got.ratios[4] == 0.0
            assert got.kl[4] == float("inf") and want["kl"][4] == np.inf
            close(got.kl[to_dev(others, torch.bool)], want["kl"][others], 8 * LSE + U * 8, "kl")
            if kl_coef:
                assert got.loss == float("inf") and want["loss"] == np.inf
            else:
                close(got.loss, want["loss"], coef.sum() + 2 * U * abs(want["loss"]), "loss")
        # dloss/dlp of the row is infinite with the KL term, and 0 without
        assert want["grad"][4].any() == (kl_coef > 0)
        if kl_coef:
            assert not torch.isfinite(got.grad_logits[4]).any()
            assert not np.isfinite(want["grad"][4]).any()
        else:
            assert not got.grad_logits[4].any()
        tol = entry_tol(want["grad"], x, tok, coef, 1.0, dtype)
        close(got.grad_logits[to_dev(others, torch.bool)], want["grad"][others], tol[others],
              "gradient")


def confident_rows(rows, vocab, dtype, seed):
    """Logits whose token has 1 - p of 1e-9 .. 1e-6: the rest of the mass all
    over the row, or all within eight entries of the token."""
    import torch

    g = np.random.default_rng(seed)
    x = np.empty((rows, vocab), np.float32)
    tok = g.integers(0, vocab, rows).astype(np.int32)
    tok[:2] = 0, vocab - 1
    for r in range(rows):
        d = 10.0 ** g.uniform(-9, -6)
        if r % 2:
            x[r] = g.normal(np.log(d / vocab), 1.0, vocab)
        else:
            x[r] = g.normal(-60.0, 1.0, vocab)
            lo, hi = max(0, tok[r] - 8), min(vocab, tok[r] + 9)
            x[r, lo:hi] = np.log(d / (hi - lo)) + g.normal(0, 0.5, hi - lo)
        x[r, tok[r]] = 0.0
    t = torch.from_numpy(x).to(_dev(), torch.float32 if dtype == "fp32" else torch.bfloat16)
    return t, t.cpu().double().numpy(), tok


# Of d = 1 - p of a token: every e_j has LSE at most, so their sum has; the
# values are rounded to fp32 once.
DIGITS = LSE + 2 * U


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(6, 2), (9, 40), (40, 300), (30, 16390), (6, 33001),
                                        (12, 151936), (200, 40001), (140, 120001)])
def test_digits_next_to_probability_1(rows, vocab, dtype):
    """Where p is near 1, log-probability, entropy and the token's own gradient
    entry are right relative to 1 - p, not just next to 1."""
    import torch

    import top_sampling_amd as ts

    say("digits", dtype, rows, vocab)
    logits, x, tok = confident_rows(rows, vocab, dtype, rows + vocab)
    lp, ent = ref.score(x, tok)
    assert (np.abs(lp) < 1e-5).all()
    at = np.arange(rows)
    tk = to_dev(tok, torch.int32)
    out = ts.token_logprobs(logits, tk, entropies=True)
    plain = ts.token_logprobs(logits, tk)
    torch.cuda.synchronize()
    close(out.logprobs, lp, DIGITS * np.abs(lp), "logprobs with entropies")
    close(plain.logprobs, lp, DIGITS * np.abs(lp), "logprobs")
    # H = ln S + E[max - z], both positive; the mean's terms have LSE too
    close(out.entropies, ent, 3 * DIGITS * ent, "entropies")
    g = np.random.default_rng(5).normal(1, 0.2, rows).astype(np.float32)
    old, adv = to_dev(lp), to_dev(-g)
    wide = dict(clip_low=np.inf, clip_high=np.inf)
    want = ref.policy(x, tok, lp.astype(np.float32).astype(np.float64), -g.astype(np.float64),
                      **wide)
    pol = ts.policy_loss(logits, tk, old, adv, backward=True, **wide)
    fwd = ts.policy_loss(logits, tk, old, adv, **wide)
    close(pol.logprobs, lp, DIGITS * np.abs(lp), "policy logprobs")
    close(fwd.logprobs, lp, DIGITS * np.abs(lp), "policy logprobs without gradient")
    # 1 - p, the ratio (LSE of nearly 0) and the rounding to the type
    tol = np.abs(want["grad"][at, tok]) * (2 * DIGITS + 2 * U + HALF[dtype])
    close(pol.grad_logits[to_dev(at, torch.int64), tk.long()], want["grad"][at, tok], tol,
          "policy gradient")
    off = np.array([0, rows // 2, rows], np.int32)
    want = ref.preference(x, tok, off)
    pref = ts.preference_loss(logits, tk, to_dev(off, torch.int32), backward=True)
    close(pref.logprobs, lp, DIGITS * np.abs(lp), "preference logprobs")
    tol = np.abs(want["grad"][at, tok]) * (2 * DIGITS + 2 * U + HALF[dtype])
    close(pref.grad_logits[to_dev(at, torch.int64), tk.long()], want["grad"][at, tok], tol,
          "preference gradient")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(6, 2), (9, 40), (40, 300), (30, 16390), (12, 151936),
                                        (200, 40001)])
def test_backward_digits_next_to_probability_1(rows, vocab, dtype):
    """The token's own gradient entry from the forward pass's results, relative
    to 1 - p; and the entries of a row add up to about 0."""
    import torch

    import top_sampling_amd as ts

    say("digits backward", dtype, rows, vocab)
    logits, x, tok = confident_rows(rows, vocab, dtype, rows + vocab)
    at = np.arange(rows)
    rng = np.random.default_rng(5)
    g = rng.normal(1, 0.2, rows).astype(np.float32)
    # of the same sign as g: the two terms of the entry do not cancel, as
    # -h p (ln p + H) has the sign of -h
    h = -rng.uniform(0.1, 0.3, rows).astype(np.float32)
    tk = to_dev(tok, torch.int32)
    for ent, gh in ((False, None), (True, None), (True, h)):
        fwd = ts.token_logprobs(logits, tk, entropies=ent)
        got = ts.token_logprobs_backward(logits, tk, fwd, to_dev(g),
                                         None if gh is None else to_dev(gh))
        torch.cuda.synchronize()
        want = ref.score_gradient(x, tok, 1.0, g.astype(np.float64),
                                  None if gh is None else gh.astype(np.float64))
        own = want[at, tok]
        # 1 - p and H, each with its digits, and two roundings of fp32 inputs
        tol = np.abs(own) * (4 * DIGITS + 4 * U + HALF[dtype])
        close(got[to_dev(at, torch.int64), tk.long()], own, tol, ("own entry", ent, gh is None))


def test_backward_without_the_log_probabilities():
    """The C entry that takes none gives the same away from probability 1."""
    import torch

    import top_sampling_amd as ts

    logits, x = make_logits(9, 4099, "fp32", 0, 1, masks=False)
    tk = to_dev(allowed_tokens(x, 2), torch.int32)
    g = torch.randn(9, device=_dev())
    fwd = ts.token_logprobs(logits, tk, 0.8, entropies=True)
    with_lp = ts.token_logprobs_backward(logits, tk, fwd, g, g, 0.8)
    d = torch.full_like(logits, 7.0)
    s = torch.cuda.current_stream().cuda_stream
    assert ts.lib.token_logprobs_backward(
        logits.data_ptr(), ts.TS_F32, 9, 4099, 4099, tk.data_ptr(), 0.8, fwd.row_stats.data_ptr(),
        g.data_ptr(), fwd.entropies.data_ptr(), g.data_ptr(), d.data_ptr(), 4099, s) == ts.TS_OK
    torch.cuda.synchronize()
    assert torch.equal(d, with_lp)


def test_backward_after_the_log_probabilities_were_changed():
    """A caller that scales or masks the forward pass's log-probabilities in
    place gets the gradient at the rows' own ones."""
    import torch

    import top_sampling_amd as ts

    logits, x, tok = confident_rows(12, 4099, "fp32", 3)
    logits[6:] *= 0.3  # p from 1 down to 0.9 or less
    x = logits.cpu().double().numpy()
    tk, g = to_dev(tok, torch.int32), torch.ones(12, device=_dev())
    want = ref.score_gradient(x, tok, 1.0, np.ones(12))
    at = np.arange(12)
    for change in (lambda v: v.neg_(), lambda v: v.sub_(0.01), lambda v: v.fill_(float("nan")),
                   lambda v: v.double(), lambda v: v[:5], lambda v: v[:, None].expand(12, 2)[:, 0],
                   lambda v: v.cpu(), lambda v: None):
        fwd = ts.token_logprobs(logits, tk)
        fwd.logprobs = change(fwd.logprobs)
        got = ts.token_logprobs_backward(logits, tk, fwd, g)
        own = want[at, tok]
        # as without them: 1 - p is off by the rounding of S in fp32
        close(got[to_dev(at, torch.int64), tk.long()], own, np.abs(own) * DIGITS * 4 + 2 * U,
              "own entry")


def check_entries(got, want, x, tok, coef, temperature, dtype):
    """The gradient entry by entry, at a tolerance that entries taken as 0
    would not pass."""
    tol = entry_tol(want, x, tok, coef, temperature, dtype)
    close(got, want, tol, "gradient")
    other = np.abs(want) > 2.0 ** -100
    other[np.arange(len(x)), np.maximum(tok, 0)] = False
    if other.any():
        assert (tol < np.abs(want))[other].mean() > 0.99


LONG = [
    # one read: held on the chip, with a part that is read again, more than that
    # twice over, short rows; and two passes
    ("fp32", 96, 33000, 0), ("fp32", 96, 114688, 0), ("fp32", 97, 120001, 0),
    ("bf16", 128, 131077, 3), ("bf16", 130, 262144, 0), ("fp32", 3, 32768, 0),
    ("fp32", 95, 33001, 0), ("bf16", 127, 40000, 1), ("fp32", 2, 300000, 0),
]
ENTRIES = [(d, *s) for d in ("fp32", "bf16") for s in SHAPES]


@pytest.mark.parametrize("dtype,rows,vocab,pad", ENTRIES + LONG)
def test_policy_gradient_entries(dtype, rows, vocab, pad):
    import torch

    import top_sampling_amd as ts

    say("policy entries", dtype, rows, vocab, pad)
    logits, x = make_logits(rows, vocab, dtype, pad, rows * 3 + vocab)
    tok = allowed_tokens(x, 6)
    temperature = 0.8
    old, rf, adv, w = policy_inputs(rows, x, tok, temperature, 8)
    f = lambda a: a.astype(np.float64)  # noqa: E731
    args = (to_dev(tok, torch.int32), to_dev(old), to_dev(adv), to_dev(rf), to_dev(w))
    for kl_coef in (0.0, 0.1):
        kw = dict(clip_low=0.2, clip_high=0.28, kl_coef=kl_coef, temperature=temperature)
        want = ref.policy(x, tok, f(old), f(adv), f(rf), f(w), **kw)
        got = ts.policy_loss(logits, *args, backward=True, **kw)
        torch.cuda.synchronize()
        # dloss/dlp: the ratio is off by LSE of itself, exp(gap) too; a clipped
        # ratio does not enter
        r = want["ratios"]
        inside = np.where(adv >= 0, r <= 1.28, r >= 0.8)
        gap = np.where(want["kl"] > 0, f(rf) - want["logprobs"], 0.0)
        coef = f(w) * (np.abs(f(adv)) * r * inside + kl_coef * np.exp(gap)) * 2 * LSE / temperature
        check_entries(got.grad_logits, want["grad"], x, tok, coef, temperature, dtype)


@pytest.mark.parametrize("dtype,rows,vocab,pad", ENTRIES + [
    ("fp32", 20, 70001, 0), ("bf16", 200, 40001, 2), ("bf16", 40, 120001, 0)])
def test_preference_gradient_entries(dtype, rows, vocab, pad):
    import torch

    import top_sampling_amd as ts

    say("preference entries", dtype, rows, vocab, pad)
    logits, x = make_logits(rows, vocab, dtype, pad, rows * 5 + vocab)
    tok = allowed_tokens(x, 7)
    pairs, beta, temperature = max(1, rows // 9), 0.3, 0.8
    off = pref_offsets(rows, pairs, 11)
    lp, _ = ref.score(x, tok, temperature)
    rf = (lp + np.random.default_rng(9).normal(0, 0.2, rows)).astype(np.float32)
    for mean in (False, True):
        kw = dict(beta=beta, label_smoothing=0.1, mean=mean, temperature=temperature)
        want = ref.preference(x, tok, off, rf.astype(np.float64), **kw)
        got = ts.preference_loss(logits, to_dev(tok, torch.int32), to_dev(off, torch.int32),
                                 to_dev(rf), backward=True, **kw)
        torch.cuda.synchronize()
        # z: LSE a row, sums over the live rows; |d2l / dz2| <= 1/4
        live = tok >= 0
        n = np.array([live[off[i]:off[i + 1]].sum() for i in range(2 * pairs)])
        rho_tol = beta * LSE * (np.minimum(n, 1) if mean else n)
        dz_tol = (rho_tol[:pairs] + rho_tol[pairs:]) / 4
        coef = np.zeros(rows)
        for i in range(2 * pairs):
            coef[off[i]:off[i + 1]] = beta / pairs * (dz_tol[i % pairs] + 2 * LSE) / \
                (max(1, n[i]) if mean else 1) / temperature
        check_entries(got.grad_logits, want["grad"], x, tok, coef, temperature, dtype)


def test_more_pairs_than_one_launch_has_workgroups_for():
    """Past 2^23 pairs, where a workgroup a pair is more threads than a launch
    has: nearly all are empty, the first and the last hold a row each side."""
    import torch

    import top_sampling_amd as ts

    pairs = (1 << 23) + 5
    x, _ = make_logits(4, 300, "fp32", 0, 3, masks=False)
    tok = torch.tensor([5, 17, 200, 299], dtype=torch.int32, device=_dev())
    # rows 0 and 1: chosen answers of pairs 0 and pairs - 1; 2 and 3: rejected
    off = torch.zeros(2 * pairs + 1, dtype=torch.int32, device=_dev())
    off[1:] = 1
    off[pairs:] = 2
    off[pairs + 1:] = 3
    off[2 * pairs:] = 4
    say("pairs", pairs)
    got = ts.preference_loss(x, tok, off, beta=0.5, backward=True)
    torch.cuda.synchronize()
    lp, _ = ref.score(x.cpu().double().numpy(), tok.cpu().numpy())
    z = 0.5 * np.array([lp[0] - lp[2], lp[1] - lp[3]])
    each = np.log1p(np.exp(-z))
    close(got.pair_losses[[0, pairs - 1]], each, LSE + 2 * U * np.abs(each), "ends")
    assert ((got.pair_losses[1:-1] - np.float32(np.log(2))).abs() <= 2 * U).all()
    assert not got.rewards[1:pairs - 1].any() and not got.rewards[pairs + 1:-1].any()
    assert abs(got.loss.item() - np.log(2)) <= 2 * U + np.abs(each).max() / pairs
    want = ref.preference(x.cpu().double().numpy(), tok.cpu().numpy(), [0, 1, 2, 3, 4], beta=0.5)
    scale = 2.0 / pairs  # of the two pairs' mean
    x64 = x.cpu().double().numpy()
    coef = np.full(4, 0.5 / pairs * 3 * LSE)
    close(got.grad_logits, want["grad"] * scale,
          entry_tol(want["grad"] * scale, x64, tok.cpu().numpy(), coef, 1.0, "fp32"), "gradient")


def test_outputs_stand_on_their_own():
    """What a user's program does with a call's outputs: a loss returned by an
    autograd function and scaled in place, and one output changed in place
    while a graph still holds another."""
    import torch

    import top_sampling_amd as ts

    dev = torch.device("cuda:0")
    x = torch.randn(6, 500, device=dev)
    tok = torch.arange(6, dtype=torch.int32, device=dev)
    f = torch.randn(6, device=dev)
    off = torch.tensor([0, 3, 6], dtype=torch.int32, device=dev)

    def calls(v):
        return (ts.policy_loss(v, tok, -f.abs() - 5, f, backward=True),
                ts.preference_loss(v, tok, off, backward=True))

    for i in range(2):
        class Loss(torch.autograd.Function):
            @staticmethod
            def forward(ctx, v):
                out = calls(v)[i]
                ctx.save_for_backward(out.grad_logits)
                return out.loss

            @staticmethod
            def backward(ctx, g):
                return g * ctx.saved_tensors[0]

        leaf = x.clone().requires_grad_()
        loss = Loss.apply(leaf)
        loss /= 4
        loss.backward()
        assert torch.equal(leaf.grad, calls(x)[i].grad_logits / 4)

    w = torch.ones(6, device=dev, requires_grad=True)
    for out in (*calls(x), ts.token_logprobs(x, tok, entropies=True)):
        held = (w * out.logprobs).sum()
        for other in (getattr(out, "loss", None), getattr(out, "entropies", None), out.row_status):
            if other is not None:
                other.zero_()
        held.backward()
        changed = out.logprobs
        changed.mul_(w)
        assert changed.requires_grad


def test_one_row_in_place_by_another_view():
    """One row of a wider buffer, and the same row as a view of its own."""
    import torch

    import top_sampling_amd as ts

    wide = torch.randn(3, 700, device=_dev())
    tok = torch.tensor([5], dtype=torch.int32, device=_dev())
    one = torch.ones(1, device=_dev())
    row, same = wide[1:2, :640], wide[1, :640].clone()[None]
    want = ts.policy_loss(same, tok, -one, one, backward=True).grad_logits
    alias = wide[1, :640].unsqueeze(0)
    assert alias.data_ptr() == row.data_ptr() and alias.stride(0) != row.stride(0)
    before = wide.clone()
    ts.policy_loss(row, tok, -one, one, grad_logits=alias)
    torch.cuda.synchronize()
    # the row starts elsewhere in its cache line than the clone
    assert ((row - want).abs() <= 4 * LSE * want.abs() + 2 * LSE * (want < 0)).all()
    assert torch.equal(wide[[0, 2]], before[[0, 2]]) and torch.equal(wide[:, 640:], before[:, 640:])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("temperature", [1e20, 1e30, 1e35, 1e37, 1e38])
def test_largest_temperatures(temperature, dtype):
    """Logits as large as the temperature: log2(e) / T is a number below
    fp32's normal ones, the sums of logits pass its range, and 1 / T^2 is 0."""
    import torch

    import top_sampling_amd as ts

    say("temperature", temperature, dtype)
    g = np.random.default_rng(4)
    for vocab in (3000, 40001):
        rows = 5
        x = (g.uniform(-1.6, 1.6, (rows, vocab)) * temperature).astype(np.float32)
        x[1, g.random(vocab) < 0.5] = -np.inf
        logits = torch.from_numpy(x).to(_dev(),
                                        torch.float32 if dtype == "fp32" else torch.bfloat16)
        x = logits.cpu().double().numpy()
        tok = np.array([g.choice(np.flatnonzero(np.isfinite(r))) for r in x]).astype(np.int32)
        tk = to_dev(tok, torch.int32)
        lp, ent = ref.score(x, tok, temperature)
        out = ts.token_logprobs(logits, tk, temperature, entropies=True)
        close(out.logprobs, lp, LSE + U * np.abs(lp), "logprobs")
        close(out.entropies, ent, LSE * 32, "entropies")
        if temperature > 1e30:  # the gradients are below fp32's normal numbers
            continue
        a, h = g.normal(size=rows).astype(np.float32), g.normal(size=rows).astype(np.float32)
        want = ref.score_gradient(x, tok, temperature, a.astype(np.float64),
                                  h.astype(np.float64))
        got = ts.token_logprobs_backward(logits, tk, out, to_dev(a), to_dev(h), temperature)
        # as in test_token_logprobs; |ln p| + H < 4 + 2 ln(vocab)
        p = np.exp(ref.log_softmax(x, temperature))
        size = p * (np.abs(a) + np.abs(h) * 32)[:, None]
        size[np.arange(rows), tok] += np.abs(a) * LSE
        tol = grad_tol(want, x, temperature, dtype, 2 * LSE) + size * 2 * LSE / temperature
        close(got, want, tol, "gradient")
        assert not got[1, np.flatnonzero(np.isinf(x[1]))].any()
