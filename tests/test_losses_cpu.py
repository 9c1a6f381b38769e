"""Token scoring and the losses on the CPU: the oracle's gradients against
differences, and the refusals of the C ABI and the binding (validation runs
before any HIP call, so no GPU is needed)."""
import ctypes

import numpy as np
import pytest

import top_sampling_amd as ts
from oracle import losses as ref

FAKE = 0x100000  # aligned, never dereferenced


def _differences(f, x, step=1e-6):
    d = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        if not np.isfinite(x[i]):
            continue
        lo, hi = x.copy(), x.copy()
        lo[i] -= step
        hi[i] += step
        d[i] = (f(hi) - f(lo)) / (2 * step)
    return d


def _rows(seed, rows=6, vocab=9):
    g = np.random.default_rng(seed)
    x = g.normal(0, 2, (rows, vocab))
    x[1, 3] = -np.inf
    tokens = g.integers(0, vocab, rows)
    tokens[1] = 2
    tokens[4] = -1
    return g, x, tokens


# Central differences of step 1e-6: error ~ 1e-12 (third derivative, O(1)
# here) plus 2^-53 / 1e-6 ~ 1e-10 of cancellation, times a few terms.
DIFF_TOL = 1e-8


@pytest.mark.parametrize("temperature", [1.0, 0.6])
def test_score_gradient_against_differences(temperature):
    g, x, tokens = _rows(1)
    a, b = g.normal(size=6), g.normal(size=6)

    def f(v):
        lp, ent = ref.score(v, tokens, temperature)
        return (a * lp + b * ent).sum()

    got = ref.score_gradient(x, tokens, temperature, a, b)
    assert np.abs(got - _differences(f, x)).max() < DIFF_TOL
    assert not got[4].any()


@pytest.mark.parametrize("kl_coef", [0.0, 0.3])
def test_policy_gradient_against_differences(kl_coef):
    g, x, tokens = _rows(2)
    lp, _ = ref.score(x, tokens)
    old, rf = lp + g.normal(0, 0.4, 6), lp + g.normal(0, 0.4, 6)
    adv, w = g.normal(size=6), g.uniform(0.1, 1, 6)
    w[5] = 0
    kw = dict(clip_low=0.2, clip_high=0.28, kl_coef=kl_coef, temperature=1.0)
    got = ref.policy(x, tokens, old, adv, rf, w, **kw)
    f = lambda v: ref.policy(v, tokens, old, adv, rf, w, **kw)["loss"]  # noqa: E731
    assert np.abs(got["grad"] - _differences(f, x)).max() < DIFF_TOL
    assert not got["grad"][5].any() and not got["grad"][4].any()


@pytest.mark.parametrize("mean,smoothing", [(False, 0.0), (True, 0.1)])
def test_preference_gradient_against_differences(mean, smoothing):
    g, x, tokens = _rows(3)
    offsets = [0, 2, 2, 5, 6]  # the second chosen answer is empty
    rf = g.normal(-2, 1, 6)
    kw = dict(beta=0.7, label_smoothing=smoothing, margin=0.2, mean=mean)
    got = ref.preference(x, tokens, offsets, rf, **kw)
    f = lambda v: ref.preference(v, tokens, offsets, rf, **kw)["loss"]  # noqa: E731
    assert np.abs(got["grad"] - _differences(f, x)).max() < DIFF_TOL


def test_policy_terms_by_hand():
    """One row of two equal logits: lp = ln 1/2."""
    x = np.zeros((1, 2))
    lp = np.log(0.5)
    up = ref.policy(x, np.array([0]), np.array([lp - np.log(2)]), np.array([3.0]))
    assert np.isclose(up["ratios"][0], 2.0) and np.isclose(up["loss"], -1.2 * 3)
    assert not up["grad"].any()  # clipped
    down = ref.policy(x, np.array([0]), np.array([lp - np.log(2)]), np.array([-3.0]))
    assert np.isclose(down["loss"], 6.0)  # not clipped on this side
    assert np.allclose(down["grad"], [[3.0, -3.0]])


# ------------------------------------------------------------- refusals (C ABI)
def _score(**kw):
    a = dict(x=FAKE, kind=0, rows=4, vocab=100, ld=100, tok=FAKE, t=1.0, lp=FAKE, ent=None,
             stats=None, status=None, ws=FAKE, n=1 << 30)
    a.update(kw)
    return ts.lib.token_logprobs(*a.values(), None)


BAD_ROWS = [
    (dict(rows=-1), ts.TS_EINVAL), (dict(vocab=-1), ts.TS_EINVAL), (dict(kind=2), ts.TS_EINVAL),
    (dict(rows=1 << 31), ts.TS_EUNSUPPORTED), (dict(vocab=1 << 31), ts.TS_EUNSUPPORTED),
    (dict(t=0.0), ts.TS_EINVAL), (dict(t=float("nan")), ts.TS_EINVAL),
    (dict(t=float("inf")), ts.TS_EINVAL), (dict(vocab=0), ts.TS_EINVAL),
    (dict(ld=99), ts.TS_EINVAL), (dict(x=None), ts.TS_EINVAL), (dict(tok=None), ts.TS_EINVAL),
    (dict(x=FAKE + 2), ts.TS_EUNSUPPORTED), (dict(x=FAKE + 1, kind=1), ts.TS_EUNSUPPORTED),
    (dict(tok=FAKE + 2), ts.TS_EUNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", BAD_ROWS + [
    (dict(lp=None), ts.TS_EINVAL), (dict(ent=FAKE + 2), ts.TS_EUNSUPPORTED),
    (dict(ws=None), ts.TS_EWORKSPACE), (dict(n=8), ts.TS_EWORKSPACE),
    (dict(ws=FAKE + 64), ts.TS_EUNSUPPORTED),
])
def test_token_logprobs_refusals(kw, code):
    assert _score(**kw) == code
    assert ts.lib.ts_last_error()


def test_token_logprobs_empty_is_noop():
    assert _score(rows=0, x=None, tok=None, lp=None, ws=None) == ts.TS_OK


def _back(**kw):
    a = dict(x=FAKE, kind=0, rows=4, vocab=100, ld=100, tok=FAKE, t=1.0, stats=FAKE, g=FAKE,
             ent=None, gh=None, d=FAKE * 2, ldd=100)
    a.update(kw)
    return ts.lib.token_logprobs_backward(*a.values(), None)


@pytest.mark.parametrize("kw,code", BAD_ROWS + [
    (dict(stats=None), ts.TS_EINVAL), (dict(g=None), ts.TS_EINVAL), (dict(d=None), ts.TS_EINVAL),
    (dict(gh=FAKE), ts.TS_EINVAL), (dict(ldd=99), ts.TS_EINVAL),
    (dict(d=FAKE + 400), ts.TS_EINVAL),           # overlaps, other rows
    (dict(d=FAKE, ldd=128), ts.TS_EINVAL),        # the same start, another stride
    (dict(d=FAKE * 2 + 2), ts.TS_EUNSUPPORTED),
    # columns of one buffer that touch the logits' on either side
    (dict(ld=250, ldd=250, d=FAKE + 4 * 99), ts.TS_EINVAL),
    (dict(ld=250, ldd=250, d=FAKE + 4 * 151), ts.TS_EINVAL),
    (dict(ld=250, ldd=250, d=FAKE - 4 * 99), ts.TS_EINVAL),
])
def test_token_logprobs_backward_refusals(kw, code):
    assert _back(**kw) == code


def _policy(params=(1.0, 0.2, 0.2, 0.0), **kw):
    a = dict(x=FAKE, kind=0, rows=4, vocab=100, ld=100, tok=FAKE, params=None, old=FAKE, ref=None,
             adv=FAKE, w=None, gl=None, loss=FAKE, lp=None, ratio=None, kl=None, status=None,
             d=None, ldd=0, ws=FAKE, n=1 << 30)
    a.update(kw)
    p = ts._PolicyParams(*params) if params else None
    a["params"] = ctypes.addressof(p) if p is not None else None
    a.pop("t", None)
    return ts.lib.policy_loss(*a.values(), None)


@pytest.mark.parametrize("kw,code", [c for c in BAD_ROWS if "t" not in c[0]] + [
    (dict(params=None), ts.TS_EINVAL),
    (dict(params=(0.0, 0.2, 0.2, 0.0)), ts.TS_EINVAL),
    (dict(params=(1.0, -0.1, 0.2, 0.0)), ts.TS_EINVAL),
    (dict(params=(1.0, 0.2, float("nan"), 0.0)), ts.TS_EINVAL),
    (dict(params=(1.0, 0.2, 0.2, -1.0)), ts.TS_EINVAL),
    (dict(params=(1.0, 0.2, 0.2, float("inf"))), ts.TS_EINVAL),
    (dict(params=(1.0, 0.2, 0.2, 0.1)), ts.TS_EINVAL),      # KL without a reference
    (dict(loss=None), ts.TS_EINVAL), (dict(old=None), ts.TS_EINVAL),
    (dict(adv=None), ts.TS_EINVAL), (dict(loss=FAKE + 2), ts.TS_EUNSUPPORTED),
    (dict(w=FAKE + 1), ts.TS_EUNSUPPORTED), (dict(ws=None), ts.TS_EWORKSPACE),
    (dict(d=FAKE * 2, ldd=99), ts.TS_EINVAL), (dict(d=FAKE + 400, ldd=100), ts.TS_EINVAL),
])
def test_policy_loss_refusals(kw, code):
    assert _policy(**kw) == code


def _preference(params=(1.0, 0.1, 0.0, 0.0, 0), **kw):
    a = dict(x=FAKE, kind=0, rows=4, vocab=100, ld=100, tok=FAKE, off=FAKE, pairs=1, params=None,
             ref=None, w=None, gl=None, loss=FAKE, pl=None, rew=None, lp=None, status=None,
             d=None, ldd=0, ws=FAKE, n=1 << 30)
    a.update(kw)
    p = ts._PreferenceParams(*params) if params else None
    a["params"] = ctypes.addressof(p) if p is not None else None
    return ts.lib.preference_loss(*a.values(), None)


@pytest.mark.parametrize("kw,code", [c for c in BAD_ROWS if "t" not in c[0]] + [
    (dict(params=None), ts.TS_EINVAL),
    (dict(params=(1.0, 0.0, 0.0, 0.0, 0)), ts.TS_EINVAL),
    (dict(params=(1.0, float("inf"), 0.0, 0.0, 0)), ts.TS_EINVAL),
    (dict(params=(1.0, 0.1, 1.5, 0.0, 0)), ts.TS_EINVAL),
    (dict(params=(1.0, 0.1, -0.1, 0.0, 0)), ts.TS_EINVAL),
    (dict(params=(1.0, 0.1, 0.0, float("inf"), 0)), ts.TS_EINVAL),
    (dict(params=(1.0, 0.1, 0.0, 0.0, 2)), ts.TS_EINVAL),
    (dict(pairs=-1), ts.TS_EINVAL), (dict(pairs=1 << 30), ts.TS_EUNSUPPORTED),
    (dict(off=None), ts.TS_EINVAL), (dict(loss=None), ts.TS_EINVAL),
    (dict(off=FAKE + 2), ts.TS_EUNSUPPORTED), (dict(ws=None), ts.TS_EWORKSPACE),
    (dict(d=FAKE + 400, ldd=100), ts.TS_EINVAL),
])
def test_preference_loss_refusals(kw, code):
    assert _preference(**kw) == code


def test_workspace_queries():
    assert ts.token_logprobs_workspace_bytes(640, 151936) > 0
    assert ts.token_logprobs_workspace_bytes(-1, 10) == 0
    assert ts.token_logprobs_workspace_bytes(0, 0) == 0
    assert ts.preference_loss_workspace_bytes(10, 100, -1) == 0
    # Every size has room for its records: one of 24 bytes a row at least.
    for rows in (1, 7, 640, 100000):
        for vocab in (1, 255, 4097, 151936, 1 << 20):
            assert ts.token_logprobs_workspace_bytes(rows, vocab) >= rows * (24 + 16 + 8)


# ------------------------------------------------------------ refusals (binding)
def test_binding_refusals():
    import torch

    x, tok = torch.zeros(3, 8), torch.zeros(3, dtype=torch.int32)
    f = torch.zeros(3)
    with pytest.raises(ValueError, match="on the GPU"):
        ts.token_logprobs(x, tok)
    for bad in (x.double(), x[0], x.t()[:3], x[:1].expand(3, 8)):
        with pytest.raises(ValueError):
            ts.token_logprobs(bad, tok)
    with pytest.raises(ValueError, match="token_ids"):
        ts.token_logprobs(x, tok.long())
    with pytest.raises(ValueError, match="token_ids"):
        ts.token_logprobs(x, tok[:2])
    with pytest.raises(ValueError, match="old_logprobs"):
        ts.policy_loss(x, tok, f[:2], f)
    with pytest.raises(ValueError, match="advantages"):
        ts.policy_loss(x, tok, f, f.double())
    with pytest.raises(ValueError, match="seq_offsets"):
        ts.preference_loss(x, tok, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="seq_offsets"):
        ts.preference_loss(x, tok, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="grad_logits"):
        ts._grad_rows(torch.zeros(3, 7), x)
    with pytest.raises(ValueError, match="grad_logits"):
        ts._grad_rows(torch.zeros(1, 8).expand(3, 8), x)


def test_preference_terms_of_factor_0():
    """A masked token in one answer: z is +-inf, and only a term whose factor
    is above 0 can make the loss infinite."""
    x = np.zeros((2, 4))
    x[1, 3] = -np.inf
    tok = np.array([0, 3])
    for order, sign in (([0, 1], 1), ([1, 0], -1)):
        rows = np.array(order)
        for eps in (0.0, 0.1, 1.0):
            got = ref.preference(x[rows], tok[rows], [0, 1, 2], label_smoothing=eps)
            # -(1 - eps) ln sigmoid(z) is 0 at z = inf, and so the other way
            factor = eps if sign > 0 else 1 - eps
            assert got["pair_losses"][0] == got["loss"] == (np.inf if factor else 0.0)
            assert np.isfinite(got["grad"]).all() and got["grad"].any() == (factor > 0)


@pytest.mark.parametrize("kl_coef", [0.0, 0.3])
def test_policy_kl_of_a_masked_token(kl_coef):
    """lp = -inf and a finite reference: e^g - g - 1 at g = inf is inf."""
    x = np.zeros((1, 3))
    x[0, 1] = -np.inf
    a = (x, np.array([1]), np.array([-1.0]), np.array([2.0]), np.array([-1.5]))
    with np.errstate(invalid="ignore"):
        got = ref.policy(*a, kl_coef=kl_coef)
    assert got["kl"][0] == np.inf and got["ratios"][0] == 0.0
    assert got["loss"] == (np.inf if kl_coef else 0.0)
    assert not (np.isfinite(got["grad"]).any() if kl_coef else got["grad"].any())


@pytest.mark.parametrize("kw,code", BAD_ROWS + [
    (dict(stats=None), ts.TS_EINVAL), (dict(g=None), ts.TS_EINVAL), (dict(d=None), ts.TS_EINVAL),
    (dict(gh=FAKE), ts.TS_EINVAL), (dict(ldd=99), ts.TS_EINVAL),
    (dict(lp=FAKE + 2), ts.TS_EUNSUPPORTED), (dict(stats=FAKE + 2), ts.TS_EUNSUPPORTED),
    (dict(d=FAKE + 400), ts.TS_EINVAL),
])
def test_token_logprobs_backward_ex_refusals(kw, code):
    a = dict(x=FAKE, kind=0, rows=4, vocab=100, ld=100, tok=FAKE, t=1.0, stats=FAKE, lp=FAKE,
             g=FAKE, ent=None, gh=None, d=FAKE * 2, ldd=100)
    a.update(kw)
    assert ts.lib.token_logprobs_backward_ex(*a.values(), None) == code
    assert ts.lib.ts_last_error()


def test_import_without_private_torch_names():
    """The package imports where torch has neither of the two private calls it
    prefers (a build without a GPU), and uses the public ones."""
    import os
    import subprocess
    import sys

    code = ("import torch\n"
            "for n in ('_cuda_getDevice', '_cuda_getCurrentRawStream'):\n"
            "    delattr(torch._C, n)\n"
            "import top_sampling_amd as ts\n"
            "class S: cuda_stream = 77\n"
            "torch.cuda.current_stream = lambda device: S() if device == 3 else None\n"
            "torch.cuda.current_device = lambda: 5\n"
            "assert ts._current_device() == 5 and ts._current_stream(3) == 77\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]


def test_one_row_has_no_leading_dimension():
    """A single row's gradient may replace it whatever the strides say; gets as
    far as the missing workspace."""
    assert _policy(rows=1, d=FAKE, ldd=128, ws=None) == ts.TS_EWORKSPACE
    assert _preference(rows=1, ld=300, d=FAKE, ldd=100, ws=None) == ts.TS_EWORKSPACE
    assert _policy(rows=2, d=FAKE, ldd=128, ws=None) == ts.TS_EINVAL
    assert _policy(rows=1, d=FAKE + 4, ldd=128, ws=None) == ts.TS_EINVAL
