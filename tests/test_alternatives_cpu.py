"""Scoring with alternatives and listed tokens on the CPU: the oracle by hand
and against differences, and the refusals of the C ABI and the binding
(validation runs before any HIP call)."""
import ctypes

import numpy as np
import pytest

import top_sampling_amd as ts
from oracle import alternatives as ref

FAKE = 0x100000  # aligned, never dereferenced
F64 = ctypes.c_double


def test_topn_by_hand():
    x = np.log(np.array([[1.0, 4.0, 4.0, 7.0, 16.0], [1, 1, 1, 1, 1]]))
    x[1, 1:4] = -np.inf
    out = ref.topn(x, np.array([2, 2]), 4)
    assert out["ids"].tolist() == [[4, 3, 1, 2], [0, 4, 1, 2]]
    assert out["ranks"].tolist() == [4, 4]
    assert np.allclose(np.exp(out["top"]), [[0.5, 7 / 32, 1 / 8, 1 / 8], [0.5, 0.5, 0, 0]])
    assert np.allclose(np.exp(out["logprobs"]), [1 / 8, 0])
    assert np.isclose(out["entropies"][1], np.log(2))
    assert ref.topn(x, None, 7)["ids"][0].tolist() == [4, 3, 1, 2, 0, -1, -1]
    bad = ref.topn(np.array([[1.0, np.nan], [1.0, 2.0], [1.0, 2.0]]), np.array([0, 5, -1]), 1)
    assert bad["status"].tolist() == [2, 1, 0] and np.isnan(bad["top"][:2]).all()
    assert bad["ids"].tolist() == [[-1], [-1], [-1]] and bad["top"][2, 0] == -np.inf


@pytest.mark.parametrize("temperature", [1.0, 0.6])
def test_listed_gradient_against_differences(temperature):
    g = np.random.default_rng(0)
    x = g.normal(size=(3, 7))
    ids = np.array([[3, 0, 3, -1], [6, 5, 1, 2], [-1, -1, -1, -1]])
    a, h = g.normal(size=ids.shape), g.normal(size=3)

    def value(x):
        lp, ent, _ = ref.listed(x, ids, temperature)
        return (a * lp).sum() + (h * ent).sum()

    want = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = 1e-5
        want[i] = (value(x + e) - value(x - e)) / 2e-5
    # central differences: 1e-10 of the third derivative and 1e-16 / 1e-5
    assert np.abs(ref.listed_gradient(x, ids, temperature, a, h) - want).max() < 1e-8


def test_listed_of_one_is_the_single_token():
    from oracle import losses

    g = np.random.default_rng(1)
    x, tok = g.normal(size=(4, 9)), np.array([3, -1, 0, 8])
    lp, ent = losses.score(x, tok, 0.8)
    got_lp, got_ent, _ = ref.listed(x, tok[:, None], 0.8)
    assert np.allclose(got_lp[:, 0], lp) and np.allclose(got_ent, ent)
    a, h = g.normal(size=4), g.normal(size=4)
    assert np.allclose(ref.listed_gradient(x, tok[:, None], 0.8, a[:, None], h),
                       losses.score_gradient(x, tok, 0.8, a, h))


def _topn(**kw):
    a = dict(x=FAKE, type=ts.TS_F32, rows=4, vocab=64, ld=64, tok=FAKE, t=1.0, n=5, lp=FAKE,
             ranks=FAKE, ent=None, ids=FAKE, top=FAKE, stats=None, status=None, ws=FAKE,
             bytes=1 << 30)
    a.update(kw)
    return ts.lib.token_logprobs_topn(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), ts.TS_EINVAL), (dict(vocab=-1), ts.TS_EINVAL), (dict(type=7), ts.TS_EINVAL),
    (dict(rows=1 << 31), ts.TS_EUNSUPPORTED), (dict(vocab=1 << 31), ts.TS_EUNSUPPORTED),
    (dict(t=0.0), ts.TS_EINVAL), (dict(t=float("nan")), ts.TS_EINVAL),
    (dict(t=float("inf")), ts.TS_EINVAL), (dict(vocab=0), ts.TS_EINVAL), (dict(ld=63), ts.TS_EINVAL),
    (dict(x=None), ts.TS_EINVAL), (dict(n=-1), ts.TS_EINVAL),
    (dict(n=ts.TS_MAX_LOGPROBS + 1), ts.TS_EUNSUPPORTED), (dict(lp=None), ts.TS_EINVAL),
    (dict(tok=None), ts.TS_EINVAL), (dict(tok=None, lp=None), ts.TS_EINVAL),
    (dict(ids=None), ts.TS_EINVAL), (dict(top=None), ts.TS_EINVAL),
    (dict(x=FAKE + 2), ts.TS_EUNSUPPORTED), (dict(tok=FAKE + 2), ts.TS_EUNSUPPORTED),
    (dict(lp=FAKE + 1), ts.TS_EUNSUPPORTED), (dict(ranks=FAKE + 2), ts.TS_EUNSUPPORTED),
    (dict(ent=FAKE + 2), ts.TS_EUNSUPPORTED), (dict(ids=FAKE + 2), ts.TS_EUNSUPPORTED),
    (dict(top=FAKE + 2), ts.TS_EUNSUPPORTED), (dict(stats=FAKE + 2), ts.TS_EUNSUPPORTED),
    (dict(status=FAKE + 2), ts.TS_EUNSUPPORTED), (dict(ws=None), ts.TS_EWORKSPACE),
    (dict(bytes=16), ts.TS_EWORKSPACE), (dict(ws=FAKE + 128), ts.TS_EUNSUPPORTED),
])
def test_topn_refusals(kw, code):
    assert _topn(**kw) == code
    assert ts.lib.ts_last_error()


def _listed(**kw):
    a = dict(x=FAKE, type=ts.TS_F32, rows=4, vocab=64, ld=64, ids=FAKE, n=5, t=1.0, lp=FAKE,
             ent=None, stats=None, status=None, ws=FAKE, bytes=1 << 30)
    a.update(kw)
    return ts.lib.token_logprobs_listed(*a.values(), None)


def _listed_backward(**kw):
    a = dict(x=FAKE, type=ts.TS_F32, rows=4, vocab=64, ld=64, ids=FAKE, n=5, t=1.0, stats=FAKE,
             lp=FAKE, glp=FAKE, ent=None, gent=None, grad=FAKE, ldg=64)
    a.update(kw)
    return ts.lib.token_logprobs_listed_backward(*a.values(), None)


@pytest.mark.parametrize("call", [_listed, _listed_backward])
@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), ts.TS_EINVAL), (dict(vocab=-1), ts.TS_EINVAL), (dict(type=7), ts.TS_EINVAL),
    (dict(rows=1 << 31), ts.TS_EUNSUPPORTED), (dict(vocab=1 << 31), ts.TS_EUNSUPPORTED),
    (dict(t=0.0), ts.TS_EINVAL), (dict(vocab=0), ts.TS_EINVAL), (dict(ld=63), ts.TS_EINVAL),
    (dict(x=None), ts.TS_EINVAL), (dict(ids=None), ts.TS_EINVAL), (dict(n=0), ts.TS_EINVAL),
    (dict(n=-3), ts.TS_EINVAL), (dict(n=ts.TS_MAX_LISTED + 1), ts.TS_EUNSUPPORTED),
    (dict(lp=None), ts.TS_EINVAL), (dict(x=FAKE + 2), ts.TS_EUNSUPPORTED),
    (dict(ids=FAKE + 2), ts.TS_EUNSUPPORTED), (dict(lp=FAKE + 1), ts.TS_EUNSUPPORTED),
    (dict(ent=FAKE + 2), ts.TS_EUNSUPPORTED), (dict(stats=FAKE + 2), ts.TS_EUNSUPPORTED),
])
def test_listed_refusals(call, kw, code):
    assert call(**kw) == code
    assert ts.lib.ts_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(stats=None), ts.TS_EINVAL), (dict(glp=None), ts.TS_EINVAL), (dict(grad=None), ts.TS_EINVAL),
    (dict(gent=FAKE), ts.TS_EINVAL), (dict(glp=FAKE + 2), ts.TS_EUNSUPPORTED),
    (dict(gent=FAKE + 2, ent=FAKE), ts.TS_EUNSUPPORTED), (dict(ldg=63), ts.TS_EINVAL),
    (dict(grad=FAKE + 2), ts.TS_EUNSUPPORTED), (dict(grad=FAKE + 4), ts.TS_EINVAL),
    (dict(ldg=65), ts.TS_EINVAL),
])
def test_listed_backward_refusals(kw, code):
    assert _listed_backward(**kw) == code
    assert ts.lib.ts_last_error()


def test_listed_workspace_refusals():
    assert _listed(ws=None) == ts.TS_EWORKSPACE
    assert _listed(bytes=16) == ts.TS_EWORKSPACE
    assert _listed(ws=FAKE + 128) == ts.TS_EUNSUPPORTED
    assert _listed(status=FAKE + 2) == ts.TS_EUNSUPPORTED


def test_empty_is_noop():
    assert _topn(rows=0, x=None, tok=None, lp=None, ws=None) == ts.TS_OK
    assert _listed(rows=0, x=None, ids=None, lp=None, ws=None) == ts.TS_OK
    assert _listed_backward(rows=0, x=None, ids=None, grad=None) == ts.TS_OK


def test_workspace_queries():
    for query in (ts.token_logprobs_topn_workspace_bytes, ts.token_logprobs_listed_workspace_bytes):
        assert query(-1, 100) == 0 and query(4, -1) == 0 and query(1 << 31, 4) == 0
        assert query(0, 100) == 0
        assert query(640, 151936) > query(64, 151936) / 4 > 0
    # a record a row at least, and a group's largest entry for 128 entries
    assert ts.token_logprobs_topn_workspace_bytes(640, 151936) >= 640 * 4 * 151936 // 128


def test_header_constant_matches_binding():
    import os
    import re

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "top_sampling.h")).read()
    assert re.search(rf"#define TS_MAX_LISTED {ts.TS_MAX_LISTED}\b", text)


def test_binding_refusals():
    import torch

    x = torch.zeros(4, 64)
    tok = torch.zeros(4, dtype=torch.int32)
    ids = torch.zeros(4, 3, dtype=torch.int32)
    for args in ((x[0], tok, 5), (x.half(), tok, 5), (x.t(), tok, 5), (x, tok[:3], 5),
                 (x, tok.long(), 5), (x, tok, -1), (x, tok, ts.TS_MAX_LOGPROBS + 1)):
        with pytest.raises(ValueError):
            ts.token_logprobs_topn(*args)
    fwd = ts.TokenLogprobs(torch.zeros(4, 3), None, torch.zeros(4, 2), None)
    for args in ((x[0], ids), (x.half(), ids), (x, ids[:3]), (x, ids.long()), (x, tok),
                 (x, ids[:, :0]), (x, torch.zeros(4, ts.TS_MAX_LISTED + 1, dtype=torch.int32)),
                 (x, ids.t().contiguous().t())):
        with pytest.raises(ValueError):
            ts.token_logprobs_listed(*args)
        with pytest.raises(ValueError):
            ts.token_logprobs_listed_backward(*args, fwd, torch.zeros(4, 3))
    for change in (dict(grad_logprobs=None), dict(grad_logprobs=torch.zeros(4, 2)),
                   dict(grad_entropies=torch.zeros(3)),
                   dict(forward=ts.TokenLogprobs(None, None, torch.zeros(4, 2), None)),
                   dict(forward=ts.TokenLogprobs(torch.zeros(4, 3), None, None, None)),
                   dict(forward=ts.TokenLogprobs(torch.zeros(4, 2), None, torch.zeros(4, 2), None))):
        kw = dict(forward=fwd, grad_logprobs=torch.zeros(4, 3))
        kw.update(change)
        with pytest.raises(ValueError):
            ts.token_logprobs_listed_backward(x, ids, **kw)
    # Right in all but the device.
    for call in (lambda: ts.token_logprobs_topn(x, tok, 5),
                 lambda: ts.token_logprobs_listed(x, ids),
                 lambda: ts.token_logprobs_listed_backward(x, ids, fwd, torch.zeros(4, 3))):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_alternatives_are_not_taken_for_the_tokens():
    """With one alternative a row the given tokens' log-probabilities have the size of the
    listed ones and would pass for them."""
    import torch

    x, one = torch.zeros(4, 64), torch.zeros(4, dtype=torch.int32)
    top = ts.TokenLogprobsTopn(torch.zeros(4), one, None, one[:, None], torch.zeros(4, 1),
                               torch.zeros(4, 2), one)
    with pytest.raises(ValueError, match="topn_logprobs"):
        ts.token_logprobs_listed_backward(x, top.topn_ids, top, torch.zeros(4, 1))
    fwd = ts.TokenLogprobs(top.topn_logprobs, top.entropies, top.row_stats, top.row_status)
    with pytest.raises(ValueError, match="GPU"):  # right in all but the device
        ts.token_logprobs_listed_backward(x, top.topn_ids, fwd, torch.zeros(4, 1))
