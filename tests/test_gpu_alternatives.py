"""Scoring with alternatives and listed tokens with their gradient on the GPU
against the float64 oracle (oracle/alternatives.py).

Ids, ranks and statuses are equal.  Tolerances of the floats are those derived in
test_gpu_losses.py: LSE of ln S, fp32's rounding of a log-probability, and a
gradient entry's own terms.
"""
import numpy as np
import pytest
import test_gpu_losses as base
from test_gpu_losses import LSE, SHAPES, U, allowed_tokens, close, grad_tol, make_logits, say, to_dev

from oracle import alternatives as ref
from oracle.losses import log_softmax

pytestmark = pytest.mark.gpu


def _ids(t):
    return t.cpu().numpy().astype(np.int64)


def as_fp32(lp):
    """Log-probabilities below fp32's lowest number by half a step and more (logits
    of the type's lowest value at temperatures below 1) round to -inf."""
    return np.where(lp <= -(2.0 ** 128 - 2.0 ** 103), -np.inf, lp)


def check_topn(got, want, what, entropies=True):
    assert np.array_equal(_ids(got.topn_ids), want["ids"]), what
    assert np.array_equal(_ids(got.row_status), want["status"]), what
    top = as_fp32(want["top"])
    size = np.where(np.isfinite(top), np.abs(top), 0.0)
    close(got.topn_logprobs, top, LSE + U * size, (what, "alternatives"))
    if got.logprobs is not None:
        assert np.array_equal(_ids(got.ranks), want["ranks"]), what
        lp = as_fp32(want["logprobs"])
        close(got.logprobs, lp, LSE + U * np.where(np.isfinite(lp), np.abs(lp), 0.0), what)
    if entropies:
        close(got.entropies, want["entropies"], LSE * (2 + 30), (what, "entropies"))
    else:
        assert got.entropies is None


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,vocab,pad", SHAPES)
def test_topn(rows, vocab, pad, dtype):
    import torch

    import top_sampling_amd as ts

    logits, x = make_logits(rows, vocab, dtype, pad, rows * 5 + vocab)
    tok = allowed_tokens(x, 7)
    tk = to_dev(tok, torch.int32)
    for n, temperature, entropies in ((0, 1.0, True), (1, 0.37, False), (5, 1.0, True),
                                      (20, 0.8, True), (67, 1.0, False)):
        say("topn", rows, vocab, pad, dtype, n, temperature)
        got = ts.token_logprobs_topn(logits, tk, n, temperature, entropies=entropies)
        torch.cuda.synchronize()
        check_topn(got, ref.topn(x, tok, n, temperature), (n, temperature), entropies)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(3, 700), (5, 3000), (2, 50000), (40, 9001), (200, 20001)])
@pytest.mark.parametrize("n", [256, 257, 600, 1024])
def test_topn_long_lists(rows, vocab, n, dtype):
    import torch

    import top_sampling_amd as ts

    logits, x = make_logits(rows, vocab, dtype, 0, rows + vocab + n)
    tok = allowed_tokens(x, 8)
    got = ts.token_logprobs_topn(logits, to_dev(tok, torch.int32), n, entropies=True)
    torch.cuda.synchronize()
    check_topn(got, ref.topn(x, tok, n), n)


def _rows_with_ties(vocab, g):
    """Rows whose order hangs on the ids: all equal, two values, equal ones beside
    a few larger, in rising and falling order, masked but for a few, one allowed."""
    rows = [np.zeros(vocab), g.integers(0, 2, vocab), np.zeros(vocab), np.arange(vocab) / 64.0,
            -np.arange(vocab) / 64.0, np.full(vocab, -np.inf), np.full(vocab, -np.inf),
            np.full(vocab, -3.3e38), np.where(g.random(vocab) < 0.5, 0.0, -0.0)]
    rows[2][g.integers(0, vocab, 7)] = 1.0
    rows[5][g.integers(0, vocab, 3)] = g.normal(size=3)
    rows[6][vocab - 1] = -5.0
    rows[7][vocab // 2] = 1.0
    return np.stack(rows).astype(np.float32)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("vocab", [1, 2, 40, 257, 4096, 30011, 140000])
def test_topn_ties(vocab, dtype):
    import torch

    import top_sampling_amd as ts

    g = np.random.default_rng(vocab)
    logits = to_dev(_rows_with_ties(vocab, g), torch.float32 if dtype == "fp32" else torch.bfloat16)
    x = logits.cpu().double().numpy()
    # A token in the middle of the equal ones, masked ones among them; the last.
    for tok in (g.integers(0, vocab, len(x)), np.full(len(x), vocab - 1)):
        for n in (1, 20, 300):
            got = ts.token_logprobs_topn(logits, to_dev(tok, torch.int32), n, entropies=True)
            torch.cuda.synchronize()
            check_topn(got, ref.topn(x, tok, n), n)


def test_topn_ranks_of_every_token():
    import torch

    import top_sampling_amd as ts

    for dtype in ("fp32", "bf16"):
        logits, x = make_logits(1, 2100, dtype, 0, 3, masks=False)
        x[0, 5:9] = x[0, 2000]
        logits.copy_(torch.from_numpy(x))
        tok = torch.arange(2100, dtype=torch.int32, device="cuda")
        got = ts.token_logprobs_topn(logits.expand(2100, 2100).contiguous(), tok, 3)
        order = np.lexsort((np.arange(2100), -x[0]))
        want = np.empty(2100, np.int64)
        want[order] = np.arange(1, 2101)
        assert np.array_equal(_ids(got.ranks), want)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(4, 5000), (4, 60000), (300, 40000)])
def test_topn_without_tokens(rows, vocab, dtype):
    import torch

    import top_sampling_amd as ts

    logits, x = make_logits(rows, vocab, dtype, 1, rows)
    got = ts.token_logprobs_topn(logits, None, 9, 0.7, entropies=True)
    torch.cuda.synchronize()
    assert got.logprobs is None and got.ranks is None
    check_topn(got, ref.topn(x, None, 9, 0.7), "no tokens")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(6, 3001), (6, 90001), (300, 40001)])
def test_bad_and_left_out_rows(rows, vocab, dtype):
    """A NaN or +inf anywhere, no finite logit, an id past the vocabulary; rows
    that are left out may hold anything."""
    import torch

    import top_sampling_amd as ts

    logits, x = make_logits(rows, vocab, dtype, 0, 11, masks=False)
    tok = allowed_tokens(x, 12, skip=0.0)
    x[0, vocab - 1] = np.nan
    x[1, 0] = np.inf
    x[2] = -np.inf
    tok[3] = vocab
    tok[4] = -7
    x[4] = np.nan
    logits.copy_(torch.from_numpy(x))
    got = ts.token_logprobs_topn(logits, to_dev(tok, torch.int32), 4, entropies=True)
    torch.cuda.synchronize()
    check_topn(got, ref.topn(x, tok, 4), "bad rows")
    ids = np.stack([tok, np.full(rows, -1), np.where(tok >= 0, 5, -2)], 1)
    lp, ent, status = ref.listed(x, ids)
    for h in (None, np.ones(rows, np.float32)):
        out = ts.token_logprobs_listed(logits, to_dev(ids, torch.int32), entropies=True)
        a = np.ones((rows, 3), np.float32)
        a[5] = [1.0, 9.0, -1.0]  # adds up to 0
        a[1] = 0.0
        grad = ts.token_logprobs_listed_backward(logits, to_dev(ids, torch.int32), out, to_dev(a),
                                                 None if h is None else to_dev(h))
        torch.cuda.synchronize()
        assert np.array_equal(_ids(out.row_status), status)
        close(out.logprobs, lp, LSE + U * np.abs(np.nan_to_num(lp)), "listed")
        close(out.entropies, ent, LSE * 32, "entropies")
        want = ref.listed_gradient(x, ids, 1.0, a.astype(np.float64), h)
        g = grad.cpu().double().numpy()
        assert np.array_equal(np.isnan(g), np.isnan(want))
        assert np.isnan(g[0]).all() and not g[4].any()


def _some_ids(x, n, seed):
    """Ids of allowed tokens, some several times, masked ones, unused places, and
    rows of none."""
    g = np.random.default_rng(seed)
    rows, vocab = x.shape
    ids = g.integers(0, vocab, (rows, n))
    for r in range(rows):
        fine = np.flatnonzero(np.isfinite(x[r]) & (x[r] > -1e38))
        keep = g.random(n) < 0.7
        ids[r, keep] = g.choice(fine, keep.sum())
        ids[r, g.random(n) < 0.3] = x[r].argmax()
    ids[g.random((rows, n)) < 0.15] = -3
    ids[g.random(rows) < 0.1] = -1
    ids[0, 0] = x[0].argmax()
    return ids


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,vocab,pad", SHAPES)
def test_listed(rows, vocab, pad, dtype):
    import torch

    import top_sampling_amd as ts

    for n, temperature, entropy in ((1, 1.0, False), (6, 0.37, True), (33, 1.0, True)):
        say("listed", rows, vocab, pad, dtype, n, temperature)
        logits, x = make_logits(rows, vocab, dtype, pad, rows + 2 * vocab)
        ids = _some_ids(x, n, rows + n)
        lp, ent, status = ref.listed(x, ids, temperature)
        lp = as_fp32(lp)
        tk = to_dev(ids, torch.int32)
        out = ts.token_logprobs_listed(logits, tk, temperature, entropies=entropy)
        torch.cuda.synchronize()
        assert not status.any() and not out.row_status.any()
        close(out.logprobs, lp, LSE + U * np.where(np.isfinite(lp), np.abs(lp), 0.0), "listed")
        if entropy:
            close(out.entropies, ent, LSE * (2 + 30), "entropies")
        g = np.random.default_rng(n)
        a, h = g.normal(size=(rows, n)).astype(np.float32), g.normal(size=rows).astype(np.float32)
        h[: rows // 2] = 0.0
        if rows > 3:
            a[rows - 2:] = 0.0
        if not entropy:
            h = None
        want = ref.listed_gradient(x, ids, temperature, a.astype(np.float64),
                                   None if h is None else h.astype(np.float64))
        wide = torch.full((rows, vocab + 2), 7.0, dtype=logits.dtype, device=logits.device)
        got = ts.token_logprobs_listed_backward(logits, tk, out, to_dev(a),
                                                None if h is None else to_dev(h), temperature,
                                                grad_logits=wide[:, :vocab])
        torch.cuda.synchronize()
        assert (wide[:, vocab:] == 7.0).all()
        # Terms of several ids and of the entropy cancel: LSE of their sizes.
        logp = log_softmax(x, temperature)
        p = np.exp(logp)
        total = np.abs(np.where(ids >= 0, a, 0.0)).sum(-1)
        size = total[:, None] * p
        if h is not None:
            far = np.where(p > 0, np.abs(np.where(p > 0, logp, 0.0)), 0.0)
            size = size + np.abs(h)[:, None] * p * (far + np.abs(ent)[:, None] + 32)
        listed = np.zeros_like(x)
        for r in range(rows):
            np.add.at(listed[r], ids[r][ids[r] >= 0], np.abs(a[r][ids[r] >= 0]))
        tol = grad_tol(want, x, temperature, dtype, 2 * LSE) + \
            (size * (2 * LSE) + listed * LSE) / temperature
        # An e_j below 2^-126 may be taken as 0 (grad_tol counts that for factors
        # below 64).  Its factor is |a + b log2 e_j| <= (sum |g| + |h| (|H| + ln S
        # + |ln e_j|)) / (S T), with S >= 1, ln S < 13 and -ln e_j below 88 at
        # 2^-126; where it is smaller still, e_j |ln e_j| is too.
        factor = total if h is None else total + np.abs(h) * (np.abs(ent) + 13 + 88)
        tol = tol + (2.0 ** -126 * factor / temperature)[:, None]
        close(got, want, tol, ("gradient", n, entropy))
        assert not got[to_dev((ids < 0).all(-1), torch.bool)].any()
        same = logits.clone()
        ts.token_logprobs_listed_backward(same, tk, out, to_dev(a),
                                          None if h is None else to_dev(h), temperature,
                                          grad_logits=same)
        other = logits.clone()
        beside = ts.token_logprobs_listed_backward(logits, tk, out, to_dev(a),
                                                   None if h is None else to_dev(h), temperature,
                                                   grad_logits=other)
        assert torch.equal(same, beside)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_listed_most_ids(dtype):
    """TS_MAX_LISTED ids, all the same one and all different."""
    import torch

    import top_sampling_amd as ts

    rows, vocab, n = 3, 5000, ts.TS_MAX_LISTED
    logits, x = make_logits(rows, vocab, dtype, 0, 21, masks=False)
    ids = np.stack([np.full(n, 17), np.arange(n) * 4, np.arange(n)[::-1] + 3000])
    out = ts.token_logprobs_listed(logits, to_dev(ids, torch.int32))
    lp, _, _ = ref.listed(x, ids)
    close(out.logprobs, lp, LSE + U * np.abs(lp), "listed")
    a = np.random.default_rng(2).normal(size=(rows, n)).astype(np.float32)
    want = ref.listed_gradient(x, ids, 1.0, a.astype(np.float64))
    got = ts.token_logprobs_listed_backward(logits, to_dev(ids, torch.int32), out, to_dev(a))
    p = np.exp(log_softmax(x, 1.0))
    listed = np.zeros_like(x)
    for r in range(rows):
        np.add.at(listed[r], ids[r], np.abs(a[r]))
    tol = grad_tol(want, x, 1.0, dtype, 2 * LSE) + \
        np.abs(a).sum(-1)[:, None] * p * 2 * LSE + listed * LSE
    close(got, want, tol, "gradient")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(2, 700), (5, 20000), (3, 151936), (300, 40000)])
def test_digits_next_to_probability_1(rows, vocab, dtype):
    """1 - p down to 1e-9: every term of S - 1 is relatively within LSE, and so is
    ln S = -lp; the gradient's own entry is g (1 - p)."""
    import torch

    import top_sampling_amd as ts

    logits, x = make_logits(rows, vocab, dtype, 0, 31, masks=False)
    g = np.random.default_rng(32)
    tok = g.integers(0, vocab, rows)
    x[np.arange(rows), tok] = np.round(x.max(-1) + np.log(vocab) + g.uniform(5, 20, rows))
    logits.copy_(torch.from_numpy(x))
    x = logits.cpu().double().numpy()
    z = x - x.max(-1, keepdims=True)
    z[np.arange(rows), tok] = -np.inf
    rest = np.exp(z).sum(-1)
    lp = -np.log1p(rest)
    tk = to_dev(tok, torch.int32)
    # S = 1 + (1 - p) is a sum in double: at most 100 additions lie on the token's
    # way (a thread's batches, lanes, waves, a row's records), each off by 2^-53.
    tol = np.abs(lp) * (LSE + 2 * U) + 100 * 2.0 ** -53
    for n in (0, 1, 5):
        out = ts.token_logprobs_topn(logits, tk, n)
        torch.cuda.synchronize()
        close(out.logprobs, lp, tol, ("token", n))
        if n:
            close(out.topn_logprobs[:, 0], lp, tol, ("first alternative", n))
    # With another token asked for, the first alternative still has its digits.
    out = ts.token_logprobs_topn(logits, to_dev((tok + 1) % vocab, torch.int32), 2)
    close(out.topn_logprobs[:, 0], lp, tol, "beside another token")
    ids = np.stack([(tok + 1) % vocab, tok, np.full(rows, -1)], 1)
    out = ts.token_logprobs_listed(logits, to_dev(ids, torch.int32))
    close(out.logprobs[:, 1], lp, tol, "listed")
    a = np.zeros((rows, 3), np.float32)
    a[:, 1] = 1.5
    grad = ts.token_logprobs_listed_backward(logits, to_dev(ids, torch.int32), out, to_dev(a))
    own = grad[torch.arange(rows), tk.long()]
    want = 1.5 * rest / (1 + rest)
    close(own, want, want * (LSE + 4 * U + base.HALF[dtype]) + 150 * 2.0 ** -53, "own entry")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_every_alignment(dtype):
    """Rows that start at every place of a cache line, and odd leading dimensions."""
    import torch

    import top_sampling_amd as ts

    t = torch.float32 if dtype == "fp32" else torch.bfloat16
    per = 128 // t.itemsize
    for vocab in (1, 37, 1100, 5003):
        wide = torch.randn(3, vocab + per + 7, device="cuda").to(t)
        keep = wide.clone()
        for start in range(0, per, 3):
            logits = wide[:, start:start + vocab]
            x = logits.cpu().double().numpy()
            tok = np.array([0, vocab - 1, vocab // 2])
            got = ts.token_logprobs_topn(logits, to_dev(tok, torch.int32), 4, entropies=True)
            torch.cuda.synchronize()
            check_topn(got, ref.topn(x, tok, 4), (vocab, start))
            ids = np.stack([tok, tok[::-1]], 1)
            out = ts.token_logprobs_listed(logits, to_dev(ids, torch.int32))
            a = np.array([[1.0, 2.0], [0.5, -1.0], [1.0, 1.0]], np.float32)
            buf = torch.full_like(wide, 3.0)
            ts.token_logprobs_listed_backward(logits, to_dev(ids, torch.int32), out, to_dev(a),
                                              grad_logits=buf[:, start:start + vocab])
            want = ref.listed_gradient(x, ids, 1.0, a.astype(np.float64))
            tol = grad_tol(want, x, 1.0, dtype, 2 * LSE) + \
                np.exp(log_softmax(x, 1.0)) * 6 * LSE + 3 * LSE * (want != 0)
            close(buf[:, start:start + vocab], want, tol, (vocab, start))
            assert (buf[:, :start] == 3).all() and (buf[:, start + vocab:] == 3).all()
        assert torch.equal(wide, keep)


def test_one_long_row_past_32_bits():
    """The last row starts past 2^31 entries; a row of 2^24 entries."""
    import torch

    import top_sampling_amd as ts

    x = torch.zeros(3, (1 << 30) + 7, dtype=torch.bfloat16, device="cuda")
    part = x[:, :300]
    part.copy_(torch.randn(3, 300))
    want = ref.topn(part.cpu().double().numpy(), np.array([1, 2, 3]), 5)
    got = ts.token_logprobs_topn(part, torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda"), 5,
                                 entropies=True)
    check_topn(got, want, "far rows")
    del x, part
    x = torch.randn(1, 1 << 24, device="cuda")
    tok = x.argsort(dim=-1, descending=True, stable=True)[:, 41].to(torch.int32)
    got = ts.token_logprobs_topn(x, tok, 50)
    top = x.sort(dim=-1, descending=True, stable=True).indices[:, :50]
    assert torch.equal(got.topn_ids.long(), top) and int(got.ranks) == 42
    lp = (x.double() - torch.logsumexp(x.double(), -1, keepdim=True)).gather(1, top)
    close(got.topn_logprobs, lp.cpu().numpy(), LSE + 30 * U, "long row")


def test_streams_and_graphs():
    """On a stream of the caller's; captured, with a workspace that two graphs
    share, and replayed on new inputs with eager work between."""
    import torch

    import top_sampling_amd as ts

    rows, vocab, n = 9, 20011, 7
    logits, x = make_logits(rows, vocab, "fp32", 0, 41)
    tok = to_dev(allowed_tokens(x, 42), torch.int32)
    ids = to_dev(_some_ids(x, n, 43), torch.int32)
    a = torch.randn(rows, n, device="cuda")
    ws = torch.empty(max(ts.token_logprobs_topn_workspace_bytes(rows, vocab),
                         ts.token_logprobs_listed_workspace_bytes(rows, vocab)),
                     dtype=torch.uint8, device="cuda")

    def top():
        return ts.token_logprobs_topn(logits, tok, n, 0.9, entropies=True, workspace=ws)

    def back():
        out = ts.token_logprobs_listed(logits, ids, 0.9, workspace=ws)
        return out.logprobs, ts.token_logprobs_listed_backward(logits, ids, out, a,
                                                               temperature=0.9)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = ts.token_logprobs_topn(logits, tok, n, 0.9, entropies=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    here = top()
    assert torch.equal(other.topn_ids, here.topn_ids)
    assert torch.equal(other.topn_logprobs, here.topn_logprobs)
    back()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        c1 = top()
    with torch.cuda.graph(g2):
        c2 = back()
    for k in range(4):
        fresh, _ = make_logits(rows, vocab, "fp32", 0, 50 + k)
        logits.copy_(fresh)
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        held = [t.clone() for t in (c1.topn_ids, c1.topn_logprobs, c1.ranks, c1.logprobs,
                                    c1.entropies, *c2)]
        e1, e2 = top(), back()
        torch.cuda.synchronize()
        for got, want in zip(held, (e1.topn_ids, e1.topn_logprobs, e1.ranks, e1.logprobs,
                                    e1.entropies, *e2)):
            assert torch.equal(got.view(torch.int32), want.view(torch.int32)), k


def test_two_streams_at_once():
    import torch

    import top_sampling_amd as ts

    cases = []
    for k, (rows, vocab) in enumerate([(5, 60000), (300, 9000)]):
        logits, x = make_logits(rows, vocab, "bf16", 0, k)
        cases.append((logits, to_dev(allowed_tokens(x, k), torch.int32)))
    want = [ts.token_logprobs_topn(*c, 12, entropies=True) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(20):
        for k, (c, s) in enumerate(zip(cases, streams)):
            got[k].append(ts.token_logprobs_topn(*c, 12, entropies=True, stream=s))
    torch.cuda.synchronize()
    for k in range(2):
        for o in got[k]:
            assert torch.equal(o.topn_ids, want[k].topn_ids)
            assert torch.equal(o.topn_logprobs, want[k].topn_logprobs)
            assert torch.equal(o.ranks, want[k].ranks)


def test_row_stats_serve_the_other_backward_passes():
    import torch

    import top_sampling_amd as ts

    logits, x = make_logits(7, 9000, "fp32", 0, 61, masks=False)
    tok = to_dev(allowed_tokens(x, 62, skip=0.0), torch.int32)
    top = ts.token_logprobs_topn(logits, tok, 6)
    one = ts.token_logprobs(logits, tok)
    assert torch.equal(top.logprobs, one.logprobs) and torch.equal(top.row_stats, one.row_stats)
    a = torch.randn(7, 6, device="cuda")
    fwd = ts.TokenLogprobs(top.topn_logprobs, None, top.row_stats, None)
    got = ts.token_logprobs_listed_backward(logits, top.topn_ids, fwd, a)
    mine = ts.token_logprobs_listed(logits, top.topn_ids)
    assert torch.equal(got, ts.token_logprobs_listed_backward(logits, top.topn_ids, mine, a))
    g = torch.randn(7, device="cuda")
    single = ts.token_logprobs_listed(logits, tok[:, None].contiguous())
    grad = ts.token_logprobs_listed_backward(logits, tok[:, None].contiguous(), single, g[:, None].contiguous())
    close(grad, ts.token_logprobs_backward(logits, tok, one, g).cpu().double().numpy(),
          2 * LSE * g.abs().max().item(), "one listed token")


def test_outputs_stand_on_their_own():
    import torch

    import top_sampling_amd as ts

    logits, x = make_logits(4, 999, "fp32", 0, 71, masks=False)
    tok = to_dev(allowed_tokens(x, 72, skip=0.0), torch.int32)
    out = ts.token_logprobs_topn(logits, tok, 3, entropies=True)
    held = out.topn_logprobs.clone()
    versions = out.topn_logprobs._version
    out.logprobs.add_(1.0)
    out.topn_ids.zero_()
    assert torch.equal(out.topn_logprobs, held) and out.topn_logprobs._version == versions


SELECT = ("plain", "15 left", "500 at the lowest", "whole numbers", "two halves", "rising")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("vocab", (1000, 3001, 33000, 100277, 151936))
@pytest.mark.parametrize("n", (1, 48, 49, 128, 129, 257, 700, 1024))
def test_selection(dtype, vocab, n):
    """The alternatives' ids are exact, ties by id: few tokens left, equal logits in
    great number, order of ids against the order of the logits."""
    import torch

    import top_sampling_amd as ts

    say("selection", dtype, vocab, n)
    to = {"fp32": torch.float32, "bf16": torch.bfloat16}[dtype]
    gen = torch.Generator().manual_seed(vocab + n)
    rows = 3
    for kind in SELECT:
        x = 2.0 * torch.randn(rows, vocab, generator=gen)
        shut = torch.rand(rows, vocab, generator=gen).argsort(-1)
        if kind == "15 left":
            x.scatter_(1, shut[:, 15:], float("-inf"))
        elif kind == "500 at the lowest":
            x.scatter_(1, shut[:, 500:], torch.finfo(to).min)
        elif kind == "whole numbers":
            x = x.round()
        elif kind == "two halves":
            x = (torch.arange(vocab) >= vocab // 2).float().expand(rows, vocab)
        elif kind == "rising":
            x = torch.arange(vocab).float().expand(rows, vocab)
        x = x.to(to).contiguous()
        got = ts.token_logprobs_topn(x.cuda(), None, n).topn_ids.cpu()
        k = min(n, vocab)
        want = (-x.double() + 0.0).argsort(dim=-1, stable=True)[:, :k].int()
        assert torch.equal(got[:, :k], want), kind
        assert (got[:, k:] == -1).all(), kind


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [7, 140])
def test_many_long_rows(dtype, n):
    import torch

    import top_sampling_amd as ts

    rows, vocab = 520, 33333
    say("many long rows", dtype, n)
    logits, x = make_logits(rows, vocab, dtype, 3, n)
    tok = allowed_tokens(x, 5)
    tok[::50] = -1
    got = ts.token_logprobs_topn(logits, to_dev(tok, torch.int32), n, 0.7, entropies=True)
    torch.cuda.synchronize()
    check_topn(got, ref.topn(x, tok, n, 0.7), n)


@pytest.mark.parametrize("rows", [0, 3])
def test_outputs_that_are_not_asked_for(rows):
    """None without tokens and without entropies, whatever the number of rows."""
    import torch

    import top_sampling_amd as ts

    logits = torch.zeros(rows, 70, device="cuda")
    got = ts.token_logprobs_topn(logits, None, 2)
    assert got.logprobs is None and got.ranks is None and got.entropies is None
    assert got.topn_ids.shape == got.topn_logprobs.shape == (rows, 2)
    tok = torch.zeros(rows, dtype=torch.int32, device="cuda")
    got = ts.token_logprobs_topn(logits, tok, 2, entropies=True)
    assert got.logprobs.shape == got.ranks.shape == got.entropies.shape == (rows,)
    assert got.row_stats.shape == (rows, 2) and got.row_status.shape == (rows,)
