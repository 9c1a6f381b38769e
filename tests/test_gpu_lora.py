"""The adapter projection on the GPU against the float64 oracle.

Tolerance.  An fp32 sum of n products of random signs and size s is off by
about 0.41 u n s (u = 2^-24: a rounding of u / sqrt(3) at each of the n partial
sums, which grow as sqrt(i) s); six times that is allowed, for the base sum
(n = H), for u (n = H, carried through B) and for the sum over the rank.  The
three bf16 parts of u keep 24 bits, and the sum and the result are rounded
once more.  A u that were rounded to bf16 would be off by 2^-9 of the
adapter's share, hundreds of times as much.
"""
import numpy as np
import pytest

from oracle import losses as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def say(*a):
    print(*a, flush=True)


def _dev():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda:0")


def make(rows, hidden, vocab, rank, n, seed, pad=0):
    """Device tensors (rows `pad` * 8 elements apart from dense) and scales."""
    import torch

    g = torch.Generator(device="cpu")
    g.manual_seed(seed)

    def bf(*shape, std):
        wide = torch.zeros(*shape[:-1], shape[-1] + 8 * pad, dtype=torch.bfloat16)
        wide[..., :shape[-1]] = (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)
        return wide.to(_dev())[..., :shape[-1]]

    return (bf(rows, hidden, std=1.0), bf(vocab, hidden, std=0.05),
            bf(n, rank, hidden, std=hidden ** -0.5), bf(n, vocab, rank, std=0.2),
            (torch.rand(n, generator=g) * 3 + 0.1).to(_dev()))


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def check(got, x, w, a, b, ids, scales):
    n, rank = a.shape[:2]
    xs, ws, as_, bs = f64(x), f64(w), f64(a), f64(b)
    sc = np.ones(n) if scales is None else f64(scales)
    want = ref.lora_logits(xs, ws, as_, bs, ids, sc)
    hidden = xs.shape[1]
    rms = lambda m: np.sqrt((m * m).mean())  # noqa: E731
    six = 6 * 0.41 * U
    row = np.sqrt((xs * xs).mean(1))
    tol = (six * hidden * row * rms(ws))[:, None] + 2 * U * np.abs(want)
    live = (ids >= 0) & (ids < n)
    u = np.zeros((len(ids), rank))
    for r in np.flatnonzero(live):
        u[r] = sc[ids[r]] * (as_[ids[r]] @ xs[r])
    du = np.where(live, six * hidden * row * rms(as_) * sc[np.clip(ids, 0, n - 1)], 0)
    # carried through B at random signs, and the sum over the rank
    size = rms(bs)
    tol += (6 * du * size * np.sqrt(rank) + six * (rank + 4) * np.abs(u).max(1) * size
            + 8 * U * np.abs(u).max(1) * np.abs(bs).max() * np.sqrt(rank))[:, None]
    got = got.double().cpu().numpy()
    both = np.isnan(got) & np.isnan(want)
    off = np.where(both, 0, np.abs(got - want) - tol)
    off = np.where(np.isnan(off), np.inf, off)
    i = np.unravel_index(off.argmax(), off.shape)
    assert off[i] <= 0, (i, got[i], want[i], tol[i] if tol.shape == off.shape else tol[i[0]])


def some_ids(kind, rows, n, seed):
    g = np.random.default_rng(seed)
    ids = {"random": lambda: g.integers(-1, n, rows), "none": lambda: np.full(rows, -1),
           "one": lambda: np.full(rows, n - 1), "sorted": lambda: np.sort(g.integers(-1, n, rows)),
           "bad": lambda: g.choice([-1, 0, n - 1, n, -2, 2 ** 31 - 1, -2 ** 31], rows),
           "runs": lambda: np.repeat(g.integers(-1, n, rows // 5 + 1), 5)[:rows]}[kind]()
    return ids.astype(np.int64)


CASES = [
    # rows, hidden, vocab, rank, adapters, pad, ids
    (1, 64, 1, 8, 1, 0, "one"), (1, 256, 1000, 16, 4, 0, "random"), (3, 128, 7, 8, 2, 1, "random"),
    (33, 256, 130, 24, 5, 0, "random"), (64, 4096, 515, 16, 32, 0, "random"),
    (64, 64, 300, 256, 3, 0, "runs"), (65, 192, 129, 64, 70, 0, "random"),
    (128, 512, 257, 40, 9, 1, "sorted"), (128, 64, 64, 8, 128, 0, "random"),
    (200, 320, 511, 16, 3, 0, "none"), (300, 256, 260, 32, 300, 0, "random"),
    (320, 128, 400, 16, 1, 0, "one"), (640, 256, 700, 32, 16, 0, "runs"),
    (641, 128, 100, 48, 7, 0, "random"), (50, 128, 90, 16, 4, 0, "bad"),
    (700, 64, 33, 8, 6, 0, "bad"),
    # wider vocabularies, for every tile shape: 64 x 128 and 128 x 128 with many
    # stages and with two, of few tiles and of many, 256 and 320 rows
    (60, 128, 25001, 16, 9, 0, "random"), (90, 192, 22300, 40, 12, 0, "runs"),
    (64, 320, 33100, 24, 64, 0, "random"), (5, 64, 40000, 8, 2, 0, "bad"),
    (100, 128, 66000, 16, 7, 0, "random"), (133, 192, 31040, 64, 9, 0, "bad"),
    (256, 128, 60001, 32, 256, 0, "random"), (320, 128, 60000, 24, 20, 1, "runs"),
    (310, 64, 60100, 8, 3, 0, "bad"), (250, 64, 60002, 16, 1, 0, "none"),
    # 64 x 64, 128 x 128 with many rows
    (60, 192, 10001, 16, 9, 0, "random"), (130, 64, 3333, 24, 130, 1, "bad"),
    (320, 448, 9500, 40, 30, 0, "runs"), (64, 64, 11000, 256, 64, 0, "random"),
    # 192 x 128, 192 x 256, one round of 128 x 128, two row tiles of 320
    (150, 128, 22100, 16, 9, 0, "random"), (190, 192, 60001, 24, 40, 1, "bad"),
    (192, 64, 40010, 72, 192, 0, "random"), (300, 64, 18993, 8, 30, 0, "random"),
    (640, 64, 30001, 16, 64, 0, "runs"),
    # several row tiles of 64 x 128, 192 x 128, 192 x 256 and 256 x 256
    (90, 64, 9500, 16, 9, 0, "random"), (370, 128, 16001, 24, 30, 0, "random"),
    (384, 64, 60001, 16, 7, 0, "bad"), (512, 64, 31000, 8, 5, 0, "runs"),
    # hidden sizes that are no multiple of 64
    (5, 72, 33, 8, 2, 0, "random"), (70, 200, 300, 24, 9, 1, "runs"), (260, 136, 140, 64, 5, 0, "bad"),
]


@pytest.mark.parametrize("rows,hidden,vocab,rank,n,pad,kind", CASES)
def test_lora_logits(rows, hidden, vocab, rank, n, pad, kind):
    import torch

    import top_sampling_amd as ts

    say("lora", rows, hidden, vocab, rank, n, pad, kind)
    x, w, a, b, scales = make(rows, hidden, vocab, rank, n, rows + hidden, pad)
    ids = some_ids(kind, rows, n, 7)
    dev_ids = torch.from_numpy(ids.astype(np.int32)).to(_dev())
    wide = torch.full((rows, vocab + 3), 7.0, device=_dev())
    got = ts.lmhead_logits_local_lora(x, w, a, b, dev_ids, scales, out=wide[:, :vocab])
    torch.cuda.synchronize()
    assert (wide[:, vocab:] == 7.0).all()
    check(got, x, w, a, b, ids, scales)
    dense = ts.lmhead_logits_local_lora(x, w, a, b, dev_ids, scales)
    same = ts.lmhead_logits_local_lora(x, w, a, b, dev_ids, scales)
    torch.cuda.synchronize()
    nan = torch.isnan(dense)
    assert torch.equal(torch.isnan(got), nan) and torch.equal(dense[~nan], same[~nan])
    assert torch.equal(dense[~nan], got[~nan])
    # rows without an adapter are exactly the shared projection
    base = ts.lmhead_logits_local(x, w)
    none = torch.from_numpy(ids == -1).to(_dev())
    assert torch.equal(dense[none], base[none])
    if n > 1:
        check(ts.lmhead_logits_local_lora(x, w, a, b, dev_ids), x, w, a, b, ids, None)


def test_vocabulary_slices_and_strides():
    """A rank's vocabulary slice of the lm_head and of every adapter's B, in
    place, written into its columns of a wider buffer."""
    import torch

    import top_sampling_amd as ts

    rows, hidden, vocab, rank, n = 70, 256, 900, 16, 6
    x, w, a, b, scales = make(rows, hidden, vocab, rank, n, 1)
    ids = torch.from_numpy(some_ids("random", rows, n, 2).astype(np.int32)).to(_dev())
    whole = ts.lmhead_logits_local_lora(x, w, a, b, ids, scales)
    parts = torch.empty_like(whole)
    for lo, hi in ((0, 300), (300, 301), (301, 900)):
        ts.lmhead_logits_local_lora(x, w[lo:hi], a, b[:, lo:hi], ids, scales,
                                    out=parts[:, lo:hi])
    torch.cuda.synchronize()
    assert torch.equal(whole, parts)


@pytest.mark.parametrize("hidden", [256, 264])
def test_rows_do_not_reach_each_other(hidden):
    """A row's logits are bit for bit those of its own call, whatever stands
    beside it: other adapters, in any order, with infinities and NaN."""
    import torch

    import top_sampling_amd as ts

    rows, vocab, rank, n = 90, 333, 24, 5
    x, w, a, b, scales = make(rows, hidden, vocab, rank, n, 3)
    ids = torch.from_numpy(some_ids("random", rows, n, 4).astype(np.int32)).to(_dev())
    clean = ts.lmhead_logits_local_lora(x, w, a, b, ids, scales)
    order = torch.randperm(rows, device=_dev())
    mixed = ts.lmhead_logits_local_lora(x[order].contiguous(), w, a, b, ids[order].contiguous(),
                                        scales)
    assert torch.equal(mixed, clean[order])
    b[1] = float("nan")
    a[2, 3] = float("inf")
    x[11] = float("nan")
    got = ts.lmhead_logits_local_lora(x, w, a, b, ids, scales)
    torch.cuda.synchronize()
    keep = (ids != 1) & (ids != 2)
    keep[11] = False
    assert torch.equal(got[keep], clean[keep])
    assert torch.isnan(got[ids == 1]).all() and torch.isnan(got[11]).all()


@pytest.mark.parametrize("rows,vocab", [(5, 300), (5, 40000), (60, 10001), (60, 25001), (64, 33100),
                                        (90, 22300), (100, 66000), (150, 22100), (190, 60001),
                                        (300, 18993), (256, 60001), (640, 30001)])
def test_infinities_in_b(rows, vocab):
    """On every tile shape: an infinity in an adapter's B makes that entry of
    its rows infinite with u's sign, and changes no other bit."""
    import torch

    import top_sampling_amd as ts

    rank, n = 24, 7
    x, w, a, b, scales = make(rows, 64, vocab, rank, n, rows)
    ids = torch.from_numpy(some_ids("random", rows, n, 2).astype(np.int32)).to(_dev())
    clean = ts.lmhead_logits_local_lora(x, w, a, b, ids, scales)
    cols = torch.tensor([0, 17, vocab // 2, vocab - 1], device=_dev())
    b[1, cols, 19] = float("inf")
    got = ts.lmhead_logits_local_lora(x, w, a, b, ids, scales)
    own = ids == 1
    u = x[own].double() @ a[1, 19].double()
    want = clean.clone()
    want[own.nonzero(), cols] = (u.sign() * float("inf")).float()[:, None]
    assert torch.equal(got, want)


@pytest.mark.parametrize("hidden", [128, 136])
def test_infinite_inner_sums(hidden):
    """An infinity in A makes u infinite, and the logits infinite with B's sign
    (NaN where B is 0), as the formula has it."""
    import torch

    import top_sampling_amd as ts

    rows, vocab, rank, n = 40, 150, 8, 2
    x, w, a, b, _ = make(rows, hidden, vocab, rank, n, 9)
    a[1, 5, 7] = float("inf")
    x[:, 7] = x[:, 7].abs() + 0.5
    b[1, 3:9] = 0
    ids = torch.arange(rows, dtype=torch.int32, device=_dev()) % 2
    got = ts.lmhead_logits_local_lora(x, w, a, b, ids).cpu()
    sign = b[1, :, 5].float().cpu()
    assert torch.isfinite(got[::2]).all()
    want = torch.where(sign == 0, float("nan"), sign * float("inf"))
    assert torch.equal(torch.isnan(got[1::2]), torch.isnan(want).expand(rows // 2, -1))
    assert torch.equal(got[1::2].nan_to_num(0.0), want.expand(rows // 2, -1).nan_to_num(0.0))


def test_streams_and_graph():
    import torch

    import top_sampling_amd as ts

    rows, hidden, vocab, rank, n = 20, 256, 4099, 16, 4
    x, w, a, b, scales = make(rows, hidden, vocab, rank, n, 5)
    ids = torch.from_numpy(some_ids("random", rows, n, 6).astype(np.int32)).to(_dev())
    plain = ts.lmhead_logits_local_lora(x, w, a, b, ids, scales)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ts.lmhead_logits_local_lora(x, w, a, b, ids, scales, stream=side)
    side.synchronize()
    assert torch.equal(plain, got)
    static_x, static_ids = x.clone(), ids.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ts.lmhead_logits_local_lora(static_x, w, a, b, static_ids, scales)
    for i in range(4):
        static_x.copy_(x * (1 + i))
        static_ids.copy_((ids + i) % n)
        graph.replay()
        want = ts.lmhead_logits_local_lora(static_x, w, a, b, static_ids, scales)
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def test_adapter_offsets_pass_32_bits():
    """Adapters 2^31 elements and more apart in one buffer (9 GB)."""
    import torch

    import top_sampling_amd as ts

    rows, hidden, vocab, rank, n = 9, 64, 200, 16, 3
    x, w, a, b, scales = make(rows, hidden, vocab, rank, n, 8)
    ids = torch.tensor([0, 1, 2, 2, -1, 1, 0, 2, 1], dtype=torch.int32, device=_dev())
    want = ts.lmhead_logits_local_lora(x, w, a, b, ids, scales)
    step = (1 << 31) + 64
    buf = torch.empty(2 * step + vocab * rank, dtype=torch.bfloat16, device=_dev())
    far = buf.as_strided((n, vocab, rank), (step, rank, 1))
    far.copy_(b)
    got = ts.lmhead_logits_local_lora(x, w, a, far, ids, scales)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_sampler_reports_a_bad_adapter():
    import torch

    import top_sampling_amd as ts
    import workloads

    rows, hidden, vocab = 6, 128, 4096
    x, w, a, b, scales = make(rows, hidden, vocab, 16, 2, 9)
    ids = torch.tensor([0, 5, -1, 1, -7, 0], dtype=torch.int32, device=_dev())
    logits = ts.lmhead_logits_local_lora(x, w, a, b, ids, scales)
    params = np.zeros(rows, dtype=workloads.PARAMS_DTYPE)
    params["temperature"], params["top_p"] = 1.0, 1.0
    out = ts.sampler_sample(logits, ts.params_to_device(params, _dev()))
    torch.cuda.synchronize()
    assert out.row_status.tolist() == [0, ts.TS_ROW_BAD_LOGITS, 0, 0, ts.TS_ROW_BAD_LOGITS, 0]


@pytest.mark.parametrize("rows,vocab", [(5, 300), (5, 40000), (60, 10001), (60, 25001), (64, 33100),
                                        (90, 22300), (100, 66000), (150, 22100), (190, 60001),
                                        (300, 18993), (256, 60001), (640, 30001)])
@pytest.mark.parametrize("hidden", [64, 72])
def test_infinite_inner_sums_and_infinities_in_b(rows, vocab, hidden):
    """On every tile shape, and in the second pass of other hidden sizes: an
    infinite u and infinite entries of B, of the same rank and of others, give
    what the formula has, the sum of the products' infinities (NaN where two of
    them differ in sign, or where one meets a 0)."""
    import torch

    import top_sampling_amd as ts

    rank, n = 24, 7
    x, w, a, b, scales = make(rows, hidden, vocab, rank, n, rows)
    ids = torch.from_numpy(some_ids("random", rows, n, 2).astype(np.int32)).to(_dev())
    a[1, 5, 7] = float("inf")
    x[:, 7] = x[:, 7].abs() + 0.5
    # column 0: B infinite at the rank of the infinite u; 17: at another rank
    # whose u is finite; the middle: both; the last: infinite at the first, and
    # 0 at the infinite u's
    mid, end = vocab // 2, vocab - 1
    b[1, 0, 5] = -float("inf")
    b[1, 17, 19] = float("inf")
    b[1, mid, 5], b[1, mid, 19] = float("inf"), float("inf")
    b[1, end, 0], b[1, end, 5] = float("inf"), 0.0
    got = ts.lmhead_logits_local_lora(x, w, a, b, ids, scales)
    torch.cuda.synchronize()
    own = ids == 1
    # the same rows' finite u, from the formula in float64
    u = x[own].double() @ a[1].double().t()
    assert torch.isinf(u[:, 5]).all() and torch.isfinite(u[:, [0, 19]]).all()
    terms = u[:, None, :] * b[1].double()[None, [0, 17, mid, end, 1]]
    want = torch.where(torch.isfinite(terms), 0.0, terms).sum(-1)
    # a base sum is finite: infinities decide
    at = got[own][:, [0, 17, mid, end, 1]].double()
    assert torch.equal(torch.isnan(at), torch.isnan(want))
    assert torch.equal(at.nan_to_num(0.0), want.nan_to_num(0.0))
    # every other column has the sign of B's entry at the infinite u
    rest = torch.ones(vocab, dtype=torch.bool, device=_dev())
    rest[[0, 17, mid, end]] = False
    sign = b[1, rest, 5].float()
    sign = torch.where(sign == 0, float("nan"), sign * float("inf")).expand(int(own.sum()), -1)
    assert torch.equal(got[own][:, rest].nan_to_num(0.0), sign.nan_to_num(0.0))
    # and rows of other adapters keep their bits (x[:, 7] is theirs too)
    a[1, 5, 7], b[1] = 0.0, 0.0
    clean = ts.lmhead_logits_local_lora(x, w, a, b, ids, scales)
    assert torch.equal(got[~own], clean[~own])


@pytest.mark.parametrize("rows,hidden,vocab,rank,n", [
    # many row tiles, ranks above 64, and more rows than a launch of the down
    # step or of the second pass has workgroups for
    (3000, 192, 70, 256, 9), (5001, 64, 300, 8, 40), (2050, 136, 130, 136, 3),
    (70001, 72, 5, 16, 6), (70001, 64, 5, 16, 6), ((1 << 18) + 77, 64, 3, 8, 5),
])
def test_many_rows(rows, hidden, vocab, rank, n):
    import torch

    import top_sampling_amd as ts

    say("lora rows", rows, hidden, vocab, rank, n)
    x, w, a, b, scales = make(rows, hidden, vocab, rank, n, 4)
    ids = torch.from_numpy(some_ids("bad", rows, n, 7).astype(np.int32)).to(_dev())
    got = ts.lmhead_logits_local_lora(x, w, a, b, ids, scales)
    torch.cuda.synchronize()
    xs, want = x.double(), x.double() @ w.double().t()
    u = torch.zeros(rows, rank, dtype=torch.float64, device=_dev())
    for i in range(n):
        mine = (ids == i).nonzero()[:, 0]
        u[mine] = scales[i].double() * (xs[mine] @ a[i].double().t())
        want[mine] += u[mine] @ b[i].double().t()
    out = (ids < -1) | (ids >= n)
    assert torch.isnan(got[out]).all()
    # the bound of check(), row by row
    six = 6 * 0.41 * U
    rms = lambda m: m.double().square().mean().sqrt()  # noqa: E731
    row = xs.square().mean(1).sqrt()
    top = u.abs().amax(1)
    du = torch.where((ids >= 0) & ~out, six * hidden * row * rms(a) *
                     scales.double()[ids.clamp(0, n - 1).long()], 0.0)
    tol = six * hidden * row * rms(w) + 6 * du * rms(b) * rank ** 0.5 + \
        six * (rank + 4) * top * rms(b) + 8 * U * top * b.double().abs().max() * rank ** 0.5
    off = (got.double() - want).abs() - tol[:, None] - 2 * U * want.abs()
    assert (off[~out] <= 0).all()
