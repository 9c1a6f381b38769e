"""4-bit rows (OCP MX FP4) and the projection from them on the GPU, against
oracle/e2m1.py.

Codes, scales and the values they stand for are equal bit for bit.  Logits are
equal bit for bit where every partial sum is a whole number below 2^24 times one
power of two (nothing is rounded then, in any order), and otherwise within
K * 2^-23 * sum |x w|: K additions of exact products, each off by at most a step
of 2^-23 of a partial sum, which is at most sum |x w|.
"""
import numpy as np
import pytest
import torch

import top_sampling_amd as ts
from oracle import e2m1 as ref

pytestmark = pytest.mark.gpu

TILES = ["", "1", "2", "3", "4", "5"]


@pytest.fixture(params=TILES)
def tile(request, monkeypatch):
    if request.param:
        monkeypatch.setenv("TS_GEMM_TILE", request.param)
    else:
        monkeypatch.delenv("TS_GEMM_TILE", raising=False)
    return request.param


def _np(t):
    return t.cpu().to(torch.float64).numpy() if t.is_floating_point() else t.cpu().numpy()


def _check_quantize(x):
    """x on the GPU: codes, scales and values against the oracle."""
    codes, scales = ts.quantize_groups_e2m1(x)
    want_codes, want_scales = ref.quantize(_np(x))
    assert (_np(scales) == want_scales).all()
    assert (ref.unpack(_np(codes)) == want_codes).all()
    want = ref.values(want_codes, want_scales)
    for dtype in (torch.float32, torch.bfloat16):
        got = _np(ts.dequantize_groups_e2m1(codes, scales, dtype=dtype))
        assert np.array_equal(got, want, equal_nan=True)
        assert (np.signbit(got) == np.signbit(want))[~np.isnan(want)].all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (257, 64), (5, 2048), (33, 4128)])
def test_quantize(rows, cols, dtype):
    gen = torch.Generator(device="cuda").manual_seed(rows * cols)
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x *= torch.exp2(torch.randint(-20, 20, (rows, cols // 32), generator=gen, device="cuda")
                    .float()).repeat_interleave(32, 1)
    _check_quantize(x.to(dtype))


def test_quantize_every_bf16():
    """Every bf16 number in a group of scale 1, 2^-127, 2^124 and in one of its own."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = bits[torch.isfinite(bits)].cuda()
    for top in (7.0, 2.0 ** -126, 6.0 * 2.0 ** 124):
        part = x[x.abs() <= top]
        part = part[: part.numel() // 31 * 31].reshape(-1, 31)
        first = torch.full((part.shape[0], 1), top, dtype=torch.bfloat16, device="cuda")
        _check_quantize(torch.cat([first, part], 1))
    _check_quantize(x[: x.numel() // 32 * 32].reshape(-1, 32))


def test_quantize_ties_and_borders():
    """fp32 numbers at and one step beside every border between codes and scales."""
    at = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0])
    near = torch.cat([at, torch.nextafter(at, torch.zeros(9)),
                      torch.nextafter(at, torch.full((9,), 9.0))])
    for scale in (1.0, 2.0 ** -100, 2.0 ** 100):
        for top in (7.0, 6.0, 4.0):
            rows = []
            for v in near[near <= top]:
                row = torch.zeros(32)
                row[0], row[1], row[2] = top, v, -v
                rows.append(row)
            _check_quantize((torch.stack(rows) * scale).cuda())
    # The largest magnitude at the border between two scales.
    rows = torch.zeros(27, 32)
    rows[:, 5] = near
    _check_quantize(rows.cuda())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_special_groups(dtype):
    x = torch.ones(6, 96)
    x[0, 40] = float("nan")
    x[1, 3] = float("inf")
    x[2, 95] = -float("inf")
    x[3, 32:64] = 0.0
    x[4, 32:64] = -0.0
    x[5, :32] = 1e-44  # below the smallest scale's steps (0 in bf16)
    x[5, 64:] = torch.finfo(torch.bfloat16).max
    _check_quantize(x.to(dtype).cuda())


def test_dequantize_every_scale():
    codes = torch.arange(16, dtype=torch.uint8, device="cuda")
    packed = (codes | (codes.flip(0) << 4)).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8, device="cuda")[:, None].contiguous()
    want = ref.values(ref.unpack(_np(packed)), _np(scales))
    want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)
    for dtype in (torch.float32, torch.bfloat16):
        got = _np(ts.dequantize_groups_e2m1(packed, scales, dtype=dtype))
        assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_strides(dtype):
    """Columns of wider buffers at odd places; what lies around them stays."""
    wide = torch.randn(7, 101, device="cuda").to(dtype)
    x = wide[:, 3:67]
    codes = torch.full((7, 60), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((7, 5), 0xCD, dtype=torch.uint8, device="cuda")
    ts.quantize_groups_e2m1(x, codes=codes[:, 4:36], scales=scales[:, 1:3])
    want_codes, want_scales = ref.quantize(_np(x))
    assert (ref.unpack(_np(codes[:, 4:36])) == want_codes).all()
    assert (_np(scales[:, 1:3]) == want_scales).all()
    assert (codes[:, :4] == 0xAB).all() and (codes[:, 36:] == 0xAB).all()
    assert (scales[:, :1] == 0xCD).all() and (scales[:, 3:] == 0xCD).all()
    out = torch.full((7, 101), 9.0, device="cuda").to(dtype)
    ts.dequantize_groups_e2m1(codes[:, 4:36], scales[:, 1:3], out=out[:, 5:69])
    assert np.array_equal(_np(out[:, 5:69]), ref.values(want_codes, want_scales))
    assert (out[:, :5] == 9).all() and (out[:, 69:] == 9).all()


# ------------------------------------------------------------- projection
SHAPES = [(1, 32, 1), (1, 4096, 531), (2, 64, 33), (5, 2560, 257), (15, 96, 300), (16, 8192, 95),
          (17, 544, 129), (31, 4128, 70), (32, 256, 1000), (33, 1024, 260), (64, 160, 511),
          (65, 96, 257), (130, 2592, 300), (300, 64, 513), (321, 320, 258), (7, 8224, 40),
          # one to three parts of a row, whole and not, and several tiles a workgroup
          (64, 6144, 300), (45, 4640, 133), (20, 9216, 77), (9, 10240, 50), (3, 1024, 70),
          (30, 512, 9001), (64, 2048, 9001), (48, 4096, 4500), (16, 1536, 17000), (33, 8192, 4200)]


def _codes(rows, cols, gen, low=120, high=135):
    packed = torch.randint(0, 256, (rows, cols // 2), generator=gen, dtype=torch.uint8)
    scales = torch.randint(low, high, (rows, cols // 32), generator=gen, dtype=torch.uint8)
    return packed.cuda(), scales.cuda()


@pytest.mark.parametrize("rows,h,vocab", SHAPES)
def test_projection_whole_numbers(rows, h, vocab, tile):
    """Hidden entries 0, +-1, +-2 and scales 1 and 2: twice every partial sum is
    a whole number of at most 10240 * 2 * 12 * 2 < 2^24."""
    gen = torch.Generator().manual_seed(rows * h + vocab)
    w, s = _codes(vocab, h, gen, 127, 129)
    x = torch.randint(-2, 3, (rows, h), generator=gen).to(torch.bfloat16).cuda()
    got = ts.lmhead_logits_local_e2m1(x, w, s)
    assert np.array_equal(_np(got), ref.logits(_np(x), ref.unpack(_np(w)), _np(s)))


@pytest.mark.parametrize("rows,h,vocab", SHAPES)
def test_projection(rows, h, vocab, tile):
    gen = torch.Generator().manual_seed(rows + h * vocab)
    w, s = _codes(vocab, h, gen)
    x = torch.randn(rows, h, generator=gen).to(torch.bfloat16).cuda()
    got = _np(ts.lmhead_logits_local_e2m1(x, w, s))
    v = ref.values(ref.unpack(_np(w)), _np(s))
    assert (np.abs(got - _np(x) @ v.T) <= h * 2.0 ** -23 * (np.abs(_np(x)) @ np.abs(v).T)).all()


@pytest.mark.parametrize("rows", [3, 20, 70])
def test_projection_strides(rows, tile):
    """Leading dimensions wider than the rows, an output of odd alignment; what
    lies beside the logits stays, and what lies beside the inputs is not read as
    such."""
    gen = torch.Generator().manual_seed(5)
    h, vocab = 224, 149
    w, s = _codes(vocab, h + 32, gen, 127, 129)
    s[:, -1] = 255
    x = torch.randint(-2, 3, (rows, h + 8), generator=gen).to(torch.bfloat16).cuda()
    x[:, h:] = float("nan")
    out = torch.full((rows, vocab + 6), 7.0, device="cuda")
    got = ts.lmhead_logits_local_e2m1(x[:, :h], w[:, :h // 2], s[:, :h // 32], out=out[:, 3:-3])
    want = ref.logits(_np(x[:, :h]), ref.unpack(_np(w[:, :h // 2])), _np(s[:, :h // 32]))
    assert np.array_equal(_np(got), want)
    assert (out[:, :3] == 7).all() and (out[:, -3:] == 7).all()


@pytest.mark.parametrize("rows", [2, 18, 66])
def test_projection_special_values(rows, tile):
    """NaN and infinities stay in their own rows and columns; scales at both ends."""
    gen = torch.Generator().manual_seed(6)
    h, vocab = 96, 70  # a last step of one group
    w, s = _codes(vocab, h, gen, 127, 129)
    x = torch.randint(-2, 3, (rows, h), generator=gen).to(torch.bfloat16).cuda()
    s[7, 2] = 255
    x[0, 95] = float("inf")
    x[1, 3] = float("nan")
    got = _np(ts.lmhead_logits_local_e2m1(x, w, s))
    with np.errstate(invalid="ignore"):
        want = ref.logits(_np(x), ref.unpack(_np(w)), _np(s))
    assert np.array_equal(got, want, equal_nan=True)
    assert np.isnan(got[:, 7]).all() and np.isnan(got[1]).all()
    assert np.isfinite(np.delete(got[2:], 7, axis=1)).all()
    # One entry each: 2^-127 with hidden 2^126, 2^120 with 2^-120.
    w.zero_()
    s.fill_(127)
    x.zero_()
    w[0, 0], s[0, 0], x[0, 0] = 1, 0, 2.0 ** 126      # 0.5 * 2^-127 * 2^126
    w[1, 16], s[1, 1], x[0, 32] = 7, 247, 2.0 ** -120  # 6 * 2^120 * 2^-120
    got = _np(ts.lmhead_logits_local_e2m1(x, w, s))
    assert got[0, 0] == 0.25 and got[0, 1] == 6.0 and not got[0, 2:].any() and not got[1:].any()


def test_projection_places_past_32_bits():
    """Codes and logits whose places in their buffers pass 2^31 bytes and entries."""
    gen = torch.Generator().manual_seed(8)
    h, vocab = 64, 40
    w, s = _codes(vocab, h, gen, 127, 129)
    x = torch.randint(-2, 3, (3, h), generator=gen).to(torch.bfloat16).cuda()
    far = torch.zeros(vocab, (1 << 27) + 16, dtype=torch.uint8, device="cuda")
    far[:, :h // 2] = w
    out = torch.zeros(3, (1 << 30) + 5, device="cuda")
    got = ts.lmhead_logits_local_e2m1(x, far[:, :h // 2], s, out=out[:, :vocab])
    assert np.array_equal(_np(got), ref.logits(_np(x), ref.unpack(_np(w)), _np(s)))


def test_other_stream_and_graph():
    """On a stream of the caller's, and captured and replayed on new inputs."""
    gen = torch.Generator().manual_seed(9)
    w, s = _codes(300, 256, gen, 127, 129)
    x = torch.zeros(5, 256, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(5, 300, device="cuda")
    back = torch.zeros(300, 256, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ts.lmhead_logits_local_e2m1(x, w, s, out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    codes, scales = torch.empty_like(w), torch.empty_like(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ts.dequantize_groups_e2m1(w, s, out=back)
        ts.quantize_groups_e2m1(back, codes=codes, scales=scales)
        ts.lmhead_logits_local_e2m1(x, codes, scales, out=out)
    for k in range(3):
        x.copy_(torch.randint(-2, 3, (5, 256), generator=gen))
        w2, s2 = _codes(300, 256, gen, 127, 129)
        w.copy_(w2)
        s.copy_(s2)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(_np(out), ref.logits(_np(x), ref.unpack(_np(w)), _np(s)))


@pytest.mark.parametrize("groups", range(7, 42))
def test_projection_every_row_length(groups, tile):
    """Whole numbers, as above; every remainder of a row's scales over what is
    loaded of them at a time, the last rows at the buffer's end."""
    gen = torch.Generator().manual_seed(groups)
    for rows, vocab in ((40, 70), (70, 300)):
        w, s = _codes(vocab, 32 * groups, gen, 127, 129)
        x = torch.randint(-2, 3, (rows, 32 * groups), generator=gen).to(torch.bfloat16).cuda()
        got = ts.lmhead_logits_local_e2m1(x, w, s)
        assert np.array_equal(_np(got), ref.logits(_np(x), ref.unpack(_np(w)), _np(s))), rows


# (rows, H, V): parts of a row x waves, whole or not, and the most tiles of 16 columns that
# one of 256 workgroups takes.
PARTS = [(9, 10240, 21001),  # 2 x 5 whole, 6 tiles
         (5, 8224, 8300),    # 2 x 5, 3
         (20, 9216, 13001),  # 3 x 6 whole, 4
         (31, 4128, 25001),  # 2 x 5, 7
         (18, 14336, 4500),  # 4 x 7 whole, 2
         (2, 25600, 4200)]   # 4 x 7, 2


@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("rows,h,vocab", PARTS)
def test_projection_parts_of_rows(rows, h, vocab, pad, monkeypatch):
    """Few rows whose entries the waves do not hold at once: the sums of one part come
    back from the logits in the next, over several tiles a workgroup with a ragged last
    one, into rows that take whole stores and rows that do not.  Whole numbers, as above:
    twice a partial sum is at most 25600 * 2 * 12 * 2 < 2^24."""
    monkeypatch.delenv("TS_GEMM_TILE", raising=False)
    gen = torch.Generator().manual_seed(rows * h + vocab + pad)
    w, s = _codes(vocab, h, gen, 127, 129)
    x = torch.randint(-2, 3, (rows, h), generator=gen).to(torch.bfloat16).cuda()
    wide = torch.full((rows, vocab + 2 * pad), float("nan"), device="cuda")
    out = wide[:, pad:pad + vocab]
    first = ts.lmhead_logits_local_e2m1(x, w, s, out=out).clone()
    # Over the finished logits of another call, as a buffer that is used again.
    ts.lmhead_logits_local_e2m1(x, w, s, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    if pad:
        assert torch.isnan(wide[:, :pad]).all() and torch.isnan(wide[:, -pad:]).all()
    for at in range(0, vocab, 2048):
        part = slice(at, min(at + 2048, vocab))
        want = ref.logits(_np(x), ref.unpack(_np(w[part])), _np(s[part]))
        assert np.array_equal(_np(first[:, part]), want), at


@pytest.mark.parametrize("rows", [2, 40, 70])
def test_projection_ends_of_the_numbers(rows, tile):
    """Entries past the largest number are infinite, as dequantize_groups_e2m1 gives them,
    and the largest below are not; hidden entries below 2^-126 keep their value."""
    h, vocab = 64, 70
    w = torch.zeros(vocab, h // 2, dtype=torch.uint8, device="cuda")
    s = torch.full((vocab, h // 32), 127, dtype=torch.uint8, device="cuda")
    # 2 and 1 times 2^127, 6 and 3 times 2^126, -4 times 2^126, 1 times 2^120
    for v, (code, byte) in enumerate([(4, 254), (2, 254), (7, 253), (5, 253), (14, 253), (2, 247)]):
        w[v, 0], s[v, 0] = code, byte
    x = torch.zeros(rows, h, dtype=torch.bfloat16, device="cuda")
    x[0, 0], x[1, 0] = 2.0 ** -30, -(2.0 ** -133)
    values = ts.dequantize_groups_e2m1(w, s)
    assert torch.isinf(values[[0, 2, 4], 0]).all() and torch.isfinite(values[[1, 3, 5]]).all()
    with np.errstate(invalid="ignore"):
        want = _np(x) @ _np(values).T
    got = _np(ts.lmhead_logits_local_e2m1(x, w, s))
    assert np.array_equal(got, want, equal_nan=True)
    assert got[0, 1] == 2.0 ** 97 and got[1, 5] == -(2.0 ** -13) and np.isnan(got[rows - 1, 0]) \
        == (rows > 2)
