"""4-bit rows on the CPU: the oracle by hand, and the refusals of the C ABI and
the binding (validation runs before any HIP call)."""
import numpy as np
import pytest

import top_sampling_amd as ts
from oracle import e2m1 as ref

FAKE = 0x100000  # aligned, never dereferenced


def _group(*first):
    x = np.zeros((1, 32))
    x[0, :len(first)] = first
    return x


def test_oracle_by_hand():
    # 7 fits scale 1 and saturates at 6; just above it takes scale 2.
    codes, scales = ref.quantize(_group(7.0, -6.0, 5.0, 0.25, 0.75, -0.1))
    assert scales[0, 0] == 127
    # 5 lies between 4 (even code 6) and 6; 0.25 between 0 and 0.5; 0.75 between 0.5 and 1
    assert codes[0, :6].tolist() == [7, 15, 6, 0, 2, 8]
    codes, scales = ref.quantize(_group(7.5, 3.0))
    assert scales[0, 0] == 128 and codes[0, :2].tolist() == [6, 3]
    assert ref.values(codes, scales)[0, :2].tolist() == [8.0, 3.0]
    codes, scales = ref.quantize(_group())
    assert scales[0, 0] == 127 and not codes.any()
    codes, scales = ref.quantize(_group(1.0, np.nan))
    assert scales[0, 0] == 255 and not codes.any() and np.isnan(ref.values(codes, scales)).all()
    codes, scales = ref.quantize(_group(2.0 ** -140))
    assert scales[0, 0] == 0


def test_oracle_packing_and_logits():
    codes = np.arange(64, dtype=np.uint8).reshape(2, 32) % 16
    assert (ref.unpack(ref.pack(codes)) == codes).all()
    assert ref.pack(codes)[0, 1] == 0x32
    scales = np.array([[127], [130]], np.uint8)
    hidden = np.ones((1, 32))
    hidden[0, 16:] = 0.0
    # entries 0..15 hold every value and its negative
    hidden[0, 15] = 2.0  # doubles -6
    assert ref.logits(hidden, codes, scales).tolist() == [[-6.0, -48.0]]


def _quantize(**kw):
    a = dict(x=FAKE, type=ts.TS_BF16, rows=4, cols=64, ldx=64, codes=FAKE, ldc=32, scales=FAKE,
             lds=2)
    a.update(kw)
    return ts.lib.quantize_groups_e2m1(*a.values(), None)


def _dequantize(**kw):
    a = dict(codes=FAKE, rows=4, cols=64, ldc=32, scales=FAKE, lds=2, x=FAKE, type=ts.TS_BF16,
             ldx=64)
    a.update(kw)
    return ts.lib.dequantize_groups_e2m1(*a.values(), None)


@pytest.mark.parametrize("call", [_quantize, _dequantize])
@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), ts.TS_EINVAL), (dict(cols=-32), ts.TS_EINVAL), (dict(type=2), ts.TS_EINVAL),
    (dict(rows=1 << 31), ts.TS_EUNSUPPORTED), (dict(cols=1 << 31), ts.TS_EUNSUPPORTED),
    (dict(cols=48), ts.TS_EUNSUPPORTED), (dict(x=None), ts.TS_EINVAL),
    (dict(codes=None), ts.TS_EINVAL), (dict(scales=None), ts.TS_EINVAL),
    (dict(ldx=63), ts.TS_EINVAL), (dict(ldc=31), ts.TS_EINVAL), (dict(lds=1), ts.TS_EINVAL),
    (dict(x=FAKE + 1), ts.TS_EUNSUPPORTED), (dict(x=FAKE + 2, type=ts.TS_F32), ts.TS_EUNSUPPORTED),
    (dict(codes=FAKE + 2), ts.TS_EUNSUPPORTED), (dict(ldc=34), ts.TS_EUNSUPPORTED),
])
def test_conversion_refusals(call, kw, code):
    assert call(**kw) == code
    assert ts.lib.ts_last_error()


def _project(**kw):
    a = dict(x=FAKE, rows=4, h=256, ldx=256, w=FAKE, ws=FAKE, vocab=64, ldw=128, lds=8, out=FAKE,
             ldo=64)
    a.update(kw)
    return ts.lib.lmhead_logits_local_e2m1(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), ts.TS_EINVAL), (dict(vocab=-1), ts.TS_EINVAL), (dict(h=-32), ts.TS_EINVAL),
    (dict(rows=1 << 31), ts.TS_EUNSUPPORTED), (dict(h=1 << 31), ts.TS_EUNSUPPORTED),
    (dict(h=0), ts.TS_EINVAL), (dict(x=None), ts.TS_EINVAL), (dict(w=None), ts.TS_EINVAL),
    (dict(ws=None), ts.TS_EINVAL), (dict(out=None), ts.TS_EINVAL), (dict(ldx=248), ts.TS_EINVAL),
    (dict(ldw=112), ts.TS_EINVAL), (dict(lds=7), ts.TS_EINVAL), (dict(ldo=63), ts.TS_EINVAL),
    (dict(ldx=(1 << 21) + 8), ts.TS_EUNSUPPORTED), (dict(h=240, ldx=256), ts.TS_EUNSUPPORTED), (dict(ldx=260), ts.TS_EUNSUPPORTED),
    (dict(ldw=136), ts.TS_EUNSUPPORTED), (dict(x=FAKE + 8), ts.TS_EUNSUPPORTED),
    (dict(w=FAKE + 4), ts.TS_EUNSUPPORTED), (dict(out=FAKE + 2), ts.TS_EUNSUPPORTED),
    (dict(vocab=(1 << 31) - 1023, ldo=1 << 31), ts.TS_EUNSUPPORTED),
    (dict(rows=1 << 25, vocab=1 << 20, ldo=1 << 20), ts.TS_EUNSUPPORTED),
])
def test_projection_refusals(kw, code):
    assert _project(**kw) == code
    assert ts.lib.ts_last_error()


def test_empty_is_noop():
    assert _quantize(rows=0, x=None, codes=None, scales=None) == ts.TS_OK
    assert _quantize(cols=0, x=None, codes=None, scales=None) == ts.TS_OK
    assert _dequantize(rows=0, x=None, codes=None, scales=None) == ts.TS_OK
    assert _project(rows=0, x=None, out=None) == ts.TS_OK
    assert _project(vocab=0, w=None, ws=None) == ts.TS_OK


def test_binding_refusals():
    import torch

    def u8(*shape):
        return torch.zeros(*shape, dtype=torch.uint8)

    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for bad in (x[0], x.half(), torch.zeros(4, 48), x.expand(3, 4, 64)[:, 0].t()):
        with pytest.raises(ValueError):
            ts.quantize_groups_e2m1(bad)
    for bad in (u8(4, 32)[0], u8(4, 24), torch.zeros(4, 32)):
        with pytest.raises(ValueError):
            ts.dequantize_groups_e2m1(bad, u8(4, 2))
    for bad in (u8(4, 3), u8(3, 2), torch.zeros(4, 2), u8(2, 4).t()):
        with pytest.raises(ValueError):
            ts.dequantize_groups_e2m1(u8(4, 32), bad)
    with pytest.raises(ValueError):
        ts.dequantize_groups_e2m1(u8(4, 32), u8(4, 2), dtype=torch.float16)
    for args in ((x.float(), u8(9, 32), u8(9, 2)), (x, u8(9, 16), u8(9, 2)),
                 (x, u8(9, 32), u8(9, 1)), (x, torch.zeros(9, 32), u8(9, 2)),
                 (x[0], u8(9, 32), u8(9, 2)), (x[:, :48], u8(9, 24), u8(9, 1))):
        with pytest.raises(ValueError):
            ts.lmhead_logits_local_e2m1(*args)
    # Right in all but the device.
    for call in (lambda: ts.quantize_groups_e2m1(x),
                 lambda: ts.dequantize_groups_e2m1(u8(4, 32), u8(4, 2)),
                 lambda: ts.lmhead_logits_local_e2m1(x, u8(9, 32), u8(9, 2))):
        with pytest.raises(ValueError, match="GPU"):
            call()
