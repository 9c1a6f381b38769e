"""Adapter projection on the CPU: the oracle by hand, and the refusals of the C
ABI and the binding (validation runs before any HIP call)."""
import numpy as np
import pytest

import top_sampling_amd as ts
from oracle import losses as ref

FAKE = 0x100000  # aligned, never dereferenced


def test_oracle_by_hand():
    x = np.array([[1.0, 2.0], [3.0, -1.0], [1.0, 1.0]])
    w = np.array([[1.0, 0.0], [0.0, 1.0], [1.0, 1.0]])
    a = np.array([[[1.0, 1.0]], [[2.0, 0.0]]])             # 2 adapters of rank 1
    b = np.array([[[1.0], [0.0], [2.0]], [[0.0], [1.0], [1.0]]])
    got = ref.lora_logits(x, w, a, b, [1, -1, 2], [0.5, 10.0])
    # row 0: adapter 1, u = 2, B u = (0, 2, 2), times 10
    assert np.array_equal(got[0], [1.0, 22.0, 23.0])
    assert np.array_equal(got[1], [3.0, -1.0, 2.0])
    assert np.isnan(got[2]).all()


def _lora(**kw):
    a = dict(x=FAKE, rows=4, h=256, ldx=256, w=FAKE, vocab=64, ldw=256, a=FAKE, sa=256 * 16,
             lda=256, b=FAKE, sb=64 * 16, ldb=16, n=3, rank=16, scales=None, ids=FAKE, out=FAKE,
             ldo=64, ws=FAKE, bytes=1 << 30)
    a.update(kw)
    return ts.lib.lmhead_logits_local_lora(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), ts.TS_EINVAL), (dict(vocab=-1), ts.TS_EINVAL), (dict(h=-8), ts.TS_EINVAL),
    (dict(n=-1), ts.TS_EINVAL), (dict(n=0), ts.TS_EINVAL), (dict(rank=0), ts.TS_EINVAL),
    (dict(rank=-8), ts.TS_EINVAL), (dict(rank=12, ldb=16), ts.TS_EUNSUPPORTED),
    (dict(rank=264, ldb=264), ts.TS_EUNSUPPORTED), (dict(rows=1 << 31), ts.TS_EUNSUPPORTED),
    (dict(n=1 << 31), ts.TS_EUNSUPPORTED),
    (dict(rows=ts.TS_MAX_LORA_ROWS + 1), ts.TS_EUNSUPPORTED), (dict(h=0), ts.TS_EINVAL),
    (dict(x=None), ts.TS_EINVAL), (dict(w=None), ts.TS_EINVAL), (dict(a=None), ts.TS_EINVAL),
    (dict(b=None), ts.TS_EINVAL), (dict(ids=None), ts.TS_EINVAL), (dict(out=None), ts.TS_EINVAL),
    (dict(ldx=248), ts.TS_EINVAL), (dict(ldw=248), ts.TS_EINVAL), (dict(lda=248), ts.TS_EINVAL),
    (dict(ldb=8), ts.TS_EINVAL), (dict(ldo=63), ts.TS_EINVAL), (dict(sa=-8), ts.TS_EINVAL),
    (dict(sb=-8), ts.TS_EINVAL), (dict(h=252), ts.TS_EUNSUPPORTED),
    (dict(ldx=260), ts.TS_EUNSUPPORTED), (dict(ldb=20), ts.TS_EUNSUPPORTED),
    (dict(sa=4097), ts.TS_EUNSUPPORTED), (dict(sb=1025), ts.TS_EUNSUPPORTED),
    (dict(x=FAKE + 8), ts.TS_EUNSUPPORTED), (dict(b=FAKE + 2), ts.TS_EUNSUPPORTED),
    (dict(out=FAKE + 2), ts.TS_EUNSUPPORTED), (dict(ids=FAKE + 2), ts.TS_EUNSUPPORTED),
    (dict(scales=FAKE + 1), ts.TS_EUNSUPPORTED), (dict(ws=None), ts.TS_EWORKSPACE),
    (dict(bytes=16), ts.TS_EWORKSPACE), (dict(ws=FAKE + 128), ts.TS_EUNSUPPORTED),
])
def test_refusals(kw, code):
    assert _lora(**kw) == code
    assert ts.lib.ts_last_error()


def test_empty_is_noop():
    assert _lora(rows=0, x=None, ids=None, out=None, ws=None) == ts.TS_OK
    assert _lora(vocab=0, w=None, b=None) == ts.TS_OK


def test_workspace_query():
    assert ts.lmhead_lora_workspace_bytes(-1, 16) == 0
    assert ts.lmhead_lora_workspace_bytes(4, 1000) == 0
    # three bf16 parts of every u, the row and its adapter
    assert ts.lmhead_lora_workspace_bytes(640, 16) >= 640 * (3 * 16 * 2 + 8)


def test_header_constants_match_binding():
    import os
    import re

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "top_sampling.h")).read()
    for name in ("TS_MAX_LORA_RANK", "TS_MAX_LORA_ROWS", "TS_PREFERENCE_MEAN"):
        assert re.search(rf"#define {name} {getattr(ts, name)}\b", text), name
    assert re.search(rf"TS_F32 = {ts.TS_F32}, TS_BF16 = {ts.TS_BF16}\b", text)


def test_binding_refusals():
    import torch

    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    x, w, a, b = bf(4, 64), bf(10, 64), bf(2, 8, 64), bf(2, 10, 8)
    ids = torch.zeros(4, dtype=torch.int32)
    call = ts.lmhead_logits_local_lora
    with pytest.raises(ValueError, match="on the GPU"):
        call(x, w, a, b, ids)
    with pytest.raises(ValueError, match="sizes do not fit"):
        call(x, w, a, bf(2, 9, 8), ids)
    with pytest.raises(ValueError, match="sizes do not fit"):
        call(x, bf(10, 56), a, b, ids)
    with pytest.raises(ValueError, match="3-D"):
        call(x, w, a[0], b, ids)
    with pytest.raises(TypeError, match="lora_a"):
        call(x, w, a.float(), b, ids)
    with pytest.raises(ValueError, match="inner stride"):
        call(x, w, a, bf(2, 8, 10).transpose(1, 2), ids)
    with pytest.raises(ValueError, match="adapter_ids"):
        call(x, w, a, b, ids.long())
    with pytest.raises(ValueError, match="adapter_scales"):
        call(x, w, a, b, ids, torch.ones(3))


@pytest.mark.parametrize("rows,vocab,hidden,fits", [
    (1, (1 << 30) - 1024, 64, True), (1, (1 << 30) - 1023, 64, False), (64, 1 << 30, 64, False),
    (65, (1 << 30) - 1024, 64, True), (129, 1 << 29, 64, False), (129, (1 << 29) - 512, 64, True),
    (ts.TS_MAX_LORA_ROWS, 1 << 20, 64, False), (1, (1 << 31) - 1, 64, False),
    (1, (1 << 31) - 257, 72, True), (1, (1 << 31) - 256, 72, False), (65, 1 << 31, 72, False),
    (257, (1 << 31) - 4096, 72, True), (513, (1 << 31) - 4096, 72, False),
])
def test_more_tiles_than_a_launch_has(rows, vocab, hidden, fits):
    """Refused before anything is enqueued; a size that fits gets as far as the
    missing workspace."""
    code = _lora(rows=rows, vocab=vocab, h=hidden, ldo=vocab, sb=0, ws=None)
    assert code == (ts.TS_EWORKSPACE if fits else ts.TS_EUNSUPPORTED)
    assert ts.lib.ts_last_error()
