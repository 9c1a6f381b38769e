"""A 4-bit draft head beside its full one, as they are used together: the head is
quantised, its logits sampled from, the sampled tokens scored with the full head's
alternatives, and the draft's logits get the gradient of the cross-entropy over
those alternatives.  Each step against its float64 oracle on the step's own inputs.
"""
import numpy as np
import pytest
import test_gpu_losses as base
from test_gpu_alternatives import check_topn
from test_gpu_losses import LSE, U, close, grad_tol

import top_sampling_amd as ts
import workloads
from oracle import alternatives as ref
from oracle import e2m1
from oracle.losses import log_softmax

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _greedy(rows, n):
    p = np.zeros(rows, dtype=workloads.PARAMS_DTYPE)
    p["temperature"], p["top_k"], p["top_p"] = 1.0, 1, 1.0
    p["n_logprobs"] = n
    return p


@pytest.mark.parametrize("rows", [3, 48, 200])
def test_draft_head(rows):
    n, hidden, vocab = 12, 256, 5003
    gen = torch.Generator().manual_seed(rows)
    head = (torch.randn(vocab, hidden, generator=gen) / 4).to(torch.bfloat16).cuda()
    x = torch.randn(rows, hidden, generator=gen).to(torch.bfloat16).cuda()
    base.say("draft head", rows)

    # the head in 4 bits, and both heads' logits
    codes, scales = ts.quantize_groups_e2m1(head)
    want_codes, want_scales = e2m1.quantize(_np(head[:40]))
    assert np.array_equal(e2m1.unpack(codes[:40].cpu().numpy()), want_codes)
    assert np.array_equal(scales[:40].cpu().numpy(), want_scales)
    back = ts.dequantize_groups_e2m1(codes, scales, dtype=torch.bfloat16)
    # 4-bit values times a power of two are bf16 values, so the draft is a bf16 head too
    values = e2m1.values(e2m1.unpack(codes.cpu().numpy()), scales.cpu().numpy())
    assert np.array_equal(_np(back), values)
    draft = ts.lmhead_logits_local_e2m1(x, codes, scales)
    teacher = ts.lmhead_logits_local(x, head)
    room = hidden * 2.0 ** -23 * (np.abs(_np(x)) @ np.abs(values).T)
    assert (np.abs(_np(draft) - _np(x) @ values.T) <= room).all()
    same = ts.lmhead_logits_local(x, back)
    assert (np.abs(_np(draft) - _np(same)) <= 2 * room).all()

    # the draft's tokens, scored by the full head with its alternatives
    params = ts.params_to_device(_greedy(rows, n), "cuda")
    sampled = ts.sampler_sample(draft, params, 0, n)
    own = ts.token_logprobs_topn(draft, sampled.token_ids, n, entropies=True)
    check_topn(own, ref.topn(_np(draft), sampled.token_ids.cpu().numpy(), n), "draft")
    assert torch.equal(own.topn_ids, sampled.topn_ids)
    assert (own.ranks == 1).all() and torch.equal(own.topn_ids[:, 0], sampled.token_ids)
    scored = ts.token_logprobs_topn(teacher, sampled.token_ids, n, entropies=True)
    want = ref.topn(_np(teacher), sampled.token_ids.cpu().numpy(), n)
    check_topn(scored, want, "teacher")

    # their cross-entropy: L = -sum_i q_i lp_i, q the full head's probabilities
    ids = scored.topn_ids
    q = scored.topn_logprobs.exp()
    listed = ts.token_logprobs_listed(draft, ids)
    grad = ts.token_logprobs_listed_backward(draft, ids, listed, -q)
    lp, _, _ = ref.listed(_np(draft), ids.cpu().numpy())
    close(listed.logprobs, lp, LSE + U * np.abs(lp), "listed")
    wanted = ref.listed_gradient(_np(draft), ids.cpu().numpy(), 1.0, -_np(q))
    # Terms of the listed tokens cancel: LSE of their sizes.
    size = _np(q).sum(-1)[:, None] * np.exp(log_softmax(_np(draft), 1.0))
    np.put_along_axis(size, ids.cpu().numpy().astype(np.int64),
                      np.take_along_axis(size, ids.cpu().numpy().astype(np.int64), 1) + _np(q), 1)
    close(grad, wanted, grad_tol(wanted, _np(draft), 1.0, "fp32", 2 * LSE) + size * 2 * LSE, "grad")

    # scoring's own statistics serve the same backward pass
    again = ts.TokenLogprobs(listed.logprobs, None, own.row_stats, None)
    assert torch.equal(ts.token_logprobs_listed_backward(draft, ids, again, -q), grad)


def test_a_step_down_the_gradient():
    """L = sum_i q_i lp_i at z + d v and z - d v, v of length 1, against the gradient
    times the step between them (as it was rounded).  With G = sum_i q_i:
    L is off by at most G (LSE + 16 U) on each side (|lp| < 16); the gradient's terms,
    G p_j and q_i, by 2 LSE of their sizes, which is less than 2 LSE G over a step
    of 2 d < 1/2; the third derivative is G times a third cumulant of v's entries,
    within a range of 2, so the difference leaves out at most d^3 / 3 * 8 G; and the
    two halves of the rounded step differ by 2^-20 at most, 32 U G with the second
    derivative below 2 G."""
    rows, vocab, n, d = 5, 3001, 9, 2.0 ** -5
    gen = torch.Generator().manual_seed(1)
    z = (2 * torch.randn(rows, vocab, generator=gen)).cuda()
    ids = torch.randint(0, vocab, (rows, n), generator=gen, dtype=torch.int32).cuda()
    q = torch.rand(rows, n, generator=gen).cuda()
    v = torch.zeros(rows, vocab, device="cuda")
    v.scatter_(1, ids.long(), 1.0)
    v[:, 0] -= 2.0
    v /= v.norm(dim=-1, keepdim=True)
    up, down = z + d * v, z - d * v
    step = (up.double() - down.double())  # as it was rounded
    grad = ts.token_logprobs_listed_backward(z, ids, ts.token_logprobs_listed(z, ids), q)
    rise = (q.double() * ts.token_logprobs_listed(up, ids).logprobs.double()).sum(-1) - \
        (q.double() * ts.token_logprobs_listed(down, ids).logprobs.double()).sum(-1)
    slope = (grad.double() * step).sum(-1)
    room = q.double().sum(-1) * (4 * LSE + 64 * U + 8 * d ** 3 / 3)
    assert ((rise - slope).abs() <= room).all()
