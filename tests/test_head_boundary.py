"""Refusals of the single-exit LM-head operators.  Argument checks run before
any device call, so these need no GPU and launch nothing."""
import ctypes

import pytest
import torch

from lm_head_loss_junction_b200 import _lib, token_logprobs_workspace, topk_distill_workspace
from lm_head_loss_junction_b200 import token_logprobs_bwd_workspace

FAKE = 0x10000  # never dereferenced: validation fails first
BIG = 1 << 40
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def score(T=8, D=128, V=1000, N=1, ids=FAKE, h=FAKE, W=FAKE, dt=_lib.MLS_BF16, logp=FAKE, stats=FAKE, K=4,
          top_ids=FAKE, top_logp=FAKE, ws=FAKE, ws_bytes=BIG):
    return _lib.lib().mls_token_logprobs(T, D, V, N, ids, h, W, dt, logp, stats, K, top_ids, top_logp, ws, ws_bytes,
                                         None, None)


def score_bwd(T=8, D=128, V=1000, N=1, ids=FAKE, h=FAKE, W=FAKE, dt=_lib.MLS_BF16, stats=FAKE, g=FAKE, ge=FAKE,
              dh=FAKE, dW=FAKE, dW_dt=_lib.MLS_F32, acc=0, ws=FAKE, ws_bytes=BIG):
    return _lib.lib().mls_token_logprobs_bwd(T, D, V, N, ids, h, W, dt, stats, g, ge, dh, dW, dW_dt, acc, ws,
                                             ws_bytes, None, None)


def distill(T=8, D=128, V=1000, K=4, y=FAKE, tid=FAKE, tl=FAKE, w=FAKE, h=FAKE, W=FAKE, alpha=0.3,
            dt=_lib.MLS_BF16, losses=FAKE, stats=FAKE, ws=FAKE, ws_bytes=BIG):
    return _lib.lib().mls_topk_distill_fwd(T, D, V, K, y, tid, tl, w, h, W, alpha, dt, losses, stats, ws, ws_bytes,
                                           None, None)


def distill_bwd(T=8, D=128, V=1000, K=4, y=FAKE, tid=FAKE, tl=FAKE, w=FAKE, h=FAKE, W=FAKE, alpha=0.3,
                dt=_lib.MLS_BF16, stats=FAKE, scale=1.0, dh=FAKE, dW=FAKE, dW_dt=_lib.MLS_F32, acc=0, ws=FAKE,
                ws_bytes=BIG):
    return _lib.lib().mls_topk_distill_bwd(T, D, V, K, y, tid, tl, w, h, W, alpha, dt, stats, scale, dh, dW, dW_dt,
                                           acc, ws, ws_bytes, None, None)


CALLS = [score, score_bwd, distill, distill_bwd]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("bad,code", [
    (dict(T=0), INVALID), (dict(T=-1), INVALID), (dict(D=0), INVALID), (dict(V=0), INVALID), (dict(dt=2), INVALID),
    (dict(D=100), UNSUPPORTED), (dict(D=65536 + 64), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED),
    (dict(V=1 << 31), UNSUPPORTED), (dict(h=None), INVALID), (dict(W=None), INVALID), (dict(h=FAKE + 8), UNSUPPORTED),
    (dict(W=FAKE + 2), UNSUPPORTED), (dict(stats=None), INVALID), (dict(stats=FAKE + 2), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=64), WORKSPACE), (dict(ws=FAKE + 8), UNSUPPORTED),
])
def test_common_refusals(call, bad, code):
    assert call(**bad) == code


@pytest.mark.parametrize("bad,code", [
    (dict(N=-1), INVALID), (dict(N=0, K=0), INVALID), (dict(N=65), UNSUPPORTED), (dict(ids=None), INVALID),
    (dict(logp=None), INVALID), (dict(K=-1), INVALID), (dict(K=65), UNSUPPORTED), (dict(K=4, V=3), UNSUPPORTED),
    (dict(top_ids=None), INVALID), (dict(top_logp=None), INVALID), (dict(ids=FAKE + 1), UNSUPPORTED),
    (dict(V=(1 << 21) + 1), UNSUPPORTED),
])
def test_score_refusals(bad, code):
    assert score(**bad) == code


@pytest.mark.parametrize("bad,code", [
    (dict(N=0), INVALID), (dict(N=65), UNSUPPORTED), (dict(ids=None), INVALID), (dict(g=None), INVALID),
    (dict(dh=None, dW=None), INVALID), (dict(dh=FAKE + 8), UNSUPPORTED), (dict(dW=FAKE + 8), UNSUPPORTED),
    (dict(dW_dt=5), INVALID), (dict(dW_dt=_lib.MLS_BF16, dt=_lib.MLS_F32), UNSUPPORTED),
    (dict(dW_dt=_lib.MLS_BF16, acc=1), UNSUPPORTED), (dict(ge=FAKE + 2), UNSUPPORTED),
])
def test_score_backward_refusals(bad, code):
    assert score_bwd(**bad) == code


@pytest.mark.parametrize("call", [distill, distill_bwd])
@pytest.mark.parametrize("bad,code", [
    (dict(K=0), INVALID), (dict(K=65), UNSUPPORTED), (dict(y=None), INVALID), (dict(tid=None), INVALID),
    (dict(tl=None), INVALID), (dict(alpha=float("nan")), INVALID), (dict(alpha=float("inf")), INVALID),
    (dict(w=FAKE + 1), UNSUPPORTED),
])
def test_distill_refusals(call, bad, code):
    assert call(**bad) == code


def test_distill_own_refusals():
    assert distill(losses=None) == INVALID
    assert distill_bwd(scale=float("nan")) == INVALID
    assert distill_bwd(dh=None, dW=None) == INVALID
    assert distill_bwd(dW_dt=_lib.MLS_BF16, acc=1) == UNSUPPORTED


def test_valid_calls_without_a_gpu_report_no_device():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for call in CALLS:
        assert call() == 7
        assert call(dt=_lib.MLS_F32, D=33) == 7
    assert score(N=0, ids=None, logp=None) == 7
    assert score(K=0, top_ids=None, top_logp=None) == 7
    assert score_bwd(dW=None) == 7 and score_bwd(dh=None) == 7 and score_bwd(ge=None) == 7
    assert distill(w=None) == 7 and distill_bwd(w=None, dW_dt=_lib.MLS_BF16) == 7


def test_fp32_operands_need_four_bytes():
    f32 = dict(dt=_lib.MLS_F32, D=33)
    for call in CALLS:
        assert call(h=FAKE + 4, **f32) in (0, 7) if not torch.cuda.is_available() else True
        assert call(h=FAKE + 2, **f32) == UNSUPPORTED and call(W=FAKE + 1, **f32) == UNSUPPORTED
    assert score_bwd(dh=FAKE + 2, **f32) == UNSUPPORTED and distill_bwd(dW=FAKE + 2, **f32) == UNSUPPORTED


def test_workspace_queries():
    bf, f32 = torch.bfloat16, torch.float32
    # without alternatives the logits are never stored: 16 bytes per token and 128 columns, not 4 per logit
    n, least = token_logprobs_workspace(8192, 2304, 49152, 1, 0, bf)
    assert least < n < 8192 * 49152
    # with them a block of tokens' logits fits the budget of 1.5 GiB
    n, least = token_logprobs_workspace(32768, 2304, 49152, 1, 20, bf)
    assert 256 * 49152 * 4 < least < n <= 3 << 29
    n, least = token_logprobs_workspace(1, 2304, 49152, 1, 20, bf)
    assert n == least < 1 << 20
    # the backward pass holds at most a chunk of the gradient
    n, least = token_logprobs_bwd_workspace(32768, 1024, 49152, 1, bf)
    assert least < n <= 3 << 29
    f, f_min, b, b_min = topk_distill_workspace(8192, 1024, 49152, 64, bf)
    assert f_min <= f and 8192 * 49152 * 2 < b <= 3 << 29 and b_min < b
    f, f_min, b, b_min = topk_distill_workspace(256, 64, 512, 8, f32)
    assert b_min <= b and f == f_min
    for bad in [(0, 64, 10, 1, 0), (4, 64, 10, 0, 0), (4, 64, 10, -1, 3), (4, 64, 10, 1, 11), (4, 63, 10, 1, 1)]:
        with pytest.raises(_lib.MLSError):
            token_logprobs_workspace(*bad, bf)
    assert _lib.lib().mls_token_logprobs_workspace(4, 64, 10, 1, 1, _lib.MLS_BF16, None, None) == INVALID
    one = ctypes.c_size_t()
    assert _lib.lib().mls_topk_distill_workspace(4, 64, 10, 1, _lib.MLS_BF16, ctypes.byref(one), None,
                                                 ctypes.byref(one), None) == 0
    assert _lib.lib().mls_topk_distill_workspace(4, 64, 10, 1, _lib.MLS_BF16, ctypes.byref(one), None, None,
                                                 None) == INVALID


@pytest.mark.parametrize("T", [1, 255, 256, 257, 1000, 5000, 70000])
@pytest.mark.parametrize("V", [1, 127, 128, 257, 50021])
def test_every_workspace_from_the_minimum_up_is_a_valid_size(T, V):
    """The minimum never exceeds what the query returns, for any shape."""
    for dt in (torch.bfloat16, torch.float32):
        for K in (0, 1):
            n, least = token_logprobs_workspace(T, 64, V, 1, K, dt)
            assert 0 < least <= n
        f, f_min, b, b_min = topk_distill_workspace(T, 64, V, 3, dt)
        assert 0 < f_min <= f and 0 < b_min <= b


def test_status_needs_a_word():
    """An empty view would have its flags set in its neighbour's memory."""
    from lm_head_loss_junction_b200.api import _head_status
    cpu, words = torch.device("cpu"), torch.zeros(4, dtype=torch.int32)
    for good in (None, words, words[1:2], words[0]):
        _head_status(good, cpu)
    for bad, error in ((words[2:2], ValueError), (torch.zeros(0, dtype=torch.int32), ValueError)):
        with pytest.raises(error):
            _head_status(bad, cpu)
