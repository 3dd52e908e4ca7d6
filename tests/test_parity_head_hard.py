"""Single-exit LM-head operators where they can go wrong: peaked rows whose gradient is small."""
import functools

import numpy as np
import pytest
import torch

from lm_head_loss_junction_b200 import token_logprobs, token_logprobs_bwd, topk_distill_bwd, topk_distill_fwd
from oracle import head as oh
from tests.head_helpers import Bounds, half_step, within
from tests.test_parity_head import gpu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


# ---------------------------------------------------------------- gradients of peaked rows
@functools.lru_cache(maxsize=None)
def peaked(T, D, V, seed=0):
    """Rows that are nearly certain of one token: q_y from 0.99 to 0.9997, and W with a mean row as long as its
    spread, so that what is lost of a row's small probabilities does not average out."""
    rng = np.random.Generator(np.random.PCG64(seed))
    W = rng.normal(size=(V, D)) * 2.0 / np.sqrt(D)
    mean = rng.normal(size=D) * 2.0 / np.sqrt(D)
    W = torch.from_numpy((W + mean).astype(np.float32)).to(BF)
    Wd = W.double().numpy()
    y = rng.choice(V, size=T, replace=False).astype(np.int32)
    h, to = rng.normal(size=(T, D)) * 0.5, Wd[y] - mean
    base, lean = h @ Wd.T, to @ Wd.T
    target = np.resize([0.99, 0.995, 0.9975, 0.999, 0.9997], T)
    lo, hi = np.zeros(T), np.full(T, 60.0)
    for _ in range(24):
        mid = (lo + hi) / 2
        logq, _ = oh.log_softmax(base + mid[:, None] * lean)
        low = np.exp(logq[np.arange(T), y]) < target
        lo, hi = np.where(low, mid, lo), np.where(low, hi, mid)
    return torch.from_numpy((h + lo[:, None] * to).astype(np.float32)).to(BF), W, y


@pytest.mark.parametrize("T,D,V", [(150, 128, 49152), (520, 192, 33001), (200, 128, 131072)])
@pytest.mark.parametrize("op", ["score", "distill"])
def test_gradients_of_peaked_rows(T, D, V, op):
    """Every token's dh and every untouched token's dW row keep their own relative precision.

    Bound of an entry of G: both passes form the same logits bit for bit here, so with dl the error of a logit
    (2 dl of a difference) an entry of a small probability is off by 2 dl + 2^-19 (exp, log) of itself and 2^-11
    (fp16); what is lost below fp16's smallest number is 2^-25 of a row stored between 2^13 and 2^15 times its largest
    coefficient: 2^-38 s.  The target's own entry is minus the sum of the others, formed from the fp32 log-sum-exp:
    the others' errors, 2^-24 |lse| and 2^-20 s."""
    h, W, y = peaked(T, D, V)
    b = Bounds(h, W)
    rows = np.arange(T)
    logq, lse = oh.log_softmax(b.h @ b.W.T)
    assert 0.985 < np.exp(logq[rows, y]).min() and np.exp(logq[rows, y]).max() < 0.9999
    hg, Wg, yg = gpu(h, W, y)
    if op == "score":
        _, stats, _, _ = token_logprobs(yg, hg, Wg)
        dh, dW = token_logprobs_bwd(yg, hg, Wg, stats, torch.full((T,), -1.0 / T, device="cuda"))
    else:
        z = torch.zeros(T, 1, device="cuda")
        _, stats = topk_distill_fwd(yg, yg[:, None].contiguous(), z, hg, Wg)
        dh, dW = topk_distill_bwd(yg, yg[:, None].contiguous(), z, hg, Wg, stats)
    G = np.exp(logq) / T
    G[rows, y] = 0.0
    G[rows, y] = -G.sum(axis=1)
    s = 1.0 / T
    rel = 2.0 ** -11 + 2 * b.dl + 2.0 ** -19
    e = rel[:, None] * np.abs(G) + 2.0 ** -38 * s
    e[rows, y] += s * (2.0 ** -24 * np.abs(lse) + 2.0 ** -20)
    aG = np.abs(G)
    exp = G @ b.W
    within(dh, exp, e @ np.abs(b.W) + (V / 16 + 32) * 2.0 ** -23 * (aG @ np.abs(b.W)) + half_step(BF) * np.abs(exp), "dh")
    rare = np.setdiff1d(np.arange(V), y)
    exp = G.T[rare] @ b.h
    # h is copied to fp16 over at most twice its largest value: 2^-38 of that below fp16's normal range
    copy = 2.0 ** -37 * np.abs(b.h).max() * aG.T[rare].sum(axis=1, keepdims=True)
    within(dW[torch.from_numpy(rare).cuda()], exp, e.T[rare] @ np.abs(b.h) + copy +
           ((T / 16 + 32) * 2.0 ** -23) * (aG.T[rare] @ np.abs(b.h)) + half_step(F32) * np.abs(exp), "dW of other tokens")
