"""Single-exit LM-head operators in numpy fp64: log probabilities of given
tokens with entropy and top alternatives, and distillation from a teacher's
top logits, with their gradients.  Plain restatements of the definitions in
include/mls.h; one matrix product per block of logits, nothing online or
chunked."""
from __future__ import annotations

import numpy as np

from .loss import _f64 as f64


def head_logits(h, W):
    return f64(h) @ f64(W).T


def log_softmax(l):
    m = l.max(axis=1, keepdims=True)
    lse = m[:, 0] + np.log(np.exp(l - m).sum(axis=1))
    return l - lse[:, None], lse


def _there(ids, V):
    ids = np.asarray(ids, dtype=np.int64)
    return (ids >= 0) & (ids < V), np.clip(ids, 0, V - 1)


def token_logprobs(ids, h, W, top_k=0):
    """dict: logp [T, N], lse [T], entropy [T], top_ids and top_logp [T, top_k]."""
    logq, lse = log_softmax(head_logits(h, W))
    q = np.exp(logq)
    entropy = -np.sum(np.where(q > 0, q * logq, 0.0), axis=1)
    out = {"lse": lse, "entropy": entropy}
    if ids is not None:
        ok, at = _there(ids, logq.shape[1])
        out["logp"] = np.where(ok, np.take_along_axis(logq, at, axis=1), 0.0)
    if top_k:
        order = np.argsort(-logq, axis=1, kind="stable")[:, :top_k]
        out["top_ids"] = order
        out["top_logp"] = np.take_along_axis(logq, order, axis=1)
    return out


def token_logprobs_grad(ids, h, W, g_logp, g_entropy=None):
    """dL/dl [T, V]."""
    logq, _ = log_softmax(head_logits(h, W))
    q = np.exp(logq)
    ok, at = _there(ids, logq.shape[1])
    g = np.where(ok, np.nan_to_num(f64(g_logp), nan=0.0), 0.0)
    G = -q * g.sum(axis=1, keepdims=True)
    if g_entropy is not None:
        entropy = -np.sum(q * logq, axis=1, keepdims=True)
        G -= f64(g_entropy)[:, None] * q * (logq + entropy)
    rows = np.arange(G.shape[0])
    for n in range(at.shape[1]):
        G[rows, at[:, n]] += g[:, n]
    return G


def teacher_probs(teacher_ids, teacher_logits, V):
    """p [T, K] over the present teacher tokens (rows without any: zeros)."""
    ok, at = _there(teacher_ids, V)
    z = np.where(ok, f64(teacher_logits), -np.inf)
    top = z.max(axis=1, keepdims=True)
    some = top > -np.inf
    e = np.where(some, np.exp(z - np.where(some, top, 0.0)), 0.0)
    s = e.sum(axis=1, keepdims=True)
    return e / np.where(s > 0, s, 1.0), at, some[:, 0]


def topk_distill(y, teacher_ids, teacher_logits, h, W, alpha_d=0.3, weights=None, grad_scale=1.0):
    """dict: losses [3], stats [3, T], and G = d(grad_scale * losses[2])/dl [T, V]."""
    logq, lse = log_softmax(head_logits(h, W))
    T, V = logq.shape
    rows = np.arange(T)
    w = np.ones(T) if weights is None else f64(weights)
    y = np.asarray(y, dtype=np.int64)
    inside = (y >= 0) & (y < V)
    counted = (w != 0) & inside
    yc = np.clip(y, 0, V - 1)
    p, at, some = teacher_probs(teacher_ids, teacher_logits, V)
    ce = np.where(inside, -logq[rows, yc], 0.0)
    kd = np.where(inside, -np.sum(p * np.take_along_axis(logq, at, axis=1), axis=1), 0.0)
    w = np.where(counted, w, 0.0)
    means = [np.mean(w * ce), np.mean(w * kd)]
    G = np.exp(logq) * ((1 - alpha_d) + alpha_d * some)[:, None]
    G[rows, yc] -= 1 - alpha_d
    for k in range(at.shape[1]):
        G[rows, at[:, k]] -= alpha_d * p[:, k]
    G *= (w * grad_scale / T)[:, None]
    return {"losses": np.array([means[0], means[1], (1 - alpha_d) * means[0] + alpha_d * means[1]]),
            "stats": np.stack([lse, ce, kd]), "G": G}
