"""The LM-head operators as calls with inputs, sizes and plain forms, for timing and comparison.

Three passes a user of the library makes with the hidden states h [T, D] of one exit and its head W [V, D]:

score    token_logprobs: log probabilities of given tokens, the entropy of each next-token distribution and its
         top alternatives (a decoding step's log probabilities; a teacher's top tokens, written down once).
policy   token_logprobs and token_logprobs_bwd: the same with the gradients of log probabilities and entropy,
         as a policy-gradient step takes them.
distill  topk_distill_fwd and topk_distill_bwd: next-token cross-entropy mixed with the cross-entropy to a
         teacher of which only its top logits are at hand, and the gradients.
"""
import math

import torch

own = False

# Columns beyond the wanted ones whose logits are computed again in 64 bits before they are ranked.
_MORE = 8


def listed():
    return [
        # one decoding step of one sequence, log probability of the drawn token and its alternatives
        dict(name="score_one_token", op="score", T=1, V=49152, D=2304, N=1, K=8, dtype="bf16"),
        # one decoding step of a small batch on the smallest exit
        dict(name="score_decode_batch", op="score", T=24, V=49152, D=1024, N=1, K=20, dtype="bf16"),
        # ranking a few continuations of a ragged batch of prompts, odd vocabulary
        dict(name="score_ragged", op="score", T=1001, V=50021, D=640, N=3, K=5, dtype="bf16"),
        # writing down a teacher's top tokens for two sequences of 2048
        dict(name="score_teacher", op="score", T=4096, V=49152, D=2304, N=1, K=32, dtype="bf16"),
        # the small single-precision suite
        dict(name="score_f32", op="score", T=256, V=512, D=192, N=2, K=4, dtype="f32"),
        # a policy-gradient step on a few short answers
        dict(name="policy_short", op="policy", T=130, V=32768, D=512, N=1, K=0, dtype="bf16"),
        # a policy-gradient step on two sequences of 2048
        dict(name="policy_main", op="policy", T=4096, V=49152, D=1024, N=1, K=0, dtype="bf16"),
        dict(name="policy_f32", op="policy", T=256, V=512, D=128, N=1, K=0, dtype="f32"),
        # distillation steps: the small single-precision suite, a ragged batch with an odd vocabulary,
        # the smallest and the middle exit on four sequences of 2048
        dict(name="distill_f32", op="distill", T=256, V=512, D=64, N=1, K=8, dtype="f32"),
        dict(name="distill_ragged", op="distill", T=777, V=32771, D=1024, N=1, K=50, dtype="bf16"),
        dict(name="distill_small_exit", op="distill", T=8192, V=49152, D=1024, N=1, K=64, dtype="bf16"),
        dict(name="distill_middle_exit", op="distill", T=8192, V=49152, D=2304, N=1, K=32, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["score", "score", "policy", "distill", "distill"])
    if rng.random() < 0.15:
        # the single-precision path is for small suites
        T, V, D, dtype = _log_int(rng, 1, 700), _log_int(rng, 70, 2000), rng.randint(5, 200), "f32"
    else:
        V, D, dtype = _log_int(rng, 500, 66000), 64 * _log_int(rng, 1, 36), "bf16"
        T = _log_int(rng, 1, min(8192, int(8192 * 49152 * 2304 / (V * D))))
    if op == "score":
        return dict(op=op, T=T, V=V, D=D, N=rng.choice([1, 1, 2, 5]), K=_log_int(rng, 1, 40), dtype=dtype)
    if op == "policy":
        return dict(op=op, T=T, V=V, D=D, N=1, K=0, dtype=dtype)
    return dict(op=op, T=T, V=V, D=D, N=1, K=_log_int(rng, 1, 64), dtype=dtype)


def _inputs(case, seed):
    """h as after a final norm, W so that logits spread by about 2, and each h leaning towards its token's row by
    a random amount: from a uniform guess to a nearly certain one, as a trained head's rows are."""
    T, V, D = case["T"], case["V"], case["D"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = (torch.randn(V, D, generator=g, device="cuda") * (2.0 / math.sqrt(D))).to(dt)
    y = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    lean = torch.rand(T, 1, generator=g, device="cuda") * 4.0
    h = (torch.randn(T, D, generator=g, device="cuda") + lean * W[y.long()].float()).to(dt)
    return g, dt, h, W, y


def prepare(case, seed):
    T, V, N, K = case["T"], case["V"], case["N"], case["K"]
    g, dt, h, W, y = _inputs(case, seed)
    s = dict(op=case["op"], h=h, W=W, K=K)
    if case["op"] == "distill":
        # the teacher's tokens: the target first (nine times in ten), then others, no token twice in a row
        step = torch.randint(1, max(2, V // (K + 1)), (T, 1), generator=g, device="cuda")
        ids = (y.long()[:, None] + step * torch.arange(K, device="cuda")) % V
        miss = torch.rand(T, generator=g, device="cuda") < 0.1
        ids[:, 0] = torch.where(miss, (y.long() + step[:, 0] * K) % V, ids[:, 0])
        gaps = -torch.log(torch.rand(T, K, generator=g, device="cuda") + 1e-9) * 0.5
        logits = 14.0 - torch.cumsum(gaps, 1)
        # one row in eight kept fewer tokens, some of them none: absent ones have id -1 and no meaningful logit
        short = torch.rand(T, 1, generator=g, device="cuda") < 0.125
        kept = torch.randint(0, K + 1, (T, 1), generator=g, device="cuda")
        gone = short & (torch.arange(K, device="cuda") >= kept)
        s["teacher_ids"] = torch.where(gone, torch.full_like(ids, -1), ids).to(torch.int32)
        s["teacher_logits"] = torch.where(gone, torch.full_like(logits, float("nan")), logits)
        # padding at the end of the batch has weight 0, the other tokens share T
        real = max(1, T - T // 9)
        s["weights"] = torch.where(torch.arange(T, device="cuda") < real, T / real, 0.0).float()
        s["y"], s["alpha"], s["scale"] = y, 0.3, 1.0
        return s
    ids = torch.randint(0, V, (T, N), generator=g, device="cuda", dtype=torch.int32)
    ids[:, 0] = y
    if T > 8:
        ids[T - T // 9:, N - 1] = -1            # no token there: padding
    s["ids"] = ids
    if case["op"] == "policy":
        s["g_logp"] = torch.randn(T, N, generator=g, device="cuda") / T
        s["g_entropy"] = torch.full((T,), 0.01 / T, device="cuda")
    return s


def run(s):
    if own:
        return _own(s)
    if s["op"] == "score":
        return _plain_score(s["ids"], s["h"], s["W"], s["K"])
    if s["op"] == "policy":
        return _plain_policy(s["ids"], s["h"], s["W"], s["g_logp"], s["g_entropy"])
    return _plain_distill(s)


def _own(s):
    import lm_head_loss_junction_b200 as mls
    h, W = s["h"], s["W"]
    if s["op"] == "score":
        logp, stats, top_ids, top_logp = mls.token_logprobs(s["ids"], h, W, top_k=s["K"])
        return dict(logp=logp, stats=stats, top_ids=top_ids, top_logp=top_logp)
    if s["op"] == "policy":
        logp, stats, _, _ = mls.token_logprobs(s["ids"], h, W)
        dh, dW = mls.token_logprobs_bwd(s["ids"], h, W, stats, s["g_logp"], s["g_entropy"], dW_dtype=W.dtype)
        return dict(logp=logp, stats=stats, dh=dh, dW=dW)
    t = (s["y"], s["teacher_ids"], s["teacher_logits"], h, W)
    losses, stats = mls.topk_distill_fwd(*t, alpha_d=s["alpha"], token_weights=s["weights"])
    dh, dW = mls.topk_distill_bwd(*t, stats, alpha_d=s["alpha"], grad_scale=s["scale"], token_weights=s["weights"],
                                  dW_dtype=W.dtype)
    return dict(losses=losses, stats=stats, dh=dh, dW=dW)


# ---------------------------------------------------------------- plain forms, in 32 bits
def _log_sum_exp(x):
    m = x.max(dim=1, keepdim=True).values
    return (m + torch.log(torch.exp(x - m).sum(dim=1, keepdim=True)))[:, 0]


def _logits_stats(h, W):
    logits = h.float() @ W.float().T
    lse = _log_sum_exp(logits)
    logq = logits - lse[:, None]
    entropy = -(torch.exp(logq) * logq).sum(dim=1)
    return logits, lse, entropy


def _pick(logits, lse, ids):
    there = ids >= 0
    at = torch.where(there, ids, 0).long()
    return torch.where(there, logits.gather(1, at) - lse[:, None], 0.0), there, at


def _plain_score(ids, h, W, K):
    logits, lse, entropy = _logits_stats(h, W)
    logp, _, _ = _pick(logits, lse, ids)
    # the candidates near the border are ranked by products in 64 bits, equal ones by the lower index
    near = torch.topk(logits, min(K + _MORE, logits.shape[1]), dim=1).indices.sort(dim=1).values
    fine = (W[near].double() @ h.double()[:, :, None])[:, :, 0]
    order = torch.sort(fine, dim=1, descending=True, stable=True).indices[:, :K]
    top = near.gather(1, order)
    return dict(logp=logp, stats=torch.stack([lse, entropy]), top_ids=top.to(torch.int32),
                top_logp=logits.gather(1, top) - lse[:, None])


def _gradients(G, h, W):
    return (G @ W.float()).to(h.dtype), (G.T @ h.float()).to(W.dtype)


def _plain_policy(ids, h, W, g_logp, g_entropy):
    logits, lse, entropy = _logits_stats(h, W)
    logp, there, at = _pick(logits, lse, ids)
    g = torch.where(there, g_logp, 0.0)
    logq = logits - lse[:, None]
    G = -torch.exp(logq) * (g.sum(dim=1, keepdim=True) + g_entropy[:, None] * (logq + entropy[:, None]))
    G.scatter_add_(1, at, g)
    dh, dW = _gradients(G, h, W)
    return dict(logp=logp, stats=torch.stack([lse, entropy]), dh=dh, dW=dW)


def _plain_distill(s):
    h, W, w, alpha = s["h"], s["W"], s["weights"], s["alpha"]
    T = h.shape[0]
    logits = h.float() @ W.float().T
    lse = _log_sum_exp(logits)
    there = s["teacher_ids"] >= 0
    at = torch.where(there, s["teacher_ids"], 0).long()
    z = torch.where(there, s["teacher_logits"], -torch.inf)
    some = there.any(dim=1, keepdim=True)
    top = torch.where(some, z.max(dim=1, keepdim=True).values, 0.0)
    p = torch.where(there, torch.exp(z - top), 0.0)
    p = p / torch.where(some, p.sum(dim=1, keepdim=True), 1.0)
    y = s["y"].long()[:, None]
    ce = lse - logits.gather(1, y)[:, 0]
    kd = (p * (lse[:, None] - logits.gather(1, at))).sum(dim=1)
    ce_mean, kd_mean = (w * ce).sum() / T, (w * kd).sum() / T
    losses = torch.stack([ce_mean, kd_mean, (1 - alpha) * ce_mean + alpha * kd_mean])
    G = torch.exp(logits - lse[:, None]) * ((1 - alpha) + alpha * some.float())
    G.scatter_add_(1, y, torch.full_like(y, -(1 - alpha), dtype=G.dtype))
    G.scatter_add_(1, at, -alpha * p)
    G *= (w * (s["scale"] / T))[:, None]
    dh, dW = _gradients(G, h, W)
    return dict(losses=losses, stats=torch.stack([lse, ce, kd]), dh=dh, dW=dW)


# ---------------------------------------------------------------- work
def work(case):
    T, V, D, N, K = (case[k] for k in ("T", "V", "D", "N", "K"))
    b = 2 if case["dtype"] == "bf16" else 4
    rows, head = T * D * b, V * D * b
    if case["op"] == "score":       # h, W, ids in; logp, lse, entropy, the alternatives out
        return dict(bytes=rows + head + T * (8 * N + 8 + 8 * K), flops=2 * T * V * D)
    if case["op"] == "policy":      # logits once; dh and dW are a product each
        return dict(bytes=2 * (rows + head) + T * (12 * N + 12), flops=6 * T * V * D)
    return dict(bytes=2 * (rows + head) + T * (8 * K + 4 + 4 + 12), flops=6 * T * V * D)


# ---------------------------------------------------------------- from the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    h, W = s["h"].double(), s["W"].double()
    T, V = h.shape[0], W.shape[0]
    logq = torch.log_softmax(h @ W.T, dim=1)
    rows = torch.arange(T, device=h.device)
    lse = (h[:, None, :] @ W[:1].T[None])[:, 0, 0] - logq[:, 0]
    if case["op"] == "distill":
        target = torch.zeros(T, V, dtype=torch.float64, device=h.device)
        kd = torch.zeros(T, dtype=torch.float64, device=h.device)
        z = s["teacher_logits"].double().masked_fill(s["teacher_ids"] < 0, -torch.inf)
        p = torch.nan_to_num(torch.softmax(z, dim=1), nan=0.0)
        for k in range(case["K"]):
            ids = s["teacher_ids"][:, k].long().clamp(min=0)
            kd -= p[:, k] * logq[rows, ids]
            target[rows, ids] += s["alpha"] * p[:, k]
        ce = -logq[rows, s["y"].long()]
        target[rows, s["y"].long()] += 1 - s["alpha"]
        w = s["weights"].double()
        losses = torch.stack([(w * ce).mean(), (w * kd).mean(), (w * ((1 - s["alpha"]) * ce + s["alpha"] * kd)).mean()])
        G = (logq.exp() * target.sum(dim=1, keepdim=True) - target) * (w * s["scale"] / T)[:, None]
        return dict(losses=losses, stats=torch.stack([lse, ce, kd]), dh=G @ W, dW=G.T @ h)
    q = logq.exp()
    entropy = -(q * logq).sum(dim=1)
    there = s["ids"] >= 0
    logp = logq[rows[:, None], s["ids"].long().clamp(min=0)].masked_fill(~there, 0.0)
    out = dict(logp=logp, stats=torch.stack([lse, entropy]))
    if case["op"] == "score":
        top = torch.sort(logq, dim=1, descending=True, stable=True)
        return dict(out, top_ids=top.indices[:, :case["K"]].to(torch.int32), top_logp=top.values[:, :case["K"]])
    g = s["g_logp"].double().masked_fill(~there, 0.0)
    G = -q * (logq + entropy[:, None]) * s["g_entropy"].double()[:, None]
    for n in range(case["N"]):
        G -= q * g[:, n:n + 1]
        G[rows, s["ids"][:, n].long().clamp(min=0)] += g[:, n]
    return dict(out, dh=G @ W, dW=G.T @ h)
