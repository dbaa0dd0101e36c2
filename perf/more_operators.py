"""Timed cases of the losses over the vocabulary that sit behind a hashed N-gram memory's model.

The model's last hidden states h [N, d] meet the rows of an output table W [V, d] (the token
embedding's own table where the two are tied): logits z[i, v] = scale * <h_i, W_v>. Four operators,
none of which hands the logits [N, V] out:

  vocab_ce            softmax cross entropy of one target a row:
                      lse_i = log sum_v exp(z[i, v]);  loss_i = lse_i - z[i, t_i] + z_loss * lse_i^2
  vocab_ce_grad       the loss, and the gradients of sum_i w_i loss_i with respect to h and W
  vocab_distill       distillation from a teacher's top logits u[i, k] of the tokens j[i, k]: with
                      p_i = softmax(u_i / T) over the listed tokens, q_i = softmax(z_i / T) over the
                      vocabulary, loss_i = sum_k p_ik (log p_ik - log q_i[j_ik])
  vocab_distill_grad  the loss, and the gradients of sum_i w_i loss_i with respect to h and W

A target or a listed token outside [0, V) is padding: a row without a target (or whose list is all
padding) has loss 0, lse 0 and no gradient. A token listed twice counts with both of its weights.

`run` computes each in elementary torch operations, or, where `own` is set, through the library's
calls.
"""
import types

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
CODES = {"f32": 0, "bf16": 1}  # the library's dtype codes
MOST = 65536 * 50304 * 768     # N V d of the largest cases, about


# ------------------------------------------------------------------------------- cases


def listed():
    return [
        # scoring 8 sequences' next tokens in a decode step of the Engram-27B width: reads the table once
        _ce("ce-8x128000x2560", "ce", 8, 128000, 2560, "bf16", "bf16", pad=0.0),
        # the tiny fp32 setting: 4096 tokens, vocabulary 1024
        _ce("ce-4096x1024x256-f32", "ce", 4096, 1024, 256, "f32", "f32", pad=0.0),
        # perplexity over 16 x 1024 tokens at the 200M-parameter setting
        _ce("ce-16384x50304x768", "ce", 16384, 50304, 768, "bf16", "bf16", pad=0.01),
        # a toy model's whole training batch: the launch-bound end
        _ce("ce-grad-512x1024x96-f32", "ce_grad", 512, 1024, 96, "f32", "f32", pad=0.0, gh="f32", gw="f32"),
        # ragged sequences, an odd vocabulary and width, fp32 gradient of the table for fp32 master weights
        _ce("ce-grad-3001x32003x515", "ce_grad", 3001, 32003, 515, "bf16", "bf16", pad=0.1, gh="bf16", gw="f32", weights=True),
        # a training batch of 64 x 1024 tokens at the 200M-parameter setting
        _ce("ce-grad-65536x50304x768", "ce_grad", 65536, 50304, 768, "bf16", "bf16", pad=0.0, gh="bf16", gw="bf16"),
        # two of the 4096-token sequences at the Engram-27B width, with the square of the log-partition
        _ce("ce-grad-8192x128000x2560", "ce_grad", 8192, 128000, 2560, "bf16", "bf16", pad=0.0, gh="bf16", gw="bf16", z_loss=1e-4),
        # a few positions scored against a teacher
        _distill("distill-16x50304x768-20", "distill", 16, 50304, 768, 20, "bf16", "bf16", 1.0),
        # validation of a distilled model: 4 x 1024 tokens, 64 teacher logits each
        _distill("distill-4096x50304x768-64", "distill", 4096, 50304, 768, 64, "bf16", "bf16", 1.0),
        # a small student trained in fp32, softened teacher
        _distill("distill-grad-1024x1024x256-f32", "distill_grad", 1024, 1024, 256, 16, "f32", "f32", 2.0, gh="f32", gw="f32"),
        # 8 x 1024 tokens at the 200M-parameter setting, teacher lists of up to 32
        _distill("distill-grad-8192x50304x768-32", "distill_grad", 8192, 50304, 768, 32, "bf16", "bf16", 2.0, gh="bf16", gw="bf16"),
        # one 4096-token sequence at the Engram-27B width, teacher lists of up to 100
        _distill("distill-grad-4096x128000x2560-100", "distill_grad", 4096, 128000, 2560, 100, "bf16", "bf16", 1.0, gh="bf16", gw="bf16"),
    ]


def _ce(name, op, N, V, d, h, w, pad, gh="", gw="", z_loss=0.0, weights=False):
    return {"name": name, "op": op, "N": N, "V": V, "d": d, "h": h, "w": w, "gh": gh, "gw": gw, "K": 0, "pad": pad,
            "z_loss": z_loss, "T": 1.0, "weights": weights}


def _distill(name, op, N, V, d, K, h, w, T, gh="", gw="", pad=0.0, weights=False):
    return {"name": name, "op": op, "N": N, "V": V, "d": d, "h": h, "w": w, "gh": gh, "gw": gw, "K": K, "pad": pad,
            "z_loss": 0.0, "T": T, "weights": weights}


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["ce", "ce_grad", "ce_grad", "distill", "distill_grad"])
    V = _log(rng, 500, 128000)
    d = _log(rng, 32, 2560)
    if rng.random() < 0.7:
        d = max(32, d // 8 * 8)
    h = rng.choice(["bf16", "bf16", "f32"])
    w = h if rng.random() < 0.8 else rng.choice(["bf16", "f32"])
    # fp32 operands are for smaller models: an eighth of the most work
    most = MOST // (8 if "f32" in (h, w) else 1) // (1 if op.endswith("grad") else 2)
    N = _log(rng, 1, max(1, min(65536, most // (V * d))))
    pad = rng.choice([0.0, 0.0, rng.uniform(0.01, 0.3)])
    weights = rng.random() < 0.3
    gh = gw = ""
    if op.endswith("grad"):
        gh = rng.choice([h, h, "bf16"])
        gw = rng.choice([w, w, "f32"])
    if op.startswith("ce"):
        c = _ce("", op, N, V, d, h, w, pad, gh, gw, rng.choice([0.0, 1e-4]), weights)
    else:
        c = _distill("", op, N, V, d, _log(rng, 1, 128), h, w, rng.choice([1.0, 2.0, rng.uniform(0.5, 4.0)]), gh, gw, pad, weights)
    del c["name"]
    return c


# ------------------------------------------------------------------------------ inputs


def _ids(gen, shape, vocab, zipf=1.05):
    cdf = torch.arange(1, vocab + 1, device="cuda", dtype=torch.float64).pow_(-zipf).cumsum_(0)
    u = torch.rand(shape, device="cuda", dtype=torch.float64, generator=gen) * cdf[-1]
    return torch.searchsorted(cdf, u, right=True).clamp_(max=vocab - 1).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 29)
    N, V, d, K = case["N"], case["V"], case["d"], case["K"]
    s = types.SimpleNamespace(case=case, kept=None)
    s.scale = 1.0
    std = 0.02
    W = torch.randn((V, d), device="cuda", generator=gen) * std
    s.targets = _ids(gen, (N,), V)
    # normed hidden states that lean towards their target's row, from not at all to confidently
    lean = torch.rand((N, 1), device="cuda", generator=gen) * (12.0 / (std * std * d))
    h = torch.randn((N, d), device="cuda", generator=gen) + lean * W[s.targets.long()]
    s.h, s.W = h.to(DTYPES[case["h"]]), W.to(DTYPES[case["w"]])
    if K:
        # the teacher's list: its best guess is mostly the target, the others are common tokens; a token drawn
        # twice leaves its second place empty, as a shorter list would
        ids = _ids(gen, (N, K), V)
        ids[:, 0] = s.targets
        ids, order = torch.sort(ids, dim=1)
        twice = torch.zeros_like(ids, dtype=torch.bool)
        twice[:, 1:] = ids[:, 1:] == ids[:, :-1]
        u = torch.randn((N, K), device="cuda", generator=gen) * 2.0
        u[:, 0] += 4.0
        s.teacher_logits = torch.gather(u, 1, order).contiguous()
        s.teacher_ids = torch.where(twice, -1, ids).to(torch.int32)
    if case["pad"]:
        gone = torch.rand(N, device="cuda", generator=gen) < case["pad"]
        s.targets[gone] = -1
        if K:
            s.teacher_ids[gone] = -1
    s.grad_scale = 1.0 / N
    s.weights = torch.rand(N, device="cuda", generator=gen) + 0.5 if case["weights"] else None
    return s


# ----------------------------------------------------------------------------- passes


def run(s):
    return (_own if own else _plain)[s.case["op"]](s)


def _plain_logits(s):
    return (s.h.float() @ s.W.float().T).mul_(s.scale / s.case["T"])


def _plain_grads(s, g, valid):
    """Gradients with respect to h and W from those with respect to the logits (without the rows' weights)."""
    w = torch.full_like(g[:, 0], s.grad_scale * s.scale / s.case["T"])
    if s.weights is not None:
        w = w * s.weights
    g *= torch.where(valid, w, 0)[:, None]
    return (g @ s.W.float()).to(DTYPES[s.case["gh"]]), (g.T @ s.h.float()).to(DTYPES[s.case["gw"]])


def _plain_ce(s, grad=False):
    z = _plain_logits(s)
    t = s.targets.long()
    valid = (t >= 0) & (t < s.case["V"])
    at = torch.where(valid, t, 0)[:, None]
    zt = z.gather(1, at)[:, 0]
    m = z.amax(1)
    e = z.sub_(m[:, None]).exp_()
    total = e.sum(1)
    lse = m + total.log()
    loss = torch.where(valid, lse - zt + s.case["z_loss"] * lse * lse, 0)
    if not grad:
        return loss, torch.where(valid, lse, 0)
    g = e.mul_(((1 + 2 * s.case["z_loss"] * lse) / total)[:, None])
    g.scatter_add_(1, at, torch.full_like(zt, -1.0)[:, None])
    return (loss, *_plain_grads(s, g, valid))


def _plain_distill(s, grad=False):
    z = _plain_logits(s)
    ids = s.teacher_ids.long()
    there = (ids >= 0) & (ids < s.case["V"])
    valid = there.any(1)
    at = torch.where(there, ids, 0)
    u = torch.where(there, s.teacher_logits.float() / s.case["T"], float("-inf"))
    u = torch.where(valid[:, None], u, 0)
    logp = u - u.amax(1, keepdim=True)
    logp = logp - logp.exp().sum(1, keepdim=True).log()
    p = torch.where(there, logp.exp(), 0)
    zt = z.gather(1, at)
    m = z.amax(1)
    e = z.sub_(m[:, None]).exp_()
    total = e.sum(1)
    lse = m + total.log()
    terms = torch.where(p > 0, p * (logp - (zt - lse[:, None])), 0)
    loss = torch.where(valid, terms.sum(1), 0)
    if not grad:
        return loss, torch.where(valid, lse, 0)
    g = e.mul_((1 / total)[:, None])
    g.scatter_add_(1, at, -p)
    return (loss, *_plain_grads(s, g, valid))


_plain = {"ce": _plain_ce, "ce_grad": lambda s: _plain_ce(s, True), "distill": _plain_distill,
          "distill_grad": lambda s: _plain_distill(s, True)}


def _own_buffers(s, size):
    """Outputs and workspace that a user's program keeps; size: the call's workspace query."""
    if s.kept is None:
        c = s.case
        N = c["N"]
        new = lambda shape, t: torch.empty(shape, device="cuda", dtype=t)  # noqa: E731
        first = new(N, torch.float32)
        if c["op"].endswith("grad"):
            rest = new((N, c["d"]), DTYPES[c["gh"]]), new((c["V"], c["d"]), DTYPES[c["gw"]])
        else:
            rest = (new(N, torch.float32),)
        s.kept = (first, *rest, new(size(), torch.uint8))
    return s.kept


def _own_ce(s):
    from hashed_head_gram_gb300 import pg

    c = s.case
    loss, lse, ws = _own_buffers(s, lambda: pg.vocab_ce_workspace_size(c["N"], c["V"], c["d"], CODES[c["h"]], CODES[c["w"]]))
    pg.vocab_ce(s.h, s.W, s.targets, loss, ws, scale=s.scale, z_loss=c["z_loss"], lse=lse)
    return loss, lse


def _own_ce_grad(s):
    from hashed_head_gram_gb300 import pg

    c = s.case
    loss, gh, gw, ws = _own_buffers(s, lambda: pg.vocab_ce_grad_workspace_size(
        c["N"], c["V"], c["d"], CODES[c["h"]], CODES[c["w"]], CODES[c["gh"]], CODES[c["gw"]]))
    pg.vocab_ce_grad(s.h, s.W, s.targets, loss, gh, gw, ws, scale=s.scale, z_loss=c["z_loss"], grad_scale=s.grad_scale,
                     row_weight=s.weights)
    return loss, gh, gw


def _own_distill(s):
    from hashed_head_gram_gb300 import pg

    c = s.case
    loss, lse, ws = _own_buffers(s, lambda: pg.vocab_distill_workspace_size(
        c["N"], c["V"], c["d"], c["K"], CODES[c["h"]], CODES[c["w"]]))
    pg.vocab_distill(s.h, s.W, s.teacher_ids, s.teacher_logits, loss, ws, scale=s.scale, temperature=c["T"], lse=lse)
    return loss, lse


def _own_distill_grad(s):
    from hashed_head_gram_gb300 import pg

    c = s.case
    loss, gh, gw, ws = _own_buffers(s, lambda: pg.vocab_distill_grad_workspace_size(
        c["N"], c["V"], c["d"], c["K"], CODES[c["h"]], CODES[c["w"]], CODES[c["gh"]], CODES[c["gw"]]))
    pg.vocab_distill_grad(s.h, s.W, s.teacher_ids, s.teacher_logits, loss, gh, gw, ws, scale=s.scale, temperature=c["T"],
                          grad_scale=s.grad_scale, row_weight=s.weights)
    return loss, gh, gw


_own = {"ce": _own_ce, "ce_grad": _own_ce_grad, "distill": _own_distill, "distill_grad": _own_distill_grad}


# ------------------------------------------------------------------------ work and exact


def work(case):
    size = {"f32": 4, "bf16": 2}
    N, V, d, K = case["N"], case["V"], case["d"], case["K"]
    grad = case["op"].endswith("grad")
    b = N * d * size[case["h"]] + V * d * size[case["w"]] + N * (8 * K if K else 4) + (4 * N if case["weights"] and grad else 0)
    if grad:
        return {"bytes": b + 4 * N + N * d * size[case["gh"]] + V * d * size[case["gw"]], "flops": 6 * N * V * d}
    return {"bytes": b + 8 * N, "flops": 2 * N * V * d}


def exact(case, seed):
    """The definitions in 64 bits, a block of rows at a time."""
    N, V, d = case["N"], case["V"], case["d"]
    grad = case["op"].endswith("grad")
    if (6 if grad else 2) * N * V * d > 1.2e13:
        return None  # more than some 20 seconds of 64-bit products
    s = prepare(case, seed)
    W = s.W.double()
    loss = torch.zeros(N, device="cuda", dtype=torch.float64)
    lse = torch.zeros_like(loss)
    gh = torch.zeros((N, d), device="cuda", dtype=torch.float64) if grad else None
    gw = torch.zeros((V, d), device="cuda", dtype=torch.float64) if grad else None
    wide = s.scale / case["T"]
    for lo in range(0, N, 2048):
        rows = slice(lo, min(N, lo + 2048))
        h = s.h[rows].double()
        z = wide * (h @ W.T)
        lse[rows] = torch.logsumexp(z, 1)
        if case["K"]:
            q = torch.zeros_like(z)  # the teacher's distribution over the vocabulary
            n = z.shape[0]
            ids, u = s.teacher_ids[rows].cpu().numpy().astype(np.int64), s.teacher_logits[rows].double().cpu().numpy() / case["T"]
            ok = (ids >= 0) & (ids < V)
            has = ok.any(1)
            top = np.where(ok, u, -np.inf).max(1, initial=-np.inf)
            p = np.where(ok, np.exp(u - np.where(has, top, 0.0)[:, None]), 0.0)
            p /= np.where(has, p.sum(1), 1.0)[:, None]
            entropy = np.where(p > 0, p * np.log(np.where(p > 0, p, 1.0)), 0.0).sum(1)
            r, k = np.nonzero(ok)
            r, c = torch.from_numpy(r).cuda(), torch.from_numpy(ids[r, k]).cuda()
            q.index_put_((r, c), torch.from_numpy(p[ok]).cuda(), accumulate=True)
            keep = torch.from_numpy(has).cuda()
            loss[rows] = torch.where(keep, torch.from_numpy(entropy).cuda() - (q * z).sum(1) + lse[rows], 0.0)
            beta = torch.ones(n, device="cuda", dtype=torch.float64)
        else:
            t = s.targets[rows].long()
            keep = (t >= 0) & (t < V)
            at = torch.nonzero(keep)[:, 0]
            q = torch.zeros_like(z)
            q[at, t[at]] = 1.0
            loss[rows][at] = lse[rows][at] - z[at, t[at]] + case["z_loss"] * lse[rows][at] ** 2
            beta = 1.0 + 2.0 * case["z_loss"] * lse[rows]
        if not grad:
            lse[rows] *= keep
            continue
        w = s.grad_scale * wide * keep.double()
        if s.weights is not None:
            w = w * s.weights[rows].double()
        g = (beta[:, None] * torch.softmax(z, 1) - q) * w[:, None]
        gh[rows] = g @ W
        gw += g.T @ h
    return (loss, gh, gw) if grad else (loss, lse)
