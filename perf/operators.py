"""Timed cases of the operators that train a hashed N-gram memory and the token embedding it sits on.

Four operators:

  embed          out[t] = scale * E[P[x_t]]: token embedding lookup with scaling, through the
                 canonical map P when there is one
  embed_grad     dE[v] = scale * sum_{t: P[x_t] = v} dout[t], dense over the vocabulary
  lookup_grad    the gradient of the hashed multi-head lookup's table: per distinct table row
                 that the batch read, the sum of the signed head gradients of every read of it;
                 rows ascending, their count beside them
  orthogonalize  the orthogonalised update of a stack of weight matrices: X_0 = G / (|G|_F + eps),
                 then `steps` times A = X X^T, X <- a X + (b A + c A A) X on the shorter side

`run` computes each in elementary torch operations, or, where `own` is set, through the
library's calls. A token outside [0, vocab) is padding to the embedding (a zero row, no
gradient), and reads as ID 0 in the hashed lookup.
"""
import types

import numpy as np
import torch

own = False

MASK32 = 0xFFFFFFFF
GOLDEN = 0x9E3779B97F4A7C15
FLAT, ENGRAM, PAGEGRAM = 0, 1, 2
COEFFS = (3.4445, -4.7750, 2.0315)  # the quintic's usual coefficients
STEPS = 5
EPS = 1e-7
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------- cases


def listed():
    return [
        # one decode step's input rows: 8 new tokens, Engram-27B width, canonical IDs
        _embed("embed-decode8-2560", 8, 128000, 98010, 2560, "bf16", "bf16", 0.0),
        # a training batch of 64 x 1024 tokens at the 200M-parameter setting; fp32 master weights
        _embed("embed-65536-768", 65536, 50304, 0, 768, "f32", "bf16", 0.0),
        # a toy model's whole batch: the launch-bound end
        _embed_grad("embed-grad-512-96", 512, 1024, 0, 96, "f32", "f32", 0.0, 0.0),
        # the 64 x 1024 batch with Zipf(1.1) IDs: one ID takes a tenth of the batch
        _embed_grad("embed-grad-65536-768", 65536, 50304, 0, 768, "bf16", "f32", 1.1, 0.0),
        # 7 ragged sequences padded to 4681, canonical IDs, gradient kept in bf16
        _embed_grad("embed-grad-32767-2560", 32767, 128000, 98010, 2560, "bf16", "bf16", 1.05, 0.03),
        # the tiny fp32 setting: 4096 tokens on 64 + 64 pages
        _lookup("lookup-grad-tiny", 1, 4096, 1024, 0, 0.0, PAGEGRAM, "2,3", 8, 4, 64, 64, "f32", "f32"),
        # PageGram, 200M parameters, 64 x 1024 tokens: a million row reads
        _lookup("lookup-grad-pagegram", 64, 1024, 50304, 0, 1.1, PAGEGRAM, "2,3", 8, 4, 64, 48823, "bf16", "f32"),
        # Engram-27B-shaped subtables, 8 x 4096 tokens, 80-wide heads
        _lookup("lookup-grad-engram", 8, 4096, 128000, 98010, 1.05, ENGRAM, "2,3", 8, 1, 80, 2226562, "bf16", "f32"),
        # the flat 200M control: two 768-wide rows a token sharing one gradient
        _lookup("lookup-grad-flat", 64, 1024, 50304, 0, 1.1, FLAT, "2,3", 1, 1, 768, 130208, "bf16", "f32"),
        # the tiny setting's projection
        _ortho("ortho-256x1024", 1, 256, 1024, "f32"),
        # the 200M setting's projection
        _ortho("ortho-768x1024", 1, 768, 1024, "bf16"),
        # the Engram-27B-shaped module's W_V and four W_K
        _ortho("ortho-5x2560x1280", 5, 2560, 1280, "bf16"),
    ]


def _embed(name, N, vocab, canon, d, table, out, pad):
    return {"name": name, "op": "embed", "N": N, "vocab": vocab, "canon": canon, "d": d, "table": table, "out": out,
            "zipf": 1.05, "pad": pad}


def _embed_grad(name, N, vocab, canon, d, grad, out, zipf, pad):
    return {"name": name, "op": "embed_grad", "N": N, "vocab": vocab, "canon": canon, "d": d, "grad": grad, "out": out,
            "zipf": zipf, "pad": pad}


def _lookup(name, B, L, vocab, canon, zipf, mode, orders, K, S, r, span, grad, out):
    """span: pages an order (PageGram), rows a subtable (Engram) or an order (flat); each next one is a little smaller."""
    return {"name": name, "op": "lookup_grad", "B": B, "L": L, "vocab": vocab, "canon": canon, "zipf": zipf, "mode": mode,
            "orders": orders, "K": K, "S": S, "r": r, "span": span, "grad": grad, "out": out}


def _ortho(name, batch, m, n, grad):
    return {"name": name, "op": "orthogonalize", "batch": batch, "m": m, "n": n, "grad": grad}


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "lookup_grad", "orthogonalize"])
    kind = lambda: rng.choice(["f32", "bf16"])  # noqa: E731
    if op in ("embed", "embed_grad"):
        vocab = _log(rng, 500, 128000)
        canon = rng.choice([0, max(1, int(vocab * rng.uniform(0.6, 0.99)))])
        d = _log(rng, 32, 2560)
        if rng.random() < 0.7:
            d = max(32, d // 8 * 8)
        N = _log(rng, 1, min(65536, 65536 * 768 // d))
        pad = rng.choice([0.0, 0.0, rng.uniform(0.01, 0.3)])
        c = (_embed if op == "embed" else _embed_grad)("", N, vocab, canon, d, kind(), kind(), *((pad,) if op == "embed" else (0.0, pad)))
        c["zipf"] = rng.choice([0.0, rng.uniform(0.9, 1.3)])
    elif op == "lookup_grad":
        mode = rng.choice([FLAT, ENGRAM, PAGEGRAM])
        orders = rng.choice(["2", "2,3", "2,3", "1,2,3", "3,4", "1,2,3,4"])
        count = len(orders.split(","))
        K = 1 if mode == FLAT else rng.randint(1, 8)
        r = 8 * _log(rng, 1, 96) if mode == FLAT else 8 * rng.randint(1, 16)
        most = max(1, min(65536, 65536 * 1024 // (count * K * max(r, 32))))
        B = rng.randint(1, min(16, most))
        L = _log(rng, 1, max(1, most // B))
        S = rng.choice([1, 3, 4, 8, 15]) if mode == PAGEGRAM else 1
        span = _log(rng, 50, {FLAT: 130208, ENGRAM: 2226562, PAGEGRAM: 48823}[mode])
        vocab = _log(rng, 500, 128000)
        c = _lookup("", B, L, vocab, rng.choice([0, int(vocab * 0.77)]), rng.choice([0.0, rng.uniform(0.9, 1.3)]), mode, orders, K, S, r,
                    span, kind(), rng.choice(["f32", "f32", "bf16"]))
    else:
        c = _ortho("", rng.randint(1, 5), _log(rng, 24, 2560), _log(rng, 24, 1280), kind())
        if rng.random() < 0.5:
            c["m"], c["n"] = c["n"], c["m"]
        if rng.random() < 0.5:
            c["m"], c["n"] = max(24, c["m"] // 8 * 8), max(24, c["n"] // 8 * 8)
    del c["name"]
    return c


# ------------------------------------------------------------------------------ inputs


def _ids(gen, shape, vocab, zipf):
    if not zipf:
        return torch.randint(0, vocab, shape, device="cuda", dtype=torch.int32, generator=gen)
    cdf = torch.arange(1, vocab + 1, device="cuda", dtype=torch.float64).pow_(-zipf).cumsum_(0)
    u = torch.rand(shape, device="cuda", dtype=torch.float64, generator=gen) * cdf[-1]
    return torch.searchsorted(cdf, u, right=True).clamp_(max=vocab - 1).to(torch.int32)


def _canon_map(gen, vocab, canon):
    """uint32 values in int32: IDs below `canon` keep their value, the rest fold into them."""
    if not canon:
        return None
    m = torch.arange(vocab, device="cuda", dtype=torch.int32)
    m[canon:] = torch.randint(0, canon, (vocab - canon,), device="cuda", dtype=torch.int32, generator=gen)
    return m


def _normal(gen, shape, dtype, std=1.0):
    return (torch.randn(shape, device="cuda", generator=gen) * std).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    s = types.SimpleNamespace(case=case, kept=None)
    op = case["op"]
    if op in ("embed", "embed_grad"):
        s.rows = case["canon"] or case["vocab"]
        s.scale = float(case["d"]) ** 0.5
        s.tokens = _ids(gen, (case["N"],), case["vocab"], case["zipf"])
        if case["pad"]:
            s.tokens[torch.rand(case["N"], device="cuda", generator=gen) < case["pad"]] = -1
        s.canon = _canon_map(gen, case["vocab"], case["canon"])
        if op == "embed":
            s.table = _normal(gen, (s.rows, case["d"]), DTYPES[case["table"]], 0.02)
        else:
            s.grad = _normal(gen, (case["N"], case["d"]), DTYPES[case["grad"]], 1e-3)
    elif op == "lookup_grad":
        s.plan = _plan(case)
        s.tokens = _ids(gen, (case["B"], case["L"]), case["vocab"], case["zipf"])
        s.canon = _canon_map(gen, case["vocab"], case["canon"])
        s.grad = _normal(gen, (case["B"] * case["L"], s.plan.width), DTYPES[case["grad"]], 1e-3)
    else:  # momentum of gradients: noise with a few strong directions
        b, m, n = case["batch"], case["m"], case["n"]
        g = torch.randn((b, m, n), device="cuda", generator=gen)
        u = torch.randn((b, m, 4), device="cuda", generator=gen)
        v = torch.randn((b, 4, n), device="cuda", generator=gen)
        s.G = ((g + 0.25 * (u @ v)) * 1e-3).to(DTYPES[case["grad"]])
    return s


def _plan(case):
    """The table's descriptor (sizes and a hash seed) and its constants as device tensors."""
    orders = [int(o) for o in case["orders"].split(",")]
    O, K, S, span, mode = len(orders), case["K"], case["S"], case["span"], case["mode"]
    div = np.array([[max(1, span - 2 * (o * K + k)) for k in range(K)] for o in range(O)], np.int64)
    if mode == PAGEGRAM:
        div = np.repeat(div[:, :1], K, axis=1)
        size = div[:, :1] * K * S
        base = np.repeat(np.cumsum(size) - size[:, 0], K).reshape(O, K) + np.arange(K) * S
    else:
        base = (np.cumsum(div) - div.reshape(-1)).reshape(O, K)
    seed = 0x5DEECE66D
    kind, o, k, j = np.meshgrid(np.arange(3), np.arange(O), np.arange(K), np.arange(4), indexing="ij")
    fid = (((kind * 4 + o) * 64 + k) * 4 + j).astype(np.uint64)
    fid[0] = fid[0][:, :1]  # one page hash an order
    mult = _mix64_np(np.uint64(seed) + np.uint64(GOLDEN) * (fid + np.uint64(1))) | np.uint64(1)
    mult[:, np.arange(4)[None, None, :].repeat(O, 0).repeat(K, 1) >= np.array(orders)[:, None, None]] = 0  # positions past an order
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    r = case["r"]
    return types.SimpleNamespace(
        mode=mode, hash_kind=0, orders=orders, K=K, S=S, r=r, row_dtype=1 if case["grad"] == "bf16" else 0, hash_seed=seed,
        pages=[int(x) for x in div[:, 0]] if mode == PAGEGRAM else [],
        rows=[] if mode == PAGEGRAM else [[int(x) for x in row] for row in div],
        width=r if mode == FLAT else O * K * r, mult=dev(mult.view(np.int64)), div=dev(div), base=dev(base))


def _mix64_np(z):
    z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
    z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
    return z ^ (z >> np.uint64(31))


# ----------------------------------------------------------------------------- passes


def run(s):
    return (_own if own else _plain)[s.case["op"]](s)


def _plain_rows(s):
    """Embedding row of each position; -1 where it has none."""
    t = s.tokens.long()
    ok = (t >= 0) & (t < s.case["vocab"])
    t = torch.where(ok, t, 0)
    if s.canon is not None:
        t = s.canon[t].long()
    return torch.where(ok & (t < s.rows), t, -1)


def _plain_embed(s):
    rows = _plain_rows(s)
    x = s.table[rows.clamp(min=0)].float() * s.scale
    return torch.where(rows[:, None] >= 0, x, 0).to(DTYPES[s.case["out"]])


def _plain_embed_grad(s):
    rows = _plain_rows(s)
    g = torch.zeros((s.rows + 1, s.case["d"]), device="cuda")
    g.index_add_(0, torch.where(rows >= 0, rows, s.rows), s.grad.float())
    return (g[:-1] * s.scale).to(DTYPES[s.case["out"]])


def _shr(z, k):
    return (z >> k) & ((1 << (64 - k)) - 1)


def _mix64(z):
    z = (z ^ _shr(z, 30)) * (0xBF58476D1CE4E5B9 - (1 << 64))
    z = (z ^ _shr(z, 27)) * (0x94D049BB133111EB - (1 << 64))
    return z ^ _shr(z, 31)


def _plain_hash(s):
    """(rows int64 [N, O, K], sign hashes int64 [N, O, K]) of every head read."""
    p, B, L = s.plan, s.case["B"], s.case["L"]
    t = s.tokens.long()
    t = torch.where((t >= 0) & (t < s.case["vocab"]), t, 0)
    if s.canon is not None:
        t = s.canon[t].long()
    t = torch.nn.functional.pad(t, (3, 0), value=MASK32)
    c = torch.stack([t[:, 3 - j:3 - j + L] for j in range(4)], -1).reshape(B * L, 1, 1, 4)
    h = [c[..., 0] * m[..., 0] ^ c[..., 1] * m[..., 1] ^ c[..., 2] * m[..., 2] ^ c[..., 3] * m[..., 3] for m in p.mult]
    page, head = ((x ^ _shr(x, 32)) & MASK32 for x in h[:2])
    if p.mode == PAGEGRAM:
        return p.base + page % p.div * (p.K * p.S) + head % p.S, h[2]
    return p.base + head % p.div, h[2]


def _plain_lookup_grad(s):
    p, r = s.plan, s.case["r"]
    rows, hs = _plain_hash(s)
    words = -(-r // 64)
    q = torch.arange(1, words + 1, device="cuda") * (GOLDEN - (1 << 64))
    bits = _mix64(hs[..., None] + q)[..., None] >> torch.arange(64, device="cuda") & 1
    sign = (1 - 2 * bits.to(torch.int8)).reshape(*hs.shape, -1)[..., :r]
    g = s.grad.view(-1, 1, 1, r) if p.mode == FLAT else s.grad.view(-1, len(p.orders), p.K, r)
    g = (g * sign).float().reshape(-1, r)
    uniq, where = torch.unique(rows.reshape(-1), sorted=True, return_inverse=True)
    n = rows.numel()
    rows_out = torch.full((n,), -1, device="cuda", dtype=torch.int32)
    rows_out[:uniq.numel()] = uniq.to(torch.int32)
    sums = torch.zeros((n, r), device="cuda").index_add_(0, where, g)
    return rows_out, sums.to(DTYPES[s.case["out"]]), torch.tensor([uniq.numel()], device="cuda", dtype=torch.int32)


def _plain_orthogonalize(s):
    a, b, c = COEFFS
    x = s.G.float()
    flip = x.shape[1] > x.shape[2]
    x = x.mT if flip else x
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    for _ in range(STEPS):
        y = x @ x.mT
        x = a * x + (b * y + c * (y @ y)) @ x
    return (x.mT if flip else x).to(torch.bfloat16).contiguous()


_plain = {"embed": _plain_embed, "embed_grad": _plain_embed_grad, "lookup_grad": _plain_lookup_grad, "orthogonalize": _plain_orthogonalize}


def _own_embed(s):
    from hashed_head_gram_gb300 import pg

    if s.kept is None:
        s.kept = torch.empty((s.case["N"], s.case["d"]), device="cuda", dtype=DTYPES[s.case["out"]])
    pg.embed(s.tokens, s.table, s.kept, s.case["vocab"], scale=s.scale, canon_map=s.canon)
    return s.kept


def _own_embed_grad(s):
    from hashed_head_gram_gb300 import pg

    if s.kept is None:
        ws = pg.embed_grad_workspace_size(s.case["N"], s.rows, s.case["d"])
        s.kept = (torch.empty((s.rows, s.case["d"]), device="cuda", dtype=DTYPES[s.case["out"]]),
                  torch.empty(ws, device="cuda", dtype=torch.uint8))
    out, ws = s.kept
    pg.embed_grad(s.tokens, s.grad, out, s.case["vocab"], ws, scale=s.scale, canon_map=s.canon)
    return out


def _own_lookup_grad(s):
    from hashed_head_gram_gb300 import pg

    if s.kept is None:
        N, n = s.grad.shape[0], s.grad.shape[0] * len(s.plan.orders) * s.plan.K
        desc = pg.table_desc(s.plan, s.case["vocab"], s.case["canon"] or None)
        s.kept = (desc, torch.empty(n, device="cuda", dtype=torch.int32),
                  torch.empty((n, s.case["r"]), device="cuda", dtype=DTYPES[s.case["out"]]),
                  torch.empty(1, device="cuda", dtype=torch.int32),
                  torch.empty(pg.lookup_grad_workspace_size(desc, N), device="cuda", dtype=torch.uint8))
    desc, rows, sums, count, ws = s.kept
    pg.lookup_grad(desc, s.tokens, s.grad, rows, sums, count, ws, canon_map=s.canon)
    return rows, sums, count


def _own_orthogonalize(s):
    from hashed_head_gram_gb300 import pg

    if s.kept is None:
        ws = pg.orthogonalize_workspace_size(*s.G.shape)
        s.kept = (torch.empty(s.G.shape, device="cuda", dtype=torch.bfloat16), torch.empty(ws, device="cuda", dtype=torch.uint8))
    out, ws = s.kept
    pg.orthogonalize(s.G, out, ws, steps=STEPS, coeffs=COEFFS, eps=EPS)
    return out


_own = {"embed": _own_embed, "embed_grad": _own_embed_grad, "lookup_grad": _own_lookup_grad, "orthogonalize": _own_orthogonalize}


# ------------------------------------------------------------------------ work and exact


def work(case):
    size = {"f32": 4, "bf16": 2}
    op = case["op"]
    if op == "embed":
        N, d = case["N"], case["d"]
        return {"bytes": N * (4 + d * (size[case["table"]] + size[case["out"]])), "flops": N * d}
    if op == "embed_grad":
        N, d, rows = case["N"], case["d"], case["canon"] or case["vocab"]
        return {"bytes": N * (4 + d * size[case["grad"]]) + rows * d * size[case["out"]], "flops": N * d}
    if op == "lookup_grad":
        N, r = case["B"] * case["L"], case["r"]
        items = len(case["orders"].split(",")) * case["K"]
        width = r if case["mode"] == FLAT else items * r
        return {"bytes": N * (4 + width * size[case["grad"]]) + N * items * (4 + r * size[case["out"]]) + 4, "flops": N * items * r}
    b, p, q = case["batch"], min(case["m"], case["n"]), max(case["m"], case["n"])
    # A = X X^T and A A are symmetric: half of each is enough
    return {"bytes": b * p * q * (size[case["grad"]] + 2), "flops": b * STEPS * (p * p * q + p * p * p + 2 * p * p * q)}


def exact(case, seed):
    """The definitions in 64 bits: hashing in numpy's unsigned integers, sums and products in float64."""
    s = prepare(case, seed)
    op = case["op"]
    if op in ("embed", "embed_grad"):
        t = s.tokens.cpu().numpy().astype(np.int64)
        ok = (t >= 0) & (t < case["vocab"])
        ids = np.where(ok, t, 0)
        if s.canon is not None:
            ids = s.canon.cpu().numpy().view(np.uint32).astype(np.int64)[ids]
        ok &= ids < s.rows
        at = torch.from_numpy(np.flatnonzero(ok)).cuda()
        ids = torch.from_numpy(ids).cuda()[at]
        if op == "embed":
            out = torch.zeros((case["N"], case["d"]), device="cuda", dtype=torch.float64)
            out[at] = s.table[ids].double() * s.scale
            return out
        out = torch.zeros((s.rows, case["d"]), device="cuda", dtype=torch.float64)
        return out.index_add_(0, ids, s.grad[at].double()).mul_(s.scale)
    if op == "orthogonalize":
        a, b, c = COEFFS
        outs = []
        for g in s.G.double():
            x = g / (torch.linalg.norm(g) + EPS)
            for _ in range(STEPS):
                if x.shape[0] <= x.shape[1]:
                    k = x @ x.T
                    x = a * x + b * (k @ x) + c * (k @ (k @ x))
                else:
                    k = x.T @ x
                    x = a * x + b * (x @ k) + c * ((x @ k) @ k)
            outs.append(x)
        return torch.stack(outs)
    return _exact_lookup_grad(s)


def _exact_lookup_grad(s):
    case, p, u = s.case, s.plan, np.uint64
    t = s.tokens.cpu().numpy().astype(np.int64)
    t[(t < 0) | (t >= case["vocab"])] = 0
    ids = t.astype(u) if s.canon is None else s.canon.cpu().numpy().view(np.uint32).astype(u)[t]
    B, L, r = case["B"], case["L"], case["r"]
    K = case["K"]

    def hashed(kind, o, k, n):
        h = np.zeros((B, L), u)
        for j in range(n):
            m = _mix64_np(np.array([(p.hash_seed + GOLDEN * (1 + ((kind * 4 + o) * 64 + k) * 4 + j)) & (2 ** 64 - 1)], u)) | u(1)
            c = np.full((B, L), MASK32, u)
            c[:, j:] = ids[:, :L - j] if j < L else 0
            h ^= c * m
        return h.reshape(-1)

    fold = lambda h: ((h ^ (h >> u(32))) & u(MASK32)).astype(np.int64)  # noqa: E731
    rows, grads, start = [], [], 0
    for o, n in enumerate(p.orders):
        for k in range(K):
            head = fold(hashed(1, o, k, n))
            if p.mode == PAGEGRAM:
                row = start + (fold(hashed(0, o, 0, n)) % p.pages[o] * K + k) * p.S + head % p.S
            else:
                row = start + head % p.rows[o][k]
                start += p.rows[o][k]
            word = hashed(2, o, k, n)
            bits = np.stack([_mix64_np(word + u(GOLDEN * (q + 1) & (2 ** 64 - 1))) for q in range(-(-r // 64))], 1)
            neg = np.unpackbits(bits.astype("<u8").view(np.uint8).reshape(len(word), -1), axis=1, bitorder="little")[:, :r]
            at = 0 if p.mode == FLAT else (o * K + k) * r
            rows.append(torch.from_numpy(row).cuda())
            grads.append(torch.where(torch.from_numpy(neg).cuda() > 0, -s.grad[:, at:at + r].double(), s.grad[:, at:at + r].double()))
        if p.mode == PAGEGRAM:
            start += p.pages[o] * K * p.S
    rows, order = torch.sort(torch.cat(rows))
    first = torch.ones_like(rows, dtype=torch.bool)
    first[1:] = rows[1:] != rows[:-1]
    n, count = rows.numel(), int(first.sum())
    rows_out = torch.full((n,), -1, device="cuda", dtype=torch.int32)
    rows_out[:count] = rows[first].to(torch.int32)
    sums = torch.zeros((n, r), device="cuda", dtype=torch.float64)
    sums.index_add_(0, torch.cumsum(first, 0) - 1, torch.cat(grads)[order])
    return rows_out, sums, torch.tensor([count], device="cuda", dtype=torch.int32)
