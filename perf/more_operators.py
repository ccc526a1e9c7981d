"""The two ends of a language model's training step, and the dropout between its
sublayers, measured: the embedding lookup and its gradient, dropout whose mask
is never stored, and log probabilities of given tokens (with the distribution's
entropy and its most likely tokens) and their gradient.

A case is one call on inputs like those of a training or serving step.  `run`
computes it in plain torch operations, in 32 bits, where `own` is false, and
through the library (fsdp_emulated_ranks_gb300.cr) where it is true.

Dropout's random numbers are the words of Philox4x32-10 (Salmon, Moraes, Dror
and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011): the counter
{column / 8, row, offset's low word, offset's high word} under a 64-bit seed
gives eight 16-bit numbers for eight columns, low halves first, and an element
is kept where its number is at least round(65536 p).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # One generated token on its way in: the latency of a small call.
        {"name": "embed_token", "op": "embed", "tokens": 1, "vocab": 32000, "dim": 2048, "dtype": "bf16", "out": "bf16"},
        # A micro-batch of 8192 tokens at the benchmark transformer's vocabulary and width.
        {"name": "embed_step", "op": "embed", "tokens": 8192, "vocab": 32000, "dim": 2048, "dtype": "bf16", "out": "bf16"},
        # The embedding's gradient in the same step, dense, as the gradient collectives take it.
        {"name": "embed_back_step", "op": "embed_back", "tokens": 8192, "vocab": 32000, "dim": 2048, "dtype": "bf16",
         "out": "bf16", "base": False, "pad": 0.0},
        # fp32 gradients of a padded micro-batch at odd sizes, added to those of the micro-batches before.
        {"name": "embed_back_odd", "op": "embed_back", "tokens": 3001, "vocab": 50257, "dim": 1111, "dtype": "f32",
         "out": "f32", "base": True, "pad": 0.2},
        # A sublayer's output on its way into the residual stream.
        {"name": "dropout_step", "op": "dropout", "rows": 8192, "cols": 2048, "dtype": "bf16", "residual": True, "p": 0.1},
        # The backward pass of one without a residual, fp32, at a width that is not a multiple of anything.
        {"name": "dropout_odd", "op": "dropout", "rows": 1777, "cols": 4099, "dtype": "f32", "residual": False, "p": 0.25},
        # One generated token: its distribution's 20 most likely tokens.
        {"name": "logp_token", "op": "logp", "rows": 1, "vocab": 32000, "dtype": "bf16", "top": 20, "temp": 0.7, "masked": False},
        # A batch of generated tokens with a large vocabulary.
        {"name": "logp_batch", "op": "logp", "rows": 64, "vocab": 131072, "dtype": "bf16", "top": 5, "temp": 1.0, "masked": False},
        # The loss of a training step.
        {"name": "logp_step", "op": "logp", "rows": 8192, "vocab": 32000, "dtype": "bf16", "top": 0, "temp": 1.0, "masked": False},
        # Scores of a prompt in fp32, most tokens ruled out by a grammar, at an odd vocabulary.
        {"name": "logp_odd", "op": "logp", "rows": 1531, "vocab": 50257, "dtype": "f32", "top": 8, "temp": 1.0, "masked": True},
        # The loss's gradient in the training step.
        {"name": "logp_back_step", "op": "logp_back", "rows": 8192, "vocab": 32000, "dtype": "bf16", "temp": 1.0,
         "entropy": False, "masked": False},
        # A policy gradient with an entropy term, fp32, a ragged micro-batch at an odd vocabulary.
        {"name": "logp_back_odd", "op": "logp_back", "rows": 515, "vocab": 50257, "dtype": "f32", "temp": 0.9,
         "entropy": True, "masked": True},
    ]


def _size(rng, lo, hi):
    """A size between lo and hi, even over the logarithm; odd numbers and multiples of 128 among them."""
    k = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    kind = rng.randrange(3)
    if kind == 0 and k >= 128:
        k -= k % 128
    elif kind == 1 and k < hi:
        k |= 1
    return max(lo, min(hi, k))


def draw(rng):
    op = rng.choice(["embed", "embed_back", "dropout", "logp", "logp_back"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("embed", "embed_back"):
        tokens, vocab, dim = _size(rng, 1, 16384), _size(rng, 256, 131072), _size(rng, 64, 8192)
        while tokens * dim > 8192 * 2048:
            tokens = max(1, tokens // 2)
        while vocab * dim > 65536 * 2048:
            vocab = max(256, vocab // 2)
        c = {"op": op, "tokens": tokens, "vocab": vocab, "dim": dim, "dtype": dtype, "out": rng.choice(["bf16", dtype])}
        if op == "embed_back":
            c["base"], c["pad"] = rng.random() < 0.3, rng.choice([0.0, 0.1, 0.5])
        return c
    if op == "dropout":
        rows, cols = _size(rng, 1, 16384), _size(rng, 64, 8192)
        while rows * cols > 8192 * 4096:
            rows = max(1, rows // 2)
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "residual": rng.random() < 0.5,
                "p": rng.choice([0.05, 0.1, 0.2, 0.5])}
    rows, vocab = _size(rng, 1, 8192), _size(rng, 256, 262144)
    while rows * vocab * (2 if dtype == "f32" else 1) > 8192 * 32000:
        rows = max(1, rows // 2)
    c = {"op": op, "rows": rows, "vocab": vocab, "dtype": dtype, "temp": rng.choice([0.7, 1.0, 1.3]), "masked": rng.random() < 0.3}
    if op == "logp":
        c["top"] = rng.choice([0, 1, 5, 20, 32])
    else:
        c["entropy"] = rng.random() < 0.5
    return c


def _bytes(dtype):
    return 4 if dtype == "f32" else 2


def work(case):
    op = case["op"]
    if op == "embed":
        t, d = case["tokens"], case["dim"]
        rows = _distinct(t, case["vocab"])  # a row that several tokens name is read once
        return {"bytes": 8 * t + rows * d * _bytes(case["dtype"]) + t * d * _bytes(case["out"]), "flops": t * d}
    if op == "embed_back":
        t, d, v = case["tokens"], case["dim"], case["vocab"]
        used = t - int(t * case["pad"])
        moved = v * d * _bytes(case["out"]) * (2 if case["base"] else 1)
        return {"bytes": 8 * t + used * d * _bytes(case["dtype"]) + moved, "flops": used * d + v * d}
    if op == "dropout":
        n, e = case["rows"] * case["cols"], _bytes(case["dtype"])
        # ten rounds of two 32 x 32-bit products for eight elements, a product, a sum
        return {"bytes": n * e * (3 if case["residual"] else 2), "flops": n * 20 // 8 + 2 * n}
    r, v, e = case["rows"], case["vocab"], _bytes(case["dtype"])
    if op == "logp":
        return {"bytes": r * v * e + r * (8 + 12 + 8 * case["top"]), "flops": 5 * r * v}
    return {"bytes": 2 * r * v * e + r * (8 + 16), "flops": 6 * r * v}


def _ids(n, vocab, g):
    """Token ids whose frequency falls as 1 / (id + 1), as in a vocabulary sorted by use."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    return (torch.exp(u * math.log(vocab + 1)) - 1.0).long().clamp(0, vocab - 1)


def _distinct(n, vocab):
    """How many different ids n of _ids have, on average."""
    k = np.arange(vocab)
    return round(float(-np.expm1(n * np.log1p(-np.log1p(1 / (k + 1.0)) / math.log(vocab + 1))).sum()))


def _logits(r, v, dt, masked, g):
    """Logits of rows of different sharpness (made in blocks of rows, to spare memory), of which a
    mask leaves one token in 16 where it is wanted; and targets that it leaves."""
    x = torch.empty(r, v, dtype=dt, device="cuda")
    targets = torch.randint(0, v, (r,), generator=g, device="cuda")
    for lo in range(0, r, 1024):
        part = torch.randn(min(1024, r - lo), v, generator=g, device="cuda")
        part *= torch.exp(torch.randn(part.shape[0], 1, generator=g, device="cuda") * 0.5 + 0.5)
        rows = torch.arange(part.shape[0], device="cuda")
        # most targets are likely tokens
        part[rows, targets[lo:lo + 1024]] += 4.0
        if masked:
            off = torch.rand(part.shape[0], v, generator=g, device="cuda") < 15 / 16
            off[rows, targets[lo:lo + 1024]] = False
            part.masked_fill_(off, -math.inf)
        x[lo:lo + 1024] = part
    return x, targets


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dev = torch.device("cuda")

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev) * std

    s = dict(case)
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op in ("embed", "embed_back"):
        t, v, d, out = case["tokens"], case["vocab"], case["dim"], DTYPES[case["out"]]
        s["ids"] = _ids(t, v, g)
        s["scale"] = math.sqrt(d)
        if op == "embed":
            s["table"] = normal(v, d, std=d ** -0.5).to(dt)
            s["y"] = torch.empty(t, d, dtype=out, device=dev)
            return s
        if case["pad"]:  # the batch's last places hold no token
            s["ids"][t - int(t * case["pad"]):] = -1
        s["dy"] = normal(t, d, std=1e-3).to(dt)
        s["sum"] = normal(v, d, std=1e-3).to(out) if case["base"] else None
        s["dtable"] = torch.empty(v, d, dtype=out, device=dev)
        # the library's workspace: every token once and a few numbers, and fp32 sums
        s["work"] = torch.empty(64 * t + 8 * t * d + (8 << 20), dtype=torch.uint8, device=dev)
        return s
    if op == "dropout":
        r, c = case["rows"], case["cols"]
        s["x"] = normal(r, c).to(dt)
        s["res"] = normal(r, c).to(dt) if case["residual"] else None
        # seed and offset, where a captured step can find and move them
        s["rng"] = torch.tensor([(int(seed) * 0x9E3779B97F4A7C15 + 12345) % (1 << 63), 1000 + int(seed) % 977],
                                dtype=torch.int64, device=dev)
        s["layer"] = 3
        s["y"] = torch.empty(r, c, dtype=dt, device=dev)
        return s
    r, v = case["rows"], case["vocab"]
    s["scale"] = 1.0 / case["temp"]
    s["x"], s["t"] = _logits(r, v, dt, case["masked"], g)
    if op == "logp":
        for name in ("logp", "ent", "lse"):
            s[name] = torch.empty(r, device=dev)
        s["ti"] = torch.empty(r, case["top"], dtype=torch.int32, device=dev)
        s["tl"] = torch.empty(r, case["top"], device=dev)
        return s
    # what the forward pass kept of every row
    s["lse"], s["ent"] = torch.empty(r, device=dev), torch.empty(r, device=dev)
    for lo in range(0, r, 1024):
        z = s["x"][lo:lo + 1024].double() * s["scale"]
        lse = torch.logsumexp(z, 1)
        logp = z - lse[:, None]
        s["lse"][lo:lo + 1024] = lse
        s["ent"][lo:lo + 1024] = -(torch.exp(logp) * torch.where(torch.isfinite(logp), logp, torch.zeros_like(logp))).sum(1)
    s["dlogp"] = normal(r) / r if case["entropy"] else torch.full((r,), -1.0 / r, device=dev)
    s["dent"] = torch.full((r,), -0.01 / r, device=dev) if case["entropy"] else None
    s["dlse"] = 2e-4 / r * s["lse"] if case["entropy"] else None
    s["dx"] = torch.empty(r, v, dtype=dt, device=dev)
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


# ---- plain form: 32 bits, rounded once at the end ----------------------------------

_LOW = 0xFFFFFFFF


def _philox(c0, c1, c2, c3, k0, k1):
    """The four words of Philox4x32-10 for int64 tensors (or numbers) of 32-bit values."""
    for _ in range(10):
        # int64 products wrap modulo 2^64, which keeps all 64 bits of them
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & _LOW) ^ c1 ^ k0, b & _LOW, ((a >> 32) & _LOW) ^ c3 ^ k1, a & _LOW
        k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
    return c0, c1, c2, c3


def _kept(s):
    """Where dropout keeps an element, and what it multiplies there."""
    r, c, dev = s["rows"], s["cols"], s["x"].device
    groups = -(-c // 8)
    col = torch.arange(groups, device=dev).expand(r, groups)
    row = torch.arange(r, device=dev)[:, None].expand(r, groups)
    off = s["rng"][1] + s["layer"]
    key = s["rng"][0]
    words = _philox(col, row, off & _LOW, (off >> 32) & _LOW, key & _LOW, (key >> 32) & _LOW)
    halves = torch.stack([part for w in words for part in (w & 0xFFFF, w >> 16)], -1).view(r, groups * 8)[:, :c]
    limit = round(65536 * s["p"])
    return halves >= limit, 65536.0 / (65536 - limit)


def _run_plain(s):
    op = s["op"]
    if op == "embed":
        v, out = s["vocab"], DTYPES[s["out"]]
        held = (s["ids"] >= 0) & (s["ids"] < v)
        rows = s["table"][s["ids"].clamp(0, v - 1)].float() * s["scale"]
        return {"y": torch.where(held[:, None], rows, torch.zeros_like(rows)).to(out)}
    if op == "embed_back":
        v, out = s["vocab"], DTYPES[s["out"]]
        ids = torch.where((s["ids"] >= 0) & (s["ids"] < v), s["ids"], torch.full_like(s["ids"], v))
        acc = torch.zeros(v + 1, s["dim"], device=ids.device).index_add_(0, ids, s["dy"].float())[:v] * s["scale"]
        if s["sum"] is not None:
            acc = acc + s["sum"].float()
        return {"dtable": acc.to(out)}
    if op == "dropout":
        keep, by = _kept(s)
        x = s["x"].float() * by
        y = torch.where(keep, x, torch.zeros_like(x))
        if s["res"] is not None:
            y = y + s["res"].float()
        return {"y": y.to(s["x"].dtype)}
    z = s["x"].float() * s["scale"]
    at = s["t"][:, None]
    if op == "logp":
        z = z - z.amax(1, keepdim=True)
        e = torch.exp(z)
        total = e.sum(1)
        log_total = torch.log(total)
        logp = z.gather(1, at)[:, 0] - log_total
        ent = log_total - (e * torch.where(e > 0, z, torch.zeros_like(z))).sum(1) / total
        lse = s["x"].amax(1).float() * s["scale"] + log_total
        out = {"logp": logp, "ent": ent, "lse": lse}
        if s["top"]:
            order = torch.sort(s["x"], dim=1, descending=True, stable=True).indices[:, :s["top"]]
            out["ti"] = order.to(torch.int32)
            out["tl"] = z.gather(1, order) - log_total[:, None]
        return out
    logp = z - s["lse"][:, None]
    p = torch.exp(logp)
    by = -s["dlogp"][:, None]
    if s["entropy"]:
        by = by + s["dlse"][:, None] - s["dent"][:, None] * (logp.clamp_min(-1e30) + s["ent"][:, None])
    dz = p * by
    dz.scatter_add_(1, at, s["dlogp"][:, None])
    return {"dx": (dz * s["scale"]).to(s["x"].dtype)}


# ---- the library's calls -----------------------------------------------------------

def _run_own(s):
    from fsdp_emulated_ranks_gb300 import cr
    op = s["op"]
    if op == "embed":
        cr.cr_embedding(s["table"], s["vocab"], s["ids"], s["tokens"], s["dim"], s["dtype"], s["scale"], s["y"], s["out"])
        return {"y": s["y"]}
    if op == "embed_back":
        cr.cr_embedding_backward(s["dy"], s["dtype"], s["ids"], s["tokens"], s["vocab"], s["dim"], s["scale"], s["sum"],
                                 s["dtable"], s["out"], s["work"], s["work"].numel())
        return {"dtable": s["dtable"]}
    if op == "dropout":
        cr.cr_dropout(s["x"], s["res"], s["rows"], s["cols"], s["dtype"], s["p"], s["rng"], s["layer"], 0, s["y"])
        return {"y": s["y"]}
    if op == "logp":
        top = s["top"]
        cr.cr_log_probs(s["x"], s["t"], s["rows"], s["vocab"], s["dtype"], s["scale"], s["logp"], s["ent"], s["lse"],
                        top, s["ti"] if top else None, s["tl"] if top else None)
        out = {"logp": s["logp"], "ent": s["ent"], "lse": s["lse"]}
        if top:
            out["ti"], out["tl"] = s["ti"], s["tl"]
        return out
    cr.cr_log_probs_backward(s["x"], s["t"], s["rows"], s["vocab"], s["dtype"], s["scale"], s["lse"], s["ent"],
                             s["dlogp"], s["dent"], s["dlse"], s["dx"])
    return {"dx": s["dx"]}


# ---- the definition in 64 bits -----------------------------------------------------

def _random_halves(rows, cols, seed, offset):
    """The 16-bit numbers of rows x cols elements, by 64-bit unsigned arithmetic on the host."""
    groups = (cols + 7) // 8
    low = np.uint64(0xFFFFFFFF)
    w = [np.tile(np.arange(groups, dtype=np.uint64), rows), np.repeat(np.arange(rows, dtype=np.uint64), groups),
         np.full(rows * groups, offset & 0xFFFFFFFF, np.uint64), np.full(rows * groups, offset >> 32, np.uint64)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        first, third = w[0] * np.uint64(0xD2511F53), w[2] * np.uint64(0xCD9E8D57)
        w = [(third >> np.uint64(32)) ^ w[1] ^ np.uint64(k[0]), third & low,
             (first >> np.uint64(32)) ^ w[3] ^ np.uint64(k[1]), first & low]
        k = [(k[0] + 0x9E3779B9) % (1 << 32), (k[1] + 0xBB67AE85) % (1 << 32)]
    out = np.empty((rows * groups, 8), np.int64)
    for i in range(4):
        out[:, 2 * i], out[:, 2 * i + 1] = w[i] & np.uint64(0xFFFF), w[i] >> np.uint64(16)
    return out.reshape(rows, groups * 8)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        return {"y": s["table"].double().index_select(0, s["ids"]) * s["scale"]}  # no case holds an id outside the table
    if op == "embed_back":
        acc = torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device=s["dy"].device)
        used = s["ids"] >= 0
        acc.index_add_(0, s["ids"][used], s["dy"][used].double())
        acc *= s["scale"]
        if case["base"]:
            acc += s["sum"].double()
        return {"dtable": acc}
    if op == "dropout":
        key, off = (int(k) for k in s["rng"].tolist())
        limit = int(math.floor(65536 * case["p"] + 0.5))
        kept = torch.from_numpy(_random_halves(case["rows"], case["cols"], key, off + s["layer"]) >= limit).to(s["x"].device)
        y = s["x"].double() * kept * (65536 / (65536 - limit))
        return {"y": y + s["res"].double() if case["residual"] else y}
    parts = []
    for lo in range(0, case["rows"], 1024):
        x, t = s["x"][lo:lo + 1024].double(), s["t"][lo:lo + 1024]
        z = x * s["scale"]
        if op == "logp":
            lse = torch.logsumexp(z, 1)
            logs = z - lse[:, None]
            p = torch.exp(logs)
            part = {"logp": torch.gather(logs, 1, t[:, None]).squeeze(1),
                    "ent": -torch.special.xlogy(p, p).sum(1), "lse": lse}
            if case["top"]:
                part["tl"] = torch.topk(logs, case["top"], dim=1).values
        else:
            row = slice(lo, lo + 1024)
            p = torch.exp(z - s["lse"][row, None].double())
            chosen = torch.zeros_like(p).scatter_(1, t[:, None], 1.0)
            dz = s["dlogp"][row, None].double() * (chosen - p)
            if case["entropy"]:
                # dH/dz_v = -p_v (log p_v + H)
                dz -= s["dent"][row, None].double() * (torch.special.xlogy(p, p) + p * s["ent"][row, None].double())
                dz += s["dlse"][row, None].double() * p
            part = {"dx": dz * s["scale"]}
        parts.append(part)
    out = {k: torch.cat([part[k] for part in parts]) for k in parts[0]}
    if op == "logp" and case["top"]:
        out["ti"] = None
    return out
