"""What is measured of the per-worker training operators.

The Sign-Muon step takes one gradient per (matrix, worker).  The operators
here are those of a token model around its hidden matrices, each giving one
gradient (or loss) per worker from one pass over all workers' rows:

  embed, embed_grad          rows of a table by token id, scaled; the table's gradient per worker
  norm, norm_grad            layer normalisation; its input's gradient and, per worker, its weight's and bias's
  distill_loss, distill_grad divergence from a teacher's top logits, per row and worker; with the logits' gradient

Worker m owns rows [splits[m], splits[m + 1]) of a batch.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
EPS = 1e-5


# ------------------------------------------------------------------- cases
def listed():
    return [
        # The prompt of one short request: the launch is all that counts.
        {"name": "embed-48x768-bf16", "op": "embed", "rows": 48, "vocab": 32768, "dim": 768, "dtype": "bf16", "pad": False},
        # A batch of 8 x 4096 tokens of a wide model.
        {"name": "embed-32768x4096-bf16", "op": "embed", "rows": 32768, "vocab": 50000, "dim": 4096, "dtype": "bf16",
         "pad": True},
        # Eight workers' table gradients of the small language model, 4096 tokens each: nearly all of it zero rows.
        {"name": "embed_grad-8w-32768x768-bf16", "op": "embed_grad", "workers": 8, "ragged": False, "rows": 32768,
         "vocab": 50000, "dim": 768, "dtype": "bf16", "pad": False},
        # One worker with a long batch over a small table, odd everywhere: many tokens for each row.
        {"name": "embed_grad-1w-100003x999-f32", "op": "embed_grad", "workers": 1, "ragged": False, "rows": 100003,
         "vocab": 10007, "dim": 999, "dtype": "f32", "pad": True},
        # A norm over a few tokens.
        {"name": "norm-64x768-bf16", "op": "norm", "rows": 64, "dim": 768, "dtype": "bf16", "weight": "bf16", "bias": True},
        # A norm of a wide model's batch.
        {"name": "norm-32768x4096-bf16", "op": "norm", "rows": 32768, "dim": 4096, "dtype": "bf16", "weight": "bf16",
         "bias": True},
        # Backward of one norm of the small language model, eight workers of 8192 tokens.
        {"name": "norm_grad-8w-65536x768-bf16", "op": "norm_grad", "workers": 8, "ragged": False, "rows": 65536, "dim": 768,
         "dtype": "bf16", "weight": "bf16", "bias": True},
        # Workers with unequal shares, 32-bit, no bias.
        {"name": "norm_grad-4w-9001x1000-f32", "op": "norm_grad", "workers": 4, "ragged": True, "rows": 9001, "dim": 1000,
         "dtype": "f32", "weight": "f32", "bias": False},
        # Validation of a few rows.
        {"name": "distill_loss-2w-16x32001-bf16", "op": "distill_loss", "workers": 2, "ragged": False, "rows": 16,
         "vocab": 32001, "top": 8, "dtype": "bf16", "temperature": 1.0, "holes": False},
        # Validation of a batch with 32-bit logits.
        {"name": "distill_loss-8w-2048x50000-f32", "op": "distill_loss", "workers": 8, "ragged": False, "rows": 2048,
         "vocab": 50000, "top": 64, "dtype": "f32", "temperature": 2.0, "holes": True},
        # The training loss of eight workers, 1024 tokens each.
        {"name": "distill_grad-8w-8192x50000-bf16", "op": "distill_grad", "workers": 8, "ragged": False, "rows": 8192,
         "vocab": 50000, "top": 64, "dtype": "bf16", "temperature": 2.0, "holes": True},
        # A large odd vocabulary, unequal shares, 32-bit logits.
        {"name": "distill_grad-3w-513x131101-f32", "op": "distill_grad", "workers": 3, "ragged": True, "rows": 513,
         "vocab": 131101, "top": 20, "dtype": "f32", "temperature": 1.0, "holes": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "distill_loss", "distill_grad"])
    dtype = rng.choice(["f32", "bf16"])
    case = {"op": op, "dtype": dtype}
    if op in ("embed_grad", "norm_grad", "distill_loss", "distill_grad"):
        case["workers"] = rng.choice([1, 2, 3, 4, 8, 16])
        case["ragged"] = rng.random() < 0.5
    if op.startswith("embed"):
        # Widths of real tables as often as arbitrary ones.
        case["dim"] = rng.choice([64, 256, 768, 1000, 1536, 4096]) if rng.random() < 0.5 else _log(rng, 1, 4096)
        case["vocab"] = _log(rng, 16, max(16, min(131072, (1 << 28) // (case["dim"] * case.get("workers", 1)))))
        case["rows"] = _log(rng, 1, min(131072, (1 << 26) // case["dim"]))
        case["pad"] = rng.random() < 0.5
    elif op.startswith("norm"):
        # From 4: of a row of two, the gradient is what rounding leaves of a difference that is nearly zero.
        case["dim"] = rng.choice([64, 256, 768, 1000, 1536, 4096]) if rng.random() < 0.5 else _log(rng, 4, 16384)
        case["rows"] = _log(rng, 1, min(131072, (1 << 26) // case["dim"]))
        case["weight"] = rng.choice([dtype, "f32"])
        case["bias"] = rng.random() < 0.7
    else:
        case["vocab"] = _log(rng, 32, 200000)
        case["rows"] = _log(rng, 1, min(8192, (1 << 27) // case["vocab"]))
        case["top"] = _log(rng, 1, min(256, case["vocab"]))
        case["temperature"] = rng.choice([0.5, 1.0, 2.0, 4.0])
        case["holes"] = rng.random() < 0.5
    if "workers" in case and not case["ragged"]:
        case["rows"] = -(-case["rows"] // case["workers"]) * case["workers"]
    return case


# ------------------------------------------------------------------ inputs
def _splits(case, seed):
    m, n = case["workers"], case["rows"]
    if not case["ragged"]:
        return [i * (n // m) for i in range(m + 1)]
    cuts = np.random.RandomState(seed % (1 << 31)).randint(0, n + 1, m - 1)
    return [0] + sorted(int(c) for c in cuts) + [n]


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    n, op = case["rows"], case["op"]

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=g, device=dev).mul_(std).add_(mean)

    s = {"op": op}
    if "workers" in case:
        s["splits"] = _splits(case, seed)
        s["workers"] = case["workers"]
        counts = torch.tensor(np.diff(s["splits"]), device=dev)
        s["worker"] = torch.repeat_interleave(torch.arange(case["workers"], device=dev), counts)
    if op.startswith("embed"):
        v, d = case["vocab"], case["dim"]
        # Token frequencies fall as 1 / rank; ranks are spread over the ids.
        rank = torch.exp(torch.rand(n, generator=g, device=dev, dtype=torch.float64) * math.log(v + 1)).long().sub_(1)
        ids = torch.randperm(v, generator=g, device=dev)[rank.clamp_(0, v - 1)]
        if case["pad"]:
            ids[torch.rand(n, generator=g, device=dev) < 0.05] = -1
        s["ids"], s["vocab"], s["scale"] = ids, v, math.sqrt(d)
        if op == "embed":
            s["table"] = normal(v, d, std=0.02).to(dt)
        else:
            s["dy"] = normal(n, d, std=1e-2).to(dt)
    elif op.startswith("norm"):
        d, wt = case["dim"], DTYPES[case["weight"]]
        x = normal(n, d, std=1.5, mean=0.25)
        s["x"] = x.to(dt)
        s["weight"] = normal(d, std=0.1, mean=1.0).to(wt)
        s["bias"] = normal(d, std=0.1).to(wt) if case["bias"] else None
        if op == "norm_grad":
            s["dy"] = normal(n, d, std=1e-2).to(dt)
            x = s["x"].double()
            mean = x.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = (x.sub_(mean[:, None]).square_().mean(1) + EPS).rsqrt().float()
    else:
        v, k = case["vocab"], case["top"]
        z = normal(n, v, std=2.0)
        top, idx = torch.topk(z + normal(n, v), k, dim=1)
        if case["holes"]:
            # A vocabulary padded with columns that never occur, entries that
            # a teacher did not send, and rows that do not count.
            z[:, v - v // 64:] = -math.inf
            idx[idx >= v - v // 64] = -1
            idx[torch.rand(n, k, generator=g, device=dev) < 0.05] = -1
            idx[torch.rand(n, generator=g, device=dev) < 0.05] = -1
        s["logits"], s["top_logits"], s["top_ids"] = z.to(dt), top, idx
        s["temperature"] = case["temperature"]
    return s


# ------------------------------------------------------------- plain forms
def _plain_embed(s):
    ids, table = s["ids"], s["table"]
    inside = (ids >= 0) & (ids < s["vocab"])
    rows = table[ids.clamp(0, s["vocab"] - 1)].float()
    return (rows * s["scale"] * inside[:, None]).to(table.dtype)


def _plain_embed_grad(s):
    ids, dy, v, m = s["ids"], s["dy"], s["vocab"], s["workers"]
    inside = (ids >= 0) & (ids < v)
    key = s["worker"] * v + ids.clamp(0, v - 1)
    total = torch.zeros(m * v, dy.shape[1], device=dy.device)
    total.index_add_(0, key, dy.float() * s["scale"] * inside[:, None])
    return list(total.to(dy.dtype).view(m, v, -1).unbind(0))


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    x = x - mean
    rstd = 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    y = x * rstd * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["x"].dtype), mean[:, 0], rstd[:, 0]


def _plain_norm_grad(s):
    x, dy, w, m = s["x"].float(), s["dy"].float(), s["weight"].float(), s["workers"]
    xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
    gy = dy * w
    dx = s["rstd"][:, None] * (gy - gy.mean(1, keepdim=True) - xh * (gy * xh).mean(1, keepdim=True))
    of_worker = (torch.arange(m, device=x.device)[:, None] == s["worker"]).float()
    dw = (of_worker @ (dy * xh)).to(s["weight"].dtype)
    db = (of_worker @ dy).to(s["weight"].dtype) if s["bias"] is not None else None
    out = {"dx": dx.to(s["x"].dtype), "dweight": list(dw.unbind(0))}
    if db is not None:
        out["dbias"] = list(db.unbind(0))
    return out


def _plain_distill(s, with_grad):
    z = s["logits"].float() / s["temperature"]
    t, m, v = s["temperature"], s["workers"], s["logits"].shape[1]
    idx = s["top_ids"]
    here = (idx >= 0) & (idx < v)
    counts = here.any(1)
    u = torch.where(here, s["top_logits"].float() / t, -math.inf)
    u = torch.exp(u - torch.where(counts, u.amax(1), 0.0)[:, None])
    p = u / torch.where(counts, u.sum(1), 1.0)[:, None]
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    logq = z.gather(1, idx.clamp(0, v - 1)) - top - torch.log(total)
    row = torch.where(p > 0, p * (torch.log(p) - logq), 0.0).sum(1) * (t * t)
    of_worker = (torch.arange(m, device=z.device)[:, None] == s["worker"]) & counts
    n = of_worker.sum(1).clamp(min=1).float()
    loss = (of_worker * row).sum(1) / n
    if not with_grad:
        return loss, row
    dz = (e / total).scatter_add_(1, idx.clamp(0, v - 1), -p)
    dz = dz * torch.where(counts, t / n[s["worker"]], 0.0)[:, None]
    return loss, row, dz.to(s["logits"].dtype)


# ------------------------------------------------------------------ a pass
def run(s):
    op = s["op"]
    if own:
        from sign_muon_optimizer_momentum_b200 import layers
        if op == "embed":
            return layers.embedding_forward(s["table"], s["ids"], scale=s["scale"])
        if op == "embed_grad":
            return layers.embedding_backward(s["ids"], s["dy"], s["vocab"], n_workers=s["workers"], splits=s["splits"],
                                             scale=s["scale"])
        if op == "norm":
            return layers.layer_norm_forward(s["x"], s["weight"], s["bias"], eps=EPS)
        if op == "norm_grad":
            dx, dw, db = layers.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"],
                                                    n_workers=s["workers"], splits=s["splits"],
                                                    bias=s["bias"] is not None)
            return {"dx": dx, "dweight": dw} if db is None else {"dx": dx, "dweight": dw, "dbias": db}
        distill = layers.distill_loss if op == "distill_loss" else layers.distill_loss_and_grad
        return distill(s["logits"], s["top_ids"], s["top_logits"], n_workers=s["workers"], splits=s["splits"],
                       temperature=s["temperature"])
    if op == "embed":
        return _plain_embed(s)
    if op == "embed_grad":
        return _plain_embed_grad(s)
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_grad":
        return _plain_norm_grad(s)
    return _plain_distill(s, op == "distill_grad")


# ------------------------------------------------------------------- work
def _distinct(vocab, draws):
    """Expected distinct ids among `draws` of a 1 / rank distribution."""
    r = np.arange(1, vocab + 1, dtype=np.float64)
    p = np.log((r + 1) / r) / math.log(vocab + 1)
    return float(-np.expm1(draws * np.log1p(-np.minimum(p, 1 - 1e-12))).sum())


def work(case):
    b, n, op = BYTES[case["dtype"]], case["rows"], case["op"]
    if op == "embed":
        d = case["dim"]
        return {"bytes": n * 8 + _distinct(case["vocab"], n) * d * b + n * d * b, "flops": n * d}
    if op == "embed_grad":
        d, m = case["dim"], case["workers"]
        return {"bytes": n * 8 + n * d * b + m * case["vocab"] * d * b, "flops": 2 * n * d}
    if op in ("norm", "norm_grad"):
        d = case["dim"]
        vectors = d * BYTES[case["weight"]] * (2 if case["bias"] else 1)
        if op == "norm":
            return {"bytes": 2 * n * d * b + vectors + 8 * n, "flops": 8 * n * d}
        return {"bytes": 3 * n * d * b + d * BYTES[case["weight"]] + case["workers"] * vectors + 8 * n, "flops": 14 * n * d}
    v, k = case["vocab"], case["top"]
    passes = 2 if op == "distill_grad" else 1
    return {"bytes": passes * n * v * b + 12 * n * k + 4 * n + 4 * case["workers"], "flops": (3 + 2 * (passes - 1)) * n * v}


# ------------------------------------------------- the definitions, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "embed":
        ids = s["ids"]
        y = torch.zeros(len(ids), s["table"].shape[1], dtype=torch.float64, device=ids.device)
        at = torch.nonzero((ids >= 0) & (ids < s["vocab"]))[:, 0]
        y[at] = s["table"].double()[ids[at]] * s["scale"]
        return y
    if op == "embed_grad":
        out = []
        for lo, hi in zip(s["splits"], s["splits"][1:]):
            ids, dy = s["ids"][lo:hi], s["dy"][lo:hi].double()
            at = torch.nonzero((ids >= 0) & (ids < s["vocab"]))[:, 0]
            g = torch.zeros(s["vocab"], dy.shape[1], dtype=torch.float64, device=dy.device)
            out.append(g.index_put_((ids[at],), dy[at] * s["scale"], accumulate=True))
        return out
    if op == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = (var + EPS) ** -0.5
        y = (x - mean[:, None]) * rstd[:, None] * s["weight"].double()
        return (y if s["bias"] is None else y + s["bias"].double()), mean, rstd
    if op == "norm_grad":
        d = s["x"].shape[1]
        mean, rstd = s["mean"].double()[:, None], s["rstd"].double()[:, None]
        xh, dy = (s["x"].double() - mean) * rstd, s["dy"].double()
        gy = dy * s["weight"].double()
        dx = (gy - (gy.sum(1) / d)[:, None] - xh * ((gy * xh).sum(1) / d)[:, None]) * rstd
        parts = list(zip(s["splits"], s["splits"][1:]))
        out = {"dx": dx, "dweight": [(dy[a:b] * xh[a:b]).sum(0) for a, b in parts]}
        if s["bias"] is not None:
            out["dbias"] = [dy[a:b].sum(0) for a, b in parts]
        return out
    t, v = s["temperature"], s["logits"].shape[1]
    loss = torch.zeros(s["workers"], dtype=torch.float64, device=s["logits"].device)
    row = torch.zeros(len(s["logits"]), dtype=torch.float64, device=loss.device)
    dz = torch.zeros(s["logits"].shape, dtype=torch.float64, device=loss.device) if op == "distill_grad" else None
    for m, (a, b) in enumerate(zip(s["splits"], s["splits"][1:])):
        idx = s["top_ids"][a:b]
        here = (idx >= 0) & (idx < v)
        at = torch.nonzero(here.any(1))[:, 0]
        if len(at) == 0:
            continue
        idx, here = idx[at], here[at]
        logp = torch.log_softmax((s["top_logits"][a:b][at].double() / t).masked_fill(~here, -math.inf), 1)
        logq = torch.log_softmax(s["logits"][a:b][at].double() / t, 1)
        p, safe = logp.exp(), idx.masked_fill(~here, 0)
        terms = (p * (logp - logq.gather(1, safe))).masked_fill(~here, 0.0).sum(1) * t * t
        row[a:b][at] = terms
        loss[m] = terms.sum() / len(at)
        if dz is not None:
            dz[a:b][at] = logq.exp_().scatter_add_(1, safe, -p).mul_(t / len(at))
    return (loss, row) if dz is None else (loss, row, dz)
