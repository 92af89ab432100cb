"""Cases of what stands before a mixture-of-experts layer's exchange: the norm, the router's choice and its balance loss.

``kind`` of a case:

* ``norm``          layer norm of each rank's rows, after adding a residual stream where ``residual``
* ``norm_grad``     its gradients: for the rows (plus the residual stream's) and, summed over them, for weight and bias
* ``gate``          router logits -> the k experts of each token and their gate weights; with ``balance``, in the same
                    call, the tokens of each expert and the balance loss
* ``gate_grad``     the gradient of the gate weights, and with ``balance`` of the balance loss, for the logits
* ``balance``       tokens of each expert and the balance loss of expert ids that are given
* ``balance_grad``  the gradient of that loss for the logits

With score u(l) (``softmax``: exp(l), ``sigmoid``: 1 / (1 + exp(-l))) and p_e = u(l_e) / sum_i u(l_i), the k experts are
those of the largest logits, ties to the lowest index, -1 where fewer than k logits are above -inf; a gate is
scale * u(l_e) / (sum over the chosen) where ``normalize``, else scale * p_e (softmax) or scale * u(l_e) (sigmoid).  The
loss of a rank (of all ranks' tokens where ``together``) is E / (k * T^2) * sum_e count_e * sum_t p_te over the T tokens
that have a logit above -inf; T is the last entry of ``counts``.

``run`` computes them by elementary torch operations in 32 bits, or, where ``own`` is true, by the package's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # serving: the eight tokens of one decoding step, residual added, nothing kept for a backward pass: latency
        {"name": "norm decode", "kind": "norm", "p": 1, "tokens": 8, "ragged": 0, "hidden": 7168, "dtype": "bf16", "weights": "bf16", "bias": True,
         "residual": True, "stats": False},
        # training: 8 ranks of 4096 tokens, residual added, fp32 weights as the optimizer's masters hold them
        {"name": "norm train", "kind": "norm", "p": 8, "tokens": 4096, "ragged": 0, "hidden": 7168, "dtype": "bf16", "weights": "f32", "bias": True,
         "residual": True, "stats": True},
        # training in fp32: other counts on each rank, rows off the 16-byte grid
        {"name": "norm ragged", "kind": "norm", "p": 4, "tokens": 4001, "ragged": 333, "hidden": 1019, "dtype": "f32", "weights": "f32", "bias": True,
         "residual": False, "stats": True},
        # training: the backward pass of the second case, gradients of weight and bias for the fp32 buckets
        {"name": "norm_grad train", "kind": "norm_grad", "p": 8, "tokens": 4096, "ragged": 0, "hidden": 7168, "dtype": "bf16", "weights": "f32",
         "bias": True, "residual": True, "dw": "f32"},
        # training a small layer in bf16, without bias: many narrow rows, other counts on each rank, an odd width
        {"name": "norm_grad ragged", "kind": "norm_grad", "p": 4, "tokens": 8001, "ragged": 1001, "hidden": 1019, "dtype": "bf16", "weights": "bf16",
         "bias": False, "residual": False, "dw": "bf16"},
        # serving: a decoding step's tokens choose 8 of 256 experts by sigmoid scores: latency
        {"name": "gate decode", "kind": "gate", "p": 1, "tokens": 8, "ragged": 0, "experts": 256, "k": 8, "dtype": "bf16", "score": "sigmoid",
         "normalize": True, "scale": 2.5, "dead": 0, "padded": 0, "balance": False, "together": False},
        # training: 8 ranks of 16384 tokens, top-8 of 256 experts, the balance loss in the same call
        {"name": "gate train", "kind": "gate", "p": 8, "tokens": 16384, "ragged": 0, "experts": 256, "k": 8, "dtype": "bf16", "score": "softmax",
         "normalize": True, "scale": 1.0, "dead": 0, "padded": 0, "balance": True, "together": False},
        # training: the backward pass of that
        {"name": "gate_grad train", "kind": "gate_grad", "p": 8, "tokens": 16384, "ragged": 0, "experts": 256, "k": 8, "dtype": "bf16", "score": "softmax",
         "normalize": True, "scale": 1.0, "dead": 0, "padded": 0, "balance": True, "together": False},
        # training with a padded batch of fp32 logits and experts that are out of service: top-6 of 60, every gate by itself
        {"name": "gate ragged", "kind": "gate", "p": 4, "tokens": 20001, "ragged": 3001, "experts": 60, "k": 6, "dtype": "f32", "score": "sigmoid",
         "normalize": False, "scale": 1.0, "dead": 3, "padded": 1000, "balance": False, "together": False},
        # its backward pass
        {"name": "gate_grad ragged", "kind": "gate_grad", "p": 4, "tokens": 20001, "ragged": 3001, "experts": 60, "k": 6, "dtype": "f32",
         "score": "sigmoid", "normalize": False, "scale": 1.0, "dead": 3, "padded": 1000, "balance": False, "together": False},
        # training on ids that the user's own rule chose: top-2 of 32, one loss over the tokens of all ranks
        {"name": "balance", "kind": "balance", "p": 8, "tokens": 4096, "ragged": 100, "experts": 32, "k": 2, "dtype": "f32", "score": "softmax",
         "dead": 0, "padded": 100, "together": True},
        # its gradient at training size
        {"name": "balance_grad", "kind": "balance_grad", "p": 8, "tokens": 16384, "ragged": 0, "experts": 256, "k": 8, "dtype": "f32", "score": "sigmoid",
         "dead": 0, "padded": 0, "together": False},
    ]


def _log(rng, lo, hi):
    return round(math.exp(rng.uniform(math.log(lo), math.log(hi))))


def _width(rng, lo, hi):
    """A row width: a multiple of 128 half of the time, of 8 a quarter, any number else."""
    v, u = _log(rng, lo, hi), rng.random()
    return max(128, v // 128 * 128) if u < 0.5 else max(8, v // 8 * 8) if u < 0.75 else v


def draw(rng):
    kind = rng.choice(["norm", "norm_grad", "gate", "gate_grad", "balance", "balance_grad"])
    p = rng.choice([1, 1, 2, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind in ("norm", "norm_grad"):
        hidden = _width(rng, 64, 8192)
        tokens = _log(rng, 1, max(2, min(65536, 8 * 4096 * 7168 // (p * hidden * 2))))
        c = {"kind": kind, "p": p, "tokens": tokens, "ragged": rng.choice([0, tokens // 16]), "hidden": hidden, "dtype": dtype,
             "weights": rng.choice([dtype, "f32"]), "bias": rng.random() < 0.7, "residual": rng.random() < 0.5}
        return c | ({"stats": rng.random() < 0.7} if kind == "norm" else {"dw": rng.choice(["f32", "f32", "bf16"])})
    experts = rng.choice([4, 8, 16, 32, 60, 64, 128, 160, 256, 256, 384])
    k = rng.choice([v for v in (1, 2, 4, 6, 8) if v <= experts])
    tokens = _log(rng, 1, max(2, min(65536, 8 * 16384 * 256 // (p * experts * 2))))
    c = {"kind": kind, "p": p, "tokens": tokens, "ragged": rng.choice([0, tokens // 16]), "experts": experts, "k": k, "dtype": dtype,
         "score": rng.choice(["softmax", "sigmoid"]), "dead": rng.choice([0, 0, experts // 8, experts - k + k // 2]), "padded": rng.choice([0, tokens // 10]),
         "together": rng.random() < 0.4}
    if kind in ("gate", "gate_grad"):
        c |= {"normalize": rng.random() < 0.6, "scale": rng.choice([1.0, 1.0, 2.5]), "balance": rng.random() < 0.5}
    return c


# ------------------------------------------------------------------ inputs
def _tokens(c):
    """Tokens of each rank."""
    return [max(1, c["tokens"] - r * c["ragged"]) for r in range(c["p"])]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    dt = DTYPES[c["dtype"]]

    def normal(*shape, dtype=torch.float32, scale=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale + mean).to(dtype)

    def empty(shape, dtype=torch.float32):
        return [torch.zeros(t, *shape, dtype=dtype, device="cuda") for t in _tokens(c)]

    if c["kind"] in ("norm", "norm_grad"):
        h, wt, ranks = c["hidden"], DTYPES[c["weights"]], range(c["p"])
        spread = torch.exp(normal(h, scale=0.5))  # some features of a residual stream are much larger than others
        s["x"] = [(torch.randn(t, h, generator=g, device="cuda") * spread + 0.1).to(dt) for t in _tokens(c)]
        s["weight"] = [normal(h, dtype=wt, scale=0.2, mean=1.0)] * c["p"]  # the ranks share them
        s["bias"] = [normal(h, dtype=wt, scale=0.1)] * c["p"] if c["bias"] else None
        if c["kind"] == "norm":
            s["residual"] = [normal(t, h, dtype=dt) for t in _tokens(c)] if c["residual"] else None
            s["y"] = empty((h,), dt)
            s["sum"] = empty((h,), dt) if c["residual"] else None
            s["mean"], s["rstd"] = (empty(()), empty(())) if c["stats"] else (None, None)
            return s
        # the forward pass has been made: its statistics are inputs
        wide = [x.double() for x in s["x"]]
        s["mean"] = [x.mean(1).float() for x in wide]
        s["rstd"] = [(x.var(1, correction=0) + EPS).rsqrt().float() for x in wide]
        s["dy"] = [normal(t, h, dtype=dt, scale=0.01) for t in _tokens(c)]
        s["dsum"] = [normal(t, h, dtype=dt, scale=0.01) for t in _tokens(c)] if c["residual"] else None
        s["dx"] = empty((h,), dt)
        s["dweight"] = [torch.zeros(h, dtype=DTYPES[c["dw"]], device="cuda") for _ in ranks]
        s["dbias"] = [torch.zeros_like(w) for w in s["dweight"]] if c["bias"] else None
        if own:
            from a2a_ring_ordered_gb300 import ccl

            s["workspace"] = torch.empty(ccl.ccl_layer_norm_grad_workspace_bytes(c["p"], h), dtype=torch.uint8, device="cuda")
        return s
    # a router's logits: some experts are more popular; padding and experts out of service are -inf
    e, k = c["experts"], c["k"]
    popular = normal(e, scale=0.5)
    popular[torch.randperm(e, generator=g, device="cuda")[:c["dead"]]] = -math.inf
    s["logits"] = [normal(t, e) + popular for t in _tokens(c)]
    for v in s["logits"]:
        v[max(1, v.shape[0] - c["padded"]):] = -math.inf
    s["logits"] = [v.to(dt) for v in s["logits"]]
    s["counts"] = [torch.zeros(e + 1, dtype=torch.int32, device="cuda") for _ in s["logits"]]
    s["losses"] = [torch.zeros(1, device="cuda") for _ in s["logits"]]
    if own and (c["kind"] == "balance" or c["kind"] == "gate" and c["balance"]):
        from a2a_ring_ordered_gb300 import ccl

        s["workspace"] = torch.empty(ccl.ccl_moe_balance_workspace_bytes(c["p"], e), dtype=torch.uint8, device="cuda")
    if c["kind"] == "gate":
        s["ids"] = empty((k,), torch.int32)
        s["gates"] = empty((k,))
        return s
    # the forward pass has been made: its choice is an input
    s["ids"] = [_plain_choice(v, k) for v in s["logits"]]
    if c["kind"] == "balance":
        return s
    if c["kind"] == "balance_grad" or c["balance"]:
        s["counts"] = _plain_counts(s["logits"], s["ids"], c["together"])
        s["dlosses"] = [normal(1, scale=0.01) for _ in s["logits"]]
    if c["kind"] == "gate_grad":
        s["dgates"] = [normal(t, k) for t in _tokens(c)]
    s["dlogits"] = empty((e,), dt)
    return s


# ------------------------------------------------------------- plain forms
def _plain_norm(x, residual, weight, bias):
    v = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    f = v.float()
    mean = f.mean(1, keepdim=True)
    centred = f - mean
    rstd = 1.0 / (centred.square().mean(1, keepdim=True) + EPS).sqrt()
    y = centred * rstd * weight.float()
    return (y if bias is None else y + bias.float()).to(x.dtype), v, mean[:, 0], rstd[:, 0]


def _plain_norm_grad(dy, dsum, x, weight, mean, rstd, dw):
    d, normed = dy.float(), (x.float() - mean[:, None]) * rstd[:, None]
    scaled = d * weight.float()
    dx = (scaled - scaled.mean(1, keepdim=True) - normed * (scaled * normed).mean(1, keepdim=True)) * rstd[:, None]
    if dsum is not None:
        dx = dx + dsum.float()
    return dx.to(x.dtype), (d * normed).sum(0).to(dw), d.sum(0).to(dw)


def _plain_choice(logits, k):
    """The experts of the k largest logits, in order, ties to the lowest index; -1 for -inf."""
    top, at = (logits.float() + 0.0).sort(dim=1, descending=True, stable=True)
    return torch.where(top[:, :k] == -math.inf, -1, at[:, :k]).to(torch.int32)


def _plain_scores(logits, score):
    """u(l) over a power of e that keeps the row's largest away from 0, and the logarithm of that power (0 for a row of -inf)."""
    f = logits.float()
    top = f.amax(1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    if score == "softmax":
        return torch.exp(f - top), top
    top = top.clamp(max=0.0)
    return torch.exp(f.clamp(max=0.0) - top) / (1.0 + torch.exp(-f.abs())), top


def _plain_shares(u):
    total = u.sum(1, keepdim=True)
    return u / torch.where(total == 0, 1.0, total)


def _plain_chosen(values, ids):
    return torch.where(ids < 0, 0.0, values.gather(1, ids.long().clamp(min=0)))


def _plain_gates(logits, ids, score, normalize, scale):
    u, top = _plain_scores(logits, score)
    if normalize:
        return _plain_shares(_plain_chosen(u, ids)) * scale
    return _plain_chosen(_plain_shares(u) if score == "softmax" else u * torch.exp(top), ids) * scale


def _plain_counts(logits, ids, together):
    """Tokens of each expert, then the tokens that have a logit above -inf."""
    counts = []
    for v, i in zip(logits, ids):
        flat = i.reshape(-1).long()
        got = torch.zeros(v.shape[1] + 2, dtype=torch.int64, device=v.device)
        got.index_add_(0, torch.where(flat < 0, v.shape[1] + 1, flat), torch.ones_like(flat))
        got[-2] = (v != -math.inf).any(1).sum()
        counts.append(got[:-1])
    if together:
        counts = [sum(counts)] * len(counts)
    return [n.to(torch.int32) for n in counts]


def _plain_losses(logits, counts, k, score, together):
    shares = [_plain_shares(_plain_scores(v, score)[0]).sum(0, dtype=torch.float64) for v in logits]
    if together:
        shares = [sum(shares)] * len(shares)
    out = []
    for n, s in zip(counts, shares):
        live = n[-1:].double().clamp(min=1)
        out.append(((n[:-1].double() * s).sum() * (s.numel() / k) / live / live).float())
    return out


def _plain_gate_grad(logits, ids, dgates, score, normalize, scale):
    u, top = _plain_scores(logits, score)
    d = torch.where(ids < 0, 0.0, dgates) * scale
    at = torch.where(ids < 0, logits.shape[1], ids).long()

    def spread(values):
        """To the experts' places in the row."""
        row = torch.zeros(u.shape[0], u.shape[1] + 1, device=u.device)
        return row.scatter_add_(1, at, values)[:, :-1]

    f = logits.float()
    away = torch.exp(-f.clamp(min=0.0)) / (1.0 + torch.exp(-f.abs()))  # 1 - sigmoid
    if normalize:
        share = _plain_shares(_plain_chosen(u, ids))
        got = spread(share * (d - (share * d).sum(1, keepdim=True)))
        return got if score == "softmax" else got * away
    if score == "softmax":
        share = _plain_shares(u)
        return spread(_plain_chosen(share, ids) * d) - share * (_plain_chosen(share, ids) * d).sum(1, keepdim=True)
    return spread(_plain_chosen(u * torch.exp(top), ids) * d) * away


def _plain_balance_grad(logits, counts, dloss, k, score):
    share = _plain_shares(_plain_scores(logits, score)[0])
    n, live = counts[:-1].double(), counts[-1].double().clamp(min=1)
    a = ((n - n.mean()) * (n.numel() / k) / live / live * dloss.double()).float()  # a constant taken off changes nothing
    got = share * (a - (share * a).sum(1, keepdim=True))
    if score == "softmax":
        return got
    f = logits.float()
    return got * (torch.exp(-f.clamp(min=0.0)) / (1.0 + torch.exp(-f.abs())))


def _each(s, *names):
    """What each rank holds of the lists, None for those that are not there."""
    return zip(*[s[n] if s.get(n) is not None else [None] * s["case"]["p"] for n in names])


def run(s):
    c, kind = s["case"], s["case"]["kind"]
    if own:
        return _own(s, c, kind)
    if kind == "norm":
        got = [_plain_norm(*v) for v in _each(s, "x", "residual", "weight", "bias")]
        return _norm_outputs(c, *[list(v) for v in zip(*got)])
    if kind == "norm_grad":
        got = [_plain_norm_grad(*v, DTYPES[c["dw"]]) for v in _each(s, "dy", "dsum", "x", "weight", "mean", "rstd")]
        return _norm_grad_outputs(c, *[list(v) for v in zip(*got)])
    if kind == "gate":
        ids = [_plain_choice(v, c["k"]) for v in s["logits"]]
        out = {"ids": ids, "gates": [_plain_gates(v, i, c["score"], c["normalize"], c["scale"]) for v, i in zip(s["logits"], ids)]}
        if c["balance"]:
            out["counts"] = _plain_counts(s["logits"], ids, c["together"])
            out["losses"] = _plain_losses(s["logits"], out["counts"], c["k"], c["score"], c["together"])
        return out
    if kind == "balance":
        counts = _plain_counts(s["logits"], s["ids"], c["together"])
        return {"counts": counts, "losses": _plain_losses(s["logits"], counts, c["k"], c["score"], c["together"])}
    out = [0.0] * c["p"]
    if kind == "gate_grad":
        out = [_plain_gate_grad(*v, c["score"], c["normalize"], c["scale"]) for v in _each(s, "logits", "ids", "dgates")]
    if kind == "balance_grad" or c["balance"]:
        out = [o + _plain_balance_grad(*v, c["k"], c["score"]) for o, v in zip(out, _each(s, "logits", "counts", "dlosses"))]
    return {"dlogits": [o.to(v.dtype) for o, v in zip(out, s["logits"])]}


def _norm_outputs(c, y, total, mean, rstd):
    out = {"y": y}
    if c["residual"]:
        out["sum"] = total
    if c["stats"]:
        out |= {"mean": mean, "rstd": rstd}
    return out


def _norm_grad_outputs(c, dx, dweight, dbias):
    out = {"dx": dx, "dweight": dweight}
    if c["bias"]:
        out["dbias"] = dbias
    return out


def _own(s, c, kind):
    from a2a_ring_ordered_gb300 import ccl

    if kind == "norm":
        ccl.ccl_layer_norm(s["x"], s["weight"], s["bias"], s["y"], residual=s["residual"], sum=s["sum"], mean=s["mean"], rstd=s["rstd"], eps=EPS)
        return _norm_outputs(c, s["y"], s["sum"], s["mean"], s["rstd"])
    if kind == "norm_grad":
        ccl.ccl_layer_norm_grad(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], dsum=s["dsum"], dweight=s["dweight"], dbias=s["dbias"],
                                workspace=s["workspace"])
        return _norm_grad_outputs(c, s["dx"], s["dweight"], s["dbias"])
    if kind == "gate":
        with_loss = {"counts": s["counts"], "losses": s["losses"], "together": c["together"], "workspace": s["workspace"]} if c["balance"] else {}
        ccl.ccl_moe_gate(s["logits"], s["ids"], s["gates"], score=c["score"], normalize=c["normalize"], scale=c["scale"], **with_loss)
        return {"ids": s["ids"], "gates": s["gates"]} | ({"counts": s["counts"], "losses": s["losses"]} if c["balance"] else {})
    if kind == "gate_grad":
        with_loss = {"counts": s["counts"], "dlosses": s["dlosses"]} if c["balance"] else {}
        ccl.ccl_moe_gate_grad(s["logits"], s["ids"], s["dgates"], s["dlogits"], score=c["score"], normalize=c["normalize"], scale=c["scale"], **with_loss)
        return {"dlogits": s["dlogits"]}
    if kind == "balance":
        ccl.ccl_moe_balance(s["logits"], s["ids"], s["counts"], s["losses"], score=c["score"], together=c["together"], workspace=s["workspace"])
        return {"counts": s["counts"], "losses": s["losses"]}
    ccl.ccl_moe_balance_grad(s["logits"], s["counts"], s["dlogits"], c["k"], score=c["score"], dlosses=s["dlosses"])
    return {"dlogits": s["dlogits"]}


# ------------------------------------------------------------ what it takes
def work(case):
    c = case
    t, e = sum(_tokens(c)), DTYPES[c["dtype"]].itemsize
    if c["kind"] in ("norm", "norm_grad"):
        h, w = c["hidden"], DTYPES[c["weights"]].itemsize
        vectors = 2 if c["bias"] else 1
        if c["kind"] == "norm":
            return {"bytes": t * h * e * (4 if c["residual"] else 2) + h * w * vectors + (8 * t if c["stats"] else 0), "flops": 8 * t * h}
        return {"bytes": t * h * e * (4 if c["residual"] else 3) + h * w + 8 * t + c["p"] * h * vectors * DTYPES[c["dw"]].itemsize, "flops": 14 * t * h}
    n, k = c["experts"], c["k"]
    row, choices, counted = t * n * e, t * k * 4, c["p"] * (n + 2) * 4
    if c["kind"] == "gate":
        return {"bytes": row + 2 * choices + (counted if c["balance"] else 0), "flops": 6 * t * n}
    if c["kind"] == "gate_grad":
        return {"bytes": 2 * row + 2 * choices + (counted if c["balance"] else 0), "flops": 8 * t * n}
    if c["kind"] == "balance":
        return {"bytes": row + choices + counted, "flops": 5 * t * n}
    return {"bytes": 2 * row + counted, "flops": 8 * t * n}


# ------------------------------------------------- the definitions, 64 bits
def exact(case, seed):
    c, kind = dict(case), case["kind"]
    s = prepare(case, seed)
    if kind == "norm":
        return _exact_norm(s, c)
    if kind == "norm_grad":
        return _exact_norm_grad(s, c)
    return _exact_router(s, c, kind)


def _exact_norm(s, c):
    got = {"y": [], "sum": [], "mean": [], "rstd": []}
    for x, r, w, b in _each(s, "x", "residual", "weight", "bias"):
        total = x.double() if r is None else x.double() + r.double()
        kept = total.to(x.dtype).double()  # what is normed is the sum as it is kept
        var, mean = torch.var_mean(kept, dim=1, correction=0)
        rstd = (var + EPS) ** -0.5
        y = torch.einsum("ij,i,j->ij", kept - mean[:, None], rstd, w.double())
        got["y"].append(y if b is None else y + b.double())
        got["sum"].append(total)
        got["mean"].append(mean)
        got["rstd"].append(rstd)
    return _norm_outputs(c, *got.values())


def _exact_norm_grad(s, c):
    got = {"dx": [], "dweight": [], "dbias": []}
    for dy, ds, x, w, mean, rstd in _each(s, "dy", "dsum", "x", "weight", "mean", "rstd"):
        h, d = x.shape[1], dy.double()
        z = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
        v = d * w.double()
        dx = rstd.double()[:, None] * (v - (v.sum(1)[:, None] + z * torch.einsum("ij,ij->i", v, z)[:, None]) / h)
        got["dx"].append(dx if ds is None else dx + ds.double())
        got["dweight"].append(torch.einsum("ij,ij->j", d, z))
        got["dbias"].append(d.sum(0))
    return _norm_grad_outputs(c, *got.values())


def _exact_shares(finite, score):
    return torch.softmax(finite, 1) if score == "softmax" else torch.sigmoid(finite) / torch.sigmoid(finite).sum(1, keepdim=True)


def _exact_gates(finite, at, there, c):
    """Gates of the chosen experts; a choice that is not there weighs nothing."""
    if c["score"] == "softmax":
        u = torch.softmax(finite, 1).gather(1, at) * there
    else:
        u = torch.sigmoid(finite).gather(1, at) * there
    if c["normalize"]:
        u = u / u.sum(1, keepdim=True)
    return c["scale"] * u


def _exact_router(s, c, kind):
    e, k = c["experts"], c["k"]
    ids, gates, dlogits, counts, shares = [], [], [], [], []
    for r, logits in enumerate(s["logits"]):
        wide = logits.double()
        live = (wide > -math.inf).any(1)
        finite = wide.clamp(min=-1e30)  # exp of it is 0; a row of them alone is left out below
        if kind == "gate":
            # k times the largest of what is left, the first of equal ones
            left, places = wide.clone(), []
            for _ in range(k):
                top = left.max(1, keepdim=True).values
                at = (left == top).int().argmax(1, keepdim=True)
                places.append(torch.where(top > -math.inf, at, -1))
                left.scatter_(1, at, -math.inf)
            ids.append(torch.cat(places, 1).to(torch.int32))
        else:
            ids.append(s["ids"][r])
        there, at = ids[r] >= 0, ids[r].long().clamp(min=0)
        if kind == "gate":
            gates.append(torch.where(there & live[:, None], _exact_gates(finite, at, there, c), 0.0))
        if kind in ("gate", "balance"):
            held = ids[r][there].long()
            counts.append(torch.cat([torch.bincount(held, minlength=e), live.sum()[None]]))
            shares.append(torch.where(live[:, None], _exact_shares(finite, c["score"]), 0.0).sum(0))
            continue
        with torch.enable_grad():
            leaf = finite[live].requires_grad_()
            total = leaf.sum() * 0.0
            if kind == "gate_grad":
                total = total + torch.where(there[live], _exact_gates(leaf, at[live], there[live], c) * s["dgates"][r][live].double(), 0.0).sum()
            if kind == "balance_grad" or c["balance"]:
                n = s["counts"][r].double()
                mean = _exact_shares(leaf, c["score"]).sum(0) / n[-1]
                total = total + s["dlosses"][r].double().sum() * e * (n[:-1] / (k * n[-1]) * mean).sum()
            (d,) = torch.autograd.grad(total, leaf)
        out = torch.zeros_like(wide)
        out[live] = d
        dlogits.append(out)
    if kind in ("gate_grad", "balance_grad"):
        return {"dlogits": dlogits}
    if c["together"]:
        counts, shares = [sum(counts)] * c["p"], [sum(shares)] * c["p"]
    losses = [e * (n[:-1] / (k * n[-1].double()) * (v / n[-1])).sum().reshape(1) for n, v in zip(counts, shares)]
    out = {} if kind == "balance" else {"ids": ids, "gates": gates}
    if kind == "balance" or c["balance"]:
        out |= {"counts": [n.to(torch.int32) for n in counts], "losses": losses}
    return out
