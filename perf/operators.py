"""Cases of the local half of a mixture-of-experts step and of the optimizer behind the gradient buckets.

``kind`` of a case:

* ``sort``          expert ids -> offsets and rows, then the tokens' rows in expert order
* ``back``          the experts' rows back to their tokens, with or without gate weights
* ``back_grad``     the gradient of that for the rows and for the gate weights
* ``product``       each expert's rows times its weight matrix
* ``product_grad``  the gradients of that for the rows and for the weight matrices
* ``adamw``         one AdamW step over many tensors

``run`` computes them by elementary torch operations in 32 bits, or, where ``own`` is true, by the package's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 128  # elements that share a scale in an 8-bit state
DITHER_ELEM, DITHER_STEP = 1779033703, 2654435769  # threshold of element i at step t: top 20 bits of i * a + t * b mod 2^32


def listed():
    return [
        # serving: the eight tokens of one decoding step, each with 8 of 256 experts: latency
        {"name": "sort decode", "kind": "sort", "p": 1, "tokens": 8, "ragged": 0, "k": 8, "experts": 256, "of": 256, "hidden": 7168, "dtype": "bf16"},
        # training: 8 ranks of 2048 tokens, top-8 of 256 experts, every expert on the rank
        {"name": "sort train", "kind": "sort", "p": 8, "tokens": 2048, "ragged": 0, "k": 8, "experts": 256, "of": 256, "hidden": 7168, "dtype": "bf16"},
        # after an exchange: rows of one choice, other counts on each rank, some of other ranks' experts, an odd fp32 width
        {"name": "sort received", "kind": "sort", "p": 8, "tokens": 4001, "ragged": 333, "k": 1, "experts": 24, "of": 32, "hidden": 1001, "dtype": "f32"},
        # serving: a batch of decoding tokens comes back from its experts
        {"name": "back decode", "kind": "back", "p": 1, "tokens": 64, "ragged": 0, "k": 8, "experts": 256, "of": 256, "hidden": 4096, "dtype": "bf16", "weights": True},
        # training: the gradient of the gated sum, rows and gates
        {"name": "back train grad", "kind": "back_grad", "p": 8, "tokens": 2048, "ragged": 0, "k": 8, "experts": 256, "of": 256, "hidden": 7168, "dtype": "bf16", "weights": True},
        # serving: 16 tokens' 128 rows over the 32 experts of one rank: the weights' bytes
        {"name": "product decode", "kind": "product", "p": 1, "rows": 128, "experts": 32, "empty": 0, "n": 2048, "contract": 7168, "skew": 0.5},
        # training: a rank's rows after the exchange, wide experts
        {"name": "product train", "kind": "product", "p": 1, "rows": 32768, "experts": 32, "empty": 0, "n": 2048, "contract": 7168, "skew": 0.5},
        # training: both gradients, popularity by Zipf's law, experts that nobody chose; fp32 weight gradients as the buckets hold them
        {"name": "product train grad", "kind": "product_grad", "p": 1, "rows": 16384, "experts": 32, "empty": 3, "n": 2048, "contract": 7168, "skew": 1.2, "dw": "f32"},
        # small experts of odd widths on four ranks: no row starts on 16 bytes
        {"name": "product odd grad", "kind": "product_grad", "p": 4, "rows": 333, "experts": 5, "empty": 1, "n": 77, "contract": 131, "skew": 1.2, "dw": "bf16"},
        # the norms and biases of a small model, fp32 all through
        {"name": "adamw small", "kind": "adamw", "tensors": 48, "total": 60000, "skew": 1.0, "param": "f32", "grad": "f32", "copy": False, "bits": 32, "shift": 0},
        # 24 buckets of 25 MiB in fp32 masters, averaged bf16 gradients, bf16 weights written beside
        {"name": "adamw 32-bit", "kind": "adamw", "tensors": 24, "total": 157286400, "skew": 0.0, "param": "f32", "grad": "bf16", "copy": True, "bits": 32, "shift": 0},
        # the same masters with 8-bit states, 96 tensors of uneven sizes, gradients that start off the 16-byte grid
        {"name": "adamw 8-bit", "kind": "adamw", "tensors": 96, "total": 157286400, "skew": 0.5, "param": "f32", "grad": "bf16", "copy": True, "bits": 8, "shift": 3},
    ]


def _log(rng, lo, hi):
    v = round(math.exp(rng.uniform(math.log(lo), math.log(hi))))
    return v + 1 if v == 3072 else v


def _width(rng, lo, hi):
    """A row width: a multiple of 128 half of the time, of 8 a quarter, any number else."""
    v = _log(rng, lo, hi)
    u = rng.random()
    v = max(128, v // 128 * 128) if u < 0.5 else max(8, v // 8 * 8) if u < 0.75 else v
    return v + 8 if v == 3072 else v


def draw(rng):
    kind = rng.choice(["sort", "back", "back_grad", "product", "product_grad", "adamw"])
    if kind in ("sort", "back", "back_grad"):
        p, k = rng.choice([1, 1, 2, 4, 8]), rng.choice([1, 2, 4, 6, 8])
        of = rng.choice([8, 32, 60, 128, 256])
        experts = rng.choice([of, of, max(1, of // 4)])
        hidden = _width(rng, 64, 7168)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        most = 8 * 2048 * 8 * 7168 * 2  # bytes of the rows of the largest listed case
        tokens = _log(rng, 1, max(2, min(65536, most // (p * k * hidden * 4) // 2)))
        c = {"kind": kind, "p": p, "tokens": tokens, "ragged": rng.choice([0, tokens // 16]), "k": k, "experts": experts, "of": max(of, k),
             "hidden": hidden, "dtype": dtype}
        if kind != "sort":
            c["weights"] = kind == "back_grad" or rng.random() < 0.6
        return c
    if kind in ("product", "product_grad"):
        experts = rng.choice([1, 4, 8, 13, 32, 64])
        n, contract = _width(rng, 64, 4096), _width(rng, 64, 7168)
        while experts * n * contract > 32 * 2048 * 7168:
            experts = max(1, experts // 2)
        most = 32768 * 2048 * 7168 // 4
        rows = _log(rng, 1, max(2, min(32768, most // (n * contract))))
        c = {"kind": kind, "p": rng.choice([1, 1, 2]), "rows": rows, "experts": experts, "empty": rng.choice([0, experts // 4]), "n": n, "contract": contract,
             "skew": rng.choice([0.0, 0.5, 1.2])}
        if kind == "product_grad":
            c["dw"] = rng.choice(["f32", "f32", "bf16"])
        return c
    total = _log(rng, 1000, 60000000)
    param = rng.choice(["f32", "f32", "bf16"])
    return {"kind": "adamw", "tensors": rng.choice([1, 7, 40, 150]), "total": total, "skew": rng.choice([0.0, 0.5, 1.0]), "param": param,
            "grad": rng.choice(["bf16", "f32"]), "copy": param == "f32" and rng.random() < 0.5, "bits": rng.choice([8, 8, 32]), "shift": rng.choice([0, 0, 1, 4])}


# ------------------------------------------------------------------ inputs
def _tokens(c):
    """Tokens of each rank."""
    return [max(1, c["tokens"] - r * c["ragged"]) for r in range(c["p"])]


def _first(c):
    """The first expert that each rank holds."""
    return [r * c["experts"] % max(1, c["of"] - c["experts"] + 1) for r in range(c["p"])]


def _counts(c):
    """Rows of each expert, the same for every seed: shares by Zipf's law, the popular experts spread over the list."""
    e, share = c["experts"], []
    for i in range(e):
        at = (i * 7 + 3) % e if math.gcd(7, e) == 1 else i
        share.append(0.0 if i < c["empty"] and e > c["empty"] else (at + 1.0) ** -c["skew"])
    s, got, left = sum(share), [], c["rows"]
    for i in range(e):
        got.append(min(left, int(c["rows"] * share[i] / s)))
        left -= got[-1]
    got[share.index(max(share))] += left
    return got


def _sizes(c):
    """Elements of each tensor, and the places that a flat buffer gives them (multiples of 128)."""
    n = c["tensors"]
    share = [(i + 1.0) ** -c["skew"] for i in range(n)]
    s = sum(share)
    sizes = [max(1, int(c["total"] * x / s) - (i % 2 if c["skew"] else 0)) for i, x in enumerate(share)]
    starts, at = [], 0
    for m in sizes:
        starts.append(at)
        at += -(-m // BLOCK) * BLOCK
    return sizes, starts, at


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    s = {"case": c}
    if c["kind"] in ("sort", "back", "back_grad"):
        dt, k, h = DTYPES[c["dtype"]], c["k"], c["hidden"]
        s["first"] = _first(c)
        popular = torch.arange(1, c["of"] + 1, device="cuda", dtype=torch.float32).log().neg()  # Zipf's law, exponent 1
        draws = [torch.rand(t, c["of"], generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7) for t in _tokens(c)]
        s["ids"] = [(popular - (-u.log()).log()).topk(k, dim=1).indices.to(torch.int32).contiguous() for u in draws]
        s["offsets"] = [torch.zeros(c["experts"] + 1, dtype=torch.int32, device="cuda") for _ in s["ids"]]
        s["rows"] = [torch.zeros_like(i) for i in s["ids"]]
        if c["kind"] == "sort":
            s["x"] = [normal(t, h, dtype=dt) for t in _tokens(c)]
            s["xs"] = [torch.zeros(t * k, h, dtype=dt, device="cuda") for t in _tokens(c)]
            return s
        # the sort has been made before: its rows are the inputs here
        s["rows"] = [_plain_sort(i, c["experts"], f)[1] for i, f in zip(s["ids"], s["first"])]
        s["y"] = [normal(t * k, h, dtype=dt) for t in _tokens(c)]
        gates = [torch.rand(t, k, generator=g, device="cuda") + 0.05 for t in _tokens(c)]
        s["weights"] = [w / w.sum(1, keepdim=True) for w in gates] if c["weights"] else None
        if c["kind"] == "back":
            s["out"] = [torch.zeros(t, h, dtype=dt, device="cuda") for t in _tokens(c)]
        else:
            s["dout"] = [normal(t, h, dtype=dt, scale=0.01) for t in _tokens(c)]
            s["dy"] = [torch.zeros(t * k, h, dtype=dt, device="cuda") for t in _tokens(c)]
            s["dweights"] = [torch.zeros_like(w) for w in gates]
        return s
    if c["kind"] in ("product", "product_grad"):
        p, e, n, k = c["p"], c["experts"], c["n"], c["contract"]
        s["counts"] = _counts(c)  # the exchange's counts, which its caller has read to size the buffers
        rows = sum(s["counts"])
        at = torch.tensor([0] + s["counts"], dtype=torch.int64, device="cuda").cumsum(0).to(torch.int32)
        s["offsets"] = [at.clone() for _ in range(p)]
        s["x"] = [normal(rows, k, dtype=torch.bfloat16) for _ in range(p)]
        if c["kind"] == "product":
            s["w"] = [normal(e, n, k, dtype=torch.bfloat16, scale=k ** -0.5) for _ in range(p)]
            s["y"] = [torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda") for _ in range(p)]
        else:
            s["w"] = [normal(e, n, k, dtype=torch.bfloat16, scale=k ** -0.5) for _ in range(p)]
            s["dy"] = [normal(rows, n, dtype=torch.bfloat16, scale=0.01) for _ in range(p)]
            s["dx"] = [torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda") for _ in range(p)]
            s["dw"] = [torch.zeros(e, n, k, dtype=DTYPES[c["dw"]], device="cuda") for _ in range(p)]
        return s
    # adamw: flat buffers, a tensor on each multiple of 128 elements, `shift` elements into gradients and parameters
    sizes, starts, total = _sizes(c)
    s["sizes"], s["starts"], s["step"], s["shift"] = sizes, starts, 10, c["shift"]
    s["hyper"] = {"lr": 3e-4, "betas": (0.9, 0.95), "eps": 1e-8, "weight_decay": 0.1}
    at = torch.arange(total, device="cuda")
    block_start = torch.tensor(starts, device="cuda").repeat_interleave(torch.tensor([-(-m // BLOCK) for m in sizes], device="cuda"))
    s["block_start"] = block_start
    ends = torch.tensor([a + m for a, m in zip(starts, sizes)], device="cuda").repeat_interleave(torch.tensor([-(-m // BLOCK) for m in sizes], device="cuda"))
    live = at.view(-1, BLOCK) < ends[:, None]  # what lies between the tensors is zero and stays it
    spread = torch.exp(torch.randn(total // BLOCK, 1, generator=g, device="cuda") - 7.0)  # gradients' size differs from place to place
    shift = c["shift"]

    def flat(values, dtype, off):
        b = torch.zeros(total + 8, dtype=dtype, device="cuda")
        b[off:off + total] = (values * live).reshape(-1).to(dtype)
        return b

    s["p"] = flat(normal(total // BLOCK, BLOCK, scale=0.02), DTYPES[c["param"]], shift)
    s["g"] = flat(normal(total // BLOCK, BLOCK) * spread, DTYPES[c["grad"]], shift)
    s["copy"] = flat(torch.zeros(1, 1, device="cuda"), torch.bfloat16, shift) if c["copy"] else None
    m = normal(total // BLOCK, BLOCK) * spread * 0.3 * live
    v = ((normal(total // BLOCK, BLOCK) * spread * 0.5).square() + (0.5 * spread).square()) * live
    if c["bits"] == 32:
        s["m"], s["v"], s["m_scale"], s["v_scale"] = m.reshape(-1), v.reshape(-1), None, None
    else:
        index = (at.view(-1, BLOCK) - block_start[:, None])
        s["m"], s["m_scale"] = _plain_nearest(m)
        s["v"], s["v_scale"] = _plain_dithered(v.sqrt(), v, index, s["step"])
        s["m"], s["v"] = s["m"].reshape(-1), s["v"].reshape(-1)
    if own:
        from a2a_ring_ordered_gb300 import optim

        def views(b, off=0):
            return [b[off + a:off + a + m] for a, m in zip(starts, sizes)]

        def scales(b):
            return [b[a // BLOCK:a // BLOCK + -(-m // BLOCK)] for a, m in zip(starts, sizes)]

        states = {"exp_avg": views(s["m"]), "exp_avg_sq": views(s["v"])}
        if c["bits"] == 8:
            states |= {"exp_avg_scale": scales(s["m_scale"]), "exp_avg_sq_scale": scales(s["v_scale"])}
        s["optimizer"] = optim.AdamW(views(s["p"], shift), views(s["g"], shift), **s["hyper"], state_bits=c["bits"], states=states,
                                     copies=views(s["copy"], shift) if c["copy"] else None, step=s["step"])
    return s


# ------------------------------------------------------------- plain forms
def _plain_sort(ids, experts, first):
    key = ids.reshape(-1).long() - first
    held = (key >= 0) & (key < experts)
    key = torch.where(held, key, experts)
    order = key.argsort(stable=True)
    offsets = torch.searchsorted(key[order], torch.arange(experts + 1, device=ids.device))
    rows = torch.empty_like(key)
    rows[order] = torch.arange(key.numel(), device=ids.device)
    return offsets.to(torch.int32), torch.where(held, rows, -1).to(torch.int32).view(ids.shape), order


def _plain_sorted(x, ids, experts, first):
    offsets, rows, order = _plain_sort(ids, experts, first)
    there = torch.arange(order.numel(), device=x.device) < offsets[-1]
    return offsets, rows, torch.where(there[:, None], x[order // ids.shape[1]], 0)


def _plain_rows(y, rows):
    return torch.where((rows >= 0)[..., None], y[rows.long().clamp(min=0)].float(), 0.0)


def _plain_back(y, rows, weights):
    v = _plain_rows(y, rows)
    return (v if weights is None else v * weights[..., None]).sum(1).to(y.dtype)


def _plain_back_grad(dout, y, rows, weights):
    w = torch.ones_like(rows, dtype=torch.float32) if weights is None else weights
    d = dout.float()[:, None]
    dy = torch.zeros(y.shape[0] + 1, y.shape[1], dtype=y.dtype, device=y.device)
    dy[torch.where(rows < 0, y.shape[0], rows).long()] = (w[..., None] * d).to(y.dtype)
    return dy[:-1], (_plain_rows(y, rows) * d).sum(-1)


def _plain_product(x, w, counts):
    return torch.cat([a.float() @ b.float().T for a, b in zip(x.split(counts), w)]).to(x.dtype)


def _plain_product_grad(dy, x, w, counts, dw):
    dx = torch.cat([a.float() @ b.float() for a, b in zip(dy.split(counts), w)]).to(x.dtype)
    return dx, torch.stack([a.float().T @ b.float() for a, b in zip(dy.split(counts), x.split(counts))]).to(dw)


def _plain_scale(x):
    """(448 / amax, amax / 448) of each block; a block of (nearly) nothing has scale 1 and codes 0."""
    top = x.abs().amax(1, keepdim=True)
    none = top <= 2.0 ** -100
    return torch.where(none, 0.0, 448.0 / top), torch.where(none, 1.0, top / 448.0)


def _plain_nearest(x):
    up, scale = _plain_scale(x)
    return (x * up).clamp(-448, 448).to(torch.float8_e4m3fn), scale.reshape(-1)


def _plain_dithered(root, v, index, step):
    """e4m3 of root / scale, up or down by the element's threshold at this step; never 0 where v is not."""
    up, scale = _plain_scale(root)
    threshold = ((index * DITHER_ELEM + step * DITHER_STEP) & 0xFFFFFFFF) >> 12
    bits = (root * up * 2.0 ** -120).view(torch.int32)
    code = ((bits + threshold.to(torch.int32)) >> 20).clamp(max=0x7E)
    code = torch.where((v > 0) & (up > 0), code.clamp(min=1), torch.where(up > 0, code, 0))
    return code.to(torch.uint8).view(torch.float8_e4m3fn), scale.reshape(-1)


def _plain_adamw(s):
    h, n, off = s["hyper"], s["m"].numel(), s["shift"]
    s["step"] += 1
    t, (b1, b2) = s["step"], h["betas"]
    p, g = s["p"][off:off + n].view(-1, BLOCK).float(), s["g"][off:off + n].view(-1, BLOCK).float()
    m, v = s["m"].view(-1, BLOCK).float(), s["v"].view(-1, BLOCK).float()
    if s["m_scale"] is not None:
        m, v = m * s["m_scale"][:, None], (v * s["v_scale"][:, None]).square()
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    root = v.sqrt()
    p = p * (1 - h["lr"] * h["weight_decay"]) - (m / (root * (1 - b2 ** t) ** -0.5 + h["eps"])) * (h["lr"] / (1 - b1 ** t))
    s["p"][off:off + n] = p.view(-1)
    if s["copy"] is not None:
        s["copy"][off:off + n] = p.view(-1)
    if s["m_scale"] is None:
        s["m"][:], s["v"][:] = m.view(-1), v.view(-1)
    else:
        index = torch.arange(n, device=p.device).view(-1, BLOCK) - s["block_start"][:, None]
        (a, s["m_scale"][:]), (b, s["v_scale"][:]) = _plain_nearest(m), _plain_dithered(root, v, index, t)
        s["m"][:], s["v"][:] = a.view(-1), b.view(-1)


def _adamw_outputs(s):
    out = {"param": s["p"], "exp_avg": s["m"], "exp_avg_sq": s["v"]}
    if s["copy"] is not None:
        out["copy"] = s["copy"]
    if s["m_scale"] is not None:
        out |= {"exp_avg_scale": s["m_scale"], "exp_avg_sq_scale": s["v_scale"]}
    return out


def run(s):
    c, kind = s["case"], s["case"]["kind"]
    if own:
        return _own(s, c, kind)
    if kind == "sort":
        got = [_plain_sorted(x, i, c["experts"], f) for x, i, f in zip(s["x"], s["ids"], s["first"])]
        return {"offsets": [v[0] for v in got], "rows": [v[1] for v in got], "sorted": [v[2] for v in got]}
    if kind in ("back", "back_grad"):
        weights = s["weights"] or [None] * c["p"]
        if kind == "back":
            return {"out": [_plain_back(*v) for v in zip(s["y"], s["rows"], weights)]}
        got = [_plain_back_grad(*v) for v in zip(s["dout"], s["y"], s["rows"], weights)]
        return {"dy": [v[0] for v in got], "dweights": [v[1] for v in got]}
    if kind == "product":
        return {"y": [_plain_product(x, w, s["counts"]) for x, w in zip(s["x"], s["w"])]}
    if kind == "product_grad":
        got = [_plain_product_grad(d, x, w, s["counts"], DTYPES[c["dw"]]) for d, x, w in zip(s["dy"], s["x"], s["w"])]
        return {"dx": [v[0] for v in got], "dw": [v[1] for v in got]}
    _plain_adamw(s)
    return _adamw_outputs(s)


def _own(s, c, kind):
    from a2a_ring_ordered_gb300 import ccl

    if kind == "sort":
        ccl.ccl_moe_sort(s["ids"], c["experts"], s["offsets"], s["rows"], first_expert=s["first"])
        ccl.ccl_moe_to_experts(s["x"], s["rows"], s["xs"])
        return {"offsets": s["offsets"], "rows": s["rows"], "sorted": s["xs"]}
    if kind == "back":
        ccl.ccl_moe_from_experts(s["y"], s["rows"], s["weights"], s["out"])
        return {"out": s["out"]}
    if kind == "back_grad":
        ccl.ccl_moe_from_experts_grad(s["dout"], s["y"], s["rows"], s["weights"], s["dy"], s["dweights"])
        return {"dy": s["dy"], "dweights": s["dweights"]}
    if kind == "product":
        ccl.ccl_moe_product(s["x"], s["offsets"], s["w"], s["y"])
        return {"y": s["y"]}
    if kind == "product_grad":
        ccl.ccl_moe_product_grad_input(s["dy"], s["offsets"], s["w"], s["dx"])
        ccl.ccl_moe_product_grad_weight(s["dy"], s["x"], s["offsets"], s["dw"])
        return {"dx": s["dx"], "dw": s["dw"]}
    s["optimizer"].step()
    return _adamw_outputs(s)


# ------------------------------------------------------------ what it takes
def work(case):
    c = case
    if c["kind"] in ("sort", "back", "back_grad"):
        e, k, h, t = DTYPES[c["dtype"]].itemsize, c["k"], c["hidden"], sum(_tokens(c))
        r = t * k * c["experts"] / c["of"]  # rows, while the ids are spread evenly
        index = 4 * t * k
        if c["kind"] == "sort":
            return {"bytes": 2 * index + 4 * c["p"] * (c["experts"] + 1) + (t + r) * h * e, "flops": 0}
        gates = index if c["weights"] else 0
        if c["kind"] == "back":
            return {"bytes": index + gates + (r + t) * h * e, "flops": 2 * r * h}
        return {"bytes": index + gates + index + (t + 2 * r) * h * e, "flops": 3 * r * h}
    if c["kind"] in ("product", "product_grad"):
        n, k, r = c["n"], c["contract"], c["rows"]
        held = sum(v > 0 for v in _counts(c)) * n * k  # weights of experts that have rows
        if c["kind"] == "product":
            return {"bytes": c["p"] * 2 * (r * (n + k) + held), "flops": c["p"] * 2 * r * n * k}
        return {"bytes": c["p"] * (2 * (r * (n + 2 * k) + held) + DTYPES[c["dw"]].itemsize * c["experts"] * n * k), "flops": c["p"] * 4 * r * n * k}
    n = sum(_sizes(c)[0])
    each = 2 * DTYPES[c["param"]].itemsize + DTYPES[c["grad"]].itemsize + (2 if c["copy"] else 0) + (16 if c["bits"] == 32 else 4 + 16 / BLOCK)
    return {"bytes": n * each, "flops": 15 * n}


# ------------------------------------------------- the definitions, 64 bits
def exact(case, seed):
    c, kind = dict(case), case["kind"]
    s = prepare(case, seed)
    if kind in ("sort", "back", "back_grad"):
        return _exact_moe(s, c, kind)
    if kind in ("product", "product_grad"):
        return _exact_product(s, c, kind)
    return _exact_adamw(s, c)


def _exact_moe(s, c, kind):
    k = c["k"]
    out = {"out": []} if kind == "back" else {"dy": [], "dweights": []} if kind == "back_grad" else {"offsets": [], "rows": [], "sorted": []}
    for r in range(c["p"]):
        t = _tokens(c)[r]
        token = torch.arange(t, device="cuda").repeat_interleave(k)  # of each (token, choice)
        if kind == "sort":
            ids = s["ids"][r].reshape(-1).long()
            n = [torch.nonzero(ids == s["first"][r] + e).reshape(-1) for e in range(c["experts"])]
            items = torch.cat(n)
            rows = torch.full((t * k,), -1, dtype=torch.int32, device="cuda")
            rows[items] = torch.arange(items.numel(), dtype=torch.int32, device="cuda")
            ordered = torch.zeros(t * k, c["hidden"], dtype=torch.float64, device="cuda")
            ordered[:items.numel()] = s["x"][r].double()[token[items]]
            out["offsets"].append(torch.tensor([0] + [v.numel() for v in n], device="cuda").cumsum(0).to(torch.int32))
            out["rows"].append(rows.view(t, k))
            out["sorted"].append(ordered)
            continue
        rows = s["rows"][r].reshape(-1).long()
        there = torch.nonzero(rows >= 0).reshape(-1)
        gate = s["weights"][r].reshape(-1).double() if s["weights"] else torch.ones(t * k, dtype=torch.float64, device="cuda")
        y = s["y"][r].double()
        if kind == "back":
            o = torch.zeros(t, c["hidden"], dtype=torch.float64, device="cuda")
            o.index_add_(0, token[there], y[rows[there]] * gate[there, None])
            out["out"].append(o)
            continue
        d = s["dout"][r].double()
        dy, dw = torch.zeros_like(y), torch.zeros(t * k, dtype=torch.float64, device="cuda")
        dy[rows[there]] = gate[there, None] * d[token[there]]
        dw[there] = torch.einsum("ih,ih->i", y[rows[there]], d[token[there]])
        out["dy"].append(dy)
        out["dweights"].append(dw.view(t, k))
    return out


def _exact_product(s, c, kind):
    out = {"y": []} if kind == "product" else {"dx": [], "dw": []}
    for r in range(c["p"]):
        x, at = s["x"][r], [0]
        for n in s["counts"]:
            at.append(at[-1] + n)
        if kind == "product":
            y = torch.zeros(x.shape[0], c["n"], dtype=torch.float64, device="cuda")
            for e in range(c["experts"]):
                y[at[e]:at[e + 1]] = torch.einsum("rk,nk->rn", x[at[e]:at[e + 1]].double(), s["w"][r][e].double())
            out["y"].append(y)
            continue
        dy = s["dy"][r]
        dx = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(c["experts"], c["n"], c["contract"], dtype=torch.float64, device="cuda")
        for e in range(c["experts"]):
            d = dy[at[e]:at[e + 1]].double()
            dx[at[e]:at[e + 1]] = torch.einsum("rn,nk->rk", d, s["w"][r][e].double())
            dw[e] = torch.einsum("rn,rk->nk", d, x[at[e]:at[e + 1]].double())
        out["dx"].append(dx)
        out["dw"].append(dw)
    return out


def _grid(x, up):
    """x >= 0 to the e4m3 numbers: the spacing at x, then floor of the ratio plus `up` (0.5 with ties to even where None)."""
    spacing = torch.exp2(torch.frexp(x.clamp(min=2.0 ** -6))[1].double() - 4)
    q = x / spacing
    return ((q.round() if up is None else (q + up).floor()) * spacing).clamp(max=448.0)


def _exact_adamw(s, c):
    h, t, off, n = s["hyper"], s["step"] + 1, s["shift"], s["m"].numel()
    b1, b2 = h["betas"]
    p, g = s["p"].double(), s["g"].double()
    m, v = s["m"].double(), s["v"].double()
    if c["bits"] == 8:
        m = m * s["m_scale"].double().repeat_interleave(BLOCK)
        v = (v * s["v_scale"].double().repeat_interleave(BLOCK)) ** 2
    gn = g[off:off + n]
    m = b1 * m + (1 - b1) * gn
    v = b2 * v + (1 - b2) * gn ** 2
    p[off:off + n] -= h["lr"] * h["weight_decay"] * p[off:off + n] + h["lr"] * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + h["eps"])
    out = {"param": p, "exp_avg": m, "exp_avg_sq": v}
    if c["copy"]:
        out["copy"] = p.clone()
    if c["bits"] == 8:
        root = v.sqrt()
        blocks_m, blocks_s = m.view(-1, BLOCK), root.view(-1, BLOCK)
        top_m, top_s = blocks_m.abs().amax(1), blocks_s.amax(1)
        scale_m = torch.where(top_m > 2.0 ** -100, top_m / 448, 1.0)
        scale_s = torch.where(top_s > 2.0 ** -100, top_s / 448, 1.0)
        index = torch.arange(n, device="cuda") - s["block_start"].repeat_interleave(BLOCK)
        up = ((index * DITHER_ELEM + t * DITHER_STEP) % 2 ** 32 // 4096).double() / 2 ** 20
        codes_m = torch.where(top_m[:, None] > 2.0 ** -100, blocks_m.sign() * _grid(blocks_m.abs() / scale_m[:, None], None), 0.0)
        codes_s = _grid(blocks_s / scale_s[:, None], up.view(-1, BLOCK))
        codes_s = torch.where((blocks_s > 0) & (codes_s == 0), 2.0 ** -9, codes_s)
        codes_s = torch.where(top_s[:, None] > 2.0 ** -100, codes_s, 0.0)
        out |= {"exp_avg": codes_m.reshape(-1), "exp_avg_sq": codes_s.reshape(-1), "exp_avg_scale": scale_m, "exp_avg_sq_scale": scale_s}
    return out
