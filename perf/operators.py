"""Cases and plain forms of the token rows: the row operators at a model's two ends and at its heads.

``embed``        rows of an embedding table looked up by token id, times a scale
``embed_grad``   the table's gradient: for each token the sum of its rows
``qk``           RMS norm of every q and k head with a learned weight, then the rotation of its position
``qk_grad``      the gradient of that, for q, k and both weights
``score``        log probability of a given token per row of logits, the row's entropy, its top alternatives
``score_grad``   the gradient of log probability and entropy, for the logits and their column scale

``run`` computes a case in plain torch operations in 32 bits, or, where ``own`` is true, through this
package's binding.  ``exact`` computes the same from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "bf16": 2}
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoding step of 64 sequences: the launch and the memory's latency are all there is
        {"name": "embed_decode", "op": "embed", "rows": 64, "cols": 4096, "vocab": 50304, "table": "bf16", "pad": 0.0},
        # a packed batch of prompts read from fp32 master weights, a few of its tokens padding
        {"name": "embed_prompt", "op": "embed", "rows": 32768, "cols": 4096, "vocab": 131072, "table": "fp32", "pad": 0.02},
        # one short sequence of odd length; the bf16 gradient goes on to the unit-row weight's own
        {"name": "embed_grad_short", "op": "embed_grad", "rows": 1021, "cols": 768, "vocab": 50304, "table": "bf16", "pad": 0.0},
        # a training batch: a large fp32 table, some tokens many hundred times in it
        {"name": "embed_grad_batch", "op": "embed_grad", "rows": 32768, "cols": 4096, "vocab": 131072, "table": "fp32", "pad": 0.02},
        # heads of a decoding step
        {"name": "qk_decode", "op": "qk", "rows": 16, "q_heads": 16, "k_heads": 4, "head_dim": 256},
        # heads of a long prompt, slices of one fused projection
        {"name": "qk_prompt", "op": "qk", "rows": 8192, "q_heads": 16, "k_heads": 4, "head_dim": 256},
        # a 768-wide layer's heads over one odd sequence
        {"name": "qk_grad_short", "op": "qk_grad", "rows": 1021, "q_heads": 12, "k_heads": 12, "head_dim": 64},
        # a training batch with grouped heads
        {"name": "qk_grad_batch", "op": "qk_grad", "rows": 16384, "q_heads": 32, "k_heads": 8, "head_dim": 128},
        # a decoding step that reports alternatives, a third of the vocabulary masked out by a grammar
        {"name": "score_decode", "op": "score", "rows": 7, "vocab": 131072, "type": "fp32", "scaled": True, "masked": 0.3, "top": 20, "inv_temp": 1.25},
        # scoring a batch of answers under a scaled head
        {"name": "score_batch", "op": "score", "rows": 8192, "vocab": 131072, "type": "bf16", "scaled": True, "masked": 0.0, "top": 5, "inv_temp": 1.0},
        # a small step over an odd vocabulary whose rows are not aligned
        {"name": "score_grad_odd", "op": "score_grad", "rows": 509, "vocab": 32003, "type": "bf16", "scaled": False, "masked": 0.0, "inv_temp": 1.0},
        # a training batch, with the head's scale learned
        {"name": "score_grad_batch", "op": "score_grad", "rows": 8192, "vocab": 131072, "type": "bf16", "scaled": True, "masked": 0.0, "inv_temp": 1.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "qk", "qk_grad", "score", "score_grad"])
    if op.startswith("embed"):
        return {"op": op, "rows": _log_int(rng, 1, 32768), "cols": 8 * _log_int(rng, 32, 512),
                "vocab": _log_int(rng, 1000, 131072), "table": rng.choice(["fp32", "bf16"]),
                "pad": rng.choice([0.0, 0.1])}
    if op.startswith("qk"):
        k_heads = rng.choice([1, 2, 4, 5, 8])
        return {"op": op, "rows": _log_int(rng, 1, 8192), "q_heads": k_heads * rng.choice([1, 2, 4]),
                "k_heads": k_heads, "head_dim": rng.choice([64, 80, 96, 128, 256])}
    case = {"op": op, "rows": _log_int(rng, 1, 4096), "vocab": _log_int(rng, 1000, 131072),
            "type": rng.choice(["fp32", "bf16"]), "scaled": rng.random() < 0.5,
            "masked": rng.choice([0.0, 0.25]), "inv_temp": rng.choice([1.0, 0.8, 1.5])}
    if op == "score":
        case["top"] = rng.choice([0, 1, 5, 20, 32])
    return case


# ----------------------------------------------------------------- inputs

def _tokens(g, rows, vocab, pad):
    """Token ids whose frequency falls with their rank, as in text; -1 stands for padding."""
    u = torch.rand(rows, device="cuda", generator=g, dtype=torch.float64)
    ids = (torch.exp(u * math.log(vocab + 1.0)) - 1.0).long().clamp_(0, vocab - 1)
    if pad:
        ids[torch.rand(rows, device="cuda", generator=g) < pad] = -1
    return ids


def _unlike(rows, vocab):
    """How many different tokens `rows` of those draws hold, on average."""
    p = np.diff(np.log1p(np.arange(vocab + 1, dtype=np.float64))) / math.log(vocab + 1.0)
    return float(-np.expm1(rows * np.log1p(-p)).sum())


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, rows = case["op"], case["rows"]
    s = {"case": dict(case)}

    def normal(*shape, dtype=torch.float32, sd=1.0):
        return torch.randn(*shape, device="cuda", generator=g, dtype=dtype).mul_(sd)

    def uniform(n, lo, hi):
        return torch.rand(n, device="cuda", generator=g) * (hi - lo) + lo

    if op.startswith("embed"):
        s["ids"] = _tokens(g, rows, case["vocab"], case["pad"])
        s["scale"] = math.sqrt(case["cols"])
        if op == "embed":
            s["table"] = normal(case["vocab"], case["cols"], dtype=TYPES[case["table"]], sd=0.02)
        else:
            s["dy"] = normal(rows, case["cols"], dtype=torch.bfloat16)
    elif op.startswith("qk"):
        hd, wq, wk = case["head_dim"], case["q_heads"] * case["head_dim"], case["k_heads"] * case["head_dim"]
        qkv = normal(rows, wq + 2 * wk, dtype=torch.bfloat16)      # a fused projection: q | k | v
        s["q"], s["k"] = qkv[:, :wq], qkv[:, wq:wq + wk]
        s["positions"] = torch.randint(0, 200_000, (1,), device="cuda", generator=g, dtype=torch.int32) \
            + torch.arange(rows, device="cuda", dtype=torch.int32)
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, hd, 2, device="cuda", dtype=torch.float64) / hd)).float()
        s["q_weight"], s["k_weight"] = uniform(hd, 0.5, 1.5), uniform(hd, 0.5, 1.5)
        if op == "qk_grad":
            s["dq_out"], s["dk_out"] = normal(rows, wq, dtype=torch.bfloat16), normal(rows, wk, dtype=torch.bfloat16)
    else:
        vocab = case["vocab"]
        s["labels"] = _tokens(g, rows, vocab, 0.0)
        s["logits"] = normal(rows, vocab, dtype=TYPES[case["type"]], sd=2.5)
        at = torch.arange(rows, device="cuda")
        s["logits"][at, s["labels"]] += uniform(rows, 0.0, 12.0).to(s["logits"].dtype)   # what a model has learned
        if case["masked"]:
            cols = torch.rand(vocab, device="cuda", generator=g) < case["masked"]
            s["logits"].masked_fill_(cols, -math.inf)
            s["logits"][at, s["labels"]] = 3.0
        s["scale"] = uniform(vocab, 0.8, 1.25) if case["scaled"] else None
        if op == "score_grad":
            s["dlogp"], s["dentropy"] = normal(rows), normal(rows, sd=0.01)
            lse, ent = [], []
            for i in range(0, rows, 512):                          # what the forward pass leaves behind
                z = _logits64(s, slice(i, i + 512))
                a, b = _lse_entropy64(z)
                lse.append(a.float())
                ent.append(b.float())
            s["lse"], s["entropy"] = torch.cat(lse), torch.cat(ent)
    return s


# ------------------------------------------------------------ plain forms

def _plain_embed(s):
    table, ids = s["table"], s["ids"]
    known = (ids >= 0) & (ids < table.shape[0])
    y = table[ids.clamp(0, table.shape[0] - 1)].float() * s["scale"]
    return torch.where(known[:, None], y, 0.0).bfloat16()


def _plain_embed_grad(s):
    case, ids = s["case"], s["ids"]
    vocab = case["vocab"]
    at = torch.where((ids >= 0) & (ids < vocab), ids, vocab)       # padding goes to a row of its own
    acc = torch.zeros(vocab + 1, case["cols"], device="cuda")
    acc.index_add_(0, at, s["dy"].float(), alpha=s["scale"])
    return acc[:vocab].to(TYPES[case["table"]])


def _heads(x, hd):
    return x.float().reshape(x.shape[0], -1, hd)


def _angles(s):
    t = s["positions"].double()[:, None] * s["inv_freq"].double()
    return torch.cos(t).float()[:, None], torch.sin(t).float()[:, None]


def _rotate(x, c, sn):
    a, b = x.chunk(2, dim=-1)
    return torch.cat([a * c - b * sn, b * c + a * sn], dim=-1)


def _plain_qk(s):
    hd = s["case"]["head_dim"]
    c, sn = _angles(s)
    out = {}
    for n in "qk":
        x = _heads(s[n], hd)
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s[n + "_weight"]
        out[n] = _rotate(x, c, sn).bfloat16().reshape(s[n].shape)
    return out


def _plain_qk_grad(s):
    hd = s["case"]["head_dim"]
    c, sn = _angles(s)
    out = {}
    for n in "qk":
        x = _heads(s[n], hd)
        inv = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        xn = x * inv
        dn = _rotate(_heads(s["d%s_out" % n], hd), c, -sn)
        out["d%s_weight" % n] = (dn * xn).sum(0).sum(0)
        dn = dn * s[n + "_weight"]
        dx = (dn - xn * (dn * xn).mean(-1, keepdim=True)) * inv
        out["d" + n] = dx.bfloat16().reshape(s[n].shape)
    return out


def _logits32(s):
    z = s["logits"].float()
    if s["scale"] is not None:
        z = z * s["scale"]
    return z * s["case"]["inv_temp"] if s["case"]["inv_temp"] != 1.0 else z


def _plain_score(s):
    z = _logits32(s)
    m = z.amax(-1, keepdim=True)
    d = z - m
    e = torch.exp(d)
    total = e.sum(-1)
    log_total = torch.log(total)
    lse = m[:, 0] + log_total
    out = {"logp": d.gather(1, s["labels"][:, None])[:, 0] - log_total,
           "entropy": log_total - torch.where(e > 0, e * d, 0.0).sum(-1) / total, "lse": lse}
    if s["case"]["top"]:
        # largest first, equal values by their place: one whole number that orders both
        bits = (z + 0.0).view(torch.int32)
        key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() * 2 ** 32
        key += 2 ** 32 - 1 - torch.arange(z.shape[1], device="cuda")
        ids = 2 ** 32 - 1 - (torch.topk(key, s["case"]["top"], dim=-1).values & (2 ** 32 - 1))
        out["top_ids"], out["top_logp"] = ids.int(), z.gather(1, ids) - lse[:, None]
    return out


def _plain_score_grad(s):
    z = _logits32(s)
    lp = z - s["lse"][:, None]
    p = torch.exp(lp)
    dz = -p * s["dlogp"][:, None]
    dz -= s["dentropy"][:, None] * torch.where(p > 0, p * (lp + s["entropy"][:, None]), 0.0)
    dz.scatter_add_(1, s["labels"][:, None], s["dlogp"][:, None])
    dz *= s["case"]["inv_temp"]
    if s["scale"] is None:
        return {"dlogits": dz.to(s["logits"].dtype)}
    x = s["logits"].float()
    dscale = torch.where(dz != 0, dz * x, 0.0).sum(0)
    return {"dlogits": (dz * s["scale"]).to(s["logits"].dtype), "dscale": dscale}


PLAIN = {"embed": _plain_embed, "embed_grad": _plain_embed_grad, "qk": _plain_qk, "qk_grad": _plain_qk_grad,
         "score": _plain_score, "score_grad": _plain_score_grad}


# ---------------------------------------------------- the framework's own

def _own(s):
    from scale_invariant_row_amd import binding as B
    case = s["case"]
    op = case["op"]
    if op == "embed":
        return B.ds_embed_rows(s["table"], s["ids"], s["scale"])
    if op == "embed_grad":
        return B.ds_embed_rows_backward(s["dy"], s["ids"], case["vocab"], s["scale"], dtype=TYPES[case["table"]])
    if op == "qk":
        q, k = B.ds_qk_rows_rms(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_weight"], s["k_weight"],
                                case["head_dim"], EPS)
        return {"q": q, "k": k}
    if op == "qk_grad":
        dq, dk, dqw, dkw = B.ds_qk_rows_rms_backward(
            s["q"], s["k"], s["positions"], s["inv_freq"], s["q_weight"], s["k_weight"], s["dq_out"], s["dk_out"],
            case["head_dim"], EPS)
        return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}
    if op == "score":
        r = B.ds_logprob_rows(s["logits"], s["labels"], scale=s["scale"], inv_temp=case["inv_temp"], top_k=case["top"])
        out = {"logp": r.logp, "entropy": r.entropy, "lse": r.lse}
        if case["top"]:
            out["top_ids"], out["top_logp"] = r.top_ids, r.top_logp
        return out
    dlogits, dscale = B.ds_logprob_rows_backward(
        s["logits"], s["labels"], s["lse"], s["entropy"], s["dlogp"], s["dentropy"], scale=s["scale"],
        inv_temp=case["inv_temp"])
    return {"dlogits": dlogits} if dscale is None else {"dlogits": dlogits, "dscale": dscale}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------- work

def work(case):
    op, rows = case["op"], case["rows"]
    if op.startswith("embed"):
        cols, size = case["cols"], SIZE[case["table"]]
        tokens = rows * (1 - case["pad"])
        if op == "embed":
            n = rows * 8 + _unlike(tokens, case["vocab"]) * cols * size + rows * cols * 2
        else:
            n = rows * 8 + tokens * cols * 2 + case["vocab"] * cols * size
        return {"bytes": n, "flops": tokens * cols}
    if op.startswith("qk"):
        hd = case["head_dim"]
        values = rows * (case["q_heads"] + case["k_heads"]) * hd
        tables = rows * 4 + hd * 2 + 2 * hd * 4
        if op == "qk":
            return {"bytes": values * 4 + tables, "flops": values * 7}
        return {"bytes": values * 6 + tables + 2 * hd * 4, "flops": values * 15}
    values, size = rows * case["vocab"], SIZE[case["type"]]
    columns = case["vocab"] * 4 if case["scaled"] else 0
    if op == "score":
        return {"bytes": values * size + columns + rows * (8 + 12 + 8 * case["top"]), "flops": values * 6}
    return {"bytes": values * size * 2 + columns * 2 + rows * (8 + 16), "flops": values * 8}


# -------------------------------------------- the definitions, in 64 bits

def _logits64(s, rows):
    z = s["logits"][rows].double()
    if s["scale"] is not None:
        z = z * s["scale"].double()
    return z * s["case"]["inv_temp"]


def _lse_entropy64(z):
    top = z.amax(-1, keepdim=True)
    w = torch.exp(z - top)
    n = w.sum(-1)
    mean = (w * torch.clamp(z - top, min=-1e4)).sum(-1) / n
    return top[:, 0] + torch.log(n), torch.log(n) - mean


def _exact_heads(s, name, theta):
    """x / rms(x) as [rows, heads, half, 2] (the two values that turn together), and 1 / rms."""
    hd = s["case"]["head_dim"]
    x = s[name].double().reshape(s[name].shape[0], -1, 2, hd // 2).transpose(2, 3)
    inv = ((x ** 2).sum((2, 3), keepdim=True) / hd + EPS) ** -0.5
    return x * inv, inv


def _turned(v, theta):
    """Each pair of values turned by its angle, as a product of complex numbers."""
    turn = torch.polar(torch.ones_like(theta), theta)[:, None]
    return torch.view_as_real(torch.view_as_complex(v.contiguous()) * turn)


def _pairs(v, hd):
    return v.double().reshape(v.shape[0], -1, 2, hd // 2).transpose(2, 3)


def _flat(v):
    return v.transpose(2, 3).reshape(v.shape[0], -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        y = torch.zeros(case["rows"], case["cols"], device="cuda", dtype=torch.float64)
        known = torch.nonzero(s["ids"] >= 0)[:, 0]
        y[known] = s["table"][s["ids"][known]].double() * s["scale"]
        return y
    if op == "embed_grad":
        order = torch.argsort(s["ids"], stable=True)
        order = order[s["ids"][order] >= 0]
        tokens, counts = torch.unique_consecutive(s["ids"][order], return_counts=True)
        total = torch.zeros(case["vocab"], case["cols"], device="cuda", dtype=torch.float64)
        if order.numel():
            total[tokens] = torch.segment_reduce(s["dy"][order].double(), "sum", lengths=counts) * s["scale"]
        return total
    if op.startswith("qk"):
        hd = case["head_dim"]
        theta = s["positions"].double()[:, None] * s["inv_freq"].double()
        out = {}
        for n in "qk":
            xn, inv = _exact_heads(s, n, theta)
            w = s[n + "_weight"].double().reshape(2, hd // 2).t()
            if op == "qk":
                out[n] = _flat(_turned(xn * w, theta))
                continue
            d = _turned(_pairs(s["d%s_out" % n], hd), -theta)
            out["d%s_weight" % n] = (d * xn).sum((0, 1)).t().reshape(hd)
            d = d * w
            out["d" + n] = _flat(inv * (d - xn * (d * xn).sum((2, 3), keepdim=True) / hd))
        return out
    rows, vocab = case["rows"], case["vocab"]
    parts = [slice(i, min(rows, i + 512)) for i in range(0, rows, 512)]
    if op == "score":
        got = {"logp": [], "entropy": [], "lse": [], "top_logp": []}
        for r in parts:
            z = _logits64(s, r)
            lse, ent = _lse_entropy64(z)
            got["lse"].append(lse)
            got["entropy"].append(ent)
            got["logp"].append(z.gather(1, s["labels"][r, None])[:, 0] - lse)
            if case["top"]:
                got["top_logp"].append(torch.topk(z, case["top"], dim=-1).values - lse[:, None])
        out = {k: torch.cat(v) for k, v in got.items() if v}
        if case["top"]:
            out["top_ids"] = None
        return out
    dlogits = torch.empty(rows, vocab, device="cuda", dtype=torch.float64)
    dscale = torch.zeros(vocab, device="cuda", dtype=torch.float64)
    for r in parts:
        z = _logits64(s, r)
        lse, ent = _lse_entropy64(z)
        p = torch.exp(z - lse[:, None])
        chosen = torch.zeros_like(p).scatter_(1, s["labels"][r, None], 1.0)
        surprise = torch.where(p > 0, z - lse[:, None] + ent[:, None], 0.0)
        d = (chosen - p) * s["dlogp"][r, None].double() - s["dentropy"][r, None].double() * p * surprise
        d = d * case["inv_temp"]
        if s["scale"] is not None:
            dscale += torch.where(p > 0, d * s["logits"][r].double(), 0.0).sum(0)
            d = d * s["scale"].double()
        dlogits[r] = d
    return {"dlogits": dlogits, "dscale": dscale} if s["scale"] is not None else {"dlogits": dlogits}
