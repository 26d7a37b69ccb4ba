"""Cases and plain forms of the rows of a decoding step: rotated heads, the paged cache, drafted tokens.

``rope``        q and k heads turned by their position: half or interleaved pairs, all or part of a head
``rope_grad``   the gradient of that
``append``      a step's keys and values put into a paged cache, RMS normed and rotated on the way, with its q heads
``attend``      attention of each sequence's newest tokens over the cache
``verify``      drafted tokens accepted or refused by given random numbers, and the token that follows them

``run`` computes a case in plain torch operations in 32 bits (64 where a border decides), or, where ``own`` is
true, through this package's binding.  ``exact`` computes the same from the definitions in 64 bits.
"""
import math

import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"fp32": 4, "bf16": 2, "e4m3": 1}
EPS = 1e-6
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a 768-wide layer's heads over one sequence of odd length
        {"name": "rope_short", "op": "rope", "rows": 1021, "q_heads": 12, "k_heads": 12, "head_dim": 64, "rotary": 64, "pairs": "half", "amplitude": 1.0},
        # a training batch with grouped heads, half of each head turned, in neighbouring pairs
        {"name": "rope_batch", "op": "rope", "rows": 16384, "q_heads": 32, "k_heads": 8, "head_dim": 128, "rotary": 64, "pairs": "interleaved", "amplitude": 1.0},
        # the backward pass of a long context, its angles' amplitude raised as such models do
        {"name": "rope_grad", "op": "rope_grad", "rows": 8192, "q_heads": 16, "k_heads": 4, "head_dim": 256, "rotary": 256, "pairs": "half", "amplitude": 1.1386},
        # one decoding step of 64 sequences
        {"name": "append_decode", "op": "append", "seqs": 64, "max_new": 1, "q_heads": 16, "k_heads": 4, "head_dim": 256, "rotary": 256, "pairs": "half", "type": "bf16", "page": 16, "order": "head", "normed": True},
        # a batch of prompts of different lengths, packed
        {"name": "append_prompt", "op": "append", "seqs": 24, "max_new": 1021, "q_heads": 32, "k_heads": 8, "head_dim": 128, "rotary": 128, "pairs": "half", "type": "bf16", "page": 16, "order": "token", "normed": False},
        # the same into 8 bits, with normed heads, half of each turned
        {"name": "append_prompt_8bit", "op": "append", "seqs": 24, "max_new": 1021, "q_heads": 16, "k_heads": 4, "head_dim": 256, "rotary": 128, "pairs": "interleaved", "type": "e4m3", "page": 64, "order": "head", "normed": True},
        # one user's step of a 768-wide model: latency
        {"name": "attend_one", "op": "attend", "seqs": 1, "max_len": 1021, "new": 1, "q_heads": 12, "k_heads": 12, "head_dim": 64, "type": "bf16", "page": 16, "order": "token", "window": 0},
        # a batch of sequences of very different lengths
        {"name": "attend_batch", "op": "attend", "seqs": 64, "max_len": 8192, "new": 1, "q_heads": 16, "k_heads": 4, "head_dim": 256, "type": "bf16", "page": 16, "order": "head", "window": 0},
        # a few very long contexts, the cache in 8 bits
        {"name": "attend_long_8bit", "op": "attend", "seqs": 4, "max_len": 131072, "new": 1, "q_heads": 32, "k_heads": 8, "head_dim": 128, "type": "e4m3", "page": 64, "order": "head", "window": 0},
        # a step that checks four drafted tokens of each sequence at once
        {"name": "attend_drafted", "op": "attend", "seqs": 32, "max_len": 4096, "new": 5, "q_heads": 32, "k_heads": 8, "head_dim": 128, "type": "bf16", "page": 16, "order": "token", "window": 0},
        # one user's drafts from a look-up, each drafted for certain, over an odd vocabulary
        {"name": "verify_one", "op": "verify", "seqs": 1, "drafts": 3, "vocab": 32003, "type": "fp32", "scaled": False, "certain": True, "inv_temp": 1.25},
        # a batch whose drafts come from a small model
        {"name": "verify_batch", "op": "verify", "seqs": 64, "drafts": 4, "vocab": 131072, "type": "bf16", "scaled": True, "certain": False, "inv_temp": 1.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope_grad", "append", "append", "attend", "attend", "attend", "verify"])
    if op == "verify":
        return {"op": op, "seqs": _log_int(rng, 1, 32), "drafts": rng.randint(0, 4), "vocab": _log_int(rng, 1000, 131072),
                "type": rng.choice(["fp32", "bf16"]), "scaled": rng.random() < 0.5, "certain": rng.random() < 0.4,
                "inv_temp": rng.choice([1.0, 0.8, 1.5])}
    k_heads = rng.choice([1, 2, 4, 5, 8])
    case = {"op": op, "q_heads": k_heads * rng.choice([1, 2, 4, 7]), "k_heads": k_heads,
            "head_dim": rng.choice([64, 80, 96, 128, 256])}
    if op != "attend":
        case["rotary"] = 16 * rng.randint(1, case["head_dim"] // 16)
        case["pairs"] = rng.choice(["half", "interleaved"])
    if op.startswith("rope"):
        case["rows"] = _log_int(rng, 1, 4096)
        case["amplitude"] = rng.choice([1.0, 1.2])
        return case
    case["type"] = rng.choice(["bf16", "e4m3"])
    case["page"] = rng.choice([1, 16, 32, 64, 128])
    case["order"] = rng.choice(["token", "head"])
    if op == "append":
        case["seqs"], case["max_new"] = _log_int(rng, 1, 32), _log_int(rng, 1, 256)
        case["normed"] = rng.random() < 0.5
        return case
    case["seqs"] = _log_int(rng, 1, 64)
    case["max_len"] = _log_int(rng, 1, min(131072, 2 ** 29 // (case["seqs"] * k_heads * case["head_dim"])))
    case["new"] = rng.choice([1, 1, 2, 5])
    case["window"] = rng.choice([0, 0, 1000])
    return case


# ----------------------------------------------------------------- inputs

BEFORE = 2000                                                      # tokens that a sequence may hold before it is appended to


def _lengths(longest, seqs):
    """Lengths of a batch, from short to the longest."""
    return [max(1, longest * (i + 1) // seqs) for i in range(seqs)]


def _frequencies(rotary):
    return (10000.0 ** (-torch.arange(0, rotary, 2, device="cuda", dtype=torch.float64) / rotary)).float()


def _paged(case, g, pages_of, n_pages, width, normal):
    """A cache that holds earlier tokens everywhere, and a table of `pages_of` pages a sequence, from all over it."""
    heads, hd, page = case["k_heads"], case["head_dim"], case["page"]
    shape = (n_pages, page, heads, hd) if case["order"] == "token" else (n_pages, heads, page, hd)
    s = {}
    for n in "kv":
        t = normal(*shape, dtype=torch.bfloat16).to(TYPES[case["type"]])
        s[n + "_cache"] = t if case["order"] == "token" else t.transpose(1, 2)
        s[n + "_scale"] = torch.rand(heads, device="cuda", generator=g) * 0.5 + 0.75 if case["type"] == "e4m3" else None
    at = torch.arange(width, device="cuda")
    used = at < pages_of.cuda()[:, None]
    order = torch.randperm(n_pages, device="cuda", generator=g, dtype=torch.int32)
    table = torch.full((len(pages_of), width), -1, device="cuda", dtype=torch.int32)
    table[used] = order[:int(pages_of.sum())]
    s["table"] = table
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    op = case["op"]
    s = {"case": dict(case)}

    def normal(*shape, dtype=torch.float32, sd=1.0):
        return torch.randn(*shape, device="cuda", generator=g, dtype=dtype).mul_(sd)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, device="cuda", generator=g) * (hi - lo) + lo

    if op == "verify":
        seqs, drafts, vocab, dtype = case["seqs"], case["drafts"], case["vocab"], TYPES[case["type"]]
        s["scale"] = uniform(vocab, lo=0.8, hi=1.25) if case["scaled"] else None
        target = normal(seqs, drafts + 1, vocab, sd=2.5)
        draft = (target[:, :drafts] + normal(seqs, drafts, vocab, sd=0.6)).to(dtype)   # a smaller model's view
        s["target"] = target.to(dtype).reshape(seqs * (drafts + 1), vocab)
        z = draft.float() * s["scale"] if case["scaled"] else draft.float()
        z = z * case["inv_temp"]
        z -= torch.log(-torch.log(uniform(seqs, drafts, vocab, lo=1e-30)))             # one token drawn from each row
        s["drafted"] = z.argmax(-1) if not case["certain"] else \
            (s["target"].float().reshape(seqs, drafts + 1, vocab)[:, :drafts] + normal(seqs, drafts, vocab, sd=0.3)).argmax(-1)
        s["draft"] = None if case["certain"] else draft.reshape(seqs * drafts, vocab)
        s["u_accept"], s["u_sample"] = uniform(seqs, drafts), uniform(seqs)
        return s

    hd, wq, wk = case["head_dim"], case["q_heads"] * case["head_dim"], case["k_heads"] * case["head_dim"]
    if op.startswith("rope"):
        rows = case["rows"]
        s["inv_freq"] = _frequencies(case["rotary"])
        s["positions"] = torch.randint(0, 200_000, (1,), device="cuda", generator=g, dtype=torch.int32) \
            + torch.arange(rows, device="cuda", dtype=torch.int32)
        qkv = normal(rows, wq + 2 * wk, dtype=torch.bfloat16)      # a fused projection: q | k | v
        s["q"], s["k"] = qkv[:, :wq], qkv[:, wq:wq + wk]
        return s
    seqs = case["seqs"]
    if op == "append":
        page = case["page"]
        new = torch.tensor(_lengths(case["max_new"], seqs))[torch.randperm(seqs, generator=host)]
        before = torch.randint(0, BEFORE, (seqs,), generator=host)  # what each sequence holds already
        most = -(-(BEFORE + new) // page)
        s.update(_paged(case, g, -(-(before + new) // page), int(most.sum()), int(most.max()), normal))
        rows = int(new.sum())
        s["inv_freq"] = _frequencies(case["rotary"])
        s["seqs"] = torch.repeat_interleave(torch.arange(seqs, dtype=torch.int32), new).cuda()
        first = torch.repeat_interleave(before - (new.cumsum(0) - new), new)
        s["positions"] = (first + torch.arange(rows)).int().cuda()
        qkv = normal(rows, wq + 2 * wk, dtype=torch.bfloat16)
        s["q"], s["k"], s["v"] = qkv[:, :wq], qkv[:, wq:wq + wk], qkv[:, wq + wk:]
        s["q_weight"], s["k_weight"] = (uniform(hd, lo=0.5, hi=1.5), uniform(hd, lo=0.5, hi=1.5)) if case["normed"] else (None, None)
        return s
    lens = torch.tensor(_lengths(case["max_len"], seqs))[torch.randperm(seqs, generator=host)]
    pages_of = -(-lens // case["page"])
    s.update(_paged(case, g, pages_of, int(pages_of.sum()) + 3, int(pages_of.max()), normal))
    s["lens"] = lens.int().cuda()
    s["q"] = normal(seqs * case["new"], wq + 2 * wk, dtype=torch.bfloat16, sd=1.5)[:, :wq]
    return s


# ------------------------------------------------------------ plain forms

def _angles(s):
    t = s["positions"].double()[:, None] * s["inv_freq"].double()
    amplitude = s["case"].get("amplitude", 1.0)
    return (torch.cos(t) * amplitude).float()[:, None], (torch.sin(t) * amplitude).float()[:, None]


def _turn(x, c, sn, case):
    """Heads [rows, heads, head_dim], the first `rotary` values of each turned."""
    r = case["rotary"]
    t = x[..., :r]
    if case["pairs"] == "half":
        a, b = t.chunk(2, dim=-1)
        t = torch.cat([a * c - b * sn, b * c + a * sn], dim=-1)
    else:
        a, b = t[..., ::2], t[..., 1::2]
        t = torch.stack([a * c - b * sn, b * c + a * sn], dim=-1).flatten(-2)
    return torch.cat([t, x[..., r:]], dim=-1)


def _heads(x, hd):
    return x.float().reshape(x.shape[0], -1, hd)


def _plain_rope(s):
    case = s["case"]
    c, sn = _angles(s)
    if case["op"] == "rope_grad":
        sn = -sn
    return {n: _turn(_heads(s[n], case["head_dim"]), c, sn, case).bfloat16().reshape(s[n].shape) for n in "qk"}


def _bytes_of(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _plain_append(s):
    case, hd = s["case"], s["case"]["head_dim"]
    c, sn = _angles(s)

    def normed(n):
        x = _heads(s[n], hd)
        if case["normed"]:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s[n + "_weight"]
        return _turn(x, c, sn, case)

    def stored(x, scale):
        if scale is None:
            return x.to(torch.bfloat16)
        return (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)

    pos = s["positions"].long()
    page = s["table"][s["seqs"].long(), pos // case["page"]].long()
    off = pos % case["page"]
    _bytes_of(s["k_cache"])[page, off] = _bytes_of(stored(normed("k"), s["k_scale"]))
    _bytes_of(s["v_cache"])[page, off] = _bytes_of(stored(_heads(s["v"], hd), s["v_scale"]))
    return {"q": normed("q").bfloat16().reshape(s["q"].shape), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attend(s):
    case, hd, new = s["case"], s["case"]["head_dim"], s["case"]["new"]
    seqs, heads, group = case["seqs"], case["k_heads"], case["q_heads"] // case["k_heads"]
    key = torch.arange(case["max_len"], device="cuda")
    page = s["table"].long()[:, key // case["page"]]
    off = key % case["page"]

    def gathered(n):                                               # [seqs, heads, max_len, head_dim]
        t = _bytes_of(s[n + "_cache"])[page.clamp(min=0), off].view(s[n + "_cache"].dtype).float()
        t = t * s[n + "_scale"][:, None] if s[n + "_scale"] is not None else t
        return t.transpose(1, 2)

    q = s["q"].float().reshape(seqs, new, heads, group, hd).permute(0, 2, 4, 1, 3).reshape(seqs, heads, hd, new * group)
    z = torch.matmul(gathered("k"), q) * hd ** -0.5                # [seqs, heads, max_len, new * group]
    last = s["lens"].long()[:, None] - new + torch.arange(new, device="cuda")
    seen = key[:, None] <= last[:, None, :]                        # [seqs, max_len, new]
    if case["window"]:
        seen &= key[:, None] > last[:, None, :] - case["window"]
    z = z.masked_fill_(~seen.repeat_interleave(group, dim=2)[:, None], -math.inf)
    top = z.amax(2, keepdim=True)
    w = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
    total = w.sum(2)
    w = torch.where(total[:, :, None] > 0, w / total[:, :, None], 0.0)
    out = torch.matmul(w.transpose(2, 3).contiguous(), gathered("v"))
    out = out.reshape(seqs, heads, new, group, hd).transpose(1, 2).reshape(seqs * new, -1)
    lse = (top[:, :, 0] + torch.log(total)).reshape(seqs, heads, new, group).transpose(1, 2).reshape(seqs * new, -1)
    return {"out": out.bfloat16(), "lse": lse}


def _probabilities(s, name, rows):
    """exp(z - lse) in 64 bits of the rows [seqs, rows, vocab], and z - lse itself."""
    z = s[name].float()
    if s["scale"] is not None:
        z = z * s["scale"]
    z = (z * s["case"]["inv_temp"]).double().reshape(s["case"]["seqs"], rows, -1)
    z = z - z.amax(-1, keepdim=True)
    e = torch.exp(z)
    total = e.sum(-1, keepdim=True)
    return e / total, z - torch.log(total)


def _plain_verify(s):
    case, ids = s["case"], s["drafted"]
    seqs, drafts = case["seqs"], case["drafts"]
    p, logp = _probabilities(s, "target", drafts + 1)
    if s["draft"] is not None:
        q = _probabilities(s, "draft", drafts)[0]
    else:
        q = torch.zeros_like(p[:, :drafts]).scatter_(2, ids[:, :, None], 1.0)
    pd, qd = p[:, :drafts].gather(2, ids[:, :, None])[..., 0], q.gather(2, ids[:, :, None])[..., 0]
    taken = (s["u_accept"].double() * qd < pd).long().cumprod(1)
    accepted = taken.sum(1)
    at = torch.arange(seqs, device="cuda")
    q = torch.cat([q, torch.zeros_like(p[:, :1])], dim=1)          # nothing was drafted after the last
    w = (p[at, accepted] - q[at, accepted]).clamp(min=0.0)
    past = torch.cumsum(w, -1) > s["u_sample"].double()[:, None] * w.sum(-1, keepdim=True)
    token = past.long().argmax(-1)
    place = torch.arange(drafts + 1, device="cuda")
    tokens = torch.cat([ids, ids.new_zeros(seqs, 1)], dim=1)
    tokens = torch.where(place < accepted[:, None], tokens, torch.where(place == accepted[:, None], token[:, None], -1))
    logp = logp.gather(2, tokens.clamp(min=0)[:, :, None])[..., 0]
    return {"accepted": accepted.int(), "tokens": tokens.int(), "logp": torch.where(tokens >= 0, logp, 0.0).float()}


PLAIN = {"rope": _plain_rope, "rope_grad": _plain_rope, "append": _plain_append, "attend": _plain_attend,
         "verify": _plain_verify}


# ---------------------------------------------------- the framework's own

def _own(s):
    from scale_invariant_row_amd import binding as B
    case = s["case"]
    op = case["op"]
    if op == "rope":
        q, k = B.ds_rope_rows(s["q"], s["k"], s["positions"], s["inv_freq"], case["head_dim"],
                              interleaved=case["pairs"] == "interleaved", amplitude=case["amplitude"])
        return {"q": q, "k": k}
    if op == "rope_grad":
        dq, dk = B.ds_rope_rows_backward(s["q"], s["k"], s["positions"], s["inv_freq"], case["head_dim"],
                                         interleaved=case["pairs"] == "interleaved", amplitude=case["amplitude"])
        return {"q": dq, "k": dk}
    if op == "verify":
        r = B.ds_draft_verify_rows(s["target"], s["drafted"], s["u_accept"], s["u_sample"], draft=s["draft"],
                                   scale=s["scale"], inv_temp=case["inv_temp"], draft_scale=s["scale"],
                                   draft_inv_temp=case["inv_temp"])
        return {"accepted": r.accepted, "tokens": r.tokens, "logp": r.logp}
    if "cache" not in s:                                           # the handle that a program keeps with its cache
        s["cache"] = B.KvCache(s["k_cache"], s["v_cache"], s["table"], s["k_scale"], s["v_scale"])
    cache = s["cache"]
    if op == "append":
        q = B.ds_cache_append_rows(cache, s["k"], s["v"], s["positions"], seqs=s["seqs"], inv_freq=s["inv_freq"],
                                   interleaved=case["pairs"] == "interleaved", q=s["q"],
                                   rms_eps=EPS if case["normed"] else None, q_weight=s["q_weight"], k_weight=s["k_weight"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    out, lse = B.ds_cache_attention_rows(cache, s["q"], s["lens"], window=case["window"], want_lse=True)
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "verify":
        seqs, drafts = case["seqs"], case["drafts"]
        rows = seqs * (drafts + 1) + (0 if case["certain"] else seqs * drafts)
        n = rows * case["vocab"] * SIZE[case["type"]] + (case["vocab"] * 4 if case["scaled"] else 0)
        return {"bytes": n + seqs * drafts * 12 + seqs * 8 + seqs * (drafts + 1) * 8, "flops": rows * case["vocab"] * 6}
    hd, q, k = case["head_dim"], case["q_heads"], case["k_heads"]
    if op.startswith("rope"):
        rows = case["rows"]
        return {"bytes": rows * (q + k) * hd * 4 + rows * 4 + case["rotary"] * 2,
                "flops": rows * (q + k) * case["rotary"] * 3}
    lengths = _lengths(case["max_new"] if op == "append" else case["max_len"], case["seqs"])
    tokens = sum(lengths)
    size = SIZE[case["type"]]
    if op == "append":
        return {"bytes": tokens * hd * (q * 4 + k * (4 + 2 * size)) + tokens * 12, "flops": tokens * (q + k) * hd * 7}
    if case["window"]:
        tokens = sum(min(n, case["window"] + case["new"] - 1) for n in lengths)
    rows = case["seqs"] * case["new"]
    return {"bytes": tokens * k * hd * 2 * size + rows * q * (hd * 4 + 4) + tokens / case["page"] * 4,
            "flops": tokens * case["new"] * q * hd * 4}


# -------------------------------------------- the definitions, in 64 bits

def _turned64(s, n, x, sign):
    """Heads [rows, heads, hd] in 64 bits: each pair a complex number, times its position's."""
    case = s["case"]
    r = case["rotary"]
    theta = sign * s["positions"].double()[:, None] * s["inv_freq"].double()
    turn = torch.polar(torch.full_like(theta, case.get("amplitude", 1.0)), theta)[:, None]
    lead = x[..., :r].reshape(*x.shape[:2], 2, r // 2).transpose(2, 3) if case["pairs"] == "half" \
        else x[..., :r].reshape(*x.shape[:2], r // 2, 2)
    lead = torch.view_as_real(torch.view_as_complex(lead.contiguous()) * turn)
    lead = lead.transpose(2, 3) if case["pairs"] == "half" else lead
    return torch.cat([lead.reshape(*x.shape[:2], r), x[..., r:]], dim=-1)


def _exact_rope(s):
    sign = -1.0 if s["case"]["op"] == "rope_grad" else 1.0
    return {n: _turned64(s, n, s[n].double().unflatten(1, (-1, s["case"]["head_dim"])), sign).flatten(1) for n in "qk"}


def _exact_append(s):
    case, hd = s["case"], s["case"]["head_dim"]
    made = {}
    for n in "qk":
        x = s[n].double().unflatten(1, (-1, hd))
        if case["normed"]:
            x = x / ((x ** 2).sum(2, keepdim=True) / hd + EPS).sqrt() * s[n + "_weight"].double()
        made[n] = _turned64(s, n, x, 1.0)
    made["v"] = s["v"].double().unflatten(1, (-1, hd))
    out = {"q": made["q"].flatten(1)}
    pos, seq, table = s["positions"].tolist(), s["seqs"].tolist(), s["table"].tolist()
    where = torch.tensor([[table[a][p // case["page"]], p % case["page"]] for a, p in zip(seq, pos)], device="cuda")
    for n in "kv":
        t = s[n + "_cache"].double()
        new = made[n]
        if s[n + "_scale"] is not None:
            new = torch.clamp(new / s[n + "_scale"].double()[:, None], -E4M3_MAX, E4M3_MAX)
        t[where[:, 0], where[:, 1]] = new
        out[n + "_cache"] = t
    return out


def _exact_attend(s):
    case, hd, new = s["case"], s["case"]["head_dim"], s["case"]["new"]
    group = case["q_heads"] // case["k_heads"]
    out, lse = [], []
    for a, length in enumerate(s["lens"].tolist()):
        pages = s["table"][a, :-(-length // case["page"])].long()
        kv = []
        for n in "kv":
            t = s[n + "_cache"].view(torch.uint8)[pages].view(s[n + "_cache"].dtype) if case["type"] == "e4m3" else s[n + "_cache"][pages]
            t = t.flatten(0, 1)[:length].double().repeat_interleave(group, dim=1).transpose(0, 1)
            if s[n + "_scale"] is not None:
                t = t * s[n + "_scale"].double().repeat_interleave(group)[:, None, None]
            kv.append(t)
        q = s["q"][a * new:(a + 1) * new].double().reshape(new, -1, hd)
        for j in range(new):
            hi = length - new + j + 1                              # keys below this are seen
            lo = max(0, hi - case["window"]) if case["window"] else 0
            if hi <= lo:
                out.append(torch.zeros(case["q_heads"] * hd, device="cuda", dtype=torch.float64))
                lse.append(torch.full((case["q_heads"],), -math.inf, device="cuda", dtype=torch.float64))
                continue
            z = (kv[0][:, lo:hi] @ q[j][:, :, None])[..., 0] / math.sqrt(hd)
            lse.append(torch.logsumexp(z, -1))
            out.append((torch.softmax(z, -1)[:, None] @ kv[1][:, lo:hi]).flatten())
    return {"out": torch.stack(out), "lse": torch.stack(lse)}


def _exact_verify(s):
    case = s["case"]
    drafts = case["drafts"]

    def log_p(rows):
        z = rows.float() * s["scale"] if s["scale"] is not None else rows.float()
        return torch.log_softmax((z * case["inv_temp"]).double(), -1)

    logp = []
    for a in range(case["seqs"]):
        target = log_p(s["target"][a * (drafts + 1):(a + 1) * (drafts + 1)])
        row, i = torch.zeros(drafts + 1, device="cuda", dtype=torch.float64), 0
        weight = None
        while i < drafts:
            token = int(s["drafted"][a, i])
            q = torch.zeros_like(target[i])
            if s["draft"] is None:
                q[token] = 1.0
            else:
                q = log_p(s["draft"][a * drafts + i:a * drafts + i + 1])[0].exp()
            if not float(s["u_accept"][a, i]) * float(q[token]) < math.exp(float(target[i, token])):
                weight = torch.relu(target[i].exp() - q)
                break
            row[i] = target[i, token]
            i += 1
        weight = target[i].exp() if weight is None else weight
        edge = float(s["u_sample"][a]) * float(weight.sum())
        row[i] = target[i, int(torch.searchsorted(torch.cumsum(weight, 0), edge, right=True))]
        logp.append(row)
    return {"accepted": None, "tokens": None, "logp": torch.stack(logp)}


EXACT = {"rope": _exact_rope, "rope_grad": _exact_rope, "append": _exact_append, "attend": _exact_attend,
         "verify": _exact_verify}


def exact(case, seed):
    s = prepare(case, seed)
    return EXACT[case["op"]](s)
