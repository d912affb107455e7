"""Cases of the operators around the paged KV cache: per-head norm + rotation of q and k, the append of a chunk's
keys and values to the pages, and attention of a chunk of new tokens over the pages.

``run`` computes a case in elementary torch operations where ``own`` is false, and through the library's public
entry points where it is true.  Shapes are the repository's model shapes (head counts 32/8 and 64/8, head_dim 64 and
128, contexts 2048 to 8192, pages of 16 to 128 tokens) and odd ones between them.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ---- cases ---------------------------------------------------------------------------------

def _norm_rope(name, tokens, heads, kv_heads, hd, rot, pairing, typ, far):
    return {"name": name, "op": "norm_rope", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "hd": hd,
            "rot": rot, "pairing": pairing, "in": typ, "out": typ, "norm": True, "far": far}


def _append(name, seqs, q, kv, ragged, heads, kv_heads, hd, page, typ, cache, norm, with_q, pairing, pad):
    return {"name": name, "op": "append", "seqs": seqs, "q": q, "kv": kv, "ragged": ragged, "heads": heads,
            "kv_heads": kv_heads, "hd": hd, "rot": hd, "page": page, "in": typ, "out": cache, "norm": norm,
            "with_q": with_q, "pairing": pairing, "pad": pad}


def _attend(name, seqs, q, kv, ragged, heads, kv_heads, hd, page, cache, window, lse, pad):
    return {"name": name, "op": "attend", "seqs": seqs, "q": q, "kv": kv, "ragged": ragged, "heads": heads,
            "kv_heads": kv_heads, "hd": hd, "page": page, "out": cache, "window": window, "lse": lse, "pad": pad}


def listed():
    return [
        # one decode step of eight branches, 8B shape: launch latency
        _norm_rope("norm-rope-step", 8, 32, 8, 128, 128, "adjacent", "bf16", 8192),
        # a whole prompt, 70B shape, far positions
        _norm_rope("norm-rope-prompt", 8192, 64, 8, 128, 128, "halves", "bf16", 131072),
        # fp32 activations (the type the framework's own projections give), part of the head rotated, odd count
        _norm_rope("norm-rope-f32-odd", 1021, 32, 8, 64, 32, "adjacent", "f32", 8192),
        # one token of each of 64 sequences, fp32 activations into the fp16 cache, q rotated in the same pass
        _append("append-step", 64, 1, 8192, True, 32, 8, 128, 64, "f32", "f16", False, True, "adjacent", 0),
        # the chunks of a prefill batch, packed, with normed q and k
        _append("append-prompt", 8, 1536, 6000, True, 32, 8, 128, 64, "bf16", "bf16", True, True, "halves", 5),
        # keys and values alone, odd chunk, small pages, a head_dim that is no power of two
        _append("append-odd", 5, 211, 700, True, 12, 6, 80, 16, "f16", "f16", False, False, "adjacent", 3),
        # the smallest call: one token over 2048 cached ones, 8B shape
        _attend("attend-one", 1, 1, 2048, False, 32, 8, 128, 64, "f16", 0, False, 0),
        # a serving batch of single tokens over ragged contexts, 70B shape: reads 1.3 GB of cache
        _attend("attend-step", 64, 1, 8192, True, 64, 8, 128, 64, "bf16", 0, False, 0),
        # verify passes: five drafted tokens of each of eight sequences
        _attend("attend-verify", 8, 5, 4101, True, 32, 8, 128, 32, "f16", 0, True, 0),
        # a whole prompt into an empty cache, 8B shape
        _attend("attend-prompt", 1, 8192, 8192, False, 32, 8, 128, 64, "bf16", 0, False, 0),
        # chunks and single tokens in one batch, 1B shape, small pages, a sliding window, padding rows behind
        _attend("attend-mixed", 13, 701, 4099, True, 32, 8, 64, 16, "f16", 1000, True, 7),
        # the last chunk of a long prompt, 70B shape
        _attend("attend-chunk-long", 1, 2048, 32768, False, 64, 8, 128, 128, "bf16", 0, False, 0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    heads, kv_heads = rng.choice([(32, 8), (64, 8), (4, 2), (12, 6), (16, 16), (14, 2), (40, 8), (24, 3), (8, 1)])
    op = rng.choice(["norm_rope", "append", "attend", "attend"])
    pairing = rng.choice(["adjacent", "halves"])
    if op == "norm_rope":
        hd = rng.choice([32, 64, 80, 96, 128, 256])
        c = _norm_rope("", _log(rng, 1, 8192), heads, kv_heads, hd, rng.choice([hd, hd, hd // 2 // 16 * 16]), pairing,
                       rng.choice(["f32", "f16", "bf16"]), rng.choice([4096, 131072, 1 << 22]))
        c["out"], c["norm"] = rng.choice([c["in"], "bf16"]), rng.random() < 0.7
        c["tokens"] = max(1, min(c["tokens"], (8192 * 72 * 128 * 2) // ((heads + kv_heads) * hd * BYTES[c["in"]])))
    else:
        hd = rng.choice([32, 64, 64, 80, 96, 112, 128, 128, 128])
        page, cache, seqs = rng.choice([16, 32, 64, 128, 256]), rng.choice(["f16", "bf16"]), _log(rng, 1, 64)
        q = rng.choice([1, 1, _log(rng, 2, 40), _log(rng, 2, 8192)])
        kv = max(q, _log(rng, 16, 8192))
        pad, ragged = rng.choice([0, 0, 1, 9]), rng.random() < 0.7
        if op == "append":
            c = _append("", seqs, q, kv, ragged, heads, kv_heads, hd, page, rng.choice(["f32", "f16", "bf16"]), cache,
                        rng.random() < 0.5, rng.random() < 0.5, pairing, pad)
            c["seqs"] = max(1, min(seqs, 40960 // kv, 8192 // q))
        else:
            c = _attend("", seqs, q, kv, ragged, heads, kv_heads, hd, page, cache, rng.choice([0, 0, 0, _log(rng, 1, 3000)]),
                        rng.random() < 0.5, pad)
            c["seqs"] = max(1, min(seqs, (1 << 31) // (q * kv * heads), (1 << 29) // (kv * kv_heads * hd)))
    del c["name"]
    return c


def _lengths(case):
    """[(new tokens, cached tokens with the new ones)] of each sequence: from the case alone."""
    n, q, kv = case["seqs"], case["q"], case["kv"]
    if not case["ragged"]:
        return [(q, kv)] * n
    r = random.Random(1000003 * n + 8191 * q + kv)
    got = [(q, kv)]  # one sequence has the full lengths
    for _ in range(n - 1):
        a = 1 if q > 1 and r.random() < 0.3 else r.randint((q + 1) // 2, q)
        got.append((a, max(a, r.randint((kv + 3) // 4, kv))))
    r.shuffle(got)
    return got


def _span(case, ql, kl):
    """Attended (query, key) pairs of a sequence, and the keys that at least one query attends."""
    base, w = kl - ql, case["window"]
    first = max(0, base - w + 1) if w else 0
    if not w:
        return ql * base + ql * (ql + 1) // 2, kl
    return sum(min(base + i + 1, w) for i in range(ql)), kl - first


def work(case):
    hd, heads, kv_heads = case["hd"], case["heads"], case["kv_heads"]
    if case["op"] == "norm_rope":
        n = case["tokens"] * (heads + kv_heads) * hd
        return {"bytes": n * (BYTES[case["in"]] + BYTES[case["out"]]), "flops": 6 * n}
    lengths = _lengths(case)
    if case["op"] == "append":
        n = sum(a for a, _ in lengths) * (2 * kv_heads + (heads if case["with_q"] else 0)) * hd
        return {"bytes": n * (BYTES[case["in"]] + BYTES[case["out"]]), "flops": 6 * n}
    spans = [_span(case, a, b) for a, b in lengths]
    rows = sum(a for a, _ in lengths) * heads
    return {"bytes": 2 * (2 * sum(k for _, k in spans) * kv_heads * hd + 2 * rows * hd) + (4 * rows if case["lse"] else 0),
            "flops": 4 * hd * heads * sum(p for p, _ in spans)}


# ---- inputs --------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, typ="f32", std=1.0):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(TYPES[typ])

    hd, heads, kv_heads = case["hd"], case["heads"], case["kv_heads"]
    s = {"case": case, "scale": 1.0 / math.sqrt(hd), "eps": 1e-5}
    if case["op"] != "attend":
        rot = case["rot"]
        inv = torch.arange(0, rot, 2, dtype=torch.float64).div_(max(rot, 1)).mul_(-math.log(500000.0)).exp_()
        s["inv_freq"] = inv.numpy()          # host, what the entry points take
        s["inv_freq_dev"] = inv.cuda()
        s["q_norm"] = normal(hd, std=0.1).add_(1.0) if case["norm"] else None
        s["k_norm"] = normal(hd, std=0.1).add_(1.0) if case["norm"] else None
    if case["op"] == "norm_rope":
        n = case["tokens"]
        qk = normal(n, heads + kv_heads, hd, typ=case["in"], std=1.5)   # one projection's output: q and k are views
        s["q"], s["k"] = qk[:, :heads], qk[:, heads:]
        s["positions"] = torch.randint(0, case["far"], (n,), generator=g, device="cuda", dtype=torch.int32)
        s["q_out"] = torch.zeros(n, heads, hd, device="cuda", dtype=TYPES[case["out"]])
        s["k_out"] = torch.zeros(n, kv_heads, hd, device="cuda", dtype=TYPES[case["out"]])
        return s
    lengths = _lengths(case)
    page = case["page"]
    counts = [-(-kl // page) for _, kl in lengths]
    n_pages = sum(counts) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lengths), max(counts), dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    starts = [0]
    for ql, _ in lengths:
        starts.append(starts[-1] + ql)
    rows = starts[-1] + case["pad"]           # rows behind the last sequence: padding of the batch
    s["page_table"] = table
    s["cu_q"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["kv_len"] = torch.tensor([kl for _, kl in lengths], dtype=torch.int32, device="cuda")
    s["max_q"], s["max_kv"] = max(a for a, _ in lengths), max(b for _, b in lengths)
    s["k_pages"] = normal(n_pages, kv_heads, page, hd, typ=case["out"])
    s["v_pages"] = normal(n_pages, kv_heads, page, hd, typ=case["out"])
    if case["op"] == "append":
        qkv = normal(rows, heads + 2 * kv_heads, hd, typ=case["in"], std=1.5)  # one projection's output
        s["q"] = qkv[:, :heads] if case["with_q"] else None
        s["k"], s["v"] = qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
        s["q_out"] = torch.zeros(rows, heads, hd, device="cuda", dtype=TYPES[case["out"]]) if case["with_q"] else None
    else:
        s["q"] = normal(rows, heads, hd, typ=case["out"], std=2.0)
        s["o"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(rows, heads, device="cuda") if case["lse"] else None
        if own:
            from decode_llama_step_gb300 import dls

            s["workspace"] = torch.zeros(dls.attention_chunk_workspace_bytes(hd), dtype=torch.uint8, device="cuda")
    return s


# ---- one pass ------------------------------------------------------------------------------

def _rotated(x, norm, eps, positions, inv_freq, pairing, typ):
    """x [n, heads, hd] normed per head (where norm is given) and rotated by positions [n], rounded once."""
    x = x.float()
    if norm is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * norm
    rot = 2 * inv_freq.numel()
    angle = positions.double()[:, None, None] * inv_freq       # 64 bits: far positions
    c, d = torch.cos(angle).float(), torch.sin(angle).float()
    y = x.clone()
    if pairing == "adjacent":
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * d, a * d + b * c
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * d, a * d + b * c
    return y.to(typ)


def _place(s, rows):
    """Sequence and index inside its chunk of rows 0..rows-1."""
    t = torch.arange(rows, device="cuda")
    b = torch.searchsorted(s["cu_q"][1:].contiguous(), t.to(torch.int32), right=True)
    return b, t - s["cu_q"].long()[b]


def _plain_append(s):
    case = s["case"]
    rows = s["k"].shape[0] - case["pad"]
    b, i = _place(s, rows)
    pos = (s["kv_len"][b] - s["cu_q"][b + 1] + s["cu_q"][b]).long() + i
    page = s["page_table"].long()[b, pos // case["page"]]
    typ = TYPES[case["out"]]
    s["k_pages"][page, :, pos % case["page"]] = _rotated(s["k"][:rows], s["k_norm"], s["eps"], pos, s["inv_freq_dev"],
                                                        case["pairing"], typ)
    s["v_pages"][page, :, pos % case["page"]] = s["v"][:rows].to(typ)
    if case["with_q"]:
        s["q_out"][:rows] = _rotated(s["q"][:rows], s["q_norm"], s["eps"], pos, s["inv_freq_dev"], case["pairing"], typ)
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "q_out": s["q_out"]}


def _plain_attend(s):
    case = s["case"]
    n, hd, kv_heads = case["seqs"], case["hd"], case["kv_heads"]
    group, mq, mk = case["heads"] // kv_heads, s["max_q"], s["max_kv"]
    rows = s["q"].shape[0] - case["pad"]
    table = s["page_table"].long()
    k, v = (s[x][table].permute(0, 2, 1, 3, 4).reshape(n, kv_heads, -1, hd)[:, :, :mk].float() for x in ("k_pages", "v_pages"))
    i, key = torch.arange(mq, device="cuda"), torch.arange(mk, device="cuda")
    row = (s["cu_q"].long()[:-1, None] + i).clamp_(max=rows - 1)
    q = s["q"][row].float().reshape(n, mq, kv_heads, group, hd).permute(0, 2, 3, 1, 4).reshape(n, kv_heads, group * mq, hd)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).reshape(n, kv_heads, group, mq, mk)
    at = (s["kv_len"] - s["cu_q"][1:] + s["cu_q"][:-1]).long()[:, None] + i          # position of each query
    hidden = key > at[..., None]
    if case["window"]:
        hidden |= key <= at[..., None] - case["window"]
    x.masked_fill_(hidden[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp_(min=-3e38)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(n, kv_heads, group * mq, mk), v).reshape(n, kv_heads, group, mq, hd) / total.clamp(min=1e-37)
    lse = (m + total.log())[..., 0]
    b, j = _place(s, rows)
    s["o"][:rows] = o.permute(0, 3, 1, 2, 4)[b, j].reshape(rows, -1, hd).to(s["o"].dtype)
    if case["lse"]:
        s["lse"][:rows] = lse.permute(0, 3, 1, 2)[b, j].reshape(rows, -1)
    return {"o": s["o"], "lse": s["lse"]}


def run(s):
    case = s["case"]
    if own:
        from decode_llama_step_gb300 import dls

        if case["op"] == "norm_rope":
            dls.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_out"], s["k_out"], q_norm=s["q_norm"],
                             k_norm=s["k_norm"], eps=s["eps"], pairing=case["pairing"])
            return {"q": s["q_out"], "k": s["k_out"]}
        if case["op"] == "append":
            dls.kv_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["page_table"], s["cu_q"], s["kv_len"],
                          s["inv_freq"], q=s["q"], q_out=s["q_out"], q_norm=s["q_norm"] if case["with_q"] else None,
                          k_norm=s["k_norm"], eps=s["eps"], pairing=case["pairing"])
            return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "q_out": s["q_out"]}
        dls.attention_chunk(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["cu_q"], s["kv_len"], s["o"],
                            s["workspace"], lse=s["lse"], scale=s["scale"], causal=True, window=case["window"])
        return {"o": s["o"], "lse": s["lse"]}
    if case["op"] == "norm_rope":
        typ = TYPES[case["out"]]
        return {"q": _rotated(s["q"], s["q_norm"], s["eps"], s["positions"], s["inv_freq_dev"], case["pairing"], typ),
                "k": _rotated(s["k"], s["k_norm"], s["eps"], s["positions"], s["inv_freq_dev"], case["pairing"], typ)}
    return _plain_append(s) if case["op"] == "append" else _plain_attend(s)


# ---- the definition in 64 bits ---------------------------------------------------------------

def _turned(x, norm, eps, positions, case):
    """Definition of norm and rotation: each pair as a complex number times exp(i pos theta^(-2 j / rot))."""
    x = x.double()
    if norm is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + eps).sqrt() * norm.double()
    rot = case["rot"]
    if not rot:
        return x
    j = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    turn = torch.exp(1j * positions.double()[:, None] * torch.exp(-math.log(500000.0) * 2 * j / rot))[:, None]
    head, tail = x[..., :rot], x[..., rot:]
    if case["pairing"] == "adjacent":
        z = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous()) * turn
        return torch.cat([torch.view_as_real(z).reshape(head.shape), tail], -1)
    z = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * turn
    return torch.cat([z.real, z.imag, tail], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return {"q": _turned(s["q"], s["q_norm"], s["eps"], s["positions"], case),
                "k": _turned(s["k"], s["k_norm"], s["eps"], s["positions"], case)}
    lengths, page, start = _lengths(case), case["page"], 0
    if case["op"] == "append":
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        qo = s["q_out"].double() if case["with_q"] else None
        for b, (ql, kl) in enumerate(lengths):
            pos = torch.arange(kl - ql, kl, device="cuda")
            where, slot, r = s["page_table"][b].long()[pos // page], pos % page, slice(start, start + ql)
            kp[where, :, slot] = _turned(s["k"][r], s["k_norm"], s["eps"], pos, case)
            vp[where, :, slot] = s["v"][r].double()
            if qo is not None:
                qo[r] = _turned(s["q"][r], s["q_norm"], s["eps"], pos, case)
            start += ql
        return {"k_pages": kp, "v_pages": vp, "q_out": qo}
    o, group = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64), case["heads"] // case["kv_heads"]
    lse = torch.zeros(s["q"].shape[:2], device="cuda", dtype=torch.float64)
    for b, (ql, kl) in enumerate(lengths):
        key, pos = torch.arange(kl, device="cuda"), torch.arange(kl - ql, kl, device="cuda")[:, None]
        seen = key <= pos
        if case["window"]:
            seen &= pos - key < case["window"]
        where = s["page_table"][b].long()[key // page]
        k, v = s["k_pages"][where, :, key % page].double(), s["v_pages"][where, :, key % page].double()
        for h in range(case["heads"]):
            x = s["q"][start:start + ql, h].double() @ k[:, h // group].T / math.sqrt(case["hd"])
            x = torch.where(seen, x, -math.inf)
            lse[start:start + ql, h] = torch.logsumexp(x, -1)
            o[start:start + ql, h] = torch.exp(x - lse[start:start + ql, h, None]) @ v[:, h // group]
        start += ql
    return {"o": o, "lse": lse if case["lse"] else None}
