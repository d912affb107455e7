"""Cases of a serving step over a paged cache held in 8 bits: pages reserved and rows laid out from request lengths, the
append that quantises keys and values into their blocks, attention over the 8-bit pages, and the verification of drafted
tokens against the target's probabilities.

``run`` computes a case in elementary torch operations where ``own`` is false, and through the library's public
entry points where it is true.  Shapes are the repository's model shapes (head counts 32/8 and 64/8, head_dim 64 and
128, vocabularies of 1024 and 128256, contexts 2048 to 8192, pages of 16 to 128 tokens) and odd ones between them.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CODES = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ---- cases ---------------------------------------------------------------------------------

def _reserve(name, seqs, new, kv, page, ended, short, pad):
    """ended: one sequence in twenty is over; short: the free pages do not suffice for all."""
    return {"name": name, "op": "reserve", "seqs": seqs, "new": new, "kv": kv, "page": page, "ended": ended, "short": short,
            "pad": pad}


def _append(name, seqs, q, kv, ragged, kv_heads, hd, page, block, typ, code, norm, pairing, pad):
    return {"name": name, "op": "append", "seqs": seqs, "q": q, "kv": kv, "ragged": ragged, "kv_heads": kv_heads, "hd": hd,
            "rot": hd, "page": page, "block": block, "in": typ, "code": code, "norm": norm, "pairing": pairing, "pad": pad}


def _attend(name, seqs, q, kv, ragged, heads, kv_heads, hd, page, block, typ, code, window, lse, pad):
    return {"name": name, "op": "attend", "seqs": seqs, "q": q, "kv": kv, "ragged": ragged, "heads": heads,
            "kv_heads": kv_heads, "hd": hd, "page": page, "block": block, "in": typ, "code": code, "window": window,
            "lse": lse, "pad": pad}


def _verify(name, seqs, q, ragged, vocab, typ, drawn, pad):
    """drawn: the drafts were drawn from probabilities, which are given; else they are the draft's greedy picks."""
    return {"name": name, "op": "verify", "seqs": seqs, "q": q, "ragged": ragged, "vocab": vocab, "in": typ, "drawn": drawn,
            "pad": pad}


def listed():
    return [
        # one decode step of 64 sequences: launch latency, a page or none a sequence
        _reserve("reserve-step", 64, 1, 8192, 64, True, False, 0),
        # the prompts of 211 requests admitted at once onto small pages, more than the free pages hold
        _reserve("reserve-prompts", 211, 2048, 1000, 16, True, True, 9),
        # one token of each of 64 sequences, 70B shape: blocks of a whole page grow now and then
        _append("append8-step", 64, 1, 8192, True, 8, 128, 64, 64, "bf16", "e4m3", False, "adjacent", 0),
        # the chunks of a prefill batch, normed keys, blocks finer than pages
        _append("append8-prompt", 8, 1536, 6000, True, 8, 128, 64, 32, "bf16", "e4m3", True, "halves", 5),
        # whole-number codes, odd chunk, small pages, fp32 projections, a head_dim that is no power of two
        _append("append8-odd", 5, 211, 700, True, 6, 80, 16, 16, "f32", "i8", False, "adjacent", 3),
        # the smallest call: one token over 2048 cached ones, 8B shape
        _attend("attend8-one", 1, 1, 2048, False, 32, 8, 128, 64, 64, "f16", "e4m3", 0, False, 0),
        # a serving batch of single tokens over ragged contexts, 70B shape: reads 0.7 GB of cache
        _attend("attend8-step", 64, 1, 8192, True, 64, 8, 128, 64, 64, "bf16", "e4m3", 0, False, 0),
        # verify passes (five rows of each of eight sequences), 1B shape, whole-number codes, a window
        _attend("attend8-verify", 8, 5, 4101, True, 32, 8, 64, 32, 16, "f16", "i8", 2000, True, 3),
        # the last chunk of a long prompt, 8B shape
        _attend("attend8-chunk", 1, 2048, 16384, False, 32, 8, 128, 128, 128, "bf16", "e4m3", 0, False, 0),
        # a single request: four drafted tokens, probabilities of both models
        _verify("verify-one", 1, 5, False, 128256, "f32", True, 0),
        # a serving batch with zero to six drafted tokens each
        _verify("verify-step", 64, 7, True, 128256, "f32", True, 0),
        # greedy drafts (the framework's own kind), 16-bit probabilities, odd vocabulary, padding rows behind
        _verify("verify-greedy", 29, 9, True, 50021, "bf16", False, 2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["reserve", "append", "attend", "attend", "verify"])
    pad, ragged = rng.choice([0, 0, 1, 9]), rng.random() < 0.7
    if op == "reserve":
        seqs = _log(rng, 1, 4096)
        c = _reserve("", seqs, rng.choice([1, _log(rng, 2, 16), _log(rng, 16, 4096)]), _log(rng, 1, 8192),
                     rng.choice([16, 32, 64, 128, 256]), rng.random() < 0.5, rng.random() < 0.3, pad)
        c["new"] = max(1, min(c["new"], 400000 // seqs))
    elif op == "verify":
        seqs, vocab, typ = _log(rng, 1, 128), rng.choice([1024, 128256, _log(rng, 5, 200000)]), rng.choice(["f32", "f16", "bf16"])
        c = _verify("", seqs, _log(rng, 1, 16), ragged, vocab, typ, rng.random() < 0.6, pad)
        c["q"] = max(1, min(c["q"], 64000000 // (seqs * vocab)))
        c["seqs"] = max(1, min(seqs, 64000000 // (c["q"] * vocab)))
    else:
        heads, kv_heads = rng.choice([(32, 8), (64, 8), (4, 2), (12, 6), (16, 16), (14, 2), (40, 8), (24, 3), (8, 1)])
        hd, page = rng.choice([32, 64, 64, 80, 96, 112, 128, 128, 128]), rng.choice([16, 32, 64, 128, 256])
        block = rng.choice([b for b in (16, 32, 64, 128, 256) if b <= page])
        seqs, q = _log(rng, 1, 64), rng.choice([1, 1, _log(rng, 2, 40), _log(rng, 2, 4096)])
        kv, code = max(q, _log(rng, 16, 8192)), rng.choice(["e4m3", "e4m3", "i8"])
        if op == "append":
            c = _append("", seqs, q, kv, ragged, kv_heads, hd, page, block, rng.choice(["f32", "f16", "bf16"]), code,
                        rng.random() < 0.5, rng.choice(["adjacent", "halves"]), pad)
            c["seqs"] = max(1, min(seqs, 40960 // kv, 8192 // q))
        else:
            c = _attend("", seqs, q, kv, ragged, heads, kv_heads, hd, page, block, rng.choice(["f16", "bf16"]), code,
                        rng.choice([0, 0, 0, _log(rng, 1, 3000)]), rng.random() < 0.5, pad)
            c["seqs"] = max(1, min(seqs, (1 << 30) // (q * kv * heads), (1 << 29) // (kv * kv_heads * hd)))
    del c["name"]
    return c


def _lengths(case):
    """[(new tokens, cached tokens with the new ones)] of each sequence: from the case alone."""
    n, q, kv = case["seqs"], case["q"], case.get("kv", 1 << 20)
    if not case["ragged"]:
        return [(q, kv)] * n
    r = random.Random(1000003 * n + 8191 * q + kv)
    got = [(q, kv)]  # one sequence has the full lengths
    for _ in range(n - 1):
        a = 1 if q > 1 and r.random() < 0.3 else r.randint((q + 1) // 2, q)
        got.append((a, max(a, r.randint((kv + 3) // 4, kv))))
    r.shuffle(got)
    return got


def _requests(case):
    """[(new tokens, cached tokens before, pages held)]; new -1: the request is over."""
    n, new, kv, page = case["seqs"], case["new"], case["kv"], case["page"]
    r = random.Random(1000003 * n + 8191 * new + kv)
    got = [(new, kv - 1, -(-(kv - 1) // page))]
    for _ in range(n - 1):
        a = -1 if case["ended"] and r.random() < 0.05 else 0 if r.random() < 0.03 else r.randint((new + 1) // 2, new)
        b = r.randint(0, kv)
        # one in eight still holds a page of a rejected draft
        got.append((a, b, -(-b // page) + (r.random() < 0.125)))
    r.shuffle(got)
    return got


def _pool(case):
    """(pages of the pool, pages on the free stack, entries of a table row)."""
    req, page = _requests(case), case["page"]
    held = sum(h for _, _, h in req)
    need = sum(max(0, -(-(b + a) // page) - h) for a, b, h in req if a > 0)
    free = need * 2 // 3 if case["short"] else need + 5
    return held + max(free, 1) + 2, free, max(-(-(b + max(a, 0)) // page) + 2 for a, b, _ in req)


def _span(case, ql, kl):
    """Attended (query, key) pairs of a sequence, and the keys that at least one query attends."""
    base, w = kl - ql, case["window"]
    first = max(0, base - w + 1) if w else 0
    if not w:
        return ql * base + ql * (ql + 1) // 2, kl
    return sum(min(base + i + 1, w) for i in range(ql)), kl - first


def work(case):
    if case["op"] == "reserve":
        req, page = _requests(case), case["page"]
        rows = sum(max(a, 0) for a, _, _ in req)
        if case["short"]:
            rows = rows * 2 // 3
        pages = rows // page + sum(h for a, _, h in req if a < 0)
        return {"bytes": 12 * rows + 24 * len(req) + 8 * pages + 16, "flops": 4 * rows}
    lengths = _lengths(case)
    rows = sum(a for a, _ in lengths)
    if case["op"] == "verify":
        n, size = case["seqs"], BYTES[case["in"]]
        per = case["vocab"] * size * (2 if case["drawn"] else 1)
        return {"bytes": n * per + rows * (16 + 2 * size) + 16 * n, "flops": 3 * n * case["vocab"]}
    kv_heads, hd, block = case["kv_heads"], case["hd"], case["block"]
    if case["op"] == "append":
        n = 2 * rows * kv_heads * hd
        blocks = sum(-(-b // block) - (b - a) // block for a, b in lengths)
        return {"bytes": n * (BYTES[case["in"]] + 1) + blocks * 8 * kv_heads, "flops": 8 * n}
    spans = [_span(case, a, b) for a, b in lengths]
    keys = sum(k for _, k in spans)
    return {"bytes": 2 * keys * kv_heads * hd + 8 * kv_heads * (keys // block) + 4 * rows * case["heads"] * hd
            + (4 * rows * case["heads"] if case["lse"] else 0),
            "flops": 4 * hd * case["heads"] * sum(p for p, _ in spans)}


# ---- inputs --------------------------------------------------------------------------------

def _paged(case, lengths, g):
    """Page table and batch rows of sequences with the given lengths, pages in random order."""
    page = case["page"]
    counts = [-(-kl // page) for _, kl in lengths]
    n_pages = sum(counts) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lengths), max(counts), dtype=torch.int32, device="cuda")
    at, starts = 0, [0]
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
        starts.append(starts[-1] + lengths[b][0])
    return {"page_table": table, "n_pages": n_pages, "cu_q": torch.tensor(starts, dtype=torch.int32, device="cuda"),
            "kv_len": torch.tensor([kl for _, kl in lengths], dtype=torch.int32, device="cuda"),
            "max_q": max(a for a, _ in lengths), "max_kv": max(b for _, b in lengths), "rows": starts[-1] + case["pad"]}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, typ="f32", std=1.0):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(TYPES[typ])

    s = {"case": case}
    if case["op"] == "reserve":
        req = _requests(case)
        n_pages, free, most = _pool(case)
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        held = torch.tensor([h for _, _, h in req], dtype=torch.int32, device="cuda")
        at = held.cumsum(0) - held
        j = torch.arange(most, device="cuda")
        s["page_table"] = torch.where(j < held[:, None], order[(at[:, None] + j).clamp_(max=n_pages - 1)], -1).to(torch.int32)
        s["held"], s["held_out"] = held, torch.zeros_like(held)
        s["new_len"] = torch.tensor([a for a, _, _ in req], dtype=torch.int32, device="cuda")
        s["kv_len"] = torch.tensor([b for _, b, _ in req], dtype=torch.int32, device="cuda")
        s["kv_len_out"] = torch.zeros_like(held)
        s["free_pages"] = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        s["free_pages"][:free] = order[int(held.sum()):][:free]
        s["free_count"] = torch.tensor([free], dtype=torch.int32, device="cuda")
        s["free_count_out"] = torch.zeros_like(s["free_count"])
        s["cu_q"] = torch.zeros(len(req) + 1, dtype=torch.int32, device="cuda")
        rows = sum(max(a, 0) for a, _, _ in req) + case["pad"]
        for name in ("positions", "slots", "seq_ids"):
            s[name] = torch.zeros(rows, dtype=torch.int32, device="cuda")
        return s
    lengths = _lengths(case)
    if case["op"] == "verify":
        vocab, rows = case["vocab"], sum(a for a, _ in lengths) + case["pad"]
        logits = normal(rows, vocab, std=2.5)
        s["target"] = torch.softmax(logits, -1).to(TYPES[case["in"]])
        p = torch.softmax(logits.add_(normal(rows, vocab, std=0.6)), -1)     # a draft that is near its target
        s["draft"] = p.to(TYPES[case["in"]]) if case["drawn"] else None
        picked = torch.multinomial(p, 1, generator=g)[:, 0] if case["drawn"] else p.argmax(-1)
        starts = [0]
        for a, _ in lengths:
            starts.append(starts[-1] + a)
        s["cu_q"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        s["tokens"] = torch.cat([picked[-1:], picked[:-1]]).to(torch.int32)  # a row's distribution gave the next row's token
        s["kv_len"] = torch.randint(50, 8192, (len(lengths),), generator=g, device="cuda", dtype=torch.int32)
        s["kv_len_out"] = torch.zeros_like(s["kv_len"])
        s["accept"] = torch.rand(rows, generator=g, device="cuda")
        s["pick"] = torch.rand(len(lengths), generator=g, device="cuda")
        s["out_tokens"] = torch.zeros(rows, dtype=torch.int32, device="cuda")
        s["n_accepted"] = torch.zeros(len(lengths), dtype=torch.int32, device="cuda")
        return s
    s.update(_paged(case, lengths, g))
    kv_heads, hd, page, block = case["kv_heads"], case["hd"], case["page"], case["block"]
    s["scale"], s["eps"] = 1.0 / math.sqrt(hd), 1e-5
    grid = (s["n_pages"], kv_heads, page // block)
    for name in ("k", "v"):
        x = torch.randn(s["n_pages"], kv_heads, page, hd, generator=g, device="cuda", dtype=torch.bfloat16)
        if case["code"] == "i8":  # codes near their whole range, as the largest value of a block sets the scale
            s[name + "_pages"] = x.mul_(30).round_().clamp_(-127, 127).to(torch.int8)
            size = 1 / 30
        else:
            s[name + "_pages"] = x.mul_(100).clamp_(-448, 448).to(torch.float8_e4m3fn)
            size = 1 / 100
        del x
        if case["op"] == "append":  # what appends leave: powers of two
            size = torch.exp2(torch.randint(-8, -4, grid, generator=g, device="cuda").float())
        else:                       # any scales
            size = size * torch.exp2(torch.rand(grid, generator=g, device="cuda").mul_(2).sub_(1))
        s[name + "_scales"] = size
    if case["op"] == "append":
        rot, rows = case["rot"], s["rows"]
        inv = torch.arange(0, rot, 2, dtype=torch.float64).div_(rot).mul_(-math.log(500000.0)).exp_()
        s["inv_freq"], s["inv_freq_dev"] = inv.numpy(), inv.cuda()   # host: what the entry points take
        s["k_norm"] = normal(hd, std=0.1).add_(1.0) if case["norm"] else None
        kv = normal(rows, 2 * kv_heads, hd, typ=case["in"], std=1.5)  # one projection's output: k and v are views
        s["k"], s["v"] = kv[:, :kv_heads], kv[:, kv_heads:]
        return s
    heads = case["heads"]
    s["q"] = normal(s["rows"], heads, hd, typ=case["in"], std=2.0)
    s["o"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(s["rows"], heads, device="cuda") if case["lse"] else None
    if own:
        from decode_llama_step_gb300 import dls

        s["workspace"] = torch.zeros(dls.attention_chunk_workspace_bytes(hd), dtype=torch.uint8, device="cuda")
    return s


# ---- one pass ------------------------------------------------------------------------------

def _place(s, rows):
    """Sequence and index inside its chunk of rows 0..rows-1."""
    t = torch.arange(rows, device="cuda")
    b = torch.searchsorted(s["cu_q"][1:].contiguous(), t.to(torch.int32), right=True)
    return b, t - s["cu_q"].long()[b]


def _plain_reserve(s):
    page, most = s["case"]["page"], s["page_table"].shape[1]
    new, kv, held = s["new_len"].long(), s["kv_len"].long(), s["held"].long()
    table, stack = s["page_table"], s["free_pages"]
    # ended sequences give their pages back
    give = torch.where(new < 0, held, 0)
    at = s["free_count"].long() + give.cumsum(0) - give
    j = torch.arange(most, device="cuda")
    back = (j < give[:, None])
    stack[(at[:, None] + j)[back]] = table[back]
    avail = s["free_count"].long() + give.sum()
    # pages, in the order of the sequences while they last
    fits = (new > 0) & (kv + new <= most * page)
    need = torch.where(fits, ((kv + new + page - 1) // page - held).clamp(min=0), 0)
    fits &= (need == 0) | (need.cumsum(0) <= avail)
    # rows, while they last; who gets none takes no pages
    rows = s["positions"].shape[0]
    q = torch.where(fits, new, 0)
    q = torch.where(q.cumsum(0) <= rows, q, 0)
    need = torch.where(q > 0, need, 0)
    i = j - held[:, None]
    fresh = (i >= 0) & (i < need[:, None])
    table[fresh] = stack[(avail - 1 - (need.cumsum(0) - need)[:, None] - i)[fresh]]
    s["cu_q"][1:] = q.cumsum(0)
    s["kv_len_out"].copy_(torch.where(new < 0, 0, kv + q))
    s["held_out"].copy_(torch.where(new < 0, 0, held + need))
    s["free_count_out"].copy_(avail - need.sum())
    t = torch.arange(rows, device="cuda")
    b = torch.searchsorted(s["cu_q"][1:].contiguous(), t.to(torch.int32), right=True).clamp_(max=new.numel() - 1)
    pos = kv[b] + t - s["cu_q"].long()[b]
    slot = table.long()[b, (pos // page).clamp(max=most - 1)] * page + pos % page
    live = t < s["cu_q"][-1]
    for name, x in (("positions", pos), ("slots", slot), ("seq_ids", b)):
        s[name].copy_(torch.where(live, x, s[name].long()))


def _turned_plain(s, pos):
    """The keys normed and rotated."""
    case, x = s["case"], s["k"][:pos.numel()].float()
    if s["k_norm"] is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * s["k_norm"]
    angle = pos.double()[:, None, None] * s["inv_freq_dev"]       # 64 bits: far positions
    c, d = torch.cos(angle).float(), torch.sin(angle).float()
    y, rot = x.clone(), case["rot"]
    if case["pairing"] == "adjacent":
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * d, a * d + b * c
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * d, a * d + b * c
    return y


def _coded(x, code):
    """x, already divided by its scale, to the nearest code (a tie to the even one)."""
    return x.round().clamp(-127, 127).to(torch.int8) if code == "i8" else x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _append_plain_one(s, x, pages, scales, blk, off, pos):
    """Rows x [rows, heads, hd] into block `blk` [rows] (numbered through the pool) at token `off` of it."""
    case, n, heads, hd = s["case"], pos.numel(), x.shape[1], x.shape[2]
    block, per, top = case["block"], case["page"] // case["block"], 127.0 if case["code"] == "i8" else 448.0
    where = blk // per * heads * per + blk % per                                       # of head 0, in scales
    unit = where[:, None] + torch.arange(heads, device="cuda") * per                  # [rows, heads]
    total = scales.numel()
    amax = torch.zeros(total, device="cuda").scatter_reduce_(0, unit.reshape(-1), x.abs().amax(-1).reshape(-1), "amax")
    part, exponent = torch.frexp(amax)
    top_part, top_exponent = math.frexp(top)
    need = torch.exp2((exponent - top_exponent + (part > top_part).int()).clamp(-64, 64).double()).float()
    need = torch.where(amax > 0, need, 2.0 ** -64)
    # tokens of the block that were there before: as many as the first new one's place
    before = torch.full((total,), block, device="cuda", dtype=torch.int64)
    before.scatter_reduce_(0, unit.reshape(-1), off[:, None].expand(n, heads).reshape(-1), "amin")
    touched = torch.zeros(total, device="cuda", dtype=torch.bool)
    touched[unit.reshape(-1)] = True
    old = scales.reshape(-1)
    fresh = torch.where(before > 0, torch.maximum(old, need), need)
    flat = pages.view(torch.uint8).reshape(total, block, hd)
    grown = (touched & (before > 0) & (fresh > old)).nonzero()[:, 0]
    if grown.numel():
        codes = flat[grown].view(CODES[case["code"]]).float() * (old / fresh)[grown, None, None]
        keep = torch.arange(block, device="cuda")[:, None] < before[grown, None, None]
        flat[grown] = torch.where(keep, _coded(codes, case["code"]).view(torch.uint8), flat[grown])
    flat[unit.reshape(-1), off[:, None].expand(n, heads).reshape(-1)] = \
        _coded(x / fresh[unit][..., None], case["code"]).view(torch.uint8).reshape(n * heads, hd)
    scales.copy_(torch.where(touched, fresh, old).reshape(scales.shape))


def _plain_append(s):
    case = s["case"]
    page, block = case["page"], case["block"]
    b, i = _place(s, s["k"].shape[0] - case["pad"])
    pos = (s["kv_len"][b] - s["cu_q"][b + 1] + s["cu_q"][b]).long() + i
    blk = s["page_table"].long()[b, pos // page] * (page // block) + pos % page // block
    _append_plain_one(s, _turned_plain(s, pos), s["k_pages"], s["k_scales"], blk, pos % block, pos)
    _append_plain_one(s, s["v"][:pos.numel()].float(), s["v_pages"], s["v_scales"], blk, pos % block, pos)


def _plain_attend(s):
    case = s["case"]
    n, hd, kv_heads, block = case["seqs"], case["hd"], case["kv_heads"], case["block"]
    group, mq, mk = case["heads"] // kv_heads, s["max_q"], s["max_kv"]
    rows = s["q"].shape[0] - case["pad"]
    table = s["page_table"].long()

    def cached(x):
        at = s[x + "_pages"].view(torch.uint8)[table].view(CODES[case["code"]]).float()
        at = at.reshape(*at.shape[:3], -1, block, hd) * s[x + "_scales"][table][..., None, None]
        return at.reshape(n, -1, kv_heads, case["page"], hd).permute(0, 2, 1, 3, 4).reshape(n, kv_heads, -1, hd)[:, :, :mk]

    k, v = cached("k"), cached("v")
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


def _plain_verify(s):
    case, cu, tokens = s["case"], s["cu_q"].long(), s["tokens"].long()
    n, rows = case["seqs"], s["tokens"].shape[0] - case["pad"]
    b, i = _place(s, rows)
    t = torch.arange(rows, device="cuda")
    last = cu[b + 1] - 1
    x = tokens[(t + 1).clamp(max=rows - 1)]
    p = s["target"][t, x].double()
    q = s["draft"][t, x].double() if case["drawn"] else torch.ones_like(p)
    stands = (s["accept"][:rows].double() * q < p) & (t < last)
    stop = torch.minimum(cu[1:] - 1, torch.full((n,), rows, device="cuda").scatter_reduce(0, b, torch.where(stands, rows, t), "amin"))
    rest = s["target"][stop].double()
    w = rest
    refused = (stop < cu[1:] - 1)[:, None]
    if case["drawn"]:
        w = torch.where(refused, (rest - s["draft"][stop].double()).clamp(min=0), rest)
    else:
        mine = torch.arange(case["vocab"], device="cuda") == tokens[(stop + 1).clamp(max=rows - 1)][:, None]
        w = torch.where(refused & mine, 0.0, rest)
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, rest)
    c = w.cumsum(-1)
    pick = (c <= s["pick"].double()[:, None] * c[:, -1:]).sum(-1)
    out = torch.where(t < stop[b], x, torch.where(t == stop[b], pick[b], -1))
    s["out_tokens"][:rows] = out
    s["n_accepted"].copy_(stop - cu[:-1])
    s["kv_len_out"].copy_(s["kv_len"] - (cu[1:] - 1 - stop))


def run(s):
    case = s["case"]
    if own:
        from decode_llama_step_gb300 import dls

        if case["op"] == "reserve":
            dls.kv_reserve(s["new_len"], s["kv_len"], s["held"], s["page_table"], s["free_pages"], s["free_count"],
                           s["kv_len_out"], s["held_out"], s["free_count_out"], s["cu_q"], case["page"],
                           positions=s["positions"], slots=s["slots"], seq_ids=s["seq_ids"])
        elif case["op"] == "append":
            dls.kv_append8(s["k"], s["v"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["page_table"],
                           s["cu_q"], s["kv_len"], s["inv_freq"], k_norm=s["k_norm"], eps=s["eps"], pairing=case["pairing"])
        elif case["op"] == "attend":
            dls.attention_chunk8(s["q"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["page_table"],
                                 s["cu_q"], s["kv_len"], s["o"], s["workspace"], lse=s["lse"], scale=s["scale"],
                                 causal=True, window=case["window"])
        else:
            dls.verify_draft(s["tokens"], s["target"], s["cu_q"], s["accept"], s["pick"], s["out_tokens"],
                             s["n_accepted"], draft=s["draft"], kv_len=s["kv_len"], kv_len_out=s["kv_len_out"])
    else:
        {"reserve": _plain_reserve, "append": _plain_append, "attend": _plain_attend, "verify": _plain_verify}[case["op"]](s)
    if case["op"] == "reserve":
        return {x: s[x] for x in ("page_table", "free_pages", "kv_len_out", "held_out", "free_count_out", "cu_q", "positions",
                                  "slots", "seq_ids")}
    if case["op"] == "append":
        # e4m3 codes are values as they are; whole-number ones become such
        pages = {x: s[x] if case["code"] == "e4m3" else s[x].to(torch.float16) for x in ("k_pages", "v_pages")}
        return {**pages, "k_scales": s["k_scales"], "v_scales": s["v_scales"]}
    if case["op"] == "attend":
        return {"o": s["o"], "lse": s["lse"]}
    return {x: s[x] for x in ("out_tokens", "n_accepted", "kv_len_out")}


# ---- the definition in 64 bits ---------------------------------------------------------------

def _turned(x, norm, eps, positions, case):
    """Definition of norm and rotation: each pair as a complex number times exp(i pos theta^(-2 j / rot))."""
    x = x.double()
    if norm is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + eps).sqrt() * norm.double()
    rot = case["rot"]
    j = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    turn = torch.exp(1j * positions.double()[:, None] * torch.exp(-math.log(500000.0) * 2 * j / rot))[:, None]
    if case["pairing"] == "adjacent":
        z = torch.view_as_complex(x.reshape(*x.shape[:-1], rot // 2, 2).contiguous()) * turn
        return torch.view_as_real(z).reshape(x.shape)
    z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:].contiguous()) * turn
    return torch.cat([z.real, z.imag], -1)


def _nearest(x, code):
    """The value of the code nearest to x, from the formats' definition: whole numbers up to 127; four bits of mantissa
    (one hidden) down to steps of 2^-9, up to 448."""
    if code == "i8":
        return torch.round(x).clamp(-127, 127)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_append(s):
    case, out = s["case"], {}
    page, block, top = case["page"], case["block"], 127 if case["code"] == "i8" else 448
    for name in ("k", "v"):
        pages = s[name + "_pages"].double()
        scales = s[name + "_scales"].double()
        start = 0
        for b, (ql, kl) in enumerate(_lengths(case)):
            pos = torch.arange(kl - ql, kl, device="cuda")
            x = s[name][start:start + ql].double()
            if name == "k":
                x = _turned(x, s["k_norm"], s["eps"], pos, case)
            start += ql
            first = (kl - ql) // block
            # rows by block: [blocks, block, heads, hd], nothing where no row is
            n = (kl - 1) // block + 1 - first
            rows = torch.zeros(n * block, *x.shape[1:], device="cuda", dtype=torch.float64)
            rows[pos - first * block] = x
            rows = rows.reshape(n, block, *x.shape[1:]).transpose(1, 2)                     # [blocks, heads, block, hd]
            at = torch.arange(first, first + n, device="cuda") * block
            where, part = s["page_table"][b].long()[at // page], at % page // block
            # (a logarithm a little over a whole number is that number's: 7 = 448 / 64)
            need = torch.exp2(torch.ceil(torch.log2(rows.abs().amax((-1, -2)) / top) - 1e-12).clamp(-64, 64))
            old = scales[where, :, part]
            kept = (at[0] + torch.arange(n * block, device="cuda").reshape(n, 1, block, 1)) < kl - ql
            got = torch.where(kept.any(2)[..., 0], torch.maximum(old, need), need)
            slots = torch.arange(block, device="cuda") + (at % page)[:, None]
            cells = (where[:, None, None], torch.arange(x.shape[1], device="cuda")[:, None], slots[:, None, :])
            new = (at[0] + torch.arange(n * block, device="cuda").reshape(n, 1, block, 1)) < kl
            now = pages[cells]
            mine = _nearest(torch.where(kept, now * (old / got)[..., None, None], rows / got[..., None, None]), case["code"])
            pages[cells] = torch.where(new, mine, now)
            scales[where, :, part] = got
        out[name + "_pages"], out[name + "_scales"] = pages, scales
    return out


def exact(case, seed):
    if case["op"] in ("reserve", "verify"):   # whole numbers
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    page, block, start = case["page"], case["block"], 0
    o, group = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64), case["heads"] // case["kv_heads"]
    lse = torch.zeros(s["q"].shape[:2], device="cuda", dtype=torch.float64)
    for b, (ql, kl) in enumerate(_lengths(case)):
        key, pos = torch.arange(kl, device="cuda"), torch.arange(kl - ql, kl, device="cuda")[:, None]
        seen = key <= pos
        if case["window"]:
            seen &= pos - key < case["window"]
        where, slot = s["page_table"][b].long()[key // page], key % page
        k, v = (s[x + "_pages"].view(torch.uint8)[where, :, slot].view(CODES[case["code"]]).double()
                * s[x + "_scales"][where, :, slot // block].double()[..., None] for x in ("k", "v"))
        for h in range(case["heads"]):
            x = s["q"][start:start + ql, h].double() @ k[:, h // group].T / math.sqrt(case["hd"])
            x = torch.where(seen, x, -math.inf)
            lse[start:start + ql, h] = torch.logsumexp(x, -1)
            o[start:start + ql, h] = torch.exp(x - lse[start:start + ql, h, None]) @ v[:, h // group]
        start += ql
    return {"o": o, "lse": lse if case["lse"] else None}
