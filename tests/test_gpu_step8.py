"""The calls around the 8-bit paged cache on the GPU, against plain implementations (whole numbers exactly, the others in
64 bits) at the sizes, masks and layouts where they can go wrong, and a run of them together."""
import math
import random
from fractions import Fraction

import numpy as np
import pytest
import torch

from decode_llama_step_gb300 import dls

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -24  # half a step of fp32, relative
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CODES = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}
I32 = torch.int32


def ints(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def half_step(t):
    return torch.finfo(t).eps / 2


def rounding(want, t):
    """Half a step of type t at `want`: relative, and the fixed step below the normal range."""
    return half_step(t) * want.abs() + torch.finfo(t).tiny * half_step(t)


# ---- pages and rows from lengths -----------------------------------------------------------------

def reserve_plain(new, kv, held, table, stack, count, page, max_rows):
    """The call's definition, one sequence after another; also the bits of its status word."""
    n, most, pages = len(new), len(table[0]) if table else 0, len(stack)
    table, stack, status = [list(r) for r in table], list(stack), 0
    room = most * page
    top = min(max(count, 0), pages)
    if top != count:
        status |= 4
    bad = [not (0 <= kv[b] <= room and 0 <= held[b] <= most and held[b] * page >= kv[b]) for b in range(n)]
    for b in range(n):
        if new[b] < 0 and not bad[b]:
            for j in range(held[b]):
                if top < pages:
                    stack[top] = table[b][j]
                    top += 1
                else:
                    status |= 4
    kv_out, held_out, cu, rows = [], [], [0], []
    dry = full = False
    for b in range(n):
        far = new[b] > 0 and kv[b] + new[b] > room
        if bad[b] or far:
            status |= 4
        q = 0
        fresh = 0
        if new[b] > 0 and not bad[b] and not far:
            fresh = max(0, -(-(kv[b] + new[b]) // page) - held[b])
            q = new[b]
            if fresh and (dry or fresh > top - taken(held_out, held, new)):
                dry, q, fresh = True, 0, 0
                status |= 16
            elif full or cu[-1] + q > max_rows:
                full, q, fresh = True, 0, 0
                status |= 16
        used = taken(held_out, held, new)
        for j in range(fresh):
            table[b][held[b] + j] = stack[top - 1 - used - j]
        for i in range(q):
            pos = kv[b] + i
            p = table[b][pos // page]
            ok = 0 <= p < pages
            if not ok:
                status |= 1
            rows.append((pos, p * page + pos % page if ok else -1, b))
        cu.append(cu[-1] + q)
        kv_out.append(0 if new[b] < 0 else kv[b] + q)
        held_out.append(0 if new[b] < 0 else held[b] + fresh)
    return dict(table=table, stack=stack, kv=kv_out, held=held_out, cu=cu, count=top - taken(held_out, held, new), rows=rows, status=status)


def taken(held_out, held, new):
    return sum(o - h for o, h, a in zip(held_out, held, new) if a >= 0)


class Requests:
    """A state of n sequences: pages in random order, table entries beyond the held ones poisoned."""

    def __init__(self, n, page, seed, kv=300, spare=0, most=None):
        r = random.Random(seed)
        self.kv = [r.choice([0, 1, page - 1, page, page + 1, r.randint(0, kv)]) for _ in range(n)]
        self.held = [-(-k // page) + r.choice([0, 0, 0, 1, 2]) for k in self.kv]
        self.most = most or max(self.held + [1]) + 8
        pages = sum(self.held) + spare + 3
        order = list(range(pages))
        r.shuffle(order)
        self.table, at = [], 0
        for h in self.held:
            self.table.append(order[at:at + h] + [-5] * (self.most - h))
            at += h
        free = order[at:]
        self.count = min(len(free), spare)
        self.stack = free[:self.count] + [-9] * (pages - self.count)
        self.page, self.r = page, r

    def run(self, new, max_rows, pad=0, alias=False, arrays=True, stream=None, skew=0):
        want = reserve_plain(new, self.kv, self.held, self.table, self.stack, self.count, self.page, max_rows)
        n = len(new)
        kv, held, count = ints(self.kv), ints(self.held), ints([self.count])
        out = (kv, held, count) if alias else (torch.full_like(kv, 77), torch.full_like(held, 77), torch.full_like(count, 77))
        table, stack = ints(self.table).reshape(n, self.most), ints(self.stack)
        cu = torch.full((n + 1,), 77, dtype=I32, device="cuda")
        status = ints([99])
        # skew: the arrays begin between two 16-byte boundaries
        got = [torch.full((max_rows + pad + skew,), 77, dtype=I32, device="cuda")[skew:] for _ in range(3)] if arrays else [None] * 3
        dls.kv_reserve(ints(new), kv, held, table, stack, count, *out, cu, self.page, positions=got[0], slots=got[1],
                       seq_ids=got[2], max_rows=max_rows, status=status, stream=stream)
        torch.cuda.synchronize()
        assert cu.tolist() == want["cu"]
        assert out[0].tolist() == want["kv"] and out[1].tolist() == want["held"] and out[2].tolist() == [want["count"]]
        assert table.tolist() == want["table"]
        assert stack.tolist() == want["stack"]
        if arrays:
            assert status.item() == want["status"], (status.item(), want["status"])
            rows = want["rows"]
            for k in range(3):
                assert got[k].tolist() == [x[k] for x in rows] + [77] * (max_rows + pad - len(rows))
        return want


@pytest.mark.parametrize("n,page", [(1, 16), (2, 256), (31, 64), (33, 16), (300, 32), (1023, 64), (1025, 128), (4096, 16)])
def test_reserve_single_tokens(gpu_lib, n, page):
    r = Requests(n, page, n, spare=n)
    r.run([1] * n, n)
    r.run([random.Random(b).choice([1, 1, 1, 0, -1]) for b in range(n)], n, pad=5, alias=True)


@pytest.mark.parametrize("n,page,rows", [(1, 16, 1), (1, 64, 5000), (5, 32, 700), (64, 16, 300), (211, 16, 90), (7, 256, 20000), (13, 64, 20000)])
def test_reserve_prompts(gpu_lib, n, page, rows):
    r = Requests(n, page, 7 * n + rows, spare=n * (rows // page + 2), most=rows // page + 30)
    new = [r.r.choice([rows, rows // 2 + 1, 1, 0]) for _ in range(n)]
    new[0] = rows
    want = r.run(new, sum(new), pad=3)
    assert want["status"] == 0 and want["cu"][-1] == sum(new)


@pytest.mark.parametrize("seed", range(12))
def test_reserve_when_pages_or_rows_run_out(gpu_lib, seed):
    """Requests of every kind, a stack that does not suffice, room for part of the rows."""
    n = [3, 17, 40, 128, 600, 1500][seed % 6]
    r = Requests(n, 16, 100 + seed, spare=n // 2)
    new = [r.r.choice([0, 1, 1, 2, 15, 16, 17, 40, -1, -3]) for _ in range(n)]
    total = sum(a for a in new if a > 0)
    r.run(new, total)
    r.run(new, max(1, total // 3), pad=2)
    r.run(new, 0)
    r.run(new, total, alias=True)
    r.run(new, total, arrays=False)
    r.run(new, total, skew=1, stream=torch.cuda.current_stream())


def test_reserve_states_that_cannot_be(gpu_lib):
    r = Requests(40, 16, 3, spare=60)
    new = [3] * 40
    r.kv[2], r.kv[5], r.held[7], r.held[9], r.kv[11] = -1, 16 * r.most + 1, -2, r.most + 1, r.kv[11] + 16 * r.held[11] + 1
    new[12] = 16 * r.most                       # past the table
    new[5], new[9], new[20] = -1, -1, -1        # over, two of them with a state that cannot be
    want = r.run(new, 4000)
    assert want["status"] & 4 and want["held"][9] == 0
    r.count = len(r.stack) + 4                  # a count that cannot be
    r.run(new, 4000)
    r.count = -3
    r.run(new, 4000)
    # more pages come back than the stack has room for
    r = Requests(10, 16, 4, spare=20)
    r.count = len(r.stack) - 1
    r.stack = list(range(len(r.stack)))
    r.run([-1] * 9 + [5], 100)


def test_reserve_names_no_page_outside_the_pool(gpu_lib):
    r = Requests(6, 16, 5, spare=30)
    r.table[1][:1], r.table[3][:1], r.stack[r.count - 2] = [1 << 30], [-1], 12345
    r.held[1], r.kv[1], r.held[3], r.kv[3] = max(r.held[1], 1), 3, max(r.held[3], 1), 2
    want = r.run([5, 5, 40, 5, 5, 0], 60)
    assert want["status"] == 1 and any(x[1] == -1 for x in want["rows"])


def test_reserve_without_sequences(gpu_lib):
    z, count, cu = torch.zeros(0, dtype=I32, device="cuda"), ints([4]), ints([9])
    out, status = ints([7]), ints([5])
    dls.kv_reserve(z, z, z, torch.zeros(0, 3, dtype=I32, device="cuda"), ints([1, 2, 3, 4, 0]), count, z, z, out, cu, 16, max_rows=0, status=status)
    assert (cu.item(), out.item(), status.item()) == (0, 4, 0)


def test_reserve_step_after_step_in_one_graph(gpu_lib):
    """A captured call whose outputs are its next inputs, replayed as the lengths grow, requests end and new ones come."""
    n, page = 37, 16
    r = Requests(n, page, 9, spare=400, most=60)
    kv, held, count, table, stack = ints(r.kv), ints(r.held), ints([r.count]), ints(r.table), ints(r.stack)
    new, cu, pos, slots, ids = ints([0] * n), ints([0] * (n + 1)), *(torch.full((600,), 77, dtype=I32, device="cuda") for _ in range(3))
    stream, gr = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=stream):
        dls.kv_reserve(new, kv, held, table, stack, count, kv, held, count, cu, page, positions=pos, slots=slots, seq_ids=ids,
                       stream=torch.cuda.current_stream())
    for step in range(40):
        asked = [r.r.choice([1, 1, 1, 1, 4, 0, 30, -1] if step % 5 == 0 else [1, 1, 4]) for _ in range(n)]
        want = reserve_plain(asked, r.kv, r.held, r.table, r.stack, r.count, page, 600)
        new.copy_(ints(asked))
        for t in (pos, slots, ids):
            t.fill_(77)
        gr.replay()
        torch.cuda.synchronize()
        r.kv, r.held, r.table, r.stack, r.count = want["kv"], want["held"], want["table"], want["stack"], want["count"]
        assert cu.tolist() == want["cu"] and kv.tolist() == r.kv and held.tolist() == r.held and count.item() == r.count
        assert table.tolist() == r.table and stack.tolist() == r.stack
        assert [pos.tolist(), slots.tolist(), ids.tolist()] == [[x[k] for x in want["rows"]] + [77] * (600 - len(want["rows"])) for k in range(3)]
    used = [p for b in range(n) for p in r.table[b][:r.held[b]]] + r.stack[:r.count]
    assert len(set(used)) == len(used)  # no page twice


# ---- a paged batch in 8 bits -----------------------------------------------------------------------

class Batch8:
    """Ragged lengths [(new, cached with the new)], pages in random order, all that no call may use poisoned: NaN codes
    (e4m3) and NaN scales."""

    def __init__(self, lengths, kvh, hd, page, block, code, seed, first=0, pad=0, spare=2, extra=1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g, self.lengths, self.page, self.block, self.code, self.kvh, self.hd = g, lengths, page, block, code, kvh, hd
        counts = [-(-kl // page) for _, kl in lengths]
        self.n_pages = sum(counts) + spare
        order = torch.randperm(self.n_pages, generator=g, device="cuda").tolist()
        self.max_pages = max(counts + [1]) + extra
        table = torch.full((len(lengths), self.max_pages), -1, dtype=I32)
        table[:, -1] = 1 << 30
        at, starts = 0, [first]
        for b, c in enumerate(counts):
            table[b, :c] = torch.tensor(order[at:at + c], dtype=I32)
            at += c
            starts.append(starts[-1] + lengths[b][0])
        self.starts, self.rows, self.table = starts, starts[-1] + pad, table.cuda()
        self.cu_q, self.kv_len = ints(starts), ints([kl for _, kl in lengths])
        shape = (self.n_pages, kvh, page, hd)
        self.k, self.v = (torch.full(shape, 127, dtype=torch.uint8, device="cuda").view(CODES[code]) for _ in range(2))
        self.ks, self.vs = (torch.full((self.n_pages, kvh, page // block), math.nan, device="cuda") for _ in range(2))

    def slots(self, b, lo, hi):
        pos = torch.arange(lo, hi, device="cuda")
        return self.table[b].long()[pos // self.page], pos % self.page

    def some_codes(self, n):
        x = torch.randn(n, self.kvh, self.hd, generator=self.g, device="cuda")
        return (x * 30).round().clamp(-128, 127).to(torch.int8) if self.code == "i8" else (x * 100).clamp(-448, 448).to(CODES["e4m3"])

    def fill(self, upto=None, powers=False):
        """Codes of tokens 0 .. and scales of their blocks (any, or powers of two)."""
        unit = 1 / 30 if self.code == "i8" else 1 / 100
        for b, (ql, kl) in enumerate(self.lengths):
            n = kl if upto is None else min(kl, max(0, upto[b]))
            p, s = self.slots(b, 0, n)
            for pool, scales in ((self.k, self.ks), (self.v, self.vs)):
                pool.view(torch.uint8)[p, :, s] = self.some_codes(n).view(torch.uint8)
                size = torch.rand(n, self.kvh, generator=self.g, device="cuda") * 3 - 1.5
                size = 2.0 ** (-6 + size.round()) if powers else unit * 2.0 ** size
                scales[p, :, s // self.block] = size[torch.arange(n, device="cuda") // self.block * self.block]

    def values(self, b, n, which):
        """Values of tokens 0 .. n - 1, in 64 bits: [n, heads, hd]."""
        p, s = self.slots(b, 0, n)
        pool, scales = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        return pool.view(torch.uint8)[p, :, s].view(CODES[self.code]).double() * scales[p, :, s // self.block].double()[..., None]


# ---- append ---------------------------------------------------------------------------------------

def turned(x, norm, eps, pos, freq, halves):
    """(value, length of the element's pair) of normed and rotated heads, in 64 bits."""
    x = x.double()
    if norm is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * norm.double()
    y, size = x.clone(), x.abs()
    n = 0 if freq is None else len(freq)
    if n:
        f = pos.double()[:, None, None] * torch.as_tensor(freq, device=x.device)
        ia = torch.arange(n, device=x.device) if halves else torch.arange(0, 2 * n, 2, device=x.device)
        ib = ia + (n if halves else 1)
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * f.cos() - b * f.sin(), a * f.sin() + b * f.cos()
        size[..., ia] = size[..., ib] = (a * a + b * b).sqrt()
    return y, size


def code_step(x, code):
    """Half the distance of neighbouring codes around x (in units of the scale)."""
    if code == "i8":
        return torch.full_like(x, 0.5)
    return torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))) * 2.0 ** -4


def nearest(x, code):
    if code == "i8":
        return torch.round(x).clamp(-127, 127)
    step = 2 * code_step(x, code)
    return (torch.round(x / step) * step).clamp(-448, 448)


def scale_of(amax, code):
    top = 127 if code == "i8" else 448
    e = torch.ceil(torch.log2(amax.double() / top) - 1e-12)
    return torch.exp2(torch.where(amax > 0, e, -64.0).clamp(-64, 64))


def check_append(lengths, kvh, hd, rot, page, block, tin, code, norm, pairing, first=0, pad=0, std=1.5, seed=11, stream=None):
    B = Batch8(lengths, kvh, hd, page, block, code, seed, first, pad)
    B.fill(upto=[kl - ql for ql, kl in lengths], powers=True)
    x = (torch.randn(B.rows, 2 * kvh + 1, hd, generator=B.g, device="cuda") * std).to(TYPES[tin])
    inside = torch.zeros(B.rows, dtype=torch.bool, device="cuda")
    inside[first:B.starts[-1]] = True
    x[~inside] = math.nan
    k, v = x[:, :kvh], x[:, kvh:2 * kvh]
    wk = torch.randn(hd, generator=B.g, device="cuda") if norm else None
    freq = dls.rope_inv_freq(rot, 500000.0) if rot else None
    before = [t.clone() for t in (B.k, B.v, B.ks, B.vs)]
    status = ints([99])
    torch.cuda.synchronize()
    dls.kv_append8(k, v, B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len, freq, k_norm=wk, eps=1e-6, pairing=pairing,
                   status=status, stream=stream)
    dls.attention_status(status, stream)
    codes_done = torch.zeros(B.n_pages, page, dtype=torch.bool, device="cuda")
    scales_done = torch.zeros(B.n_pages, page // block, dtype=torch.bool, device="cuda")
    for b, (ql, kl) in enumerate(lengths):
        if not ql:
            continue
        r, pos = slice(B.starts[b], B.starts[b] + ql), torch.arange(kl - ql, kl, device="cuda")
        lo = (kl - ql) // block * block                      # the first block's first token
        far = 0.0 if freq is None else kl * float(np.abs(freq).max()) * 2.0 ** -51
        for which, src, pool, scales, old_pool, old_scales in (("k", k, B.k, B.ks, before[0], before[2]), ("v", v, B.v, B.vs, before[1], before[3])):
            want, size = turned(src[r], wk, 1e-6, pos, freq, pairing == "halves") if which == "k" else (src[r].double(), src[r].double().abs() * 0)
            # the fp32 steps of norm and rotation (as in the 16-bit append's test); V is exact
            off = (32 * F32 + far) * size
            blk = pos // block - lo // block
            n_blk = int(blk[-1]) + 1
            most = torch.zeros(n_blk, kvh, dtype=torch.float64, device="cuda")
            most.scatter_reduce_(0, blk[:, None].expand(ql, kvh), want.abs().amax(-1), "amax")
            slack = torch.zeros_like(most).scatter_reduce_(0, blk[:, None].expand(ql, kvh), off.amax(-1), "amax")
            at = lo + torch.arange(n_blk, device="cuda") * block
            p, part = B.table[b].long()[at // page], at % page // block
            got = scales[p, :, part].double()
            had = old_scales[p, :, part].double()
            grown_from = (torch.arange(n_blk, device="cuda") == 0)[:, None] & torch.tensor(lo < kl - ql, device="cuda")
            low, high = scale_of(most - slack, code), scale_of(most + slack, code)
            low, high = (torch.where(grown_from, torch.maximum(had, t), t) for t in (low, high))
            assert bool(((got == low) | (got == high)).all()), which
            # new rows: half a step, and what came before it
            pp, ss = B.slots(b, kl - ql, kl)
            mine = pool.view(torch.uint8)[pp, :, ss].view(CODES[code]).double()
            sc = got[blk][..., None]
            top = 127.0 if code == "i8" else 448.0
            lim = code_step((want.abs() + off) / sc, code) * sc * (1 + 2.0 ** -20) + off
            # (the largest value may round down to the top code when its scale is the smaller of the two)
            err = (mine * sc - want).abs()
            assert bool((err <= lim).all()), (which, float((err / lim).max()))
            assert bool((mine.abs() <= top).all())
            if float(off.abs().max()) == 0:
                assert torch.equal(mine, nearest(want / sc, code))
            # earlier codes of the first block, rescaled
            if lo < kl - ql:
                op, os_ = B.slots(b, lo, kl - ql)
                was = old_pool.view(torch.uint8)[op, :, os_].view(CODES[code]).double()
                f = (had[0] / got[0])[None, :, None]
                expect = torch.where(f < 1, nearest(was * f, code), was)
                assert torch.equal(pool.view(torch.uint8)[op, :, os_].view(CODES[code]).double(), expect), which
                codes_done[op, os_] = True
            codes_done[pp, ss] = True
            scales_done[p, part] = True
    for now, was in ((B.k, before[0]), (B.v, before[1])):  # no other slot of any page
        left = ~codes_done[:, None, :, None].expand_as(now)
        assert torch.equal(now.view(torch.uint8)[left], was.view(torch.uint8)[left])
    for now, was in ((B.ks, before[2]), (B.vs, before[3])):
        left = ~scales_done[:, None, :].expand_as(now)
        assert torch.equal(now.view(I32)[left], was.view(I32)[left])
    return B


@pytest.mark.parametrize("lengths,kvh,hd,rot,page,block,tin,code,norm,pairing,first,pad", [
    ([(1, 1)], 2, 64, 64, 64, 64, "f32", "e4m3", False, "adjacent", 0, 0),
    ([(1, 17), (1, 16), (1, 1)], 8, 128, 128, 16, 16, "bf16", "e4m3", True, "adjacent", 0, 1),
    ([(16, 16), (0, 9), (15, 40), (33, 33)], 3, 80, 80, 32, 16, "f16", "i8", False, "halves", 2, 5),
    ([(5, 300), (257, 257), (64, 128)], 2, 128, 64, 64, 32, "bf16", "e4m3", True, "halves", 0, 3),
    ([(3, 2000)] * 40 + [(0, 0)] * 3 + [(7, 1025)] * 30, 1, 96, 96, 32, 32, "bf16", "i8", False, "adjacent", 1, 2),
    ([(1, 5 + b % 90) for b in range(1100)], 1, 16, 16, 64, 64, "f32", "e4m3", False, "adjacent", 0, 0),
    ([(700, 1700)], 2, 256, 0, 256, 256, "f16", "i8", True, "halves", 0, 0),
    ([(700, 1700), (1, 300), (40, 41)], 3, 128, 128, 256, 128, "f32", "e4m3", True, "adjacent", 0, 0),
    ([(31, 1000), (1, 1), (9, 77), (8, 64), (65, 65)], 5, 48, 32, 128, 64, "bf16", "i8", True, "adjacent", 3, 40),
    ([(1, 60)] * 63 + [(2048, 2048)], 2, 64, 64, 64, 64, "bf16", "e4m3", False, "halves", 0, 0),
    # blocks whose angles are too many to be held
    ([(300, 700), (1, 5), (256, 256)], 1, 256, 256, 256, 256, "bf16", "e4m3", True, "halves", 0, 0),
    ([(700, 1700), (2, 900)], 2, 128, 128, 256, 256, "f16", "i8", True, "adjacent", 1, 1),
])
def test_append8(gpu_lib, lengths, kvh, hd, rot, page, block, tin, code, norm, pairing, first, pad):
    check_append(lengths, kvh, hd, rot, page, block, tin, code, norm, pairing, first, pad)


@pytest.mark.parametrize("code", ["e4m3", "i8"])
@pytest.mark.parametrize("std", [1e-30, 1e-19, 1e-3, 30.0, 1e18, 1e25])
def test_append8_sizes_of_values(gpu_lib, code, std):
    """Values from below the smallest scale to above the largest: a scale of 2^-64 or 2^64 then, codes 0 or the top one."""
    if std >= 1e25:
        k = torch.full((3, 2, 64), std, device="cuda")
        k[1] *= -1
        B = Batch8([(3, 3)], 2, 64, 16, 16, code, 3)
        dls.kv_append8(k, k, B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len, None)
        p, s = B.slots(0, 0, 3)
        top = 127.0 if code == "i8" else 448.0
        for pool, sc in ((B.k, B.ks), (B.v, B.vs)):
            got = pool.view(torch.uint8)[p, :, s].view(CODES[code]).float()
            assert torch.equal(got, torch.sign(k) * top)
            assert bool((sc[p, :, 0] == 2.0 ** 64).all())
        return
    check_append([(5, 40), (40, 40), (1, 1)], 2, 64, 64, 32, 16, "f32", code, False, "halves", std=std)


@pytest.mark.parametrize("code", ["e4m3", "i8"])
def test_append8_zeros_nan_and_infinity(gpu_lib, code):
    B = Batch8([(4, 4), (40, 40)], 2, 64, 16, 16, code, 3)
    x = torch.randn(44, 2, 64, generator=B.g, device="cuda")
    x[:4] = 0.0
    x[4 + 3, 0, 7], x[4 + 20, 1, 9], x[4 + 21, 1, 9] = math.nan, math.inf, -math.inf
    dls.kv_append8(x, x, B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len, None)
    top = 127.0 if code == "i8" else 448.0
    for pool, sc in ((B.k, B.ks), (B.v, B.vs)):
        p, s = B.slots(0, 0, 4)
        assert bool((sc[p, :, 0] == 2.0 ** -64).all()) and not bool(pool.view(torch.uint8)[p, :, s].any())
        p, s = B.slots(1, 0, 40)
        got = pool.view(torch.uint8)[p, :, s].view(CODES[code]).float()
        rest = x[4:20, 0].clone()
        rest[3, 7] = 0.0
        want = scale_of(rest.abs().max(), code)
        assert float(sc[p[0], 0, 0]) == float(want)          # NaN does not count
        assert got[3, 0, 7].item() == 0 if code == "i8" else math.isnan(got[3, 0, 7].item())
        assert float(sc[p[20], 1, 0]) == 2.0 ** 64 and got[20, 1, 9].item() == top and got[21, 1, 9].item() == -top


@pytest.mark.parametrize("code,block,page,hd", [("e4m3", 64, 64, 128), ("i8", 64, 64, 64), ("e4m3", 16, 32, 80), ("i8", 256, 256, 128)])
def test_append8_token_by_token(gpu_lib, code, block, page, hd):
    """A block filled one token at a time, each larger than the last: the scale ends where appending all at once puts it, and a
    value is off by its own half step and, of whole numbers, the half steps of every growth: a step of the last scale."""
    n, kvh = block + 5, 2
    B = Batch8([(1, n)], kvh, hd, page, block, code, 5)
    x = torch.randn(n, kvh, hd, generator=B.g, device="cuda") * torch.exp2(torch.linspace(-3, 3, n, device="cuda"))[:, None, None]
    for i in range(n):
        dls.kv_append8(x[i:i + 1], x[i:i + 1], B.k, B.v, B.ks, B.vs, B.table, ints([0, 1]), ints([i + 1]), None)
    for which in "kv":
        got = B.values(0, n, which)
        p, s = B.slots(0, 0, n)
        sc = (B.ks if which == "k" else B.vs)[p, :, s // block].double()
        for lo, hi in ((0, block), (block, n)):
            assert torch.equal(sc[lo], scale_of(x[lo:hi].abs().amax((0, 2)), code))
        unit = x.double() / sc[..., None]
        # e4m3: a value may be rounded again where it falls below the normal range: half a step there (2^-10), each time less
        lim = torch.full_like(unit, 1.0) if code == "i8" else code_step(unit, code) * (1 + 2.0 ** -20) + 2.0 ** -9
        assert bool(((got / sc[..., None] - unit).abs() <= lim).all())


def test_append8_flags_what_does_not_fit(gpu_lib):
    def run(cu, kl, table, rows=8, pages=4):
        k = torch.ones(rows, 2, 32, device="cuda")
        kp, vp = (torch.zeros(pages, 2, 16, 32, dtype=torch.int8, device="cuda") for _ in range(2))
        ks, vs = (torch.zeros(pages, 2, 1, device="cuda") for _ in range(2))
        status = ints([0])
        dls.kv_append8(k, k, kp, vp, ks, vs, ints(table), ints(cu), ints(kl), None, status=status)
        torch.cuda.synchronize()
        assert torch.equal(kp, vp) and torch.equal(ks, vs)
        return int(status), int((kp == 64).sum()) / 64  # (1 is 64 times the scale 2^-6)

    assert run([0, 8], [8], [[0, 1]]) == (0, 8)
    assert run([0, 8], [20], [[0, 1]])[0] == 0
    assert run([0, 8], [20], [[0, -1]])[0] == 1
    assert run([0, 8], [20], [[4, 1]])[0] == 1
    assert run([0, 8], [33], [[0, 1]]) == (4, 0)
    assert run([0, 8], [-1], [[0, 1]]) == (4, 0)
    assert run([0, 8], [7], [[0, 1]]) == (4, 0)
    assert run([0, 9], [9], [[0, 1]]) == (4, 0)
    assert run([0, 5, 3], [5, 3], [[0, 1], [2, 3]])[0] == 4
    assert run([8, 0], [8], [[0, 1]])[0] == 4
    assert run([-1, 4], [8], [[0, 1]])[0] == 4


@pytest.mark.parametrize("cu,kl", [
    ([0, 8, 0, 1], [8, 0, 32]), ([0, 6, 2, 3], [6, 4, 32]), ([0, 8, 0, 1, 0], [8, 0, 32, 5]), ([8, 0, 8, 0], [8, 8, 8]),
    ([3, 1, 2, 0, 8], [32, 32, 32, 32]), ([0, 4, 4, 2, 8, 1, 5], [4, 0, 9, 17, 1, 32]), ([0, 8] * 40, [31, 32] * 39 + [32]),
])
def test_append8_where_cu_q_decreases(gpu_lib, cu, kl):
    """Codes go to slots of sequences that fit and hold the row, to no page of the table rows around the batch."""
    n, page, rows, most = len(kl), 16, 8, 2
    pages = 2 * n + 8
    table = torch.arange(pages, dtype=I32, device="cuda").flip(0).reshape(-1, most).contiguous()
    k = torch.ones(rows, 2, 32, device="cuda")
    pools = [torch.zeros(pages, 2, page, 32, dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.full((pages, 2, 1), 2.0 ** -6, device="cuda") for _ in range(2)]
    status = ints([0])
    dls.kv_append8(k, k, *pools, *scales, table[2:2 + n], ints(cu), ints(kl), None, status=status)
    torch.cuda.synchronize()
    assert int(status) == 4
    allowed = torch.zeros(pages, page, dtype=torch.bool)
    for b in range(n):
        if 0 <= cu[b] <= cu[b + 1] <= rows and cu[b + 1] - cu[b] <= kl[b] <= most * page:
            for pos in range(kl[b] - (cu[b + 1] - cu[b]), kl[b]):
                allowed[int(table[2 + b, pos // page]), pos % page] = True
    for pool, sc in zip(pools, scales):
        got = pool.cpu()
        assert bool(((got == 0) | ((got == 64) & allowed[:, None, :, None])).all())
        assert bool((sc == 2.0 ** -6).all())


# ---- attention --------------------------------------------------------------------------------------

def workspace(hd):
    return torch.zeros(dls.attention_chunk_workspace_bytes(hd), dtype=torch.uint8, device="cuda")


def attend64(B, q, heads, scale, causal, window):
    """(o, lse, sum of weights * |v|, largest scale * sum |q k|) in 64 bits; 0 and -inf where a row has no key."""
    o = torch.zeros(q.shape[0], heads, B.hd, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:1] + (heads,), -math.inf, dtype=torch.float64, device="cuda")
    mag, dot = torch.zeros_like(o), torch.zeros_like(lse)
    group = heads // B.kvh
    for b, (ql, kl) in enumerate(B.lengths):
        if not ql or not kl:
            continue
        r = slice(B.starts[b], B.starts[b] + ql)
        pos = torch.arange(kl - ql, kl, device="cuda")[:, None]
        key = torch.arange(kl, device="cuda")[None]
        seen = (key <= pos) if causal else torch.ones(ql, kl, dtype=torch.bool, device="cuda")
        if window:
            seen = seen & (pos - key < window)
        k, v = B.values(b, kl, "k"), B.values(b, kl, "v")
        dead = ~seen.any(0)                     # (NaN where a test poisoned them)
        k[dead], v[dead] = 0.0, 0.0
        x = q[r].double().reshape(ql, B.kvh, group, B.hd)
        sc = torch.einsum("qkgd,nkd->kgqn", x, k) * scale
        sc = torch.where(seen, sc, -math.inf)
        m = sc.amax(-1, keepdim=True)
        e = torch.where(seen, torch.exp(sc - torch.where(m.isfinite(), m, 0.0)), 0.0)
        tot = e.sum(-1, keepdim=True)
        w = e / torch.where(tot > 0, tot, 1.0)
        o[r] = torch.einsum("kgqn,nkd->qkgd", w, v).reshape(ql, heads, B.hd)
        mag[r] = torch.einsum("kgqn,nkd->qkgd", w, v.abs()).reshape(ql, heads, B.hd)
        lse[r] = (m + tot.log())[..., 0].permute(2, 0, 1).reshape(ql, heads)
        dot[r] = torch.where(seen, torch.einsum("qkgd,nkd->kgqn", x.abs(), k.abs()) * scale, 0.0).amax(-1).permute(2, 0, 1).reshape(ql, heads)
    return o, lse, mag, dot


def close_attend(B, got, lse, want, rows=None):
    o, wl, mag, dot = want
    typ = got.dtype
    # a score: hd products summed in fp32 (each step may truncate: 2^-23 of the sum of magnitudes), scaled by c and the
    # block's scale, its exponent rounded, log2 of V's scale (below 64 in size, added in fp32: 64 * 2^-23 at most with the
    # reference of the same size): at most (hd + 8) 2^-23 of scale * sum |q k| plus 2^-16.5 and the exponential's own 2^-21
    ds = (B.hd + 8) * 2.0 ** -23 * dot + 2.0 ** -16
    u = half_step(typ)
    keys = max([kl for _, kl in B.lengths] + [1])
    # weights rounded to q's type (u each, relative), scores off by ds in weight and in the sum, sums of `keys` terms in
    # fp32, the output's rounding
    lim = (u * (1 + 2.0 ** -6) + 2 * ds[..., None] + 2 * (keys / 64 + 64) * 2.0 ** -23) * mag + rounding(o, typ) * (1 + 2.0 ** -6)
    if typ == torch.float16:
        # below fp16's normal range half of 2^-24, against a largest weight times V's scale of at least 2^7, for codes up to
        # the largest there is: 2^-32 of the largest V that a code of its block could stand for
        top = 128.0 if B.code == "i8" else 448.0
        lim = lim + keys * 2.0 ** -32 * top * float(B.vs.nan_to_num(0.0, 0.0, 0.0).max())
    inside = torch.zeros(got.shape[0], dtype=torch.bool, device="cuda")
    inside[B.starts[0]:B.starts[-1]] = True
    if rows is not None:
        inside &= rows
    err = (got.double() - o).abs()
    assert bool((err <= lim)[inside].all()), float((err / lim)[inside].nan_to_num(math.inf).max())
    if lse is not None:
        a, w = lse.double()[inside], wl[inside]
        assert torch.equal(a == -math.inf, w == -math.inf)
        e = (a - w).abs().nan_to_num(0.0)
        assert not bool(a.isnan().any())
        assert bool((e <= ds[inside] + (keys / 64 + 64) * 2.0 ** -23 + 4 * F32 * w.abs().nan_to_num(0.0, 0.0, 0.0)).all()), float(e.max())


def check_attend(lengths, heads, kvh, hd, page, block, typ, code, causal=True, window=0, first=0, pad=0, scale=0.0, with_lse=True,
                 seed=5, qstd=1.5, ws=None, stream=None):
    B = Batch8(lengths, kvh, hd, page, block, code, seed, first, pad)
    B.fill()
    wide = torch.full((B.rows, heads + 1, hd), math.nan, dtype=TYPES[typ], device="cuda")
    q = wide[:, :heads]
    q[first:B.starts[-1]] = (torch.randn(B.starts[-1] - first, heads, hd, generator=B.g, device="cuda") * qstd).to(TYPES[typ])
    want = attend64(B, q, heads, scale or hd ** -0.5, causal, window)
    if window:  # what lies wholly before every window is gone: no table entry, NaN codes and scales
        for b, (ql, kl) in enumerate(lengths):
            gone = min(max(0, kl - ql - window + 1), kl)
            if gone:
                p, s = B.slots(b, 0, gone)
                for pool in (B.k, B.v):
                    pool.view(torch.uint8)[p, :, s] = 127
                whole = gone // block * block
                p, s = B.slots(b, 0, whole)
                B.ks[p, :, s // block] = math.nan
                B.vs[p, :, s // block] = math.nan
                B.table[b, :gone // page] = -1
    out = torch.full((B.rows, heads + 3, hd), 7.0, dtype=TYPES[typ], device="cuda")
    o = out[:, 2:2 + heads]
    lse = torch.full((B.rows, heads), 7.0, device="cuda") if with_lse else None
    status = ints([99])
    ws = workspace(hd) if ws is None else ws
    torch.cuda.synchronize()
    args = q, B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len
    dls.attention_chunk8(*args, o, ws, lse=lse, scale=scale, causal=causal, window=window, status=status, stream=stream)
    dls.attention_status(status, stream)
    close_attend(B, o, lse, want)
    inside = torch.zeros(B.rows, dtype=torch.bool, device="cuda")
    inside[first:B.starts[-1]] = True
    assert bool((out[~inside] == 7).all()) and bool((out[:, :2] == 7).all()) and bool((out[:, 2 + heads:] == 7).all())
    if with_lse:
        assert bool((lse[~inside] == 7).all())
    # the same call again: the same bits, on the workspace that the first call left
    again = torch.full_like(out, 7.0)
    dls.attention_chunk8(*args, again[:, 2:2 + heads], ws, scale=scale, causal=causal, window=window, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))
    return B, q, o


SIZES = [
    [(1, 1)],
    [(1, 2), (3, 3), (1, 64), (1, 65)],
    [(127, 127)], [(128, 128)], [(129, 129)], [(129, 300), (1, 300), (31, 31)],
    [(0, 5), (2, 7), (0, 0), (1, 128), (4, 129), (0, 3)],
    [(257, 1025), (1, 1), (64, 64)],
]


@pytest.mark.parametrize("lengths", SIZES, ids=str)
@pytest.mark.parametrize("heads,kvh,hd,page,block,typ,code", [(4, 2, 64, 64, 64, "f16", "e4m3"), (8, 1, 128, 32, 16, "bf16", "i8"),
                                                              (6, 2, 80, 16, 16, "f16", "i8"), (4, 2, 128, 128, 32, "bf16", "e4m3")])
def test_attention8_lengths(gpu_lib, lengths, heads, kvh, hd, page, block, typ, code):
    check_attend(lengths, heads, kvh, hd, page, block, typ, code, first=2, pad=3)


@pytest.mark.parametrize("heads,kvh", [(1, 1), (5, 5), (4, 2), (9, 3), (32, 8), (5, 1), (7, 1), (31, 1), (33, 1), (128, 2), (128, 1)])
def test_attention8_head_groups(gpu_lib, heads, kvh):
    check_attend([(1, 200), (3, 131), (70, 150), (1, 7)], heads, kvh, 64, 64, 32, "bf16", "e4m3")


@pytest.mark.parametrize("hd", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("page,block,typ,code", [(16, 16, "f16", "e4m3"), (32, 32, "bf16", "i8"), (64, 16, "f16", "i8"),
                                                 (128, 128, "bf16", "e4m3"), (256, 64, "f16", "e4m3"), (256, 256, "bf16", "i8")])
def test_attention8_head_dims_pages_and_blocks(gpu_lib, hd, page, block, typ, code):
    check_attend([(1, 300), (40, 260), (7, 7)], 6, 3, hd, page, block, typ, code)


@pytest.mark.parametrize("window", [1, 2, 7, 127, 128, 129, 500])
@pytest.mark.parametrize("hd,page,block", [(64, 16, 16), (128, 64, 32)])
def test_attention8_windows(gpu_lib, window, hd, page, block):
    check_attend([(1, 1000), (300, 300), (130, 900), (5, 129), (1, 1)], 8, 2, hd, page, block, "f16", "e4m3", window=window)


def test_attention8_rows_without_keys(gpu_lib):
    check_attend([(5, 3), (4, 0), (300, 10), (1, 0), (2, 2), (140, 130)], 4, 2, 64, 32, 16, "bf16", "e4m3")
    check_attend([(5, 3), (4, 0), (300, 10)], 4, 2, 128, 32, 32, "f16", "i8", window=2)
    check_attend([(5, 3), (4, 0), (1, 1)], 4, 2, 128, 32, 32, "f16", "e4m3", causal=False)


@pytest.mark.parametrize("hd,window", [(64, 0), (128, 2)])
def test_attention8_runs_of_rows_without_keys(gpu_lib, hd, window):
    lengths = ([(2, 0)] * 5 + [(5, 40), (1, 1), (0, 7), (3, 0)] * 2 + [(140, 60), (7, 0), (200, 30)]) * 16
    check_attend(lengths, 2, 2, hd, 16, 16, "f16", "e4m3", window=window)


def test_attention8_every_key(gpu_lib):
    check_attend([(5, 700), (130, 257), (300, 40), (1, 1)], 8, 4, 128, 64, 64, "bf16", "e4m3", causal=False)
    check_attend([(64, 64)] * 3, 3, 3, 64, 16, 16, "f16", "i8", causal=False)


@pytest.mark.parametrize("scale", [1e-3, 0.5, 4.0])
def test_attention8_scales_of_scores(gpu_lib, scale):
    check_attend([(1, 777), (150, 400)], 4, 2, 64, 64, 16, "bf16", "e4m3", scale=scale)


def test_attention8_long_caches(gpu_lib):
    check_attend([(1, 20011)], 8, 2, 128, 64, 64, "bf16", "e4m3")
    check_attend([(1, 9000), (1, 33), (5, 8200), (1, 16384)], 16, 2, 64, 128, 32, "f16", "i8")


def test_attention8_many_sequences(gpu_lib):
    check_attend([(1 + b % 3, 1 + (37 * b) % 90 + b % 3) for b in range(600)], 2, 1, 64, 16, 16, "f16", "e4m3")


def test_attention8_whole_prompts(gpu_lib):
    check_attend([(1500, 1500)], 8, 2, 128, 64, 64, "bf16", "e4m3")
    check_attend([(700, 1900), (1, 1200), (900, 900)], 8, 8, 64, 64, 32, "f16", "i8")


@pytest.mark.parametrize("heads,kvh,hd,page,block,typ,code", [(32, 8, 128, 32, 32, "f16", "e4m3"), (16, 2, 128, 64, 16, "bf16", "i8"),
                                                              (8, 8, 64, 16, 16, "f16", "e4m3"), (16, 8, 64, 64, 64, "bf16", "i8")])
def test_attention8_many_tiles_of_each_range(gpu_lib, heads, kvh, hd, page, block, typ, code):
    """Several tiles of several key tiles in each CTA's range, repeated: the rings run on from tile to tile."""
    B = Batch8([(5, 4101), (1, 3661), (3, 4009), (4, 1803), (1, 2951), (4, 3718), (5, 2122), (1, 2767), (60, 3001)], kvh, hd, page,
               block, code, 16)
    B.fill()
    q = (2 * torch.randn(B.rows, heads, hd, generator=B.g, device="cuda")).to(TYPES[typ])
    o, first, lse, ws = torch.empty_like(q), torch.empty_like(q), torch.empty(B.rows, heads, device="cuda"), workspace(hd)
    args = q, B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len
    dls.attention_chunk8(*args, first, ws)
    for _ in range(20):
        dls.attention_chunk8(*args, o, ws, lse=lse)
        assert torch.equal(o, first)
    close_attend(B, o, lse, attend64(B, q, heads, hd ** -0.5, True, 0))


FEW = [  # few rows a sequence: heads x new tokens of a KV head's group up to eight, or sixteen
    ([(1, 1)], 4, 1), ([(1, 300), (1, 16), (1, 17), (1, 15), (1, 129)], 8, 1), ([(1, 2500), (1, 1), (1, 777)], 16, 1),
    ([(1, 1000)] * 5, 3, 3), ([(2, 400), (2, 2), (1, 90)], 4, 1), ([(4, 600), (3, 50), (4, 4), (0, 9), (5, 1300)], 8, 2),
    ([(16, 900), (9, 40)], 2, 2), ([(1, 333)] * 40, 12, 1), ([(5, 4101)] + [(3, 700 + b) for b in range(7)], 6, 2),
    ([(0, 5)] * 30 + [(60, 500), (1, 64)] + [(0, 0)] * 30, 2, 1),   # a long one among empty ones
    ([(1, 40 + 3 * b) for b in range(300)], 10, 2),                  # planned by the block
]


@pytest.mark.parametrize("lengths,heads,kvh", FEW, ids=lambda x: f"{len(x)}seqs" if isinstance(x, list) else str(x))
@pytest.mark.parametrize("hd,page,block,typ,code", [(128, 64, 64, "bf16", "e4m3"), (64, 16, 16, "f16", "i8"), (128, 16, 16, "f16", "e4m3"),
                                                    (64, 256, 32, "bf16", "e4m3"), (128, 128, 32, "bf16", "i8"), (96, 64, 16, "f16", "e4m3"),
                                                    (80, 16, 16, "bf16", "i8"), (112, 32, 32, "f16", "e4m3"), (48, 128, 64, "bf16", "e4m3"),
                                                    (32, 64, 64, "f16", "i8"), (16, 16, 16, "bf16", "e4m3")])
def test_attention8_few_rows(gpu_lib, lengths, heads, kvh, hd, page, block, typ, code):
    check_attend(lengths, heads, kvh, hd, page, block, typ, code, first=1, pad=2)


@pytest.mark.parametrize("window", [1, 5, 16, 17, 130])
def test_attention8_few_rows_windows(gpu_lib, window):
    check_attend([(1, 1000), (2, 300), (1, 33), (3, 3), (1, 1)], 8, 2, 128, 32, 16, "f16", "e4m3", window=window)
    check_attend([(1, 1000), (2, 300), (1, 33), (3, 3), (1, 1)], 4, 2, 64, 16, 16, "bf16", "i8", window=window)
    check_attend([(1, 1000), (2, 300), (1, 33), (3, 3), (1, 1)], 4, 2, 80, 64, 16, "bf16", "e4m3", window=window)


def test_attention8_few_rows_without_keys_and_every_key(gpu_lib):
    check_attend([(2, 1), (1, 0), (3, 2), (1, 50)], 4, 2, 64, 32, 16, "bf16", "e4m3")
    check_attend([(2, 1), (1, 0), (3, 2), (1, 50)], 4, 2, 128, 32, 32, "f16", "i8", window=1)
    check_attend([(2, 700), (3, 40), (1, 1), (2, 0)], 4, 2, 128, 64, 64, "bf16", "e4m3", causal=False)


@pytest.mark.parametrize("scale", [1e-3, 0.5, 4.0])
def test_attention8_few_rows_scales_of_scores(gpu_lib, scale):
    check_attend([(1, 777), (2, 400)], 4, 2, 64, 64, 16, "bf16", "e4m3", scale=scale)
    check_attend([(1, 777), (2, 400)], 4, 2, 128, 64, 32, "f16", "e4m3", scale=scale)


@pytest.mark.parametrize("hd", [64, 112, 128])
@pytest.mark.parametrize("lengths,heads", [([(1, 9000)], 16), ([(3, 5000), (1, 3001)], 16)])
def test_attention8_rising_scores(gpu_lib, hd, lengths, heads):
    """Keys whose scores grow along the sequence: the running maximum moves at every step, by little and by much."""
    for step in (0.02, 0.5):
        B = Batch8(lengths, 2, hd, 64, 64, "e4m3", 9)
        B.fill()
        B.ks.fill_(1 / 64)
        for b, (_, kl) in enumerate(lengths):
            p, s = B.slots(b, 0, kl)
            rise = (torch.arange(kl, device="cuda") * step * 0.1 * 0.5).clamp(max=440)
            B.k.view(torch.uint8)[p, :, s, 0] = rise.to(CODES["e4m3"]).view(torch.uint8)[:, None]
        q = torch.randn(B.rows, heads, hd, generator=B.g, device="cuda").bfloat16()
        q[..., 0] = 8.0 * 64
        o, lse = torch.empty_like(q), torch.empty(B.rows, heads, device="cuda")
        dls.attention_chunk8(q, B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len, o, workspace(hd), lse=lse, scale=0.05)
        close_attend(B, o, lse, attend64(B, q, heads, 0.05, True, 0))


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("size", [1e-30, 1e-6, 3e4, 1e30])
def test_attention8_bf16_rows_of_any_size(gpu_lib, rows, size):
    """bf16 holds rows of q that halves do not: their scores are what the formula gives all the same."""
    B = Batch8([(rows, 300)], 1, 64, 16, 16, "e4m3", 19)
    B.fill()
    q = torch.randn(rows, 4, 64, generator=B.g, device="cuda")
    q[:, 1] = 0.0
    q[:, 2, 5] = 1e-4
    q = (q * size).bfloat16()
    o, lse = torch.empty_like(q), torch.empty(rows, 4, device="cuda")
    scale = min(max(0.1 / size, 1e-28), 1e28)
    dls.attention_chunk8(q, B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len, o, workspace(64), lse=lse, scale=scale)
    close_attend(B, o, lse, attend64(B, q, 4, float(np.float32(scale)), True, 0))


@pytest.mark.parametrize("lengths,heads,kvh,hd", [([(5, 4101), (1, 3661), (4, 1803), (2, 2951)], 8, 2, 128), ([(1, 2000 + 5 * b) for b in range(70)], 8, 1, 64),
                                                  ([(1, 2000 + 5 * b) for b in range(70)], 16, 2, 128)])
def test_attention8_few_rows_repeated(gpu_lib, lengths, heads, kvh, hd):
    """Several pieces in each CTA's range, cut tiles among them, repeated: the same bits."""
    B = Batch8(lengths, kvh, hd, 32, 32, "e4m3", 16)
    B.fill()
    q = (2 * torch.randn(B.rows, heads, hd, generator=B.g, device="cuda")).half()
    o, first, ws = torch.empty_like(q), torch.empty_like(q), workspace(hd)
    args = q, B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len
    dls.attention_chunk8(*args, first, ws)
    for _ in range(20):
        dls.attention_chunk8(*args, o, ws)
        assert torch.equal(o, first)
    x = q.clone()
    dls.attention_chunk8(x, *args[1:], x, ws)
    assert torch.equal(x, first)
    close_attend(B, o, None, attend64(B, q, heads, hd ** -0.5, True, 0))


@pytest.mark.parametrize("typ", ["f16", "bf16"])
def test_attention8_every_code(gpu_lib, typ):
    """One key a sequence: its value is the output, for every code that is a number."""
    for code in ("e4m3", "i8"):
        every = torch.arange(256, dtype=torch.uint8, device="cuda")
        if code == "e4m3":
            every = every[~every.view(CODES[code]).float().isnan()]
        n = -(-len(every) // 64)
        B = Batch8([(1, 1)] * n, 1, 64, 16, 16, code, 3)
        B.fill()
        codes = every[torch.arange(n * 64, device="cuda") % len(every)].reshape(n, 64)
        B.v.view(torch.uint8)[B.table[:, 0].long(), 0, 0] = codes
        B.vs[B.table[:, 0].long()] = 0.25
        q = torch.randn(n, 2, 64, device="cuda").to(TYPES[typ])
        o = torch.empty_like(q)
        dls.attention_chunk8(q, B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len, o, workspace(64))
        # the one weight is 2^7 (or a rounding away from it) and is divided by itself
        want = (codes.view(CODES[code]).double() * 0.25)[:, None].expand(n, 2, 64)
        assert bool(((o.double() - want).abs() <= 2 * rounding(want, TYPES[typ]) * (1 + 2.0 ** -6)).all())
        # and as a key: the score comes back as lse
        B.k.view(torch.uint8)[B.table[:, 0].long(), 0, 0] = codes
        B.ks[B.table[:, 0].long()] = 0.5
        lse = torch.empty(n, 2, device="cuda")
        for d in range(64):
            q.zero_()
            q[:, :, d] = 3.0
            dls.attention_chunk8(q, B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len, o, workspace(64), lse=lse, scale=1.0)
            want = codes.view(CODES[code])[:, d].double() * 1.5
            # c = log2 e times the score and back: four roundings, the sum's, and the exponential's 2^-21
            assert bool(((lse.double() - want[:, None]).abs() <= 8 * F32 * (want[:, None].abs() + 16) + 2.0 ** -20).all())


@pytest.mark.parametrize("spread", [10, 40, 64])
@pytest.mark.parametrize("typ", ["f16", "bf16"])
def test_attention8_scales_far_apart(gpu_lib, spread, typ):
    """V scales from 2^-spread to 2^spread/2 in one sequence, K scales that make the scores of a block vanish: the weights
    keep their bits in 16, and the sum of the weights is that of the small-scaled blocks too."""
    B = Batch8([(1, 500), (40, 300)], 2, 64, 32, 16, "e4m3", 21)
    B.fill()
    for b, (_, kl) in enumerate(B.lengths):
        p, s = B.slots(b, 0, kl)
        e = torch.randint(-spread, spread // 8, (kl,), generator=B.g, device="cuda").float()
        B.vs[p, :, s // 16] = torch.exp2(e[torch.arange(kl, device="cuda") // 16 * 16])[:, None]
        B.ks[p, :, s // 16] = torch.where(torch.arange(kl, device="cuda") // 16 % 3 == 0, 2.0 ** -64, 0.01)[:, None]
    q = torch.randn(B.rows, 4, 64, generator=B.g, device="cuda").to(TYPES[typ])
    o, lse = torch.empty_like(q), torch.empty(B.rows, 4, device="cuda")
    dls.attention_chunk8(q, B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len, o, workspace(64), lse=lse)
    close_attend(B, o, lse, attend64(B, q, 4, 0.125, True, 0))


def test_attention8_scales_that_are_none(gpu_lib):
    """0, negative ones and NaN count as 2^-64, more than 2^64 as that."""
    B = Batch8([(3, 100)], 2, 64, 16, 16, "i8", 22)
    B.fill()
    q = torch.randn(3, 4, 64, generator=B.g, device="cuda").half()
    p = B.table[0, :7].long()
    o, want = torch.empty_like(q), torch.empty_like(q)
    ks, vs = B.ks.clone(), B.vs.clone()
    for scales, mine in ((ks, B.ks), (vs, B.vs)):
        scales[p[1]], mine[p[1]] = 0.0, 2.0 ** -64
        scales[p[3]], mine[p[3]] = math.nan, 2.0 ** -64
        scales[p[5]], mine[p[5]] = -1.0, 2.0 ** -64
    dls.attention_chunk8(q, B.k, B.v, ks, vs, B.table, B.cu_q, B.kv_len, o, workspace(64))
    dls.attention_chunk8(q, B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len, want, workspace(64))
    assert torch.equal(o, want) and bool(o.isfinite().all())


def test_attention8_flags_what_does_not_fit(gpu_lib):
    def run(cu, kl, table, rows=8, pages=4):
        q = torch.ones(rows, 2, 64, dtype=torch.float16, device="cuda")
        kp = torch.ones(pages, 2, 16, 64, dtype=torch.int8, device="cuda")
        ks = torch.ones(pages, 2, 1, device="cuda")
        status, o, ws = ints([0]), torch.full_like(q, 7.0), workspace(64)
        dls.attention_chunk8(q, kp, kp, ks, ks, ints(table), ints(cu), ints(kl), o, ws, status=status)
        torch.cuda.synchronize()
        got = int(status)
        # the workspace serves the next call
        dls.attention_chunk8(q, kp, kp, ks, ks, ints([[0, 1]]), ints([0, 8]), ints([20]), o, ws, status=status)
        dls.attention_status(status)
        assert bool((o == 1).all())
        return got

    assert run([0, 8], [20], [[0, 1]]) == 0
    assert run([0, 8], [20], [[0, -1]]) == 1
    assert run([0, 8], [20], [[4, 1]]) == 1
    assert run([0, 8], [33], [[0, 1]]) == 4
    assert run([0, 8], [-1], [[0, 1]]) == 4
    assert run([0, 9], [9], [[0, 1]]) == 4
    assert run([0, 5, 3], [5, 3], [[0, 1], [2, 3]]) == 4
    assert run([-1, 4], [8], [[0, 1]]) == 4


def test_attention8_workspace_streams_and_in_place(gpu_lib):
    """One workspace for all shapes and both kinds of pages; a stream of its own; o = q; two calls at once."""
    ws = workspace(128)
    check_attend([(1, 5000)], 8, 2, 128, 64, 64, "bf16", "e4m3", ws=ws)
    check_attend([(300, 700)], 4, 2, 64, 16, 16, "f16", "i8", ws=ws)
    check_attend([(1, 900), (150, 300)], 8, 2, 128, 64, 32, "bf16", "i8", stream=torch.cuda.Stream(), ws=ws)
    assert not bool(ws[:4096].any())  # its counters are zero again
    made = []
    for lengths, hd in (([(1, 2000)] * 5 + [(70, 200)], 128), ([(400, 1000), (1, 3000)], 64)):
        B = Batch8(lengths, 2, hd, 32, 32, "e4m3", 13)
        B.fill()
        q = torch.randn(B.rows, 8, hd, generator=B.g, device="cuda").half()
        made.append((B, q, torch.empty_like(q), torch.empty_like(q), workspace(hd), torch.cuda.Stream()))
    for B, q, alone, _, w, _ in made:
        dls.attention_chunk8(q, B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len, alone, w)
        x = q.clone()
        dls.attention_chunk8(x, B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len, x, w)
        assert torch.equal(x, alone)
    torch.cuda.synchronize()
    for _ in range(30):
        for B, q, _, o, w, stream in made:
            dls.attention_chunk8(q, B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len, o, w, stream=stream)
    torch.cuda.synchronize()
    for _, _, alone, o, _, _ in made:
        assert torch.equal(o, alone)


def test_attention8_is_the_16_bit_call_on_values_that_both_hold(gpu_lib):
    """Scales of one: the codes are the 16-bit values, and both calls are within their roundings of the formula."""
    B = Batch8([(1, 700), (130, 400), (5, 1300)], 2, 128, 64, 64, "e4m3", 14)
    B.fill()
    B.ks.fill_(2.0 ** -7)
    B.vs.fill_(2.0 ** -7)
    q = torch.randn(B.rows, 8, 128, generator=B.g, device="cuda").bfloat16()
    o, o16 = torch.empty_like(q), torch.empty_like(q)
    k, v = ((t.float() * 2.0 ** -7).bfloat16() for t in (B.k, B.v))
    dls.attention_chunk8(q, B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len, o, workspace(128))
    dls.attention_chunk(q, k, v, B.table, B.cu_q, B.kv_len, o16, workspace(128))
    want = attend64(B, q, 8, 128 ** -0.5, True, 0)
    close_attend(B, o, None, want)
    close_attend(B, o16, None, want)


def test_pools_of_more_than_two_to_the_31_codes(gpu_lib):
    """Append and attention over the last pages of pools whose offsets pass 32 bits."""
    kvh, page, hd, heads, n_pages = 2, 128, 128, 8, 70000  # 2.3e9 codes
    pools = [torch.empty(n_pages, kvh, page, hd, dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.empty(n_pages, kvh, 4, device="cuda") for _ in range(2)]
    B = Batch8([(150, 150), (1, 300)], kvh, hd, page, 32, "i8", 31, extra=0)
    B.fill(powers=True)
    own = (B.table >= 0) & (B.table < B.n_pages)
    used = B.table[own].long()
    moved = n_pages - 1 - 3 * used
    for pool, src in zip(pools + scales, (B.k, B.v, B.ks, B.vs)):
        pool[moved] = src[used]
    table = torch.where(own, n_pages - 1 - 3 * B.table, B.table)
    x = torch.randn(B.rows, heads + 2 * kvh, hd, generator=B.g, device="cuda").bfloat16()
    q, status = x[:, :heads], ints([0])
    freq, o = dls.rope_inv_freq(hd, 500000.0), torch.empty(B.rows, heads, hd, dtype=torch.bfloat16, device="cuda")
    k, v = x[:, heads:heads + kvh], x[:, heads + kvh:]
    dls.kv_append8(k, v, *pools, *scales, table, B.cu_q, B.kv_len, freq, status=status)
    dls.attention_status(status)
    dls.attention_chunk8(q, *pools, *scales, table, B.cu_q, B.kv_len, o, workspace(hd), status=status)
    dls.attention_status(status)
    dls.kv_append8(k, v, B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len, freq)  # the small pool
    for pool, small in zip(pools + scales, (B.k, B.v, B.ks, B.vs)):
        assert torch.equal(pool[moved].view(torch.uint8), small[used].view(torch.uint8))
    close_attend(B, o, None, attend64(B, q, heads, hd ** -0.5, True, 0))


# ---- drafted tokens ----------------------------------------------------------------------------------

def units(p):
    """Probabilities (any float array) in whole numbers of 2^-45, to the nearest: p 2^45 is exact in 64 bits, and below 2^53."""
    p = np.nan_to_num(np.asarray(p, dtype=np.float64), nan=0.0).clip(0.0, 1.0)
    return np.rint(p * 2.0 ** 45).astype(np.int64)


def verify_plain(tokens, target, draft, cu, accept, pick, vocab):
    """The call's definition: [(tokens of the rows, accepted)] a sequence, in exact arithmetic."""
    got = []
    for b in range(len(cu) - 1):
        s, e = cu[b], cu[b + 1]
        if s == e:
            got.append(([], 0))
            continue
        stop = e - 1
        for r in range(s, e - 1):
            x = tokens[r + 1]
            ok = 0 <= x < vocab
            if ok:
                p, q = float(target[r][x]), float(draft[r][x]) if draft is not None else 1.0
                ok = Fraction(accept[r]) * Fraction(q) < Fraction(p) if math.isfinite(p) and math.isfinite(q) else False
            if not ok:
                stop = r
                break
        p = units(target[stop])
        w = p
        if stop < e - 1:
            if draft is not None:
                w = np.maximum(p - units(draft[stop]), 0)
            else:
                w = p.copy()
                if 0 <= tokens[stop + 1] < vocab:
                    w[tokens[stop + 1]] = 0
        if not int(w.sum()):
            w = p
        total = int(w.sum())
        if total:
            v = Fraction(min(max(float(pick[b]), 0.0), 1 - 2.0 ** -24)) if not math.isnan(float(pick[b])) else Fraction(0)
            border = int(v * total)  # floor
            t = int(np.argmax(np.cumsum(w) > border))
        else:
            t = -1
        got.append(([tokens[r + 1] for r in range(s, stop)] + [t] + [-1] * (e - 1 - stop), stop - s))
    return got


def check_verify(lengths, vocab, typ, drawn, seed, pad=0, first=0, stride=0, near=0.6, offset=0, edit=None, expect=0, stream=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = first + sum(lengths) + pad
    cu = [first]
    for n in lengths:
        cu.append(cu[-1] + n)

    def probs(x):
        wide = torch.full((rows * (vocab + stride) + offset + 8,), math.nan, dtype=TYPES[typ], device="cuda")
        t = wide[offset:offset + rows * (vocab + stride)].reshape(rows, vocab + stride)[:, :vocab]
        t.copy_(x)
        return t

    logits = torch.randn(rows, vocab, generator=g, device="cuda") * 2.5
    p = torch.softmax(logits, -1)
    q = torch.softmax(logits + near * torch.randn(rows, vocab, generator=g, device="cuda"), -1)
    picked = torch.multinomial(q, 1, generator=g)[:, 0] if drawn else q.argmax(-1)
    tokens = torch.cat([picked[-1:], picked[:-1]]).to(I32)
    s = dict(target=probs(p), draft=probs(q) if drawn else None, tokens=tokens, accept=torch.rand(rows, generator=g, device="cuda"),
             pick=torch.rand(len(lengths), generator=g, device="cuda"))
    if edit:
        edit(s, cu)
    kv = torch.randint(50, 999, (len(lengths),), generator=g, device="cuda", dtype=I32)
    kv_out, status = torch.full_like(kv, 7), ints([99])
    out, n_acc = torch.full((rows,), 77, dtype=I32, device="cuda"), torch.full((len(lengths),), 77, dtype=I32, device="cuda")
    torch.cuda.synchronize()
    dls.verify_draft(s["tokens"], s["target"], ints(cu), s["accept"], s["pick"], out, n_acc, draft=s["draft"], kv_len=kv,
                     kv_len_out=kv_out, status=status, stream=stream)
    torch.cuda.synchronize()
    want = verify_plain(s["tokens"].tolist(), s["target"].double().cpu().numpy(), None if s["draft"] is None else s["draft"].double().cpu().numpy(),
                        cu, s["accept"].tolist(), s["pick"].tolist(), vocab)
    got = out.tolist()
    for b, (toks, acc) in enumerate(want):
        assert got[cu[b]:cu[b + 1]] == toks, (b, got[cu[b]:cu[b + 1]], toks)
        assert n_acc[b].item() == acc
        assert kv_out[b].item() == kv[b].item() - (max(lengths[b] - 1, 0) - acc)
    assert got[:first] == [77] * first and got[cu[-1]:] == [77] * pad
    assert status.item() == expect
    return want


@pytest.mark.parametrize("vocab", [1, 2, 3, 31, 1000, 1024, 5003, 32000, 128256])
@pytest.mark.parametrize("typ,drawn", [("f32", True), ("bf16", False), ("f16", True), ("f32", False)])
def test_verify_vocabularies_and_types(gpu_lib, vocab, typ, drawn):
    want = check_verify([5, 1, 0, 3, 7, 2], vocab, typ, drawn, 3 + vocab, pad=2, first=1)
    assert len(want) == 6


@pytest.mark.parametrize("lengths", [[1], [2], [33], [34], [70, 1, 65], [0, 0, 4], [3] * 200, [1] * 700], ids=lambda x: f"{len(x)}of{max(x)}")
def test_verify_lengths(gpu_lib, lengths):
    check_verify(lengths, 777, "f32", True, 11, near=0.05)
    check_verify(lengths, 777, "bf16", False, 12)


@pytest.mark.parametrize("stride,offset", [(0, 1), (3, 0), (5, 2), (8, 8), (1, 7)])
@pytest.mark.parametrize("typ", ["f32", "f16"])
def test_verify_rows_anywhere(gpu_lib, stride, offset, typ):
    """Rows that begin at any element, also where rows of the two lie differently to 16 bytes."""
    check_verify([4, 2, 3], 4099, typ, True, 21, stride=stride, offset=offset)
    check_verify([4, 2, 3], 4099, typ, False, 22, stride=stride, offset=offset)

    def move(s, cu):  # the draft's rows elsewhere than the target's
        d = torch.full((s["draft"].shape[0], 4099 + 2), math.nan, dtype=s["draft"].dtype, device="cuda")[:, 1:4100]
        d.copy_(s["draft"])
        s["draft"] = d

    check_verify([4, 2, 3], 4099, typ, True, 23, stride=stride, offset=offset, edit=move)


def test_verify_borders(gpu_lib):
    """Random numbers at the ends, and picks exactly on the border of two tokens: the next one then."""
    vocab = 16

    def edges(s, cu):
        s["target"].fill_(1 / 16)
        s["draft"].fill_(1 / 16)
        s["accept"].copy_(torch.tensor([0.0, 1 - 2.0 ** -24, 0.5] * 7, device="cuda"))
        s["pick"].copy_(torch.tensor([0.0, 1 / 16, 0.5, 0.5 - 2.0 ** -25, 1 - 2.0 ** -24, 1.0, math.nan], device="cuda"))

    want = check_verify([3] * 7, vocab, "f32", True, 5, edit=edges)
    assert [w[0][w[1]] for w in want] == [0, 1, 8, 7, 15, 15, 0] and all(w[1] == 2 for w in want)

    def refuse(s, cu):  # p = q everywhere but at the draft's token, which is refused
        s["target"].fill_(1 / 32)
        s["target"][:, 5] = 0.0
        s["draft"].fill_(1 / 64)
        s["draft"][:, 5] = 0.5
        s["tokens"].fill_(5)
        s["accept"].fill_(0.0)

    want = check_verify([3] * 4, vocab, "f32", True, 6, edit=refuse)
    assert all(w[1] == 0 and w[0][0] != 5 for w in want)


def test_verify_probabilities_that_are_none(gpu_lib):
    """NaN, negative ones and more than 1; a residual without weight; a row without any; tokens outside the vocabulary."""
    def nothing_left(s, cu):
        s["draft"].copy_(s["target"])
        s["draft"][cu[0]] = 1.0              # refused for certain, and nothing over
        s["accept"].fill_(1 - 2.0 ** -24)

    want = check_verify([3, 2], 900, "f32", True, 31, edit=nothing_left)
    assert want[0][1] == 0

    def empty_row(s, cu):
        s["target"][cu[0]:cu[1]] = 0.0

    want = check_verify([3, 2], 900, "f32", True, 32, edit=empty_row, expect=2)
    assert want[0][0] == [-1, -1, -1]

    def strange(s, cu):
        s["target"][:, 3], s["target"][:, 4], s["target"][:, 6] = math.nan, -0.5, 1.5
        s["draft"][:, 5], s["draft"][:, 6] = math.nan, -1.0

    check_verify([3, 2, 6], 900, "f32", True, 33, edit=strange)

    def outside(s, cu):
        s["tokens"][cu[0] + 1] = 900
        s["tokens"][cu[1] + 1] = -1

    want = check_verify([3, 2], 900, "f32", False, 34, edit=outside, expect=2)
    assert want[0][1] == want[1][1] == 0


def test_verify_tiny_weights_and_many_borders(gpu_lib):
    """One heavy token and a tail of unlikely ones that a 32-bit sum would not tell apart, picks inside the tail."""
    vocab = 100003

    def tail(s, cu):
        s["target"].uniform_(0.5, 1.5, generator=torch.Generator(device="cuda").manual_seed(1))
        s["target"].mul_(1e-9)
        s["target"][:, 17] = 0.9999
        s["pick"].copy_(torch.linspace(0.99990, 0.999999, 40, device="cuda"))

    want = check_verify([1] * 40, vocab, "f32", False, 8, edit=tail)
    assert len({w[0][0] for w in want}) > 30


def test_verify_agrees_with_the_distribution(gpu_lib):
    """What comes out, over many draws, has the target's distribution (drafts from another one): the method's purpose."""
    n, vocab = 60000, 6
    g = torch.Generator(device="cuda").manual_seed(2)
    p = torch.tensor([0.05, 0.3, 0.1, 0.25, 0.2, 0.1], device="cuda")
    q = torch.tensor([0.3, 0.05, 0.25, 0.1, 0.1, 0.2], device="cuda")
    x = torch.multinomial(q, n, replacement=True, generator=g).to(I32)
    tokens = torch.stack([torch.zeros_like(x), x], 1).reshape(-1).contiguous()
    cu = torch.arange(n + 1, device="cuda", dtype=I32) * 2
    out, acc = torch.empty_like(tokens), torch.empty(n, dtype=I32, device="cuda")
    dls.verify_draft(tokens, p.expand(2 * n, vocab).contiguous(), cu, torch.rand(2 * n, generator=g, device="cuda"),
                     torch.rand(n, generator=g, device="cuda"), out, acc, draft=q.expand(2 * n, vocab).contiguous())
    share = torch.bincount(out[::2].long(), minlength=vocab).double() / n
    assert bool(((share - p.double()).abs() <= 5 * (p.double() * (1 - p.double()) / n).sqrt()).all())  # five standard deviations


def test_verify_on_streams_and_in_a_graph(gpu_lib):
    """Two calls at once on two streams, and a captured one replayed with other inputs, give what each gives alone."""
    made = []
    for seed, n, vocab in ((1, 9, 128256), (2, 40, 5003)):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rows = 4 * n
        s = dict(tokens=torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=I32),
                 target=torch.softmax(2 * torch.randn(rows, vocab, generator=g, device="cuda"), -1),
                 draft=torch.softmax(2 * torch.randn(rows, vocab, generator=g, device="cuda"), -1), cu=torch.arange(n + 1, device="cuda", dtype=I32) * 4,
                 accept=torch.rand(rows, generator=g, device="cuda") * 0.01, pick=torch.rand(n, generator=g, device="cuda"))
        made.append((s, [(torch.full((rows,), 7, dtype=I32, device="cuda"), torch.full((n,), 7, dtype=I32, device="cuda")) for _ in range(2)], torch.cuda.Stream()))

    def call(s, out, stream):
        dls.verify_draft(s["tokens"], s["target"], s["cu"], s["accept"], s["pick"], *out, draft=s["draft"], stream=stream)

    for s, out, _ in made:
        call(s, out[0], None)
    torch.cuda.synchronize()
    for _ in range(20):
        for s, out, stream in made:
            call(s, out[1], stream)
    torch.cuda.synchronize()
    for s, out, _ in made:
        assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    s, out, stream = made[1]
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=stream):
        call(s, out[1], torch.cuda.current_stream())
    s["target"].copy_(s["draft"].flip(0))
    s["pick"].mul_(0.5)
    call(s, out[0], None)
    torch.cuda.synchronize()
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


def test_verify_flags_rows_that_do_not_fit(gpu_lib):
    def run(cu):
        rows, n = 8, len(cu) - 1
        out, acc, status, kv = torch.full((rows,), 77, dtype=I32, device="cuda"), ints([5] * n), ints([0]), ints([40] * n)
        dls.verify_draft(torch.zeros(rows, dtype=I32, device="cuda"), torch.full((rows, 10), 0.1, device="cuda"), ints(cu),
                         torch.zeros(rows, device="cuda"), torch.zeros(n, device="cuda"), out, acc, kv_len=kv, kv_len_out=kv, status=status)
        return status.item(), acc.tolist(), out.tolist(), kv.tolist()

    assert run([0, 9]) == (4, [0], [77] * 8, [40])
    assert run([-1, 3])[0] == 4
    got = run([0, 5, 3])
    assert got[0] == 4 and got[1] == [4, 0] and got[2] == [0] * 5 + [77] * 3 and got[3] == [40, 40]
    assert run([0, 0, 8]) == (0, [0, 7], [0] * 8, [40, 40])


def test_empty_calls_clear_the_status(gpu_lib):
    B = Batch8([(1, 20)], 2, 64, 16, 16, "i8", 3)
    x, status = torch.zeros(0, 2, 64, dtype=torch.float16, device="cuda"), ints([5])
    dls.kv_append8(x, x, B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len, None, status=status)
    assert status.item() == 0
    status.fill_(5)
    dls.attention_chunk8(x, B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len, x, workspace(64), status=status)
    assert status.item() == 0
    status.fill_(5)
    z = torch.zeros(0, device="cuda")
    dls.verify_draft(z.to(I32), torch.zeros(0, 5, device="cuda"), ints([0]), z, z, z.to(I32), z.to(I32), status=status)
    assert status.item() == 0
    with pytest.raises(dls.DlsError, match="0x10") as e:
        dls.attention_status(ints([16]))
    assert e.value.code == dls.DLS_ERR_CAPACITY
    with pytest.raises(dls.DlsError) as e:
        dls.attention_status(ints([20]))
    assert e.value.code == dls.DLS_ERR_STATE


# ---- together -----------------------------------------------------------------------------------------

class Step:
    """One layer's serving step over the 8-bit cache, all lengths on the device: reserve, rotate, append, attend, verify.
    A row's "model" is its token's fixed projection; its probabilities come from the attention's output."""

    def __init__(self, n, heads, kvh, hd, page, block, code, vocab, pages, most, rows, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.n, self.heads, self.kvh, self.hd, self.page, self.block, self.code, self.vocab, self.rows = n, heads, kvh, hd, page, block, code, vocab, rows
        self.table, self.stack = torch.full((n, most), -1, dtype=I32, device="cuda"), torch.randperm(pages, generator=g, device="cuda").to(I32)
        self.count, self.kv, self.held, self.new = ints([pages]), ints([0] * n), ints([0] * n), ints([0] * n)
        self.cu, self.status = ints([0] * (n + 1)), [ints([0]) for _ in range(4)]
        self.positions, self.slots, self.ids, self.tokens, self.out = (torch.zeros(rows, dtype=I32, device="cuda") for _ in range(5))
        self.k, self.v = (torch.full((pages, kvh, page, hd), 127, dtype=torch.uint8, device="cuda").view(CODES[code]) for _ in range(2))
        self.ks, self.vs = (torch.full((pages, kvh, page // block), math.nan, device="cuda") for _ in range(2))
        self.embed = (r(vocab, heads + 2 * kvh, hd) * 1.2).bfloat16()
        self.head = r(heads * hd, vocab) * 0.3
        self.q, self.o = (torch.zeros(rows, heads, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.wk = 1 + 0.1 * r(hd)
        self.freq, self.ws = dls.rope_inv_freq(hd, 10000.0), workspace(hd)
        self.probs = torch.zeros(rows, vocab, device="cuda")
        self.accept, self.pick, self.acc = torch.zeros(rows, device="cuda"), torch.zeros(n, device="cuda"), ints([0] * n)

    def run(self, stream):
        s = dict(stream=stream)
        dls.kv_reserve(self.new, self.kv, self.held, self.table, self.stack, self.count, self.kv, self.held, self.count, self.cu,
                       self.page, positions=self.positions, slots=self.slots, seq_ids=self.ids, status=self.status[0], **s)
        x = self.embed[self.tokens.long()]
        k, v = x[:, self.heads:self.heads + self.kvh], x[:, self.heads + self.kvh:]
        dls.qk_norm_rope(x[:, :self.heads], None, self.positions, self.freq, self.q, None, pairing="halves", **s)
        dls.kv_append8(k, v, self.k, self.v, self.ks, self.vs, self.table, self.cu, self.kv, self.freq, k_norm=self.wk, pairing="halves",
                       status=self.status[1], **s)
        dls.attention_chunk8(self.q, self.k, self.v, self.ks, self.vs, self.table, self.cu, self.kv, self.o, self.ws, status=self.status[2], **s)
        self.probs.copy_(torch.softmax(self.o.float().reshape(self.rows, -1) @ self.head, -1))
        dls.verify_draft(self.tokens, self.probs, self.cu, self.accept, self.pick, self.out, self.acc, kv_len=self.kv, kv_len_out=self.kv,
                         status=self.status[3], **s)


@pytest.mark.parametrize("code,hd,captured", [("e4m3", 64, False), ("e4m3", 128, True), ("i8", 64, True)])
def test_a_serving_step_with_drafts(gpu_lib, code, hd, captured):
    """Prompts, then steps of a token and drafts a sequence, ending and new requests between them, eagerly and as one captured
    graph: what each step leaves in the tables, the cache and the outputs is what the parts' definitions give."""
    n, vocab, page, block = 9, 40, 16, 16
    S = Step(n, 4, 2, hd, page, block, code, vocab, 120, 30, 400, 7)
    stream = torch.cuda.Stream()
    if captured:
        S.run(torch.cuda.current_stream())  # (no sequence has rows: warms torch's own kernels up)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=stream):
            S.run(torch.cuda.current_stream())
    r = random.Random(4)
    history = [[] for _ in range(n)]        # tokens in the cache
    left = [r.randrange(vocab) for _ in range(n)]
    for step in range(14):
        new, rows = [], []
        for b in range(n):
            if step == 0 or (not history[b] and r.random() < 0.5):
                fed = [r.randrange(vocab) for _ in range(r.choice([1, 15, 16, 17, 40]))]
            elif history[b] and r.random() < 0.08:
                new.append(-1)
                history[b] = []
                continue
            elif r.random() < 0.1:
                fed = []
            else:
                fed = [left[b]] + [r.randrange(vocab) for _ in range(r.choice([0, 1, 3, 4]))]
            new.append(len(fed))
            rows.append((b, fed))
        flat = [t for _, fed in rows for t in fed]
        S.new.copy_(ints(new))
        S.tokens.copy_(ints(flat + [0] * (S.rows - len(flat))))
        S.accept.copy_(torch.tensor([r.random() ** 3 for _ in range(S.rows)], device="cuda"))
        S.pick.copy_(torch.tensor([r.random() for _ in range(n)], device="cuda"))
        before = S.kv.tolist()
        torch.cuda.synchronize()
        if captured:
            gr.replay()
        else:
            S.run(torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert [s.item() for s in S.status] == [0, 0, 0, 0]
        cu, out, acc, kv, held, table = S.cu.tolist(), S.out.tolist(), S.acc.tolist(), S.kv.tolist(), S.held.tolist(), S.table.tolist()
        assert len({p for b in range(n) for p in table[b][:held[b]]} | set(S.stack.tolist()[:S.count.item()])) == 120
        want = verify_plain(S.tokens.tolist(), S.probs.double().cpu().numpy(), None, cu, S.accept.tolist(), S.pick.tolist(), vocab)
        at = 0
        for b in range(n):
            fed = new[b] if new[b] > 0 else 0
            assert cu[b + 1] - cu[b] == fed
            if new[b] < 0:
                assert kv[b] == held[b] == 0
                continue
            assert (out[cu[b]:cu[b + 1]], acc[b]) == want[b]
            if not fed:
                continue
            toks = flat[at:at + fed]
            at += fed
            assert S.positions.tolist()[cu[b]:cu[b + 1]] == list(range(before[b], before[b] + fed))
            # attention of these rows over the whole history, from the tokens: within the cache's roundings
            full = history[b] + toks
            x = S.embed[torch.tensor(full, device="cuda")]
            pos = torch.arange(len(full), device="cuda")
            k, _ = turned(x[:, 4:6], S.wk, 1e-5, pos, S.freq, True)
            q, _ = turned(x[-fed:, :4], None, 0, pos[-fed:], S.freq, True)
            sc = torch.einsum("qkgd,nkd->kgqn", q.reshape(fed, 2, 2, hd), k) * hd ** -0.5
            sc = torch.where(pos[None, :] <= pos[-fed:, None], sc, -math.inf).softmax(-1)
            o = torch.einsum("kgqn,nkd->qkgd", sc, x[:, 6:].double()).reshape(fed, 4, hd)
            far = (S.o[cu[b]:cu[b + 1]].double() - o).norm() / o.norm()
            # e4m3: values off by 2^-4 of themselves at most, a third of that on average, and scores by as much; whole numbers
            # by a step of amax / 64, twice that where a block grew
            assert float(far) < 0.15, float(far)
            history[b] = full[:len(full) - (fed - 1 - acc[b])] if fed > 1 else full
            assert kv[b] == len(history[b])
            left[b] = out[cu[b] + acc[b]]
