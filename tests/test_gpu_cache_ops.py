"""The operators around the paged cache on the GPU, against their formulas in 64 bits: per-head norm + rotation, the
append of ragged chunks, and attention of ragged chunks over the pages, at the sizes, masks and layouts where they can
go wrong, and a run of the three together."""
import math

import numpy as np
import pytest
import torch

from decode_llama_step_gb300 import dls

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -24  # half a step of fp32, relative


def half_step(t):
    return torch.finfo(t).eps / 2


def rounding(want, t):
    """Half a step of type t at `want`: relative, and the fixed step below the normal range."""
    return half_step(t) * want.abs() + torch.finfo(t).tiny * half_step(t)


# ---- formulas in 64 bits ----------------------------------------------------------------------

def turned(x, norm, eps, pos, freq, halves):
    """(value, length of the element's pair) of normed and rotated heads."""
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


def close_turned(got, x, norm, eps, pos, freq, halves):
    # fp32 steps on the way: the sum of squares (16 in a lane, 4 joins, halved by the root), rsqrt, two products, the
    # rotation's two products and sum, sincospi (2 ulp) and the angle (2^-25 of a half turn = 1.6 * 2^-24 radians,
    # and 2^-53 * inv_freq * position, the double's own rounding, both here and in the formula): 32 half steps of
    # the pair's length
    want, size = turned(x, norm, eps, pos, freq, halves)
    far = 0.0 if freq is None or not len(freq) else float(pos.abs().max()) * float(np.abs(freq).max()) * 2.0 ** -51
    err = (got.double() - want).abs()
    lim = rounding(want, got.dtype) * (1 + 2.0 ** -10) + (32 * F32 + far) * size
    assert bool((err <= lim).all()), float((err / lim).max())


# ---- norm and rotation --------------------------------------------------------------------------

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.mark.parametrize("n,heads,kvh,hd,rot,pairing,tin,tout,norm", [
    (1, 4, 2, 64, 64, "adjacent", "f32", "f32", True),
    (1, 1, 0, 16, 16, "halves", "f32", "f32", True),
    (3, 0, 5, 32, 16, "adjacent", "f16", "f32", True),
    (7, 5, 3, 48, 32, "halves", "bf16", "bf16", True),
    (33, 32, 8, 128, 128, "adjacent", "f32", "f16", False),
    (65, 14, 2, 80, 80, "halves", "f16", "f16", True),
    (129, 12, 6, 96, 0, "adjacent", "bf16", "f32", True),
    (31, 9, 1, 112, 64, "adjacent", "bf16", "f16", False),
    (1000, 64, 8, 128, 128, "halves", "bf16", "bf16", True),
    (17, 3, 3, 208, 192, "adjacent", "f32", "bf16", True),
    (5000, 3, 1, 256, 256, "halves", "f16", "f32", True),
])
def test_qk_norm_rope(gpu_lib, n, heads, kvh, hd, rot, pairing, tin, tout, norm):
    g = torch.Generator(device="cuda").manual_seed(n + hd)
    qk = (torch.randn(n, heads + kvh + 1, hd, generator=g, device="cuda") * 1.5).to(TYPES[tin])
    q, k = qk[:, :heads], qk[:, heads:heads + kvh]       # views with a token stride of their own
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (n,), generator=g, device="cuda").to(torch.int32)
    pos[0] = 0 if n < 3 else -1
    pos[n // 2:] = pos[n // 2:] % 8192
    freq = dls.rope_inv_freq(rot, 10000.0) if rot else None
    wq, wk = ((torch.randn(hd, generator=g, device="cuda") if norm else None) for _ in range(2))
    qo = torch.full((n, heads + 2, hd), 7.0, device="cuda", dtype=TYPES[tout])
    ko = torch.full((n, kvh, hd), 7.0, device="cuda", dtype=TYPES[tout])
    dls.qk_norm_rope(q if heads else None, k if kvh else None, pos, freq, qo[:, 1:1 + heads] if heads else None,
                     ko if kvh else None, q_norm=wq, k_norm=wk, eps=1e-5, pairing=pairing)
    torch.cuda.synchronize()
    # positions over the whole int32 range: the formula's own angle is 2^-53 * 2^31 off
    if heads:
        close_turned(qo[:, 1:1 + heads], q, wq, 1e-5, pos, freq, pairing == "halves")
    if kvh:
        close_turned(ko, k, wk, 1e-5, pos, freq, pairing == "halves")
    assert bool((qo[:, 0] == 7).all()) and bool((qo[:, heads + 1] == 7).all())  # heads beside the output


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
def test_qk_norm_rope_in_place_and_turned_back(gpu_lib, pairing):
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(300, 6, 128, generator=g, device="cuda")
    pos = torch.randint(0, 1 << 20, (300,), generator=g, device="cuda", dtype=torch.int32)
    freq = dls.rope_inv_freq(128, 500000.0)
    want, away, x = q.clone(), torch.empty_like(q), q.clone()
    dls.qk_norm_rope(x, None, pos, freq, away, None, pairing=pairing)
    dls.qk_norm_rope(x, None, pos, freq, x, None, pairing=pairing)
    assert torch.equal(x, away)
    dls.qk_norm_rope(x, None, pos, -freq, x, None, pairing=pairing)  # the inverse turn
    assert float((x - want).abs().max()) <= 2 * 32 * F32 * float(want.abs().max()) * math.sqrt(2)


def test_qk_norm_rope_rows_of_zeros_and_infinities_stay_apart(gpu_lib):
    q = torch.randn(4, 3, 64, device="cuda")
    q[1, 1] = 0.0
    q[2, 0, 5] = math.inf
    out = torch.empty_like(q)
    w = torch.ones(64, device="cuda")
    pos = torch.arange(4, device="cuda", dtype=torch.int32)
    freq = dls.rope_inv_freq(64, 10000.0)
    dls.qk_norm_rope(q, None, pos, freq, out, None, q_norm=w, eps=1e-5)
    assert bool((out[1, 1] == 0).all())
    ok = torch.ones(4, 3, dtype=torch.bool, device="cuda")
    ok[2, 0] = False
    assert bool(out[ok].isfinite().all())
    want, size = turned(q, w, 1e-5, pos, freq, False)
    assert bool(((out.double() - want).abs()[ok] <= (33 * F32 * size)[ok] + 1e-38).all())


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
def test_negative_frequencies_are_the_turn_of_negative_positions(gpu_lib, pairing):
    """f p is the same angle as (-f)(-p), bit by bit, for the slowest frequency at the farthest positions too."""
    g = torch.Generator(device="cuda").manual_seed(17)
    q = torch.randn(2000, 2, 128, generator=g, device="cuda")
    pos = torch.randint(-(1 << 31) + 1, (1 << 31) - 1, (2000,), generator=g, device="cuda").to(torch.int32)
    freq = dls.rope_inv_freq(128, 500000.0)
    a, b = torch.empty_like(q), torch.empty_like(q)
    dls.qk_norm_rope(q, None, pos, freq, a, None, pairing=pairing)
    dls.qk_norm_rope(q, None, -pos, -freq, b, None, pairing=pairing)
    assert torch.equal(a, b)


# ---- a paged batch ----------------------------------------------------------------------------

class Batch:
    """Ragged lengths [(new, cached with the new)], pages in random order, everything no call may use poisoned."""

    def __init__(self, lengths, kvh, hd, page, typ, seed, first=0, pad=0, spare=2, extra=1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g, self.lengths, self.page, self.typ, self.kvh, self.hd = g, lengths, page, typ, kvh, hd
        counts = [-(-kl // page) for _, kl in lengths]
        self.n_pages = sum(counts) + spare
        order = torch.randperm(self.n_pages, generator=g, device="cuda").tolist()
        self.max_pages = max(counts + [1]) + extra
        self.table = torch.full((len(lengths), self.max_pages), -1, dtype=torch.int32)
        self.table[:, -1] = 1 << 30
        at, starts = 0, [first]
        for b, c in enumerate(counts):
            self.table[b, :c] = torch.tensor(order[at:at + c], dtype=torch.int32)
            at += c
            starts.append(starts[-1] + lengths[b][0])
        self.starts, self.rows = starts, starts[-1] + pad
        self.table = self.table.cuda()
        self.cu_q = torch.tensor(starts, dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor([kl for _, kl in lengths], dtype=torch.int32, device="cuda")
        self.k = torch.full((self.n_pages, kvh, page, hd), math.nan, dtype=typ, device="cuda")
        self.v = torch.full_like(self.k, math.nan)

    def slots(self, b, lo, hi):
        pos = torch.arange(lo, hi, device="cuda")
        return self.table[b].long()[pos // self.page], pos % self.page

    def fill(self, std=1.0):
        for b, (_, kl) in enumerate(self.lengths):
            p, s = self.slots(b, 0, kl)
            self.k[p, :, s] = (torch.randn(kl, self.kvh, self.hd, generator=self.g, device="cuda") * std).to(self.typ)
            self.v[p, :, s] = torch.randn(kl, self.kvh, self.hd, generator=self.g, device="cuda").to(self.typ)


def workspace(hd):
    return torch.zeros(dls.attention_chunk_workspace_bytes(hd), dtype=torch.uint8, device="cuda")


# ---- append -------------------------------------------------------------------------------------

@pytest.mark.parametrize("lengths,heads,kvh,hd,rot,page,tin,typ,norm,with_q,pairing,first,pad", [
    ([(1, 1)], 4, 2, 64, 64, 64, "f32", "f16", False, True, "adjacent", 0, 0),
    ([(1, 17), (1, 16), (1, 1)], 32, 8, 128, 128, 16, "f32", "f16", True, True, "adjacent", 0, 1),
    ([(16, 16), (0, 9), (15, 40), (33, 33)], 6, 3, 80, 80, 16, "f16", "f16", False, False, "halves", 2, 5),
    ([(5, 300), (257, 257), (64, 128)], 14, 2, 128, 64, 64, "bf16", "bf16", True, True, "halves", 0, 3),
    ([(3, 2000)] * 40 + [(0, 0)] * 3 + [(7, 1025)] * 30, 3, 1, 96, 96, 32, "bf16", "f16", False, True, "adjacent", 1, 2),
    ([(1, 5)] * 1100, 1, 1, 16, 16, 16, "f32", "bf16", False, False, "adjacent", 0, 0),
    ([(700, 1700)], 2, 2, 256, 0, 256, "f16", "bf16", True, True, "halves", 0, 0),
])
def test_kv_append(gpu_lib, lengths, heads, kvh, hd, rot, page, tin, typ, norm, with_q, pairing, first, pad):
    B = Batch(lengths, kvh, hd, page, TYPES[typ], 11, first, pad)
    x = (torch.randn(B.rows, heads + 2 * kvh, hd, generator=B.g, device="cuda") * 1.5).to(TYPES[tin])
    inside = torch.zeros(B.rows, dtype=torch.bool, device="cuda")
    inside[first:B.starts[-1]] = True
    x[~inside] = math.nan                           # padding may hold anything
    q, k, v = x[:, :heads], x[:, heads:heads + kvh], x[:, heads + kvh:]
    wq, wk = ((torch.randn(hd, generator=B.g, device="cuda") if norm else None) for _ in range(2))
    qo = torch.full((B.rows, heads, hd), 7.0, dtype=B.typ, device="cuda") if with_q else None
    freq = dls.rope_inv_freq(rot, 500000.0) if rot else None
    status = torch.full((1,), 99, dtype=torch.int32, device="cuda")
    before_k, before_v = B.k.clone(), B.v.clone()
    dls.kv_append(k, v, B.k, B.v, B.table, B.cu_q, B.kv_len, freq, q=q if with_q else None, q_out=qo, q_norm=wq if with_q else None,
                  k_norm=wk, eps=1e-6, pairing=pairing, status=status)
    dls.attention_status(status)
    written = torch.zeros(B.n_pages, page, dtype=torch.bool, device="cuda")
    for b, (ql, kl) in enumerate(lengths):
        r, pos = slice(B.starts[b], B.starts[b] + ql), torch.arange(kl - ql, kl, device="cuda")
        if not ql or (b > 8 and b < len(lengths) - 3):  # long batches: the ends
            p, s = B.slots(b, kl - ql, kl)
            written[p, s] = True
            continue
        p, s = B.slots(b, kl - ql, kl)
        written[p, s] = True
        close_turned(B.k[p, :, s], k[r], wk, 1e-6, pos, freq, pairing == "halves")
        assert torch.equal(B.v[p, :, s], v[r].to(B.typ))
        if with_q:
            close_turned(qo[r], q[r], wq, 1e-6, pos, freq, pairing == "halves")
    for now, was in ((B.k, before_k), (B.v, before_v)):  # no other slot of any page
        left = ~written[:, None, :, None].expand_as(now)
        assert torch.equal(now[left].view(torch.int16), was[left].view(torch.int16))
    if with_q:
        assert bool((qo[~inside] == 7).all())


def test_kv_append_flags_what_does_not_fit(gpu_lib):
    def run(cu, kl, table, rows=8, pages=4):
        k = torch.ones(rows, 2, 32, device="cuda")
        kp = torch.zeros(pages, 2, 16, 32, dtype=torch.float16, device="cuda")
        vp = torch.zeros_like(kp)
        qo = torch.zeros(rows, 2, 32, dtype=torch.float16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        dls.kv_append(k, k, kp, vp, torch.tensor(table, dtype=torch.int32, device="cuda"),
                      torch.tensor(cu, dtype=torch.int32, device="cuda"), torch.tensor(kl, dtype=torch.int32, device="cuda"),
                      None, q=k, q_out=qo, status=status)
        torch.cuda.synchronize()
        return int(status), float(kp.sum()) / 64, float(qo.sum()) / 64

    assert run([0, 8], [8], [[0, 1]]) == (0, 8, 8)
    assert run([0, 8], [20], [[0, 1]]) == (0, 8, 8)
    assert run([0, 8], [20], [[0, -1]]) == (1, 4, 8)      # positions 16..19 have no page: q is still there
    assert run([0, 8], [20], [[4, 1]]) == (1, 4, 8)       # a page outside the pool
    assert run([0, 8], [33], [[0, 1]]) == (4, 0, 0)       # longer than the page table
    assert run([0, 8], [-1], [[0, 1]]) == (4, 0, 0)
    assert run([0, 8], [7], [[0, 1]])[0] == 4             # the first token would stand at -1
    assert run([0, 9], [9], [[0, 1]]) == (4, 0, 0)        # more rows than there are
    assert run([0, 5, 3], [5, 3], [[0, 1], [2, 3]])[0] == 4
    assert run([8, 0], [8], [[0, 1]])[0] == 4
    assert run([-1, 4], [8], [[0, 1]])[0] == 4
    with pytest.raises(dls.DlsError):
        dls.attention_status(torch.full((1,), 4, dtype=torch.int32, device="cuda"))


def append_where(cu, kl, n_tokens, n_seqs, room):
    """{(sequence, position): row} of the rows that an append with these lengths may write: rows of sequences that fit."""
    return {(b, kl[b] - cu[b + 1] + t): t for b in range(n_seqs)
            if 0 <= cu[b] <= cu[b + 1] <= n_tokens and cu[b + 1] - cu[b] <= kl[b] <= room for t in range(cu[b], cu[b + 1])}


@pytest.mark.parametrize("cu,kl", [
    ([0, 8, 0, 1], [8, 0, 32]), ([0, 6, 2, 3], [6, 4, 32]), ([0, 8, 0, 1, 0], [8, 0, 32, 5]), ([8, 0, 8, 0], [8, 8, 8]),
    ([3, 1, 2, 0, 8], [32, 32, 32, 32]), ([0, 4, 4, 2, 8, 1, 5], [4, 0, 9, 17, 1, 32]), ([0, 8] * 40, [31, 32] * 39 + [32]),
])
def test_kv_append_where_cu_q_decreases(gpu_lib, cu, kl):
    """No row goes to a slot that is not its own, and none looks past its sequence's row of the page table: the rows of the
    table around the batch name pages of the pool too, which stay as they are."""
    n, page, rows, most = len(kl), 16, 8, 2
    pages = 2 * n + 8
    table = torch.arange(pages, dtype=torch.int32, device="cuda").flip(0).reshape(-1, most).contiguous()  # 2 spare rows at each end
    k = torch.arange(1.0, rows + 1, device="cuda")[:, None, None].expand(rows, 2, 32).contiguous()
    pools = [torch.zeros(pages, 2, page, 32, dtype=torch.float16, device="cuda") for _ in range(2)]
    qo = torch.zeros(rows, 2, 32, dtype=torch.float16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dls.kv_append(k, -k, *pools, table[2:2 + n], torch.tensor(cu, dtype=torch.int32, device="cuda"),
                  torch.tensor(kl, dtype=torch.int32, device="cuda"), None, q=2 * k, q_out=qo, status=status)
    torch.cuda.synchronize()
    assert int(status) == 4
    own = append_where(cu, kl, rows, n, most * page)
    for pool, sign in zip(pools, (1.0, -1.0)):
        allowed = torch.zeros(pages, page)
        for (b, pos), t in own.items():
            allowed[int(table[2 + b, pos // page]), pos % page] = sign * (t + 1)
        got = pool.float().cpu()
        assert torch.equal(got, got[:, :1, :, :1].expand_as(got))  # whole rows, every head
        got = got[:, 0, :, 0]
        assert bool(((got == 0) | (got == allowed)).all()), (got != 0).nonzero().tolist()
    for t in range(rows):
        x = qo[t].float().unique().tolist()
        assert x == [0.0] or (x == [2.0 * (t + 1)] and t in own.values())


@pytest.mark.parametrize("short", [0, 1, 4, 7])
def test_kv_append_skips_a_sequence_shorter_than_its_chunk(gpu_lib, short):
    """kv_len below the chunk's length is flagged, and no row of that sequence reaches a page or q_out; its neighbours do."""
    cu, kl, rows, pages = [0, 3, 11, 13], [20, short, 2], 13, 6
    table = torch.arange(pages, dtype=torch.int32, device="cuda").reshape(3, 2)
    k = torch.arange(1.0, rows + 1, device="cuda")[:, None, None].expand(rows, 2, 32).contiguous()
    pools = [torch.zeros(pages, 2, 16, 32, dtype=torch.float16, device="cuda") for _ in range(2)]
    qo = torch.zeros(rows, 2, 32, dtype=torch.float16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dls.kv_append(k, -k, *pools, table, torch.tensor(cu, dtype=torch.int32, device="cuda"),
                  torch.tensor(kl, dtype=torch.int32, device="cuda"), None, q=2 * k, q_out=qo, status=status)
    torch.cuda.synchronize()
    assert int(status) == 4
    want = torch.zeros(pages, 16)
    for (b, pos), t in append_where(cu, kl, rows, 3, 32).items():
        want[2 * b + pos // 16, pos % 16] = t + 1
    assert int((want != 0).sum()) == 5
    for pool, sign in zip(pools, (1.0, -1.0)):
        assert torch.equal(pool.float().cpu(), (sign * want)[:, None, :, None].expand(pages, 2, 16, 32))
    assert qo[:, 0, 0].tolist() == [2.0, 4.0, 6.0] + [0.0] * 8 + [24.0, 26.0]


@pytest.mark.parametrize("pairing,rot", [("adjacent", 128), ("halves", 96)])
def test_kv_append_turns_q_in_place(gpu_lib, pairing, rot):
    """q_out = q: the bits of a call with an output of its own, rows outside the sequences untouched."""
    B = Batch([(1, 40), (300, 300), (33, 65)], 2, 128, 32, torch.bfloat16, 12, first=2, pad=3)
    x = (torch.randn(B.rows, 8 + 4, 128, generator=B.g, device="cuda") * 1.5).to(B.typ)
    w = [1 + 0.1 * torch.randn(128, generator=B.g, device="cuda") for _ in range(2)]
    freq, away = dls.rope_inv_freq(rot, 500000.0), torch.full((B.rows, 8, 128), 7.0, dtype=B.typ, device="cuda")
    args = B.k, B.v, B.table, B.cu_q, B.kv_len, freq
    dls.kv_append(x[:, 8:10], x[:, 10:], *args, q=x[:, :8], q_out=away, q_norm=w[0], k_norm=w[1], pairing=pairing)
    k, v, y = B.k.clone(), B.v.clone(), x.clone()
    dls.kv_append(y[:, 8:10], y[:, 10:], *args, q=y[:, :8], q_out=y[:, :8], q_norm=w[0], k_norm=w[1], pairing=pairing)
    inside = slice(B.starts[0], B.starts[-1])
    assert torch.equal(y[inside, :8], away[inside])
    y[inside, :8] = x[inside, :8]
    assert torch.equal(y, x)  # padding rows, k and v
    for now, was in ((B.k, k), (B.v, v)):
        assert torch.equal(now.view(torch.int16), was.view(torch.int16))


# ---- attention -----------------------------------------------------------------------------------

def attend64(B, q, heads, scale, causal, window):
    """(o, lse, sum of weights * |v|, largest scale * sum |q k|) in 64 bits; 0 and -inf where a row has no key."""
    o = torch.zeros(B.rows, heads, B.hd, dtype=torch.float64, device="cuda")
    lse = torch.full((B.rows, heads), -math.inf, dtype=torch.float64, device="cuda")
    mag, dot = torch.zeros_like(o), torch.zeros_like(lse)
    group = heads // B.kvh
    for b, (ql, kl) in enumerate(B.lengths):
        if not ql or not kl:
            continue
        p, s = B.slots(b, 0, kl)
        r = slice(B.starts[b], B.starts[b] + ql)
        pos = torch.arange(kl - ql, kl, device="cuda")[:, None]
        key = torch.arange(kl, device="cuda")[None]
        seen = (key <= pos) if causal else torch.ones(ql, kl, dtype=torch.bool, device="cuda")
        if window:
            seen = seen & (pos - key < window)
        k, v = B.k[p, :, s].double(), B.v[p, :, s].double()       # NaN where a test freed a page
        dead = ~seen.any(0)
        k[dead], v[dead] = 0.0, 0.0
        for h in range(heads):
            x = q[r, h].double()
            sc = (x @ k[:, h // group].T) * scale
            sc = torch.where(seen, sc, -math.inf)
            m = sc.amax(-1, keepdim=True)
            e = torch.where(seen, torch.exp(sc - torch.where(m.isfinite(), m, 0.0)), 0.0)
            tot = e.sum(-1, keepdim=True)
            w = e / torch.where(tot > 0, tot, 1.0)
            o[r, h], mag[r, h] = w @ v[:, h // group], w @ v[:, h // group].abs()
            lse[r, h] = (m + tot.log())[:, 0]
            dot[r, h] = torch.where(seen, (x.abs() @ k[:, h // group].abs().T) * scale, 0.0).amax(-1)
    return o, lse, mag, dot


def close_attend(B, got, lse, want, heads):
    o, wl, mag, dot = want
    # a score: hd products summed in fp32 (each step may truncate: 2^-23 of the sum of magnitudes), scaled, its
    # exponent rounded: at most (hd + 8) 2^-23 of scale * sum |q k| plus the exponential's own 2^-21
    ds = (B.hd + 8) * 2.0 ** -23 * dot + 2.0 ** -21
    u = half_step(B.typ)
    keys = max([kl for _, kl in B.lengths] + [1])
    # weights rounded to the cache's type (u each, relative; below fp16's normal range half of 2^-24, against a largest
    # weight of at least 2^7), scores off by ds in weight and in the sum, sums of `keys` terms in fp32, the output's rounding
    lim = (u * (1 + 2.0 ** -6) + 2 * ds[..., None] + 2 * (keys / 64 + 64) * 2.0 ** -23) * mag + rounding(o, B.typ) * (1 + 2.0 ** -6)
    if B.typ == torch.float16:
        lim = lim + keys * 2.0 ** -32 * 6.0
    inside = torch.zeros(B.rows, dtype=torch.bool, device="cuda")
    inside[B.starts[0]:B.starts[-1]] = True
    err = (got.double() - o).abs()
    assert bool((err <= lim)[inside].all()), float((err / lim)[inside].nan_to_num(math.inf).max())
    if lse is not None:
        a, w = lse.double()[inside], wl[inside]
        assert torch.equal(a == -math.inf, w == -math.inf)
        e = (a - w).abs().nan_to_num(0.0)
        assert not bool(a.isnan().any())
        assert bool((e <= ds[inside] + (keys / 64 + 64) * 2.0 ** -23 + 4 * F32 * w.abs().nan_to_num(0.0, 0.0, 0.0)).all()), float(e.max())


def check_attend(lengths, heads, kvh, hd, page, typ, causal=True, window=0, first=0, pad=0, scale=0.0, with_lse=True, seed=5,
                 qstd=1.5, ws=None, stream=None):
    B = Batch(lengths, kvh, hd, page, TYPES[typ], seed, first, pad)
    B.fill()
    wide = torch.full((B.rows, heads + 1, hd), math.nan, dtype=B.typ, device="cuda")
    q = wide[:, :heads]
    q[first:B.starts[-1]] = (torch.randn(B.starts[-1] - first, heads, hd, generator=B.g, device="cuda") * qstd).to(B.typ)
    want = attend64(B, q, heads, scale or hd ** -0.5, causal, window)
    if window:  # pages wholly before every window are gone: no entry, NaN inside; slots before it too
        for b, (ql, kl) in enumerate(lengths):
            gone = min(max(0, kl - ql - window + 1), kl)
            if gone:
                p, s = B.slots(b, 0, gone)
                B.k[p, :, s] = math.nan
                B.v[p, :, s] = math.nan
                B.table[b, :gone // page] = -1
    out = torch.full((B.rows, heads + 3, hd), 7.0, dtype=B.typ, device="cuda")
    o = out[:, 2:2 + heads]
    lse = torch.full((B.rows, heads), 7.0, device="cuda") if with_lse else None
    status = torch.full((1,), 99, dtype=torch.int32, device="cuda")
    ws = workspace(hd) if ws is None else ws
    torch.cuda.synchronize()
    dls.attention_chunk(q, B.k, B.v, B.table, B.cu_q, B.kv_len, o, ws, lse=lse, scale=scale, causal=causal, window=window,
                        status=status, stream=stream)
    dls.attention_status(status, stream)
    close_attend(B, o, lse, want, heads)
    inside = torch.zeros(B.rows, dtype=torch.bool, device="cuda")
    inside[first:B.starts[-1]] = True
    assert bool((out[~inside] == 7).all()) and bool((out[:, :2] == 7).all()) and bool((out[:, 2 + heads:] == 7).all())
    if with_lse:
        assert bool((lse[~inside] == 7).all())
    # the same call again: the same bits, on the workspace that the first call left
    again = torch.full_like(out, 7.0)
    dls.attention_chunk(q, B.k, B.v, B.table, B.cu_q, B.kv_len, again[:, 2:2 + heads], ws, scale=scale, causal=causal,
                        window=window, stream=stream)
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
@pytest.mark.parametrize("heads,kvh,hd,page,typ", [(4, 2, 64, 64, "f16"), (8, 1, 128, 32, "bf16"), (6, 2, 80, 16, "f16")])
def test_attention_chunk_lengths(gpu_lib, lengths, heads, kvh, hd, page, typ):
    check_attend(lengths, heads, kvh, hd, page, typ, first=2, pad=3)


@pytest.mark.parametrize("heads,kvh", [(1, 1), (5, 5), (4, 2), (9, 3), (32, 8), (5, 1), (7, 1), (16, 1), (31, 1), (33, 1), (128, 2), (128, 1)])
def test_attention_chunk_head_groups(gpu_lib, heads, kvh):
    check_attend([(1, 200), (3, 131), (70, 150), (1, 7)], heads, kvh, 64, 64, "bf16")


@pytest.mark.parametrize("hd", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("page,typ", [(16, "f16"), (32, "bf16"), (64, "f16"), (128, "bf16"), (256, "f16")])
def test_attention_chunk_head_dims_and_pages(gpu_lib, hd, page, typ):
    check_attend([(1, 300), (40, 260), (7, 7)], 6, 3, hd, page, typ)


@pytest.mark.parametrize("window", [1, 2, 7, 127, 128, 129, 500])
@pytest.mark.parametrize("hd,page", [(64, 16), (128, 64)])
def test_attention_chunk_windows(gpu_lib, window, hd, page):
    check_attend([(1, 1000), (300, 300), (130, 900), (5, 129), (1, 1)], 8, 2, hd, page, "f16", window=window)


def test_attention_chunk_rows_without_keys(gpu_lib):
    # chunks longer than the cached length: the first rows have no key; no keys at all
    check_attend([(5, 3), (4, 0), (300, 10), (1, 0), (2, 2), (140, 130)], 4, 2, 64, 32, "bf16")
    check_attend([(5, 3), (4, 0), (300, 10)], 4, 2, 128, 32, "f16", window=2)
    check_attend([(5, 3), (4, 0), (1, 1)], 4, 2, 128, 32, "f16", causal=False)


@pytest.mark.parametrize("hd,window", [(64, 0), (128, 2)])
def test_attention_chunk_runs_of_rows_without_keys(gpu_lib, hd, window):
    """Many tiles in a row without any key, or with keys for one half of their rows only, between ordinary ones: the
    warps that have nothing to wait for must not get ahead of those that have."""
    lengths = ([(2, 0)] * 5 + [(5, 40), (1, 1), (0, 7), (3, 0)] * 2 + [(140, 60), (7, 0), (200, 30)]) * 16
    check_attend(lengths, 2, 2, hd, 16, "f16", window=window)


def test_attention_chunk_every_key(gpu_lib):
    check_attend([(5, 700), (130, 257), (300, 40), (1, 1)], 8, 4, 128, 64, "bf16", causal=False)
    check_attend([(64, 64)] * 3, 3, 3, 64, 16, "f16", causal=False)


@pytest.mark.parametrize("scale", [1e-3, 0.5, 4.0])
def test_attention_chunk_scales(gpu_lib, scale):
    # flat to peaked: at 4 a row's weight lies on one key
    check_attend([(1, 777), (150, 400)], 4, 2, 64, 64, "bf16", scale=scale)


def test_attention_chunk_long_cache_of_one_token(gpu_lib):
    check_attend([(1, 20011)], 8, 2, 128, 64, "bf16")
    check_attend([(1, 9000), (1, 33), (5, 8200), (1, 16384)], 16, 2, 64, 128, "f16")


def test_attention_chunk_many_sequences(gpu_lib):
    check_attend([(1 + b % 3, 1 + (37 * b) % 90 + b % 3) for b in range(600)], 2, 1, 64, 16, "f16")


def test_attention_chunk_a_whole_prompt(gpu_lib):
    check_attend([(1500, 1500)], 8, 2, 128, 64, "bf16")
    check_attend([(700, 1900), (1, 1200), (900, 900)], 8, 8, 64, 64, "f16")


def test_attention_chunk_rising_scores(gpu_lib):
    """Keys whose scores grow along the sequence: the running maximum moves at every tile, by little and by much."""
    for step in (0.02, 0.5):
        B = Batch([(3, 1500), (200, 1200)], 2, 64, 64, torch.float16, 9)
        B.fill()
        for b, (_, kl) in enumerate(B.lengths):
            p, s = B.slots(b, 0, kl)
            B.k[p, :, s, 0] = (torch.arange(kl, device="cuda", dtype=torch.float32) * step * 0.1)[:, None].half()
        q = torch.randn(B.rows, 4, 64, generator=B.g, device="cuda").half()
        q[..., 0] = 8.0
        o, lse = torch.empty_like(q), torch.empty(B.rows, 4, device="cuda")
        want = attend64(B, q, 4, 0.125, True, 0)
        dls.attention_chunk(q, B.k, B.v, B.table, B.cu_q, B.kv_len, o, workspace(64), lse=lse)
        close_attend(B, o, lse, want, 4)


def test_attention_chunk_shared_pages(gpu_lib):
    """Two sequences over the same prefix pages give what each gives alone."""
    B = Batch([(3, 200), (3, 200)], 2, 64, 32, torch.bfloat16, 4)
    B.fill()
    B.table[1, :4] = B.table[0, :4]
    q = torch.randn(B.rows, 4, 64, generator=B.g, device="cuda").to(B.typ)
    o, ws = torch.empty_like(q), workspace(64)
    want = attend64(B, q, 4, 0.125, True, 0)
    dls.attention_chunk(q, B.k, B.v, B.table, B.cu_q, B.kv_len, o, ws)
    close_attend(B, o, None, want, 4)


def test_attention_chunk_flags_what_does_not_fit(gpu_lib):
    def run(cu, kl, table, rows=8, pages=4):
        q = torch.ones(rows, 2, 64, dtype=torch.float16, device="cuda")
        kp = torch.ones(pages, 2, 16, 64, dtype=torch.float16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o, ws = torch.full_like(q, 7.0), workspace(64)
        args = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (table, cu, kl)]
        dls.attention_chunk(q, kp, kp, *args, o, ws, status=status)
        torch.cuda.synchronize()
        got = int(status)
        # the workspace serves the next call
        args = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([[0, 1]], [0, 8], [20])]
        dls.attention_chunk(q, kp, kp, *args, o, ws, status=status)
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


def test_attention_chunk_one_workspace_for_all_shapes(gpu_lib):
    ws = workspace(128)
    check_attend([(1, 5000)], 8, 2, 128, 64, "bf16", ws=ws)
    check_attend([(300, 700)], 4, 2, 64, 16, "f16", ws=ws)
    check_attend([(3, 40), (1, 3000)], 32, 1, 128, 32, "f16", ws=ws)
    check_attend([(1, 5000)], 8, 2, 128, 64, "bf16", ws=ws)
    assert not bool(ws[:4096].any())  # its counters are zero again


def test_attention_chunk_on_a_stream_of_its_own(gpu_lib):
    s = torch.cuda.Stream()
    check_attend([(1, 900), (150, 300)], 8, 2, 128, 64, "bf16", stream=s)


def test_attention_chunk_in_place(gpu_lib):
    """o = q: tiles cut among CTAs, tiles of neighbours in one load, single tokens."""
    B = Batch([(1, 3000), (300, 900), (2, 700), (77, 77)], 2, 128, 64, torch.bfloat16, 6)
    B.fill()
    q = torch.randn(B.rows, 8, 128, generator=B.g, device="cuda").to(B.typ)
    o, ws = torch.empty_like(q), workspace(128)
    dls.attention_chunk(q, B.k, B.v, B.table, B.cu_q, B.kv_len, o, ws)
    for _ in range(5):
        x = q.clone()
        dls.attention_chunk(x, B.k, B.v, B.table, B.cu_q, B.kv_len, x, ws)
        assert torch.equal(x, o)


def test_empty_calls_clear_the_status(gpu_lib):
    B = Batch([(1, 20)], 2, 64, 16, torch.float16, 3)
    x = torch.zeros(0, 2, 64, dtype=torch.float16, device="cuda")
    status = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    dls.kv_append(x, x, B.k, B.v, B.table, B.cu_q, B.kv_len, None, status=status)
    assert status.item() == 0
    status.fill_(5)
    dls.attention_chunk(x, B.k, B.v, B.table, B.cu_q, B.kv_len, x, workspace(64), status=status)
    assert status.item() == 0


def test_attention_chunk_two_calls_at_once(gpu_lib):
    """Calls on two streams, a workspace each, give what each gives alone."""
    made = []
    for lengths, hd in (([(1, 2000)] * 5 + [(70, 200)], 128), ([(400, 1000), (1, 3000)], 64)):
        B = Batch(lengths, 2, hd, 32, torch.float16, 13)
        B.fill()
        q = torch.randn(B.rows, 8, hd, generator=B.g, device="cuda").half()
        made.append((B, q, torch.empty_like(q), torch.empty_like(q), workspace(hd), torch.cuda.Stream()))
    for B, q, alone, _, ws, _ in made:
        dls.attention_chunk(q, B.k, B.v, B.table, B.cu_q, B.kv_len, alone, ws)
        torch.cuda.synchronize()
    for _ in range(30):
        for B, q, _, o, ws, stream in made:
            dls.attention_chunk(q, B.k, B.v, B.table, B.cu_q, B.kv_len, o, ws, stream=stream)
    torch.cuda.synchronize()
    for _, _, alone, o, _, _ in made:
        assert torch.equal(o, alone)


def test_a_pool_of_more_than_two_to_the_31_elements(gpu_lib):
    """Append and attention over the last pages of pools whose element offsets pass 32 bits."""
    kvh, page, hd, heads, n_pages = 2, 128, 128, 8, 70000  # 2.3e9 elements, 4.6 GB each
    pools = [torch.empty(n_pages, kvh, page, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    B = Batch([(150, 150), (1, 300)], kvh, hd, page, torch.bfloat16, 31, extra=0)
    B.fill()
    own = (B.table >= 0) & (B.table < B.n_pages)
    used = B.table[own].long()
    moved = n_pages - 1 - 3 * used                       # far pages, in another order
    for pool, src in zip(pools, (B.k, B.v)):
        pool[moved] = src[used]
    table = torch.where(own, n_pages - 1 - 3 * B.table, B.table)
    x = torch.randn(B.rows, heads + 2 * kvh, hd, generator=B.g, device="cuda").to(B.typ)
    q = torch.empty(B.rows, heads, hd, dtype=B.typ, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    freq, ws, o = dls.rope_inv_freq(hd, 500000.0), workspace(hd), torch.empty_like(q)
    dls.kv_append(x[:, heads:heads + kvh], x[:, heads + kvh:], *pools, table, B.cu_q, B.kv_len, freq, q=x[:, :heads], q_out=q,
                  status=status)
    dls.attention_status(status)
    dls.attention_chunk(q, *pools, table, B.cu_q, B.kv_len, o, ws, status=status)
    dls.attention_status(status)
    dls.kv_append(x[:, heads:heads + kvh], x[:, heads + kvh:], B.k, B.v, B.table, B.cu_q, B.kv_len, freq)  # the small pool
    for pool, small in zip(pools, (B.k, B.v)):
        assert torch.equal(pool[moved].view(torch.int16), small[used].view(torch.int16))
    close_attend(B, o, None, attend64(B, q, heads, hd ** -0.5, True, 0), heads)


def test_attention_chunk_matches_single_token_attention(gpu_lib):
    """The same rows as dls_attention_decode (fp32 q and o) on the same pages."""
    B = Batch([(1, 513), (1, 64), (1, 1300)], 8, 128, 64, torch.float16, 8, extra=0)
    B.fill()
    q = torch.randn(3, 32, 128, generator=B.g, device="cuda").half()
    o = torch.empty_like(q)
    dls.attention_chunk(q, B.k, B.v, B.table, B.cu_q, B.kv_len, o, workspace(128))
    B.k.nan_to_num_(0.0)
    B.v.nan_to_num_(0.0)
    n = dls.attention_workspace_bytes(3, 32, 8, 128, 4)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    o32 = torch.empty(3, 32, 128, device="cuda")
    dls.attention_decode(q.float(), B.k, B.v, B.table, B.kv_len, o32, ws, n, 3, 32, 8, 128, 64, B.max_pages, 4)
    close_attend(B, o32.half(), None, attend64(B, q, 32, 128 ** -0.5, True, 0), 32)
    close_attend(B, o, None, attend64(B, q, 32, 128 ** -0.5, True, 0), 32)


@pytest.mark.parametrize("cu,kl", [
    ([0, 8, 0, 1], [8, 0, 32]), ([0, 6, 2, 3], [20, 4, 32]), ([0, 300, 290, 300], [320, 7, 40]), ([8, 0, 8, 0], [8, 9, 8]),
    ([3, 1, 2, 0, 8], [32, 32, 32, 32]), ([0, 400, 8, 300, 0, 50], [400, 3, 310, 5, 200]),
])
def test_attention_chunk_where_cu_q_decreases(gpu_lib, cu, kl):
    """Flagged; rows of no sequence stay as they are, and a row that one sequence alone holds has that sequence's result."""
    rows, heads, hd = max(cu) + 2, 4, 64
    # every sequence has keys for its length; those whose rows do not fit get none of the batch
    B = Batch([(0, n) for n in kl], 2, hd, 16, torch.float16, 40)
    B.fill()
    B.cu_q = torch.tensor(cu, dtype=torch.int32, device="cuda")
    q = torch.randn(rows, heads, hd, generator=B.g, device="cuda").half()
    o, status = torch.full_like(q, 7.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    dls.attention_chunk(q, B.k, B.v, B.table, B.cu_q, B.kv_len, o, workspace(hd), status=status)
    torch.cuda.synchronize()
    assert int(status) == 4
    held = [sum(a <= t < b for a, b in zip(cu, cu[1:])) for t in range(rows)]
    assert bool((o[torch.tensor(held) == 0] == 7).all())
    for b, (first, end) in enumerate(zip(cu, cu[1:])):
        if first >= end:
            continue
        B.lengths, B.starts, B.rows = [(0, 0)] * b + [(end - first, kl[b])], [first] * (b + 1) + [end], rows
        want = attend64(B, q, heads, hd ** -0.5, True, 0)
        alone = torch.tensor([t for t in range(first, end) if held[t] == 1], device="cuda", dtype=torch.long)
        got = want[0].to(B.typ)
        got[alone] = o[alone]
        close_attend(B, got, None, want, heads)


def border_keys(B, b, window):
    """Keys of sequence b at the borders of key tiles, their halves and pages, of the cache and of its rows' windows."""
    ql, kl = B.lengths[b]
    keys = {0, kl - 1} | {j + x for j in range(0, kl, 128) for x in (0, 15, 16, 63, 64, 127)}
    for pos in (kl - ql, kl - ql // 2 - 1, kl - 1):
        keys |= {pos - 1, pos, pos + 1} | ({pos - window, pos - window + 1, pos - window + 2} if window else set())
    return sorted(k for k in keys if 0 <= k < kl)


@pytest.mark.parametrize("lengths,heads,kvh,hd,page,typ,window", [
    ([(1, 20011)], 8, 2, 128, 64, "bf16", 0),
    ([(1, 9000), (1, 33), (5, 8200)], 16, 2, 64, 128, "f16", 0),
    ([(5, 4101), (1, 3661), (4, 1803), (60, 3001)], 16, 8, 128, 32, "f16", 0),
    ([(700, 1300)], 4, 2, 128, 64, "bf16", 0),
    ([(300, 1500), (1, 1200), (130, 900)], 8, 2, 64, 16, "f16", 333),
    ([(1, 2000), (200, 1000)], 4, 4, 80, 256, "bf16", 129),
])
def test_attention_chunk_each_value_row_counts_once(gpu_lib, lengths, heads, kvh, hd, page, typ, window):
    """V with one key for each column and zeros elsewhere: an output element is one key's weight times its value, held to a
    relative bound, so that a row of V that is lost, taken twice, zeroed or taken from another place shows whatever the
    length.  Flat scores keep every weight well above the roundings."""
    B = Batch(lengths, kvh, hd, page, TYPES[typ], 33)
    B.fill()
    q = (0.3 * torch.randn(B.rows, heads, hd, generator=B.g, device="cuda")).to(B.typ)
    o, lse, ws = torch.empty_like(q), torch.empty(B.rows, heads, device="cuda"), workspace(hd)
    keys = []
    for b in range(len(lengths)):
        border = torch.tensor(border_keys(B, b, window))
        keys.append(border[torch.randperm(len(border), generator=torch.Generator().manual_seed(b))])
    value = (32.0 + torch.arange(hd, device="cuda")).to(B.typ)  # (whole numbers up to 159: exact)
    for part in range(-(-max(len(k) for k in keys) // hd)):
        for b, (_, kl) in enumerate(lengths):
            p, s = B.slots(b, 0, kl)
            B.v[p, :, s] = 0.0
            some = keys[b][torch.arange(part * hd, part * hd + hd) % len(keys[b])].cuda()
            B.v[p[some], :, s[some], torch.arange(hd, device="cuda")] = value[:, None]
        dls.attention_chunk(q, B.k, B.v, B.table, B.cu_q, B.kv_len, o, ws, lse=lse, window=window)
        want = attend64(B, q, heads, hd ** -0.5, True, window)
        close_attend(B, o, lse, want, heads)
        assert torch.equal(o == 0, want[0] == 0)  # every key that a row sees, and no other


# ---- together -------------------------------------------------------------------------------------

def serve(B, calls, heads, x, wq, wk, freq, ws):
    """One layer's cache work for each ragged call: append (q in the same pass), then attend."""
    outs = []
    for i, _ in enumerate(calls):
        xi, cu, kl, o, qo = x[i]
        kvh = B.kvh
        dls.kv_append(xi[:, heads:heads + kvh], xi[:, heads + kvh:], B.k, B.v, B.table, cu, kl, freq, q=xi[:, :heads], q_out=qo,
                      q_norm=wq, k_norm=wk, pairing="halves", stream=torch.cuda.current_stream())
        dls.attention_chunk(qo, B.k, B.v, B.table, cu, kl, o, ws, stream=torch.cuda.current_stream())
        outs.append(o)
    return outs


@pytest.mark.parametrize("captured", [False, True])
def test_prompt_chunks_then_single_tokens(gpu_lib, captured):
    """Three sequences: prompts in two ragged calls, then single tokens, each call append + attend, eagerly and as
    one captured graph replayed over a cache that was cleared; against attention of the whole sequences in 64 bits."""
    heads, kvh, hd = 8, 2, 128
    calls = [[50, 0, 131], [13, 70, 1], [1, 1, 1], [1, 1, 1]]
    total = [sum(c[b] for c in calls) for b in range(3)]
    B = Batch([(n, n) for n in total], kvh, hd, 32, torch.bfloat16, 21)
    full = torch.randn(sum(total), heads + 2 * kvh, hd, generator=B.g, device="cuda") * 1.2
    wq, wk = (1 + 0.1 * torch.randn(hd, generator=B.g, device="cuda") for _ in range(2))
    freq, ws = dls.rope_inv_freq(hd, 500000.0), workspace(hd)
    x, rows, done = [], [], [0, 0, 0]
    for c in calls:
        idx = [B.starts[b] + done[b] + i for b in range(3) for i in range(c[b])]
        for b in range(3):
            done[b] += c[b]
        rows.append(torch.tensor(idx, device="cuda"))
        cu = torch.tensor(np.concatenate([[0], np.cumsum(c)]), dtype=torch.int32, device="cuda")
        o = torch.zeros(len(idx), heads, hd, dtype=B.typ, device="cuda")
        x.append((full[rows[-1]].clone(), cu, torch.tensor(done, dtype=torch.int32, device="cuda"), o, torch.empty_like(o)))
    serve(B, calls, heads, x, wq, wk, freq, ws)
    torch.cuda.synchronize()
    if captured:
        want_o = [t[3].clone() for t in x]
        stream = torch.cuda.Stream()
        graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
        with torch.cuda.stream(stream):
            for gr, part in zip(graphs, (slice(0, 2), slice(2, 4))):  # two graphs over one workspace
                with torch.cuda.graph(gr, stream=stream):
                    serve(B, calls[part], heads, x[part], wq, wk, freq, ws)
        for _ in range(2):
            B.k.fill_(math.nan)
            B.v.fill_(math.nan)
            for t in x:
                t[3].zero_()
            torch.cuda.synchronize()
            for gr in graphs:
                gr.replay()
            torch.cuda.synchronize()
            for t, w in zip(x, want_o):
                assert torch.equal(t[3], w)
    got = torch.zeros(B.rows, heads, hd, dtype=B.typ, device="cuda")
    qs = torch.zeros_like(got)
    for r, t in zip(rows, x):
        got[r], qs[r] = t[3], t[4]
    for b in range(3):
        r, pos = slice(B.starts[b], B.starts[b + 1]), torch.arange(total[b], device="cuda")
        close_turned(qs[r], full[r, :heads], wq, 1e-5, pos, freq, True)
        p, s = B.slots(b, 0, total[b])
        close_turned(B.k[p, :, s], full[r, heads:heads + kvh], wk, 1e-5, pos, freq, True)
    close_attend(B, got, None, attend64(B, qs, heads, hd ** -0.5, True, 0), heads)


def test_a_graph_follows_the_lengths(gpu_lib):
    """A captured call replayed with other lengths, pages and inputs in the same buffers."""
    heads, kvh, hd = 8, 2, 64
    B = Batch([(1, 100), (40, 333), (1, 2500)], kvh, hd, 64, torch.float16, 3, pad=30)
    B.fill()
    q = torch.randn(B.rows, heads, hd, generator=B.g, device="cuda").half()
    o, ws = torch.zeros_like(q), workspace(hd)
    dls.attention_chunk(q, B.k, B.v, B.table, B.cu_q, B.kv_len, o, ws)
    torch.cuda.synchronize()
    stream, gr = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=stream):
        dls.attention_chunk(q, B.k, B.v, B.table, B.cu_q, B.kv_len, o, ws, stream=torch.cuda.current_stream())
    for lengths in ([(2, 90), (60, 61), (9, 2400)], [(0, 0), (1, 1), (71, 71)]):
        B.lengths = lengths
        B.starts = [0]
        for ql, _ in lengths:
            B.starts.append(B.starts[-1] + ql)
        B.cu_q.copy_(torch.tensor(B.starts))
        B.kv_len.copy_(torch.tensor([kl for _, kl in lengths]))
        q.normal_()
        o.fill_(7.0)
        torch.cuda.synchronize()
        gr.replay()
        torch.cuda.synchronize()
        close_attend(B, o, None, attend64(B, q, heads, hd ** -0.5, True, 0), heads)
        assert bool((o[B.starts[-1]:] == 7).all())


@pytest.mark.parametrize("heads,kvh,hd,page,typ", [(32, 8, 128, 32, "f16"), (16, 2, 128, 64, "bf16"), (8, 8, 64, 16, "f16")])
def test_attention_chunk_many_tiles_of_each_range(gpu_lib, heads, kvh, hd, page, typ):
    """Several tiles of several key tiles in each CTA's range, each with a partly filled last page, repeated: copies run
    ahead of the products from tile to tile."""
    B = Batch([(5, 4101), (1, 3661), (3, 4009), (4, 1803), (1, 2951), (4, 3718), (5, 2122), (1, 2767), (60, 3001)], kvh, hd, page,
              TYPES[typ], 16)
    B.fill()
    q = (2 * torch.randn(B.rows, heads, hd, generator=B.g, device="cuda")).to(B.typ)
    o, first, lse, ws = torch.empty_like(q), torch.empty_like(q), torch.empty(B.rows, heads, device="cuda"), workspace(hd)
    dls.attention_chunk(q, B.k, B.v, B.table, B.cu_q, B.kv_len, first, ws)
    for _ in range(20):
        dls.attention_chunk(q, B.k, B.v, B.table, B.cu_q, B.kv_len, o, ws, lse=lse)
        assert torch.equal(o, first)
    close_attend(B, o, lse, attend64(B, q, heads, hd ** -0.5, True, 0), heads)
