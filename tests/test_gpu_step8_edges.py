"""Edges of the calls around the 8-bit paged cache, each against the definition: inputs that are no numbers, states that
cannot be, scales of any size, lengths past a look of 32."""
import math
import os
import subprocess
import sys

import pytest
import torch

from decode_llama_step_gb300 import dls
from test_gpu_step8 import Batch8, CODES, Requests, TYPES, attend64, check_verify, close_attend, ints, rounding, scale_of, turned, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("code", ["e4m3", "i8"])
@pytest.mark.parametrize("hd,rot,pairing", [(80, 80, "adjacent"), (96, 64, "halves"), (48, 0, "adjacent"), (112, 112, "halves"),
                                            (160, 32, "adjacent"), (64, 64, "halves"), (240, 240, "halves")])
@pytest.mark.parametrize("bad", ["nan", "zero"])
def test_append8_a_row_that_is_no_number_reaches_no_other(gpu_lib, code, hd, rot, pairing, bad):
    """A NaN in one row, or a row of zeros with eps = 0 (0 / 0), in the middle of a block and in its last rows: every other
    row and every scale is what it is with a row of ones in its place (which, normed and turned, stays below the others'
    largest value, as is looked at)."""
    lengths = [(70, 70), (40, 100), (33, 35)]
    eps = 0.0 if bad == "zero" else 1e-5
    first = None
    rows = [5, 63, 69, 70 + 2, 70 + 37, 110 + 31]
    for broken in (False, True):
        B = Batch8(lengths, 3, hd, 64, 32, code, 17)
        B.fill(upto=[kl - ql for ql, kl in lengths], powers=True)
        x = torch.randn(B.rows, 6, hd, generator=B.g, device="cuda")
        norm = 1 + 0.1 * torch.randn(hd, generator=B.g, device="cuda")
        for r in rows:
            x[r] = 1.0
            if broken:
                x[r, :3] = 0.0
                if bad == "nan":
                    x[r, :3, 7] = math.nan
        freq = dls.rope_inv_freq(rot, 500000.0) if rot else None
        for b, (ql, kl) in enumerate(lengths):
            if broken:
                break
            pos = torch.arange(kl - ql, kl, device="cuda")
            y = turned(x[B.starts[b]:B.starts[b] + ql, :3], norm, eps, pos, freq, pairing == "halves")[0].abs().amax(-1)
            ones = torch.tensor([B.starts[b] + i in rows for i in range(ql)], device="cuda")
            for block in set((pos // 32).tolist()):
                here = pos // 32 == block
                assert bool((scale_of(y[here].amax(0), code) == scale_of(y[here & ~ones].amax(0), code)).all())
        status = ints([9])
        dls.kv_append8(x[:, :3], x[:, 3:], B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len,
                       freq, k_norm=norm, eps=eps, pairing=pairing, status=status)
        dls.attention_status(status)
        got = []
        for b, (ql, kl) in enumerate(lengths):
            p, s = B.slots(b, 0, kl)
            got.append([t.view(torch.uint8)[p, :, s] for t in (B.k, B.v)] + [t[p, :, s // 32] for t in (B.ks, B.vs)])
        if not broken:
            first = got
            continue
        for b, (ql, kl) in enumerate(lengths):
            start = B.starts[b]
            mine = [r - start + kl - ql for r in rows if start <= r < start + ql]
            keep = torch.ones(kl, dtype=torch.bool, device="cuda")
            keep[mine] = False
            for now, was in zip(got[b][1:], first[b][1:]):      # V, and the scales of both
                assert torch.equal(now, was)
            assert torch.equal(got[b][0][keep], first[b][0][keep])
            codes = got[b][0][mine].view(CODES[code]).float()
            assert bool((codes == 0).all()) if code == "i8" else bool(codes.isnan().all())


@pytest.mark.parametrize("n,rows", [(6, 50), (40, 20000), (300, 4000)])
def test_reserve_keeps_the_record_of_pages_that_it_cannot_take_back(gpu_lib, n, rows):
    """Requests that are over with a state that cannot be, in place: length and held pages stay, for the caller to put right
    and end again; arrays of their own hold 0."""
    page = 16
    r = Requests(n, page, 50 + n, spare=4 * n)
    bad = {1: (-7, None), 2: (page * r.most + 1, None), 4: (5 + page * max(r.held[4], 1), max(r.held[4], 1)), n - 1: (0, r.most + 1)}
    pages = {}
    for b, (kv, held) in bad.items():
        pages[b] = r.held[b]
        r.kv[b] = kv
        r.held[b] = r.held[b] if held is None else held
    new = [-1 if b in bad else 1 for b in range(n)]
    for inside in (False, True):
        kv, held, count, table, stack = ints(r.kv), ints(r.held), ints([r.count]), ints(r.table), ints(r.stack)
        kv_out, held_out = (kv, held) if inside else (torch.full_like(kv, 77), torch.full_like(held, 77))
        cu, status = ints([0] * (n + 1)), ints([0])
        dls.kv_reserve(ints(new), kv, held, table, stack, count, kv_out, held_out, count, cu, page, max_rows=rows, status=status)
        assert status.item() == 4
        taken = sum(r.kv[b] == page * r.held[b] for b in range(n) if b not in bad)
        assert count.item() == r.count - taken
        for b in range(n):
            want = (r.kv[b] + 1, r.held[b] + (r.kv[b] == page * r.held[b])) if b not in bad else (r.kv[b], r.held[b]) if inside else (0, 0)
            assert (kv_out[b].item(), held_out[b].item()) == want, b
    # the lengths put right, the same requests end: their pages are on the stack
    for b in bad:
        kv[b], held[b] = 0, pages[b]
    before = count.item()
    dls.kv_reserve(ints([-1 if b in bad else 0 for b in range(n)]), kv, held, table, stack, count, kv, held, count, cu, page,
                   max_rows=rows, status=status)
    assert status.item() == 0 and count.item() == before + sum(pages.values())
    back = stack.tolist()[before:count.item()]
    assert sorted(back) == sorted(p for b in bad for p in r.table[b][:pages[b]])


def kept_scale(had, code):
    """What a scale that is there counts as: 2^-64 to 2^64, the nearer end where it lies outside or is none."""
    return had.nan_to_num(0.0, math.inf, 0.0).clamp(2.0 ** -64, 2.0 ** 64)


def coded(x, code):
    return x.round().clamp(-127, 127).to(torch.int8) if code == "i8" else x.clamp(-448, 448).to(CODES["e4m3"])


@pytest.mark.parametrize("code", ["e4m3", "i8"])
@pytest.mark.parametrize("grows", [False, True])
@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_append8_into_blocks_of_any_scale(gpu_lib, code, grows, typ):
    """Blocks filled elsewhere, whose scales are no powers of two: new rows are divided by the scale that stays, codes of one
    that grows multiplied by old / new, both in fp32, and rounded to the nearest code."""
    kvh, hd, page, block = 2, 128, 64, 64
    lengths = [(9, 20 + b % 30) for b in range(64)]
    B = Batch8(lengths, kvh, hd, page, block, code, 23)
    B.fill(upto=[kl - ql for ql, kl in lengths])
    x = torch.empty(B.rows, 2 * kvh, hd, device="cuda")
    for b, (ql, kl) in enumerate(lengths):
        p = int(B.table[b, 0])
        if b == 0:
            B.vs[p, 0, 0] = 0.010002499
        size = torch.cat([B.ks[p, :, 0], B.vs[p, :, 0]])[None, :, None]
        # halves of codes, times the scale, rounded: quotients on and next to the borders between codes
        unit = (torch.randint(-126, 127, (ql, 2 * kvh, hd), generator=B.g, device="cuda") / 2) if code == "i8" else (
            torch.randn(ql, 2 * kvh, hd, generator=B.g, device="cuda") * 60).clamp(-220, 220)
        x[b * ql:(b + 1) * ql] = unit * size * (3.0 if grows else 1.0)
    x = x.to({"f32": torch.float32, "bf16": torch.bfloat16}[typ])
    if code == "i8" and typ == "f32" and not grows:
        x[0, kvh, 0] = 0.02500625   # 2.5 times its scale in fp32, a tie: 2; times the reciprocal it is more
    old = [t.clone() for t in (B.k, B.v, B.ks, B.vs)]
    dls.kv_append8(x[:, :kvh], x[:, kvh:], B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len, None)
    grown = 0
    for b, (ql, kl) in enumerate(lengths):
        p = int(B.table[b, 0])
        for src, pool, scales, op, os_ in ((x[:, :kvh], B.k, B.ks, old[0], old[2]), (x[:, kvh:], B.v, B.vs, old[1], old[3])):
            mine = src[b * ql:(b + 1) * ql].float()
            most = mine.abs().amax((0, 2))
            had = os_[p, :, 0]
            want = torch.maximum(had, scale_of(most, code).float())
            assert torch.equal(scales[p, :, 0], want)
            grown += int((want > had).sum())
            got = pool.view(torch.uint8)[p, :, kl - ql:kl].view(CODES[code])
            assert torch.equal(got.view(torch.uint8), coded(mine / want[:, None], code).transpose(0, 1).contiguous().view(torch.uint8))
            was = op.view(torch.uint8)[p, :, :kl - ql].view(CODES[code]).float()
            f = (had / want)[:, None, None]
            then = torch.where(f < 1, coded(was * f, code).float(), was)
            assert torch.equal(pool.view(torch.uint8)[p, :, :kl - ql].view(CODES[code]).float(), then)
    assert (grown > 100) == grows


@pytest.mark.parametrize("code", ["e4m3", "i8"])
def test_append8_into_blocks_whose_scale_is_none(gpu_lib, code):
    """A scale of 0, a negative one, NaN or one outside 2^-64..2^64 counts as the nearer end, codes as they are, as the
    attention takes it."""
    odd = [0.0, -3.0, math.nan, 2.0 ** -80, 2.0 ** 70, math.inf, 2.0 ** 64, 2.0 ** -64]
    lengths = [(1, 10)] * len(odd)
    B = Batch8(lengths, 1, 64, 16, 16, code, 29)
    B.fill(upto=[9] * len(odd))
    p = B.table[:, 0].long()
    had = torch.tensor(odd, device="cuda")
    B.ks[p, 0, 0], B.vs[p, 0, 0] = had, had
    old = B.v.clone()
    x = torch.zeros(B.rows, 1, 64, device="cuda")
    dls.kv_append8(x, x, B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len, None)
    for scales in (B.ks, B.vs):
        assert torch.equal(scales[p, 0, 0], kept_scale(had, code))
    assert torch.equal(B.v.view(torch.uint8)[p, :, :9], old.view(torch.uint8)[p, :, :9])
    assert not bool(B.v.view(torch.uint8)[p, :, 9].any())


@pytest.mark.parametrize("drawn", [False, True])
def test_verify_flags_a_strange_token_anywhere(gpu_lib, drawn):
    """A drafted token outside the vocabulary sets its bit also far behind the first draft that does not stand."""
    for at in (3, 31, 32, 33, 68):
        for token in (-1, 777, 1 << 30):
            def edit(s, cu):
                s["accept"][cu[1]] = 1e30       # the second sequence's first draft does not stand
                s["tokens"][cu[1] + at] = token

            want = check_verify([4, 70, 2], 777, "f32", drawn, 13, edit=edit, expect=2)
            assert want[1][1] == 0


FIRST_CALLS = """
import sys, time, torch
sys.path.insert(0, sys.argv[1])
from decode_llama_step_gb300 import dls
z = lambda *s, t=torch.float16: torch.zeros(*s, dtype=t, device="cuda")
i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
q, k, k8, sc = z(1, 8, 64), z(2, 2, 16, 64), z(2, 2, 16, 64, t=torch.int8), torch.ones(2, 2, 1, device="cuda")
rest = i([[0, 1]]), i([0, 1]), i([5]), torch.empty_like(q), z(dls.attention_chunk_workspace_bytes(64), t=torch.uint8)
for f, a in ((dls.attention_chunk, (q, k, k)), (dls.attention_chunk8, (q, k8, k8, sc, sc))):
    torch.cuda.synchronize()
    t = time.perf_counter()
    f(*a, *rest)
    torch.cuda.synchronize()
    print(time.perf_counter() - t)
"""


def test_a_call_over_16_bit_pages_loads_no_kernel_over_codes(gpu_lib):
    """In a process of its own the first call over 16-bit pages is short beside the first one over codes, which has ten
    times the kernels: each pays for its own."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    runs = [subprocess.run([sys.executable, "-c", FIRST_CALLS, root], capture_output=True, text=True, check=True,
                           env={**os.environ, "CUDA_MODULE_LOADING": "LAZY"}).stdout.split()
            for _ in range(3)]
    pages, codes = (min(float(r[x]) for r in runs) for x in (0, 1))
    assert codes > pages, (pages, codes)


# ---- what the header says of weights, scales and prompts in a batch --------------------------------------

def near_cancelling(lengths, kvh, hd, code, seed):
    """A batch whose values cancel: neighbours' V are each other's negatives, keys nearly alike."""
    B = Batch8(lengths, kvh, hd, 32, 32, code, seed)
    B.fill()
    for b, (_, kl) in enumerate(lengths):
        p, s = B.slots(b, 0, kl)
        sign = 1 - 2 * (torch.arange(kl, device="cuda") % 2)
        v = B.v.view(torch.uint8)[p, :, s].view(CODES[code]).float()
        v = v[:1].clamp(min=-127) * sign[:, None, None]
        B.v.view(torch.uint8)[p, :, s] = v.to(CODES[code]).view(torch.uint8)
    B.ks.mul_(0.05)
    return B


@pytest.mark.parametrize("typ", ["f16", "bf16"])
@pytest.mark.parametrize("code", ["e4m3", "i8"])
@pytest.mark.parametrize("hd,lengths", [(128, [(1, 2), (1, 3), (1, 4), (1, 6)] * 20), (64, [(1, 2), (1, 3), (1, 5)] * 20),
                                        (128, [(40, 42), (50, 51), (45, 49)] * 4), (64, [(40, 42), (50, 51), (45, 49)] * 4)])
def test_attention8_weights_are_halves(gpu_lib, typ, code, hd, lengths):
    """Weights are rounded to eleven bits whatever q's type: few keys, whose values cancel, so that the output is small beside
    what it is summed from and its own rounding hides nothing."""
    B = near_cancelling(lengths, 2, hd, code, 37)
    q = torch.randn(B.rows, 4, hd, generator=B.g, device="cuda").to(TYPES[typ])
    o, ws = torch.empty_like(q), workspace(hd)
    dls.attention_chunk8(q, B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len, o, ws)
    want, _, mag, dot = attend64(B, q, 4, hd ** -0.5, True, 0)
    # as close_attend, with a half's half step for the weights, below its normal range 2^-32 of the largest V
    ds = (hd + 8) * 2.0 ** -23 * dot + 2.0 ** -16
    top = 128.0 if code == "i8" else 448.0
    lim = (2.0 ** -11 * (1 + 2.0 ** -6) + 2 * ds[..., None] + 2 * 66 * 2.0 ** -23) * mag + rounding(want, TYPES[typ]) * (1 + 2.0 ** -6)
    lim = lim + 64 * 2.0 ** -32 * top * float(B.vs.nan_to_num(0.0).max())
    err = (o.double() - want).abs()
    assert bool((err <= lim).all()), float((err / lim).max())
    if typ == "bf16":  # the test would see weights of eight bits
        assert float((lim / (mag * 2.0 ** -9).clamp(min=1e-30))[..., 0].median()) < 1


@pytest.mark.parametrize("typ", ["f16", "bf16"])
@pytest.mark.parametrize("rows", [1, 40])
def test_attention8_scales_2_to_the_110_apart(gpu_lib, typ, rows):
    """Keys of equal weight whose V scales are 2^-50 and 2^60: all count in the sum of weights."""
    B = Batch8([(rows, 300), (rows, 64)], 2, 64, 32, 16, "e4m3", 41)
    B.fill()
    for b, (_, kl) in enumerate(B.lengths):
        p, s = B.slots(b, 0, kl)
        small = torch.arange(kl, device="cuda") // 16 % 2 == 0
        B.vs[p, :, s // 16] = torch.where(small, 2.0 ** -50, 2.0 ** 60)[:, None].expand(-1, 2)
    q = torch.randn(B.rows, 4, 64, generator=B.g, device="cuda").to(TYPES[typ])
    out = torch.empty_like(q)
    lse = torch.empty(B.rows, 4, device="cuda")
    B.v.view(torch.uint8).bitwise_and_(0x80)   # (values of 2^60 do not fit the output: zeros, the sum is what is looked at)
    dls.attention_chunk8(q, B.k, B.v, B.ks, B.vs, B.table, B.cu_q, B.kv_len, out, workspace(64), lse=lse)
    close_attend(B, out, lse, attend64(B, q, 4, 0.125, True, 0))


@pytest.mark.parametrize("typ,heads,hd", [("bf16", 8, 128), ("f16", 4, 64)])
def test_attention8_a_call_for_each_kind_of_sequence(gpu_lib, typ, heads, hd):
    """Single tokens first, chunks behind: two calls over parts of the same lengths, tables and rows are one over all, and
    the first leaves the other's rows alone."""
    n, chunks = 30, [(200, 700), (90, 90)]
    B = Batch8([(1, 50 + 40 * b) for b in range(n)] + chunks, 2, hd, 32, 32, "e4m3", 47, first=2, pad=3)
    B.fill()
    q = torch.randn(B.rows, heads, hd, generator=B.g, device="cuda").to(TYPES[typ])
    o, ws, status = torch.full_like(q, 7.0), workspace(hd), ints([9])
    pools = B.k, B.v, B.ks, B.vs
    rows = B.starts[n]
    dls.attention_chunk8(q[:rows], *pools, B.table[:n], B.cu_q[:n + 1], B.kv_len[:n], o[:rows], ws, status=status)
    dls.attention_status(status)
    assert bool((o[rows:] == 7).all()) and bool((o[:2] == 7).all()) and not bool((o[2:rows] == 7).all())
    dls.attention_chunk8(q, *pools, B.table[n:], B.cu_q[n:], B.kv_len[n:], o, ws, status=status)
    dls.attention_status(status)
    close_attend(B, o, None, attend64(B, q, heads, hd ** -0.5, True, 0))
    assert bool((o[B.starts[-1]:] == 7).all())


def test_verify_of_a_batch_with_prompts(gpu_lib):
    """accept below 0 keeps a row's next token where its probabilities are above 0: a prompt's rows go through whole, its
    length stays, and the token after it comes from its last row."""
    def prompts(s, cu):
        s["accept"][cu[1]:cu[2]] = -1.0
        s["tokens"][cu[1]:cu[2]] = torch.randint(0, 500, (cu[2] - cu[1],), device="cuda", dtype=torch.int32)

    for drawn in (False, True):
        want = check_verify([4, 90, 1, 3], 500, "f32", drawn, 43, edit=prompts)
        assert want[1][1] == 89 and want[1][0][-1] >= 0
