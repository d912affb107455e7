"""Edges of the calls around the 8-bit paged cache, each against the definition: inputs that are no numbers, states that
cannot be, scales of any size, lengths past a look of 32."""
import math

import pytest
import torch

from decode_llama_step_gb300 import dls
from test_gpu_step8 import Batch8, CODES, Requests, ints, scale_of, turned

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
