"""Argument checks of the calls around the 8-bit paged cache, on a machine without a GPU: every refusal comes before a
CUDA call."""
import math

import numpy as np
import pytest
import torch

from decode_llama_step_gb300 import dls

P = 4096  # a 16-byte aligned address that is never followed
FREQ = np.ones(64)

RESERVE = dict(new_len=P, kv_len=P, held=P, page_table=P, free_pages=P, free_count=P, kv_len_out=P, held_out=P,
               free_count_out=P, cu_q=P, positions=P, slots=P, seq_ids=P, status=0, n_seqs=4, max_rows=64, page_tokens=64,
               n_pages=100, max_pages=10)
APPEND8 = dict(k=P, v=P, k_pages=P, v_pages=P, k_scales=P, v_scales=P, k_stride=1024, v_stride=1024, k_norm=0, page_table=P,
               cu_q=P, kv_len=P, inv_freq=FREQ.ctypes.data, status=0, n_tokens=4, n_seqs=2, n_kv_heads=8, head_dim=128,
               rot_dim=128, pairing=0, in_type=1, code_type=4, page_tokens=64, block_tokens=32, n_pages=10, max_pages=5,
               eps=1e-5)
CHUNK8 = dict(q=P, k_pages=P, v_pages=P, k_scales=P, v_scales=P, page_table=P, cu_q=P, kv_len=P, o=P, lse=0, workspace=P,
              workspace_bytes=1 << 40, status=0, q_stride=4096, o_stride=4096, n_tokens=4, n_seqs=2, n_heads=32,
              n_kv_heads=8, head_dim=128, page_tokens=64, block_tokens=16, n_pages=10, max_pages=5, q_type=2, code_type=5,
              causal=1, window=0, scale=0.0)
VERIFY = dict(tokens=P, target=P, draft=P, cu_q=P, accept=P, pick=P, kv_len=P, out_tokens=P + 64, n_accepted=P, kv_len_out=P,
              status=0, target_stride=1024, draft_stride=1024, n_tokens=10, n_seqs=2, vocab=1024, prob_type=1)
CALLS = {"dls_kv_reserve": (dls._KV_RESERVE, RESERVE), "dls_kv_append8": (dls._KV_APPEND8, APPEND8),
         "dls_attention_chunk8": (dls._ATTENTION_CHUNK8, CHUNK8), "dls_verify_draft": (dls._VERIFY_DRAFT, VERIFY)}


@pytest.fixture(scope="module")
def lib():
    return dls.load()


def refused(lib, name, over, word):
    fmt, base = CALLS[name]
    d = {**base, **over}
    assert len(d) == len(base)
    rc = getattr(lib, name)(fmt.pack(*d.values()), None)
    msg = lib.dls_last_error(None).decode()
    assert rc == dls.DLS_ERR_ARG, (over, rc)
    assert msg.startswith("ERR ARG") and name[4:] + ":" in msg and word in msg, msg


@pytest.mark.parametrize("over,word", [
    (dict(page_tokens=48), "page_tokens=48"), (dict(page_tokens=8), "page_tokens=8"), (dict(n_seqs=-1), "n_seqs=-1"),
    (dict(n_seqs=4097), "n_seqs=4097"), (dict(max_rows=-1), "max_rows=-1"), (dict(max_rows=(1 << 30) + 1), "max_rows"),
    (dict(n_pages=0), "n_pages=0"), (dict(max_pages=0), "max_pages=0"), (dict(max_pages=1 << 25), "max_pages"),
    (dict(n_pages=1 << 25), "n_pages"), (dict(cu_q=0), "cu_q"), (dict(free_count=0), "free_count"),
    (dict(free_count_out=0), "free_count_out"), (dict(free_pages=0), "free_pages"), (dict(new_len=0), "new_len"),
    (dict(kv_len=0), "kv_len"), (dict(held=0), "held"), (dict(page_table=0), "page_table"), (dict(kv_len_out=0), "kv_len_out"),
    (dict(held_out=0), "held_out"), (dict(positions=P + 2), "aligned"), (dict(status=P + 1), "aligned"),
    (dict(slots=P + 3), "aligned"), (dict(held=P + 2), "aligned"),
])
def test_kv_reserve_refuses(lib, over, word):
    refused(lib, "dls_kv_reserve", over, word)


@pytest.mark.parametrize("over,word", [
    (dict(head_dim=72), "head_dim=72"), (dict(head_dim=272, rot_dim=0), "head_dim=272"), (dict(rot_dim=256), "rot_dim=256"),
    (dict(pairing=-1), "pairing=-1"), (dict(inv_freq=0), "inv_freq"), (dict(eps=math.nan), "eps="), (dict(in_type=4), "in_type=4"),
    (dict(code_type=3), "code_type=3"), (dict(page_tokens=48), "page_tokens=48"), (dict(block_tokens=8), "block_tokens=8"),
    (dict(block_tokens=128), "block_tokens=128"), (dict(block_tokens=48), "block_tokens=48"), (dict(n_tokens=-1), "n_tokens=-1"),
    (dict(n_tokens=(1 << 30) + 1), "n_tokens"), (dict(n_seqs=-2), "n_seqs=-2"), (dict(n_seqs=(1 << 30) + 1), "n_seqs"),
    (dict(n_kv_heads=0), "n_kv_heads=0"), (dict(n_kv_heads=5000), "n_kv_heads=5000"), (dict(n_pages=0), "n_pages=0"),
    (dict(max_pages=1 << 26), "max_pages"), (dict(page_table=0), "page_table"), (dict(cu_q=P + 2), "cu_q"), (dict(kv_len=0), "kv_len"),
    (dict(k=0), "aligned"), (dict(v=P + 8), "aligned"), (dict(k_stride=1020), "rows"), (dict(v_stride=1026), "aligned"),
    (dict(k_pages=P + 4), "k_pages"), (dict(v_pages=0), "v_pages"), (dict(k_scales=0), "k_scales"), (dict(v_scales=P + 2), "v_scales"),
    (dict(k_norm=P + 4), "k_norm"), (dict(status=P + 2), "status"), (dict(status=P + 2, n_tokens=0), "status"),
])
def test_kv_append8_refuses(lib, over, word):
    refused(lib, "dls_kv_append8", over, word)


@pytest.mark.parametrize("over,word", [
    (dict(head_dim=8), "head_dim=8"), (dict(head_dim=144), "head_dim=144"), (dict(page_tokens=512), "page_tokens=512"),
    (dict(block_tokens=0), "block_tokens=0"), (dict(block_tokens=128), "block_tokens=128"), (dict(q_type=1), "q_type=1"),
    (dict(code_type=0), "code_type=0"), (dict(code_type=2), "code_type=2"), (dict(n_heads=30), "n_heads=30"),
    (dict(n_heads=2048), "groups"), (dict(n_kv_heads=0), "n_kv_heads=0"), (dict(n_tokens=-1), "n_tokens=-1"),
    (dict(n_seqs=4097), "n_seqs=4097"), (dict(n_pages=0), "n_pages=0"), (dict(max_pages=1 << 25), "max_pages"),
    (dict(n_pages=1 << 22), "2^31"), (dict(causal=2), "causal=2"), (dict(window=4, causal=0), "window=4"),
    (dict(scale=math.nan), "scale="), (dict(q=0), "aligned"), (dict(o=P + 8), "aligned"), (dict(q_stride=4088), "rows"),
    (dict(o_stride=8192), "in place"), (dict(k_pages=0), "k_pages"), (dict(v_pages=P + 4), "v_pages"), (dict(k_scales=0), "k_scales"),
    (dict(v_scales=P + 1), "v_scales"), (dict(page_table=0), "page_table"), (dict(cu_q=0), "cu_q"), (dict(kv_len=P + 2), "kv_len"),
    (dict(lse=P + 2), "lse"), (dict(workspace=P + 16), "workspace"), (dict(workspace_bytes=0), "workspace"),
    (dict(n_tokens=1 << 30, n_seqs=4096), "too many"),
])
def test_attention_chunk8_refuses(lib, over, word):
    refused(lib, "dls_attention_chunk8", over, word)


@pytest.mark.parametrize("over,word", [
    (dict(prob_type=4), "prob_type=4"), (dict(n_tokens=-1), "n_tokens=-1"), (dict(n_seqs=-1), "n_seqs=-1"),
    (dict(n_seqs=(1 << 24) + 1), "n_seqs"), (dict(vocab=0), "vocab=0"), (dict(vocab=(1 << 18) + 1, target_stride=1 << 20, draft_stride=1 << 20), "vocab"), (dict(target_stride=1023), "target_stride=1023"),
    (dict(draft_stride=1000), "draft_stride=1000"), (dict(target_stride=(1 << 32) + 1), "target_stride"), (dict(cu_q=0), "cu_q"),
    (dict(n_accepted=0), "n_accepted"), (dict(kv_len=0), "both lengths"), (dict(kv_len_out=0), "both lengths"),
    (dict(tokens=0), "tokens"), (dict(target=0), "target"), (dict(accept=0), "accept"), (dict(pick=0), "pick"),
    (dict(out_tokens=0), "out_tokens"), (dict(out_tokens=P), "cannot be tokens"), (dict(tokens=P + 2), "aligned"),
    (dict(pick=P + 1), "aligned"), (dict(target=P + 2), "aligned"), (dict(prob_type=2, draft=P + 1), "aligned"), (dict(status=P + 2), "status"),
])
def test_verify_draft_refuses(lib, over, word):
    refused(lib, "dls_verify_draft", over, word)


def test_null_descriptors_and_empty_batches(lib):
    for name in CALLS:
        assert getattr(lib, name)(None, None) == dls.DLS_ERR_ARG
        assert "desc=NULL" in lib.dls_last_error(None).decode()
    for name, over in [("dls_kv_append8", dict(n_tokens=0, k=0)), ("dls_kv_append8", dict(n_seqs=0, page_table=0)),
                       ("dls_attention_chunk8", dict(n_tokens=0, o=0)), ("dls_attention_chunk8", dict(n_seqs=0, cu_q=0)),
                       ("dls_verify_draft", dict(n_seqs=0, cu_q=0, target=0))]:  # nothing to do: no pointer is looked at
        fmt, base = CALLS[name]
        assert getattr(lib, name)(fmt.pack(*{**base, **over}.values()), None) == 0


def test_frequencies_that_are_not_finite(lib):
    f = np.ones(64)
    f[5] = math.inf
    refused(lib, "dls_kv_append8", dict(inv_freq=f.ctypes.data), "inv_freq")


def test_binding_refuses_what_does_not_fit_together():
    z, i32, e4 = torch.zeros, torch.int32, torch.float8_e4m3fn
    a = dict(q=z(4, 8, 64, dtype=torch.float16), k_pages=z(5, 2, 32, 64).to(e4), v_pages=z(5, 2, 32, 64).to(e4),
             k_scales=z(5, 2, 2), v_scales=z(5, 2, 2), page_table=z(2, 3, dtype=i32), cu_q=z(3, dtype=i32), kv_len=z(2, dtype=i32),
             o=z(4, 8, 64, dtype=torch.float16), workspace=z(1 << 12, dtype=torch.uint8))
    for over, word in [
        (dict(), "one CUDA device"), (dict(o=z(4, 8, 64)), "o: type"),
        (dict(k_pages=z(5, 2, 32, 64)), "k_pages: type"), (dict(v_pages=z(5, 2, 32, 64, dtype=torch.int8)), "v_pages"),
        (dict(k_scales=z(5, 2, 3)), "k_scales: shape"), (dict(k_scales=z(4, 2, 2)), "k_scales: shape"),
        (dict(k_scales=z(5, 2)), "k_scales: shape"), (dict(v_scales=z(5, 2, 1)), "v_scales"), (dict(v_scales=z(5, 2, 2).double()), "v_scales"),
        (dict(kv_len=z(3, dtype=i32)), "kv_len"), (dict(lse=z(4, 4)), "lse"),
    ]:
        with pytest.raises(ValueError, match=word):
            dls.attention_chunk8(**{**a, **over})
    k = z(4, 2, 64)
    b = dict(k=k, v=k, inv_freq=None, **{x: a[x] for x in ("k_pages", "v_pages", "k_scales", "v_scales", "page_table", "cu_q", "kv_len")})
    for over, word in [(dict(), "one CUDA device"), (dict(v=z(4, 3, 64)), "v: shape"), (dict(v=k.half()), "v: type"),
                       (dict(k_norm=z(32)), "k_norm"), (dict(pairing="split"), "pairing"), (dict(inv_freq=np.ones((2, 2))), "inv_freq")]:
        with pytest.raises(ValueError, match=word):
            dls.kv_append8(**{**b, **over})
    n = z(3, dtype=i32)
    c = dict(new_len=n, kv_len=n, held=n, page_table=z(3, 4, dtype=i32), free_pages=z(9, dtype=i32), free_count=z(1, dtype=i32),
             kv_len_out=n, held_out=n, free_count_out=z(1, dtype=i32), cu_q=z(4, dtype=i32), page_tokens=16, positions=z(7, dtype=i32))
    for over, word in [(dict(), "one CUDA device"), (dict(cu_q=n), "cu_q"), (dict(slots=z(8, dtype=i32)), "slots"),
                       (dict(positions=None), "max_rows"), (dict(max_rows=8), "max_rows"), (dict(free_pages=z(3, 3, dtype=i32)), "free_pages"),
                       (dict(page_table=n), "page_table"), (dict(held=z(3)), "held"), (dict(free_count=n), "free_count")]:
        with pytest.raises(ValueError, match=word):
            dls.kv_reserve(**{**c, **over})
    d = dict(tokens=z(6, dtype=i32), target=z(6, 10), cu_q=n, accept=z(6), pick=z(2), out_tokens=z(6, dtype=i32),
             n_accepted=z(2, dtype=i32))
    for over, word in [(dict(), "one CUDA device"), (dict(target=z(10)), "target"), (dict(draft=z(6, 9)), "draft"),
                       (dict(draft=z(6, 10).half()), "draft"), (dict(draft=z(10, 6).T), "contiguous"), (dict(accept=z(5)), "accept"),
                       (dict(pick=z(3)), "pick"), (dict(tokens=z(6, dtype=torch.int64)), "tokens"), (dict(kv_len=n), "kv_len")]:
        with pytest.raises(ValueError, match=word):
            dls.verify_draft(**{**d, **over})
