"""Argument checks of the operators around the paged cache, on a machine without a GPU: every refusal comes before a
CUDA call."""
import math

import numpy as np
import pytest
import torch

from decode_llama_step_gb300 import dls

P = 4096  # a 16-byte aligned address that is never followed


@pytest.fixture(scope="module")
def lib():
    return dls.load()


FREQ = np.ones(64)
ROPE = dict(q=P, k=P, q_out=P + 64, k_out=P + 64, q_stride=4096, k_stride=1024, q_out_stride=4096, k_out_stride=1024,
            q_norm=0, k_norm=0, positions=P, inv_freq=FREQ.ctypes.data, n_tokens=4, n_heads=32, n_kv_heads=8, head_dim=128,
            rot_dim=128, pairing=0, in_type=3, out_type=3, eps=1e-5)
APPEND = dict(k=P, v=P, q=P, k_pages=P, v_pages=P, q_out=P + 64, k_stride=1024, v_stride=1024, q_stride=4096,
              q_out_stride=4096, k_norm=0, q_norm=0, page_table=P, cu_q=P, kv_len=P, inv_freq=FREQ.ctypes.data, status=0,
              n_tokens=4, n_seqs=2, n_heads=32, n_kv_heads=8, head_dim=128, rot_dim=128, pairing=0, in_type=1, kv_type=2,
              page_tokens=64, n_pages=10, max_pages=5, eps=1e-5)
CHUNK = dict(q=P, k_pages=P, v_pages=P, page_table=P, cu_q=P, kv_len=P, o=P, lse=0, workspace=P, workspace_bytes=1 << 40,
             status=0, q_stride=4096, o_stride=4096, n_tokens=4, n_seqs=2, n_heads=32, n_kv_heads=8, head_dim=128,
             page_tokens=64, n_pages=10, max_pages=5, kv_type=2, causal=1, window=0, scale=0.0)


def refused(lib, name, fmt, base, over, word):
    d = {**base, **over}
    assert len(d) == len(base)
    rc = getattr(lib, name)(fmt.pack(*d.values()), None)
    msg = lib.dls_last_error(None).decode()
    assert rc == dls.DLS_ERR_ARG, (over, rc)
    assert msg.startswith("ERR ARG") and name[4:] in msg and word in msg, msg


@pytest.mark.parametrize("over,word", [
    (dict(head_dim=0, rot_dim=0), "head_dim=0"), (dict(head_dim=120), "head_dim=120"),
    (dict(head_dim=272, rot_dim=0), "head_dim=272"), (dict(rot_dim=144), "rot_dim=144"), (dict(rot_dim=24), "rot_dim=24"),
    (dict(rot_dim=-16), "rot_dim=-16"), (dict(pairing=2), "pairing=2"), (dict(inv_freq=0), "inv_freq"),
    (dict(eps=-1.0), "eps=-1"), (dict(eps=math.nan), "eps="), (dict(in_type=0), "in_type=0"), (dict(out_type=4), "out_type=4"),
    (dict(n_tokens=-1), "n_tokens=-1"), (dict(n_heads=-1), "n_heads=-1"), (dict(n_kv_heads=5000), "n_kv_heads=5000"),
    (dict(positions=0), "positions"), (dict(q=0), "aligned"), (dict(k_out=P + 8), "aligned"), (dict(q_stride=4095), "rows"),
    (dict(k_out_stride=1028), "aligned"), (dict(q_stride=-4096), "rows"), (dict(q_out=P, out_type=1), "in place"),
    (dict(k_out=P, k_out_stride=2048), "in place"), (dict(n_tokens=0x7fffffff), "too many"),
])
def test_qk_norm_rope_refuses(lib, over, word):
    refused(lib, "dls_qk_norm_rope", dls._QK_NORM_ROPE, ROPE, over, word)


def test_qk_norm_rope_refuses_frequencies_that_are_not_finite(lib):
    for bad in (math.inf, math.nan):
        f = np.ones(64)
        f[63] = bad
        refused(lib, "dls_qk_norm_rope", dls._QK_NORM_ROPE, ROPE, dict(inv_freq=f.ctypes.data), "inv_freq")
        refused(lib, "dls_kv_append", dls._KV_APPEND, APPEND, dict(inv_freq=f.ctypes.data), "inv_freq")


@pytest.mark.parametrize("over,word", [
    (dict(head_dim=72), "head_dim=72"), (dict(rot_dim=256), "rot_dim=256"), (dict(pairing=-1), "pairing=-1"),
    (dict(in_type=8), "in_type=8"), (dict(kv_type=1), "kv_type=1"), (dict(page_tokens=48), "page_tokens=48"),
    (dict(page_tokens=8), "page_tokens=8"), (dict(n_tokens=-1), "n_tokens=-1"), (dict(n_seqs=-2), "n_seqs=-2"),
    (dict(n_kv_heads=0), "n_kv_heads=0"), (dict(n_heads=0), "n_heads=0"), (dict(n_pages=0), "n_pages=0"),
    (dict(max_pages=0), "max_pages=0"), (dict(max_pages=1 << 26), "max_pages"), (dict(page_table=0), "page_table"),
    (dict(cu_q=0), "cu_q"), (dict(kv_len=0), "kv_len"), (dict(k=0), "aligned"), (dict(v=P + 2), "aligned"),
    (dict(q_out=0), "aligned"), (dict(v_stride=1023), "rows"), (dict(k_pages=0), "k_pages"), (dict(v_pages=P + 8), "v_pages"),
    (dict(q_out=P), "in place"),
])
def test_kv_append_refuses(lib, over, word):
    refused(lib, "dls_kv_append", dls._KV_APPEND, APPEND, over, word)


@pytest.mark.parametrize("over,word", [
    (dict(head_dim=8), "head_dim=8"), (dict(head_dim=144), "head_dim=144"), (dict(head_dim=100), "head_dim=100"),
    (dict(page_tokens=512), "page_tokens=512"), (dict(kv_type=1), "kv_type=1"), (dict(n_heads=30), "n_heads=30"),
    (dict(n_heads=2048, n_kv_heads=8), "groups"), (dict(n_kv_heads=0), "n_kv_heads=0"), (dict(n_tokens=-1), "n_tokens=-1"),
    (dict(n_seqs=4097), "n_seqs=4097"), (dict(n_seqs=-1), "n_seqs=-1"), (dict(n_pages=0), "n_pages=0"),
    (dict(max_pages=0), "max_pages=0"), (dict(max_pages=1 << 25), "max_pages"), (dict(n_pages=1 << 22), "2^31"),
    (dict(causal=2), "causal=2"), (dict(window=-1), "window=-1"), (dict(window=4, causal=0), "window=4"),
    (dict(scale=-1.0), "scale=-1"), (dict(scale=math.inf), "scale="), (dict(scale=math.nan), "scale="), (dict(q=0), "aligned"),
    (dict(o=P + 8), "aligned"), (dict(q_stride=4088), "rows"), (dict(o_stride=4100), "aligned"), (dict(k_pages=0), "k_pages"),
    (dict(v_pages=P + 4), "v_pages"), (dict(page_table=0), "page_table"), (dict(cu_q=0), "cu_q"), (dict(kv_len=0), "kv_len"),
    (dict(workspace=0), "workspace"), (dict(workspace=P + 16), "workspace"), (dict(workspace_bytes=0), "workspace"),
])
def test_attention_chunk_refuses(lib, over, word):
    refused(lib, "dls_attention_chunk", dls._ATTENTION_CHUNK, CHUNK, over, word)


def test_null_descriptors_and_empty_batches(lib):
    for name in ("dls_qk_norm_rope", "dls_kv_append", "dls_attention_chunk"):
        assert getattr(lib, name)(None, None) == dls.DLS_ERR_ARG
        assert "desc=NULL" in lib.dls_last_error(None).decode()
    # nothing to do: no pointer is looked at
    assert lib.dls_qk_norm_rope(dls._QK_NORM_ROPE.pack(*{**ROPE, "n_tokens": 0, "q": 0, "positions": 0}.values()), None) == 0
    assert lib.dls_kv_append(dls._KV_APPEND.pack(*{**APPEND, "n_tokens": 0, "k": 0}.values()), None) == 0
    assert lib.dls_kv_append(dls._KV_APPEND.pack(*{**APPEND, "n_seqs": 0}.values()), None) == 0
    assert lib.dls_attention_chunk(dls._ATTENTION_CHUNK.pack(*{**CHUNK, "n_tokens": 0, "o": 0}.values()), None) == 0
    assert lib.dls_attention_chunk(dls._ATTENTION_CHUNK.pack(*{**CHUNK, "n_seqs": 0}.values()), None) == 0


@pytest.mark.parametrize("name,over,word", [
    # rows and weights are read 16 bytes at a time: a view that begins inside such a piece is refused
    ("dls_qk_norm_rope", dict(q_norm=P + 4), "q_norm"), ("dls_qk_norm_rope", dict(k_norm=P + 8), "k_norm"),
    ("dls_qk_norm_rope", dict(positions=P + 2), "positions"), ("dls_kv_append", dict(q_norm=P + 8), "q_norm"),
    ("dls_kv_append", dict(k_norm=P + 4), "k_norm"), ("dls_kv_append", dict(cu_q=P + 1), "cu_q"),
    ("dls_kv_append", dict(status=P + 2), "status"), ("dls_kv_append", dict(status=P + 2, n_tokens=0), "status"),
    ("dls_attention_chunk", dict(kv_len=P + 2), "kv_len"), ("dls_attention_chunk", dict(page_table=P + 2), "page_table"),
    ("dls_attention_chunk", dict(lse=P + 2), "lse"), ("dls_attention_chunk", dict(status=P + 1), "status"),
    # in place, other strides; more tiles than an int counts should cu_q decrease all the time
    ("dls_attention_chunk", dict(o_stride=8192), "in place"),
    ("dls_attention_chunk", dict(n_tokens=1 << 30, n_seqs=4096), "too many"),
    ("dls_attention_chunk", dict(n_tokens=(1 << 30) + 1), "n_tokens"),
])
def test_alignment_and_limits(lib, name, over, word):
    fmt, base = {"dls_qk_norm_rope": (dls._QK_NORM_ROPE, ROPE), "dls_kv_append": (dls._KV_APPEND, APPEND),
                 "dls_attention_chunk": (dls._ATTENTION_CHUNK, CHUNK)}[name]
    refused(lib, name, fmt, base, over, word)


@pytest.mark.parametrize("n_seqs", [(1 << 30) + 1, 0x7fffffff - 30, 0x7fffffff])
def test_kv_append_refuses_more_sequences_than_its_lookup_counts(lib, n_seqs):
    """The search over cu_q probes up to 31 entries past the end before it looks at them: those numbers have to fit an int."""
    refused(lib, "dls_kv_append", dls._KV_APPEND, APPEND, dict(n_seqs=n_seqs), f"n_seqs={n_seqs}")


def test_binding_refuses_an_unknown_pairing():
    k = torch.zeros(3, 2, 64)
    with pytest.raises(ValueError, match="pairing"):
        dls.qk_norm_rope(k, None, torch.zeros(3, dtype=torch.int32), np.ones(32), k, None, pairing="split")


def test_frequencies_of_any_kind_of_array():
    f = dls.rope_inv_freq(64, 10000.0)
    fixed = f.copy()
    fixed.flags.writeable = False
    for given in (f, fixed, f.astype(np.float32), list(f), np.repeat(f, 2)[::2]):
        a, at, rot = dls._inv_freq(given)
        assert rot == 64 and at == a.ctypes.data and np.allclose(a, f, rtol=1e-7, atol=0)
    assert dls._inv_freq(np.zeros(0))[2] == 0 and dls._inv_freq(None) == (None, 0, 0)


def test_workspace_bytes(lib):
    for bad in (0, 8, 24, 136, 256, -16):
        assert dls.attention_chunk_workspace_bytes(bad) == 0
    assert 0 < dls.attention_chunk_workspace_bytes(16) <= dls.attention_chunk_workspace_bytes(128)


def test_rope_inv_freq():
    f = dls.rope_inv_freq(64, 10000.0)
    assert f.dtype == np.float64 and f.shape == (32,)
    assert f[0] == 1.0 and abs(f[16] - 0.01) < 1e-17


def _attend(**over):
    a = dict(q=torch.zeros(4, 8, 64, dtype=torch.float16), k_pages=torch.zeros(5, 2, 32, 64, dtype=torch.float16),
             v_pages=torch.zeros(5, 2, 32, 64, dtype=torch.float16), page_table=torch.zeros(2, 3, dtype=torch.int32),
             cu_q=torch.zeros(3, dtype=torch.int32), kv_len=torch.zeros(2, dtype=torch.int32),
             o=torch.zeros(4, 8, 64, dtype=torch.float16), workspace=torch.zeros(1 << 12, dtype=torch.uint8))
    a.update(over)
    dls.attention_chunk(**a)


def test_binding_refuses_what_does_not_fit_together():
    z = torch.zeros
    for over, word in [
        (dict(), "one CUDA device"),  # host tensors
        (dict(q=z(4, 8, 32, dtype=torch.float16)), "q: shape"), (dict(q=z(4, 512, dtype=torch.float16)), "q: shape"),
        (dict(q=z(4, 8, 64)), "q: type"), (dict(q=z(4, 64, 8, dtype=torch.float16).transpose(1, 2)), "contiguous"),
        (dict(o=z(5, 8, 64, dtype=torch.float16)), "o: shape"), (dict(cu_q=z(2, dtype=torch.int32)), "cu_q"),
        (dict(kv_len=z(2, dtype=torch.int64)), "kv_len"), (dict(page_table=z(6, dtype=torch.int32)), "page_table"),
        (dict(v_pages=z(5, 2, 32, 64)), "v_pages"), (dict(k_pages=z(2, 5, 32, 64, dtype=torch.float16).transpose(0, 1)), "contiguous"),
        (dict(lse=z(4, 8, dtype=torch.float16)), "lse"), (dict(status=z(2, dtype=torch.int32)), "status"),
        (dict(k_pages=z(5, 2, 32, 64, dtype=torch.int8), v_pages=z(5, 2, 32, 64, dtype=torch.int8)), "type"),
    ]:
        with pytest.raises(ValueError, match=word):
            _attend(**over)
    k = z(3, 2, 64)
    with pytest.raises(ValueError, match="q with q_out"):
        dls.qk_norm_rope(k, k, z(3, dtype=torch.int32), None, None, k)
    with pytest.raises(ValueError, match="k: shape"):
        dls.qk_norm_rope(k, z(4, 2, 64), z(3, dtype=torch.int32), None, k, z(4, 2, 64))
    with pytest.raises(ValueError, match="positions"):
        dls.qk_norm_rope(k, None, z(3, dtype=torch.int64), None, k, None)
    with pytest.raises(ValueError, match="q_norm"):
        dls.qk_norm_rope(k, None, z(3, dtype=torch.int32), None, k, None, q_norm=z(32))
    with pytest.raises(ValueError, match="v: shape"):
        dls.kv_append(k, z(3, 2, 32), z(5, 2, 32, 64, dtype=torch.float16), z(5, 2, 32, 64, dtype=torch.float16),
                      z(1, 3, dtype=torch.int32), z(2, dtype=torch.int32), z(1, dtype=torch.int32), None)
    with pytest.raises(ValueError, match="inv_freq"):
        dls.qk_norm_rope(k, None, z(3, dtype=torch.int32), np.ones((2, 2)), k, None)
