"""Refusals of the rotated appends and the 8-bit gather: no GPU is reached."""

import pytest
import torch


@pytest.fixture(scope="module")
def B():
    from paged_decode_attention_attn_gb300 import build
    build.build()
    from paged_decode_attention_attn_gb300 import binding
    return binding


FAKE = 1 << 20      # never dereferenced: every check below fails before a CUDA call


def append(B, q8=False, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, q_stride=1024, k_stride=1024, v_stride=1024, q_out=FAKE,
             q_out_stride=1024, cu=FAKE, positions=FAKE, n=4, batch=2, hq=4, hkv=2, d=128, inv=FAKE,
             rot=128, flags=0, pool=FAKE, scales=FAKE, pool_pages=4, table=FAKE, max_pages=4)
    a.update(kw)
    head = [a[x] for x in ("q", "k", "v", "q_stride", "k_stride", "v_stride", "q_out",
                           "q_out_stride", "cu", "positions", "n", "batch", "hq", "hkv", "d", "inv",
                           "rot", "flags", "pool")]
    tail = [a["pool_pages"], a["table"], a["max_pages"], None, None]
    if q8:
        return B.lib.kv_append_rope_q8(*head, a["scales"], *tail)
    return B.lib.kv_append_rope(*head, *tail)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kw,word", [
    (dict(n=-1), "n_tokens"), (dict(batch=-1), "n_tokens"), (dict(hkv=0), "n_kv_heads"),
    (dict(hq=0), "n_q_heads"), (dict(q=None), "q_out"), (dict(q_out=None), "q_out"),
    (dict(k=None), "null"), (dict(v=None), "null"), (dict(pool=None), "null"),
    (dict(positions=None), "null"), (dict(table=None), "null"), (dict(cu=None), "cu_tokens"),
    (dict(rot=12), "rot_dim"), (dict(rot=136), "rot_dim"), (dict(rot=-8), "rot_dim"),
    (dict(inv=None), "inv_freq"), (dict(flags=2), "flags"), (dict(k=FAKE + 8), "aligned"),
    (dict(pool=FAKE + 4), "aligned"), (dict(q_out=FAKE + 2), "aligned"),
    (dict(k_stride=1028), "strides"), (dict(v_stride=248), "strides"),
    (dict(q_stride=504), "strides"), (dict(pool_pages=0), "pool_pages"),
    (dict(max_pages=0), "pool_pages")])
def test_bad_arguments_are_refused(B, q8, kw, word):
    assert append(B, q8, **kw) == B.PA_ERR_INVALID
    assert word in B.last_error()


def test_head_dims_that_are_not_built(B):
    assert append(B, d=96, rot=96) == B.PA_ERR_UNSUPPORTED
    assert append(B, True, d=64, rot=64) == B.PA_ERR_UNSUPPORTED
    assert append(B, True, scales=None) == B.PA_ERR_INVALID
    assert append(B, True, scales=FAKE + 4) == B.PA_ERR_INVALID
    g = [FAKE, FAKE, 4, FAKE, 4, FAKE, FAKE, 4, 2, 2, 128, FAKE, None, None]
    for at, bad, code in ((0, None, -1), (1, FAKE + 4, -1), (2, 0, -1), (5, None, -1), (7, -1, -1),
                          (9, 0, -1), (10, 64, -6), (11, FAKE + 8, -1), (11, FAKE + 16, -1),
                          (11, None, -1)):
        args = list(g)
        args[at] = bad
        assert B.lib.kv_gather_q8(*args) == code, (at, bad)


def test_more_rows_than_32_bits_number_are_refused(B):
    n = (1 << 30) + 1
    for q8 in (False, True):
        assert append(B, q8, n=n) == B.PA_ERR_INVALID and "n_tokens" in B.last_error()
    assert B.lib.kv_gather_q8(FAKE, FAKE, 4, FAKE, 4, FAKE, FAKE, n, 2, 2, 128, FAKE, None,
                              None) == B.PA_ERR_INVALID


def test_nothing_to_do_is_no_error(B):
    assert append(B, n=0) == B.PA_OK
    assert append(B, True, batch=0) == B.PA_OK
    assert B.lib.kv_gather_q8(0, 0, 0, 0, 0, 0, 0, 0, 3, 1, 128, 0, None, None) == B.PA_OK


def test_binding_refuses_tensors_off_the_gpu(B):
    t = torch.zeros(1, 64, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        B.kv_append_rope(None, t, t, t, t, t, None)
    with pytest.raises(ValueError, match="scales"):
        B.kv_append_rope_q8(None, t, t, t, None, t, t, None)
    with pytest.raises(ValueError, match="CUDA"):
        B.kv_gather_q8(t, t, t, t, None, t)
