"""Refusals of decode attention over the 8-bit pool: no GPU is reached."""

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def B():
    from paged_decode_attention_attn_gb300 import build
    build.build()
    from paged_decode_attention_attn_gb300 import binding
    return binding


FAKE = 1 << 20      # never dereferenced: every check below fails before a CUDA call


def call(B, tiles=[[[0, 64]]], **kw):
    arr = np.ascontiguousarray(np.asarray(tiles, dtype=np.int32))
    a = dict(q=FAKE, pool=FAKE, scales=FAKE, pages=16, table=FAKE, max_pages=8,
             tiles_ptr=arr.ctypes.data, b=arr.shape[0], t=arr.shape[1], hq=24, hkv=4, d=256,
             scale=0.0625, out=FAKE, lse=FAKE, m=None, ml=None, ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    return B.lib.paged_decode_attn_q8_lse(*a.values(), None)


@pytest.mark.parametrize("kw,word", [
    (dict(b=-1), "B and T"), (dict(hkv=0), "n_q_heads"), (dict(hq=25), "n_q_heads"),
    (dict(hq=0), "n_q_heads"), (dict(q=None), "null"), (dict(pool=None), "null"),
    (dict(scales=None), "null"), (dict(table=None), "null"), (dict(out=None), "null"),
    (dict(lse=None), "null"), (dict(ws=None), "null"), (dict(tiles_ptr=None), "null"),
    (dict(pages=0), "pool_pages"), (dict(max_pages=0), "pool_pages"), (dict(q=FAKE + 8), "q must"),
    (dict(pool=FAKE + 8), "pool must"), (dict(scales=FAKE + 4), "scales must"),
    (dict(out=FAKE + 4), "out must"), (dict(ws=FAKE + 16), "workspace"),
    (dict(ws_bytes=16), "workspace"), (dict(m=FAKE), "merged"),
    (dict(m=FAKE + 4, ml=FAKE), "merged"), (dict(pages=1 << 25), "pool too large"),
    (dict(tiles_=[[[0, 513]]]), "outside"), (dict(tiles_=[[[-1, 3]]]), "outside"),
    (dict(tiles_=[[[9, 3]]]), "outside")])
def test_bad_arguments_are_refused(B, kw, word):
    kw = dict(kw)
    tiles = kw.pop("tiles_", [[[0, 64]]])
    assert call(B, tiles, **kw) == B.PA_ERR_INVALID
    assert word in B.last_error()


def test_unsupported_geometries(B):
    assert call(B, d=64) == B.PA_ERR_UNSUPPORTED
    assert call(B, hq=36) == B.PA_ERR_UNSUPPORTED
    size = B.lib.paged_decode_attn_q8_workspace_bytes
    assert size(4, 2, 24, 4, 256) > 0 and size(4, 2, 24, 4, 128) > 0
    assert size(4, 2, 24, 4, 64) == 0 and size(4, 2, 36, 4, 256) == 0
    assert size(4, 2, 25, 4, 256) == 0 and size(-1, 2, 24, 4, 256) == 0
    assert call(B, ws_bytes=size(1, 1, 24, 4, 256) - 1) == B.PA_ERR_INVALID


def test_no_requests_is_no_error(B):
    assert call(B, b=0, q=None, pool=None) == B.PA_OK
    assert call(B, t=0, q=None, pool=None) == B.PA_OK


def test_binding_refuses_tensors_off_the_gpu(B):
    t = torch.zeros(1, 64, 512, dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="CUDA"):
        B.paged_decode_attn_q8_lse(t, t, t, t, [[[0, 1]]], 1.0, t, t, t)
