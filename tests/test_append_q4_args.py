"""Refusals of the appends with norms, of those to the 4-bit pool and of its gather: no
GPU is reached."""

import pytest
import torch


@pytest.fixture(scope="module")
def B():
    from paged_decode_attention_attn_gb300 import build
    build.build()
    from paged_decode_attention_attn_gb300 import binding
    return binding


FAKE = 1 << 20      # never dereferenced: every check below fails before a CUDA call


def append(B, q4, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, q_stride=1024, k_stride=1024, v_stride=1024, q_out=FAKE,
             q_out_stride=1024, cu=FAKE, positions=FAKE, n=4, batch=2, hq=4, hkv=2, d=128, qw=FAKE,
             kw=FAKE, eps=1e-6, inv=FAKE, rot=128, flags=0, pool=FAKE, scales=FAKE, pool_pages=4,
             table=FAKE, max_pages=4)
    a.update(kw)
    if not q4:
        del a["scales"]
    fn = B.lib.kv_append_rope_q4 if q4 else B.lib.kv_append_norm_rope
    return fn(*a.values(), None, None)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("kw,word", [
    (dict(n=-1), "n_tokens"), (dict(batch=-1), "n_tokens"), (dict(n=(1 << 30) + 1), "n_tokens"),
    (dict(hkv=0), "n_kv_heads"), (dict(hq=0), "n_q_heads"), (dict(q=None), "q_out"),
    (dict(q_out=None), "q_out"), (dict(k=None), "null"), (dict(v=None), "null"),
    (dict(pool=None), "null"), (dict(positions=None), "null"), (dict(table=None), "null"),
    (dict(cu=None), "cu_tokens"), (dict(rot=12), "rot_dim"), (dict(rot=136), "rot_dim"),
    (dict(inv=None), "inv_freq"), (dict(flags=2), "flags"), (dict(k=FAKE + 8), "aligned"),
    (dict(pool=FAKE + 4), "aligned"), (dict(k_stride=1028), "strides"),
    (dict(v_stride=248), "strides"), (dict(pool_pages=0), "pool_pages"),
    (dict(max_pages=0), "pool_pages"), (dict(kw=None), "k_weight"), (dict(qw=None), "q_weight"),
    (dict(qw=FAKE + 2), "aligned"), (dict(kw=FAKE + 1), "aligned"), (dict(eps=0.0), "eps"),
    (dict(eps=-1e-6), "eps"), (dict(eps=float("nan")), "eps"), (dict(eps=2.0), "eps")])
def test_bad_arguments_are_refused(B, q4, kw, word):
    assert append(B, q4, **kw) == B.PA_ERR_INVALID
    assert word in B.last_error()


def test_geometries_and_pools(B):
    assert append(B, False, d=96, rot=96) == B.PA_ERR_UNSUPPORTED
    assert append(B, True, d=64, rot=64) == B.PA_ERR_UNSUPPORTED
    assert append(B, True, scales=None) == B.PA_ERR_INVALID
    assert append(B, True, scales=FAKE + 4) == B.PA_ERR_INVALID
    # without weights eps is not looked at, and one weight alone is refused
    assert append(B, True, qw=None, kw=None, eps=-1.0, rot=12) == B.PA_ERR_INVALID
    assert "rot_dim" in B.last_error()
    assert append(B, True, q=None, q_out=None, qw=FAKE, kw=None) == B.PA_ERR_INVALID
    assert "k_weight" in B.last_error()


def test_gather(B):
    g = [FAKE, FAKE, 4, FAKE, 4, FAKE, FAKE, 4, 2, 2, 128, FAKE, None, None]
    for at, bad, code in ((0, None, -1), (1, FAKE + 4, -1), (1, None, -1), (2, 0, -1), (3, None, -1),
                          (5, None, -1), (6, None, -1), (7, -1, -1), (7, (1 << 30) + 1, -1),
                          (9, 0, -1), (10, 64, -6), (11, FAKE + 16, -1), (11, None, -1)):
        args = list(g)
        args[at] = bad
        assert B.lib.kv_gather_q4(*args) == code, (at, bad)


def test_nothing_to_do_is_no_error(B):
    assert append(B, False, n=0) == B.PA_OK
    assert append(B, True, batch=0) == B.PA_OK
    assert B.lib.kv_gather_q4(0, 0, 0, 0, 0, 0, 0, 0, 3, 1, 128, 0, None, None) == B.PA_OK


def test_binding_refuses_what_it_cannot_pass_on(B):
    t = torch.zeros(1, 64, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        B.kv_append_norm_rope(None, t, t, t, t, t, None, None, t)
    u = torch.zeros(1, 4, 64, 64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        B.kv_append_rope_q4(None, t, t, u, u[..., :4], t, t, None)
    with pytest.raises(ValueError, match="CUDA"):
        B.kv_gather_q4(u, u, t, t, None, t)
