"""Decode attention with more kv heads than 16 bits count, over a bf16 and an 8-bit
pool of one page, against the float64 oracle at heads on both sides of 65,536.

Tolerances: with A = scale max_j sum_d |q_d k_jd|, about 8 here, scores and
exponentials leave 2^-21 A + 2^-18 of a probability, and a row may hang on one key
(2^-16, the kernels' coarser probabilities): times max |V| for the output; the
log-sum-exp within the first.  bf16 probabilities of the bf16 kernel: 2^-8 more."""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda"
HKV, D, L = 65_600, 256, 37
HEADS = [0, 1, 1023, 1024, 65_534, 65_535, 65_536, 65_537, 65_599]


@pytest.fixture(scope="module")
def B():
    from paged_decode_attention_attn_gb300 import build
    build.build()
    from paged_decode_attention_attn_gb300 import binding
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return binding


@pytest.mark.parametrize("bits", [16, 8])
def test_heads_beyond_16_bits(B, bits):
    g = torch.Generator(device=DEV).manual_seed(bits)
    q = torch.randn(1, HKV, D, generator=g, device=DEV).bfloat16()
    pool = torch.randn(1, 64, 2 * HKV * D, generator=g, device=DEV, dtype=torch.bfloat16)
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    tiles = np.array([[[0, L]]], np.int32)
    out, lse = torch.zeros(1, 1, HKV, D, device=DEV), torch.zeros(1, 1, HKV, device=DEV)
    if bits == 16:
        ws = B.alloc_workspace(1, 1, HKV, HKV, D)
        B.paged_decode_attn_lse(q, pool, table, tiles, D ** -0.5, out, lse, ws)
    else:
        pool = pool.to(torch.float8_e4m3fn)
        scales = torch.ones(1, 2 * HKV, 4, device=DEV)
        ws = B.alloc_workspace_q8(1, 1, HKV, HKV, D)
        B.paged_decode_attn_q8_lse(q, pool, scales, table, tiles, D ** -0.5, out, lse, ws)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32).item()) == 0
    rows = pool.view(64, 2 * HKV, D)[:L]
    at = torch.tensor(HEADS, device=DEV)
    K, V = (rows.view(torch.uint8 if bits == 8 else torch.int16)[:, at + i * HKV].view(
        rows.dtype).float().double().cpu().numpy() for i in (0, 1))
    q = q[0, at].double().cpu().numpy()
    want, wl = oracle.tile_attention(q, K, V, [(0, L)], D ** -0.5)
    e = 2.0 ** -21 * 16 + 2.0 ** -18
    bound = (e + 2.0 ** -16 + (2.0 ** -8 if bits == 16 else 0)) * np.abs(V).max()
    assert np.abs(out[0, 0, at].double().cpu().numpy() - want[0]).max() <= bound
    assert np.abs(lse[0, 0, at].double().cpu().numpy() - wl[0]).max() <= e + 2.0 ** -20
