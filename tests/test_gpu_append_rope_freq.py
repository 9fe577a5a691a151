"""Frequencies that are not finite: their pairs become NaN in q, in the bf16 pool and
in the 8-bit pool, at position 0 as elsewhere, and nothing else does."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
HQ, HKV, D, ROT = 4, 2, 128, 96


@pytest.fixture(scope="module")
def B():
    from paged_decode_attention_attn_gb300 import build
    build.build()
    from paged_decode_attention_attn_gb300 import binding
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return binding


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("start", [0, 12345])
def test_pairs_of_a_frequency_that_is_not_finite(B, bad, interleaved, start):
    n, pair = 21, 7
    g = torch.Generator(device=DEV).manual_seed(start)
    qkv = torch.randn(n, HQ + 2 * HKV, D, generator=g, device=DEV).bfloat16()
    q, k, v = qkv.split([HQ, HKV, HKV], 1)
    inv = torch.from_numpy((10000.0 ** (-np.arange(ROT // 2) / (ROT // 2))).astype(np.float32)).to(DEV)
    inv[pair] = bad
    pages = (start + n) // 64 + 1
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    pos = torch.tensor([start], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    where = torch.zeros(D, dtype=torch.bool, device=DEV)
    where[[2 * pair, 2 * pair + 1] if interleaved else [pair, pair + ROT // 2]] = True
    q_out = torch.zeros(n, HQ, D, dtype=torch.bfloat16, device=DEV)
    pool = torch.zeros(pages, 64, 2 * HKV * D, dtype=torch.bfloat16, device=DEV)
    B.kv_append_rope(q, k, v, pool, table, pos, inv, q_out, cu_tokens=cu, interleaved=interleaved)
    rows = pool.view(-1, 2 * HKV, D)[start:start + n]
    assert q_out[..., where].isnan().all() and q_out[..., ~where].isfinite().all()
    assert rows[:, :HKV][..., where].isnan().all() and rows[:, :HKV][..., ~where].isfinite().all()
    assert torch.equal(rows[:, HKV:], v)
    pool8 = torch.zeros(pages, 64, 2 * HKV * D, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(pages, 2 * HKV, 4, device=DEV)
    q_out.zero_()
    B.kv_append_rope_q8(q, k, v, pool8.view(torch.float8_e4m3fn), scales, table, pos, inv, q_out,
                        cu_tokens=cu, interleaved=interleaved)
    codes = pool8.view(-1, 2 * HKV, D)[start:start + n].view(torch.float8_e4m3fn).float()
    assert q_out[..., where].isnan().all() and q_out[..., ~where].isfinite().all()
    assert codes[:, :HKV][..., where].isnan().all() and codes[:, :HKV][..., ~where].isfinite().all()
    assert codes[:, HKV:].isfinite().all() and scales.isfinite().all()
