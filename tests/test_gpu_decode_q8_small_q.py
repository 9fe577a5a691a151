"""Decode attention over 8-bit pools where K is large in channels in which q is far
below its head's largest value, against the float64 oracle.

Bounds.  K is zero where q is large, so the scores come from the small values alone:
with A = scale max_j sum_d |q_d k_jd| over those, FP32 sums and the scaling leave 8
steps of 2^-24 of A, the exponential 2^-21, and q's own representation 2^-32 of its
largest value: r = scale 2^-32 max |q| max_j sum_d |k_jd|.  d = 2^-21 A + 2^-21 + r
relative for a probability, and 2^-19 more where it is held in parts; the output is
within (d + 2^-19) sum_j p_j |V_j - out| + 2^-21 sum_j p_j |V_j| + 2^-25 max_j(p_j s_j)
sum_j |code_j| (steps of the smallest probabilities, s_j V's scale), the log-sum-exp
within d + 2^-22 of itself.
"""

import numpy as np
import pytest
import torch

from oracle import rope_q8 as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
HKV = 2


@pytest.fixture(scope="module")
def B():
    from paged_decode_attention_attn_gb300 import build
    build.build()
    from paged_decode_attention_attn_gb300 import binding
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return binding


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("below", [10, 12, 13, 14, 16, 20, 24, 28, 34])
@pytest.mark.parametrize("hq", [16, 6])
def test_small_values_of_q_keep_their_bits(B, hq, below, d):
    """Requests of several lengths (units after a CTA's first take another path), an
    eighth of the channels 2^-below under the largest, K zero in the others."""
    lengths = [1, 2, 17, 64, 130, 300] * 60
    g = torch.Generator(device=DEV).manual_seed(100 * below + d)
    n, width, G = len(lengths), -(-max(lengths) // 64), hq // HKV
    small = torch.arange(d, device=DEV) % 8 == 5
    q = torch.randn(n, hq, d, generator=g, device=DEV).clamp(-4, 4)
    q[:, :, 0] = 3.999
    q = torch.where(small, q / 2 * 2.0 ** -below, q).bfloat16()
    k = torch.randn(n * width, 64, HKV, d, generator=g, device=DEV) * 64 * small
    v = torch.randn(n * width, 64, HKV, d, generator=g, device=DEV) * 64
    pool = torch.cat([k, v], 2).to(torch.float8_e4m3fn).view(n * width, 64, 2 * HKV * d)
    scales = torch.full((n * width, 2 * HKV, 4), 2.0 ** -6, device=DEV)
    table = torch.arange(n * width, dtype=torch.int32, device=DEV).view(n, width)
    tiles = np.array([[(0, x)] for x in lengths], np.int32)
    scale = 2.0 ** below / 8
    out, lse = torch.empty(n, 1, hq, d, device=DEV), torch.empty(n, 1, hq, device=DEV)
    ws = B.alloc_workspace_q8(n, 1, hq, HKV, d)
    B.paged_decode_attn_q8_lse(q, pool, scales, table, tiles, scale, out, lse, ws)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32).item()) == 0
    kv = R.pool_values(pool.view(torch.uint8).cpu().numpy().reshape(-1, 2 * HKV, d),
                       scales.double().cpu().numpy().transpose(0, 2, 1).reshape(-1, 2 * HKV))
    kv = kv.reshape(n, -1, 2 * HKV, d)
    q, out = q.double().cpu().numpy(), out.double().cpu().numpy()
    lse = lse.double().cpu().numpy()
    for b in list(range(12)) + list(range(n - 48, n)):
        for h in range(hq):
            K, V = kv[b, :lengths[b], h // G], kv[b, :lengths[b], HKV + h // G]
            s = K @ q[b, h] * scale
            p = np.exp(s - s.max())
            x = s.max() + np.log(p.sum())
            p /= p.sum()
            want = p @ V
            A = scale * np.max(np.abs(K) @ np.abs(q[b, h]))
            held = scale * 2.0 ** -32 * np.max(np.abs(q[b, h])) * np.max(np.sum(np.abs(K), 1))
            e = 2.0 ** -21 * A + 2.0 ** -21 + held
            assert abs(lse[b, 0, h] - x) <= e + 2.0 ** -22 * abs(x), (b, h)
            bound = ((e + 2.0 ** -19) * (p @ np.abs(V - want)) + 2.0 ** -21 * (p @ np.abs(V)) +
                     np.minimum(2.0 ** -25 * p.max(), p) @ np.abs(V))
            assert np.all(np.abs(out[b, 0, h] - want) <= bound), (b, h)
