"""Decode attention over 8-bit pools in rows that hang on few keys, against the
float64 oracle.

Bounds.  With A = scale max_j sum_d |q_d k_jd|, a score is within 8 steps of 2^-24 of
A, the exponential of it within 2^-21: d = 2^-21 A + 2^-21 relative for a probability
before it is held in four parts of 4 bits and a sign: 2^-19 more.  An error d_j of the
probabilities p_j moves the output, whose sum has the same errors, by sum p_j d_j
(V_j - out), at most (d + 2^-19) sum_j p_j |V_j - out|; the rest is a few FP32
roundings, 8 of 2^-24 of sum_j p_j |V_j|.  A probability times its V scale s_j is held relative to a
power of two that is at most 2^8 times the largest of them, in steps of 2^-32 of it
where it has fewer than 19 bits above that: it is off by half such a step, 2^-25
max_i(p_i s_i), or by itself where that is less, for each |code_j|.  The log-sum-exp
has d alone, and 2^-22 of itself.  (With V scales that are no powers of two, their
reciprocal's 2^-22 joins.)
"""

import numpy as np
import pytest
import torch

from oracle import rope_q8 as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
HQ, HKV = 16, 2
G = HQ // HKV


@pytest.fixture(scope="module")
def B():
    from paged_decode_attention_attn_gb300 import build
    build.build()
    from paged_decode_attention_attn_gb300 import binding
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return binding


def run_and_check(B, lengths, d, seed, q_scale=1.0, odd_scales=False, tiles=None, same_keys=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n, width = len(lengths), -(-max(lengths) // 64)
    pool = (torch.randn(n * width, 64, 2 * HKV * d, generator=g, device=DEV) * 64).to(
        torch.float8_e4m3fn)
    if same_keys:   # equal scores in every row
        pool.view(torch.uint8).view(-1, 2, HKV * d)[:, 0] = pool.view(torch.uint8).view(
            -1, 2, HKV * d)[:1, 0].clone()
    scales = torch.exp2(torch.randint(-8, -5, (n * width, 2 * HKV, 4), generator=g,
                                      device=DEV).float())
    if same_keys:
        scales[:, :HKV] = 2.0 ** -7
    if odd_scales:
        scales[:, HKV:] *= 1 + torch.rand(n * width, HKV, 4, generator=g, device=DEV)
    table = torch.arange(n * width, dtype=torch.int32, device=DEV).view(n, width)
    q = (torch.randn(n, HQ, d, generator=g, device=DEV) * q_scale).bfloat16()
    tiles = np.array([[(0, x)] for x in lengths] if tiles is None else tiles, np.int32)
    T = tiles.shape[1]
    out, lse = torch.empty(n, T, HQ, d, device=DEV), torch.empty(n, T, HQ, device=DEV)
    merged, merged_lse = torch.empty(n, HQ, d, device=DEV), torch.empty(n, HQ, device=DEV)
    ws = B.alloc_workspace_q8(n, T, HQ, HKV, d)
    B.paged_decode_attn_q8_lse(q, pool, scales, table, tiles, d ** -0.5, out, lse, ws,
                               merged_out=merged, merged_lse=merged_lse)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32).item()) == 0
    kv = R.pool_values(pool.view(torch.uint8).cpu().numpy().reshape(-1, 2 * HKV, d),
                       scales.double().cpu().numpy().transpose(0, 2, 1).reshape(-1, 2 * HKV))
    kv = kv.reshape(n, -1, 2 * HKV, d)
    sv = scales[:, HKV:].double().cpu().numpy().transpose(0, 2, 1).reshape(-1, HKV)
    sv = np.repeat(sv, 16, 0).reshape(n, -1, HKV)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    q = q.double().cpu().numpy()
    for b in range(n):
        for t, (lo, hi) in enumerate(tiles[b]):
            if hi == lo:
                continue
            for h in range(HQ):
                K, V = kv[b, lo:hi, h // G], kv[b, lo:hi, HKV + h // G]
                s = K @ q[b, h] * d ** -0.5
                top = s.max()
                p = np.exp(s - top)
                total = p.sum()
                p /= total
                want = p @ V
                A = d ** -0.5 * np.max(np.abs(K) @ np.abs(q[b, h]))
                e = 2.0 ** -21 * A + 2.0 ** -21
                spread = p @ np.abs(V - want)
                small = p * sv[b, lo:hi, h // G]
                floor = np.minimum(2.0 ** -25 * small.max(), small) @ np.abs(
                    V / sv[b, lo:hi, h // G, None])
                bound = floor + (e + 2.0 ** -19) * spread + (2.0 ** -21 + odd_scales * 2.0 ** -22) * (
                    p @ np.abs(V))
                err = np.abs(out[b, t, h] - want)
                assert np.all(err <= bound), (b, t, h, np.max(err / bound))
                x = top + np.log(total)
                assert abs(lse[b, t, h] - x) <= e + 2.0 ** -22 * abs(x), (b, t, h)
    if T == 1:
        assert np.array_equal(merged.double().cpu().numpy(), out[:, 0])


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("odd_scales", [False, True])
def test_requests_of_one_token(B, d, odd_scales):
    """The output is V itself, to an FP32 rounding, whatever the score."""
    run_and_check(B, [1] * 200, d, seed=d, odd_scales=odd_scales)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("odd_scales", [False, True])
def test_rows_that_one_key_of_many_leads(B, d, odd_scales):
    run_and_check(B, [2, 3, 17, 64, 65, 130, 500, 900], d, seed=1, q_scale=16.0,
                  odd_scales=odd_scales)
    run_and_check(B, [2, 3, 17, 64, 65, 130, 500, 900], d, seed=2, q_scale=4.0,
                  odd_scales=odd_scales)


@pytest.mark.parametrize("d", [128, 256])
def test_rows_of_equal_keys_are_averages(B, d):
    run_and_check(B, [2, 3, 16, 48, 129, 640], d, seed=3, same_keys=True)


def test_tiles_of_one_token_and_split_rows(B):
    run_and_check(B, [300], 256, seed=4, tiles=[[(i, i + 1) for i in range(0, 300, 7)]])
    run_and_check(B, [40000], 256, seed=5, q_scale=8.0)       # a unit over many CTAs
    run_and_check(B, [40000], 128, seed=6, q_scale=8.0, odd_scales=True)
