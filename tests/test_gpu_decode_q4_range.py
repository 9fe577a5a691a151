"""The 4-bit decode where scales and scores lie far apart, against the float64 oracle's values.

Tolerances.  With A the largest of scale sum_d |q_d k_jd| over the row's keys, a probability
p_j is within e = 2^-21 A + 2^-20 of itself (FP32 scores, the exponential, the parts that a
probability is held in, their sums), so with S_d = sum_j p_j |V_jd| an output is within (e + 2^-19)
of the largest S of its group of 32 dims: this has no floor, so that groups and keys are held to
their own size.  The log-sum-exp is within e + 2^-22 |lse|."""

import numpy as np
import pytest
import torch

from oracle import rope_q4 as Q

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


class Rows:
    """One request of n tokens in order over its pages: `kv` codes' bytes [n][2 Hkv][D / 2] and
    `scales` bytes [n][2 Hkv][D / 32] are put there by run()."""

    def __init__(self, n, d, seed=0, groups=4):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.n, self.d, self.hq = n, d, HKV * groups
        self.codes = torch.randint(0, 256, (n, 2 * HKV, d // 2), generator=g, device=DEV,
                                   dtype=torch.uint8)
        self.scales = torch.full((n, 2 * HKV, d // 32), 126, dtype=torch.uint8, device=DEV)
        self.q = torch.randn(1, self.hq, d, generator=g, device=DEV).bfloat16()
        self.scale = d ** -0.5

    def run(self, B, behind=255):
        n, d, pages = self.n, self.d, -(-self.n // 64)
        pool = torch.zeros(pages * 64, 2 * HKV, d // 2, dtype=torch.uint8, device=DEV)
        scales = torch.full((pages * 64, 2 * HKV, d // 32), behind, dtype=torch.uint8, device=DEV)
        pool[:n], scales[:n] = self.codes, self.scales
        pool, scales = (x.view(pages, 64, 2 * HKV, -1).transpose(1, 2).contiguous()
                        for x in (pool, scales))
        table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
        self.out = torch.empty(1, 1, self.hq, d, device=DEV)
        self.lse = torch.empty(1, 1, self.hq, device=DEV)
        ws = B.alloc_workspace_q4(1, 1, self.hq, HKV, d)
        B.paged_decode_attn_q4_lse(self.q, pool, scales, table, [[[0, n]]], self.scale, self.out,
                                   self.lse, ws)
        torch.cuda.synchronize()
        assert int(ws[:4].view(torch.int32).item()) == 0

    def check(self):
        kv = Q.values(self.codes.cpu().numpy(), self.scales.cpu().numpy())
        q = self.q[0].double().cpu().numpy()
        G = self.hq // HKV
        for h in range(self.hq):
            k, v = kv[:, h // G], kv[:, HKV + h // G]
            x = self.scale * (k @ q[h])
            A = self.scale * np.max(np.abs(k) @ np.abs(q[h]))
            e = 2.0 ** -21 * A + 2.0 ** -20
            lse = np.max(x) + np.log(np.sum(np.exp(x - np.max(x))))
            p = np.exp(x - lse)
            S = np.repeat((p @ np.abs(v)).reshape(-1, 32).max(1), 32)
            err = np.abs(self.out[0, 0, h].double().cpu().numpy() - p @ v)
            assert np.all(err <= (e + 2.0 ** -19) * S), (h, np.max(err / np.maximum(S, 1e-300)), e)
            assert abs(float(self.lse[0, 0, h]) - lse) <= e + 2.0 ** -22 * abs(lse), h


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("n,at", [(2, 1), (300, 7), (300, 299), (9000, 4000), (9000, 8999)])
@pytest.mark.parametrize("p_exp,v_exp", [(-104, 105), (-104, 106), (-108, 109), (-110, 110),
                                         (-100, 60), (-60, 100)])
def test_a_key_of_little_weight_and_far_larger_values(B, d, n, at, p_exp, v_exp):
    """Key 0 has the largest score and V near 2^-30, key `at` the probability 2^p_exp and V 2^v_exp
    times as large; the others' scores lie as far below again."""
    r = Rows(n, d, seed=at)
    r.q[:] = 1.0
    r.scale = -p_exp * np.log(2.0) / d
    r.codes[:, :HKV] = 0xAA                               # minus ones
    r.codes[0, :HKV], r.codes[at, :HKV] = 0x22, 0         # ones, zeros
    r.scales[:, :HKV] = 127
    r.scales[:, HKV:] = 127 - 30
    r.scales[at, HKV:] = 127 - 30 + v_exp
    r.run(B)
    r.check()


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("top,low,v_exp", [(104, 0, 96), (106, 4, 112), (106, 4, 105), (107, 3, 111)])
def test_a_page_of_little_weight_and_far_larger_values(B, d, top, low, v_exp):
    """The same with a whole page of such keys, alike in scale, behind the first in one CTA's
    part of a long history: scores of top and -low top / 128 in powers of two."""
    r = Rows(80_000, d, seed=3)
    r.q[:] = 1.0
    r.scale = top * np.log(2.0) / d
    r.codes[:, :HKV] = 0xAA
    r.codes[0, :HKV], r.codes[512:576, :HKV] = 0x22, 0
    r.codes[512:576, :HKV, :low * d // 256] = 0xAA
    r.scales[:, :HKV] = 127
    r.scales[:, HKV:] = 127 - 30
    r.scales[512:576, HKV:] = 127 - 30 + v_exp
    r.run(B)
    r.check()


def times(x, e):
    """bf16 x * 2^e for any e in range."""
    return (x.float() * 2.0 ** (e // 2) * 2.0 ** (e - e // 2)).bfloat16()


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("k_exp,q_exp", [(112, -113), (113, -114), (112, -118), (119, -125),
                                         (106, -107), (126, -131), (-60, 60), (60, -66),
                                         (-60, 110), (-127, 122), (-126, 121), (-100, 90),
                                         (112, -107), (112, -105), (126, -106), (120, -40),
                                         (111, 0)])
def test_scores_within_range_from_factors_far_apart(B, d, k_exp, q_exp):
    """K's scale and q far from 1, the scores near it."""
    r = Rows(200, d, seed=k_exp + 200)
    r.scales[:, :HKV] = 127 + k_exp
    r.q = times(r.q, q_exp)
    r.scale *= 2.0 ** -(q_exp + k_exp)
    r.run(B)
    r.check()


@pytest.mark.parametrize("d", [128, 256])
def test_a_few_keys_of_large_scales(B, d):
    """Every 17th key is large, the others small beside it; a head of q is zero."""
    r = Rows(700, d, seed=5)
    r.scales[:, :HKV] = 127 + 100
    r.scales[::17, :HKV] = 127 + 110
    r.q = times(r.q, -111)
    r.q[0, 3] = 0
    r.run(B)
    r.check()


@pytest.mark.parametrize("d", [128, 256])
def test_far_scores_stay_finite(B, d):
    """Scores of 10^34: finite, and the key of the largest has the whole weight."""
    r = Rows(70, d, seed=6)
    r.codes[:, :HKV] = 0x77                               # sixes
    r.codes[::2, :HKV] = 0xFF
    r.codes[41, :HKV], r.codes[40, :HKV] = 0x77, 0xFF
    r.scales[:, :HKV] = 127 + 106
    r.scales[41, :HKV] = 127 + 107
    r.q[:] = 1.0
    r.scale = 1 / 16
    r.run(B)
    v = Q.values(*(x[41, HKV:].cpu().numpy() for x in (r.codes, r.scales)))
    assert np.array_equal(r.out[0, 0].double().cpu().numpy(), np.repeat(v, 4, 0))
    want = d * 6 * 2.0 ** 107 / 16
    assert torch.all((r.lse.double() / want - 1).abs() <= 2.0 ** -21)


@pytest.mark.parametrize("d", [128, 256])
def test_rows_that_are_not_live_do_not_reach_the_bits_of_others(B, d):
    outs = []
    for behind in (255, 254, 0, 127):
        r = Rows(130, d, seed=7)
        r.run(B, behind)
        r.check()
        outs.append((r.out, r.lse))
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, outs[0]))


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("at,gap", [(-60, 20), (-60, 27), (-80, 24), (-60, 18), (-127, 30), (-60, 70)])
@pytest.mark.parametrize("n,every", [(70, 3), (700, 64), (3000, 2999)])
def test_small_groups_beside_larger_ones_of_other_keys(B, d, at, gap, n, every):
    """The last group of dims has the scale 2^at in every key, the others too but for the first, and
    each `every`-th key after it, where they are 2^gap times as large."""
    r = Rows(n, d, seed=gap)
    r.scales[:, HKV:] = 127 + at
    r.scales[::every, HKV:, :-1] = 127 + at + gap
    r.run(B)
    r.check()


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("byte", [0, 67, 100])
def test_groups_of_zeros_of_any_scale(B, d, byte):
    """Groups without codes do not change a bit of the others, whatever their scale."""
    outs = []
    for b in (byte, 126):
        r = Rows(1000, d, seed=8)
        r.codes[:, HKV:, -32:] = 0
        r.scales[:, HKV:, -2:] = b
        r.run(B)
        assert torch.all(r.out[..., -64:] == 0)
        r.check() if b == 126 else None
        outs.append((r.out, r.lse))
    assert all(torch.equal(x, y) for x, y in zip(*outs))


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("offsets", [[0, 20], [0, 30], [0, 50, 20, 30], [0, 0, 0, 70], [0, 16], [0, 17]])
@pytest.mark.parametrize("n", [3, 64, 1000])
def test_groups_of_fixed_distances_in_every_key(B, d, offsets, n):
    """Groups of dims 2^offset below the first in all keys alike: each is held to its own size."""
    r = Rows(n, d, seed=n)
    e = torch.tensor((offsets * 8)[: d // 32], dtype=torch.uint8, device=DEV)
    r.scales[:, HKV:] = 127 + 20 - e
    r.run(B)
    r.check()


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("at", [0, 100, 9_999, 19_999])
@pytest.mark.parametrize("groups", [slice(None), slice(0, 1), slice(2, 3)])
def test_one_key_of_far_larger_values_in_a_long_history(B, d, at, groups):
    """Its pages, and those that its team has after it, go in fp32."""
    r = Rows(20_000, d, seed=at)
    r.scales[at, HKV:, groups] = 127 + 22
    r.run(B)
    r.check()
