"""Decode attention over 8-bit pools whose V scales span the whole documented
range, [2^-100, 2^120] and zero, against the float64 oracle.

Tolerances as in test_gpu_decode_q8.py: with A = scale max_j sum_d |q_d k_jd|, a
probability is within e = 2^-21 A + 2^-18 relative and the output within (e +
2^-16) max |V|; the log-sum-exp, which V's scales have no part in, within e + 2^-22
|lse|.
"""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda"
HQ, HKV = 6, 2
G = HQ // HKV


@pytest.fixture(scope="module")
def B():
    from paged_decode_attention_attn_gb300 import build
    build.build()
    from paged_decode_attention_attn_gb300 import binding
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return binding


class Rows:
    """One request of whole blocks: codes, and a K and a V exponent per block (None: a
    scale of zero), the same for every head."""

    def __init__(self, k_exp, v_exp, d=128, seed=0, q_scale=1.0, tiles=None, scale=None):
        n = 16 * len(v_exp)
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.n, self.d, self.scale = n, d, d ** -0.5 if scale is None else scale
        self.tiles = [(0, n)] if tiles is None else tiles
        pages = -(-n // 64)
        self.q = (torch.randn(1, HQ, d, generator=g, device=DEV) * q_scale).bfloat16()
        codes = torch.randn(pages, 64, 2 * HKV * d, generator=g, device=DEV) * 64
        self.pool = codes.to(torch.float8_e4m3fn)
        value = lambda e: [0.0 if x is None else 2.0 ** x for x in e] + [1.0] * (4 * pages - len(e))
        both = torch.tensor([value(k_exp), value(v_exp)], device=DEV)       # [K | V][block]
        self.scales = both.view(2, pages, 1, 4).permute(1, 0, 2, 3).expand(
            pages, 2, HKV, 4).reshape(pages, 2 * HKV, 4).contiguous()
        self.table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]

    def run(self, B):
        T = len(self.tiles)
        self.out = torch.empty(1, T, HQ, self.d, device=DEV)
        self.lse = torch.empty(1, T, HQ, device=DEV)
        self.merged = torch.empty(1, HQ, self.d, device=DEV)
        self.merged_lse = torch.empty(1, HQ, device=DEV)
        ws = B.alloc_workspace_q8(1, T, HQ, HKV, self.d)
        B.paged_decode_attn_q8_lse(self.q, self.pool, self.scales, self.table,
                                   np.array([self.tiles], np.int32), self.scale, self.out, self.lse,
                                   ws, merged_out=self.merged, merged_lse=self.merged_lse)
        torch.cuda.synchronize()
        assert int(ws[:4].view(torch.int32).item()) == 0

    def values(self):
        by = self.scales.double().permute(0, 2, 1).repeat_interleave(16, 1)   # [page][token][head]
        kv = self.pool.float().double().view(-1, 64, 2 * HKV, self.d) * by[..., None]
        kv = kv.view(-1, 2 * HKV, self.d)[:self.n].cpu().numpy()
        return self.q[0].double().cpu().numpy(), kv[:, :HKV], kv[:, HKV:]

    def check(self):
        q, K, V = self.values()
        outs, lses = oracle.tile_attention(q, K, V, self.tiles, self.scale)
        want = list(zip(outs, lses)) + [oracle.lse_merge(outs, lses)]
        got = [(self.out[0, t], self.lse[0, t]) for t in range(len(self.tiles))]
        spans = list(self.tiles) + [(0, self.n)]
        for (o, l), (wo, wl), (lo, hi) in zip(got + [(self.merged[0], self.merged_lse[0])], want,
                                              spans):
            for h in range(HQ):
                A = self.scale * np.max(np.abs(K[lo:hi, h // G]) @ np.abs(q[h]))
                e = 2.0 ** -21 * A + 2.0 ** -18
                assert abs(float(l[h]) - wl[h]) <= e + 2.0 ** -22 * abs(wl[h]), (h, lo, hi)
                err = np.max(np.abs(o[h].double().cpu().numpy() - wo[h]))
                assert err <= (e + 2.0 ** -16) * np.max(np.abs(V[lo:hi, h // G])), (h, lo, hi)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("near,far", [(-100, 40), (-60, 99), (-100, 120), (None, 99), (None, 120),
                                      (-100, -30)])
@pytest.mark.parametrize("order", ["up", "down", "far last", "far in the other group"])
def test_v_scales_as_far_apart_as_they_may_be(B, near, far, order, d):
    """A key's place in the sum does not depend on its V scale, nor on which of them
    comes first: in the same step, in a later one, or in the other group's."""
    v = {"up": [near] * 48 + [far] * 48, "down": [far] * 48 + [near] * 48,
         "far last": [near] * 95 + [far], "far in the other group": [near] * 8 + [far] * 8}[order]
    r = Rows([-7] * len(v), v, d=d, seed=len(v))
    r.run(B)
    r.check()


@pytest.mark.parametrize("exp", [-100, -60, 60, 99, 110, 118])
def test_small_probabilities_beside_large_v_scales(B, exp):
    """One key far above the others, which together weigh as much: none of them is
    lost, whatever the scale that V has."""
    n = 4096
    r = Rows([-7] * (n // 16), [exp] * (n // 16), seed=5)
    r.q[0] = 0
    r.q[0, :, 0] = 1.0
    codes = torch.zeros_like(r.pool.view(-1, 2 * HKV, 128), dtype=torch.float32)
    codes[:, :HKV, 0] = -224.0                   # -1.75: far below the first key's score
    codes[0, :HKV, 0] = 224.0
    rest = r.pool.view(-1, 2 * HKV, 128).float()[:, HKV:]
    codes[:, HKV:] = rest / 4
    r.pool = codes.to(torch.float8_e4m3fn).view(r.pool.shape)
    r.scale = np.log(n - 1.0) / 3.5              # the others' probabilities sum to the first's
    r.run(B)
    _, wl = oracle.tile_attention(*r.values()[:1], *r.values()[1:], r.tiles, r.scale)
    r.scale = float(r.scale)
    r.check()
    # the other keys are half of the sum
    assert np.allclose(wl[0], 1.75 * r.scale + np.log(2.0), atol=1e-9)


def test_ramps_and_cut_units(B):
    """V scales that climb and fall through the range by turns, scores that do the same,
    in tiles and split over CTAs."""
    rng = np.random.default_rng(8)
    v = np.concatenate([np.arange(-100, 121, 2), np.arange(120, -101, -4), rng.integers(-100, 121, 600)])
    k = rng.integers(-12, -3, len(v))
    n = 16 * len(v)
    for tiles in ([(0, n)], [(0, 1000), (1000, 1001), (1001, n)]):
        r = Rows(k.tolist(), v.tolist(), d=256, seed=9, tiles=tiles)
        r.run(B)
        r.check()


def test_the_largest_rows_an_append_can_write(B):
    """bf16 values up to the type's largest give V scales up to 2^120: what the append
    writes is what the decode reads."""
    n, d = 200, 128
    g = torch.Generator(device=DEV).manual_seed(6)
    k = torch.randn(n, HKV, d, generator=g, device=DEV).bfloat16()
    v = (torch.randn(n, HKV, d, generator=g, device=DEV).clamp(-3, 3) * 2.0 ** 126).bfloat16()
    v[0, 0, 0] = torch.finfo(torch.bfloat16).max
    r = Rows([0] * 16, [0] * 16, seed=7)
    r.n, r.tiles = n, [(0, n)]
    B.kv_append_rope_q8(None, k, v, r.pool, r.scales, r.table,
                        torch.zeros(1, dtype=torch.int32, device=DEV), None,
                        cu_tokens=torch.tensor([0, n], dtype=torch.int32, device=DEV))
    assert float(r.scales[:, HKV:].max()) == 2.0 ** 120
    r.run(B)
    r.check()


@pytest.mark.parametrize("k_exp,q_exp", [(112, -113), (113, -114), (112, -118), (119, -125),
                                         (104, -110), (-60, 60), (60, -66), (-60, 110)])
def test_scores_within_range_from_factors_far_apart(B, k_exp, q_exp):
    """K's scale and q far from 1, their product near it."""
    n = 20
    r = Rows([k_exp] * n, [-6] * n, seed=k_exp + 200)
    r.q = (r.q.float() * 2.0 ** min(q_exp, 100)).bfloat16()
    if q_exp > 100:
        r.q = (r.q.float() * 2.0 ** (q_exp - 100)).bfloat16()
        r.scale *= 2.0 ** -(q_exp + k_exp + 6)
    r.run(B)
    r.check()
    assert r.out.isfinite().all()


def test_rows_of_zeros_in_a_block_of_a_large_scale(B):
    """K codes of zero under a scale near the top, and q large: their scores are 0."""
    n = 8
    r = Rows([119] * n, [-6] * n, seed=17)
    r.pool.view(torch.uint8).view(-1, 2, HKV * r.d)[:, 0] = 0
    r.q = (r.q.float() * 2.0 ** 30).bfloat16()
    r.run(B)
    r.check()
    assert r.out.isfinite().all() and torch.allclose(r.lse, torch.log(torch.tensor(16.0 * n)))


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("apart", [6, 9, 12, 14, 16, 20, 26, 32])
def test_probabilities_beside_a_larger_v_scale_count_in_full(B, apart, d):
    """A block whose V scale is 2^apart below the next one's: what its keys' products lose
    to the parts' smallest step does not change what they weigh."""
    for seed in range(4):
        r = Rows([-7] * 9, [40 - apart] * 4 + [40] + [40 - apart] * 4, d=d, seed=apart + 50 * seed,
                 q_scale=[1.0, 4.0, 2.0, 0.1][seed], tiles=[(0, 144), (63, 70), (50, 144)])
        r.run(B)
        r.check()


@pytest.mark.parametrize("exp", [-140, -127, -120])
def test_v_scales_below_the_range_are_as_good_as_zero(B, exp):
    """Beside scales of 1: the keys count, their values do not show."""
    for v in ([exp] * 16 + [0] * 16, [0] * 16 + [exp] * 16, [exp] * 31 + [0]):
        r = Rows([-7] * 32, v, seed=3)
        r.run(B)
        assert r.out.isfinite().all() and r.merged.isfinite().all()
        r.check()
