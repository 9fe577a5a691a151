"""Appends with norms (bf16 and 4-bit pools) and the gather of 4-bit rows, against the
float64 oracle.

Tolerances.  A normed value carries the sum of squares (at most 16 additions in a lane
and 5 between lanes, half their relative error through the root), the root's two units
in the last place and three products: 2^-20 relative in all.  A rotated one 4e-7 (|x1|
+ |x2|) for sine, cosine, two products and a sum.  With u the sum of both over a
rotated value's pair, a bf16 result is within u plus half a step (2^-8 relative) of the
exact value, a 4-bit value within u plus half a step of e2m1 at its scale: 0.25, 0.5 or 1
below 2, 4 and 6 (1 at most by saturation inside u).  A scale may be the one of any group
within u.  Values that are neither normed nor rotated are exact.
"""

import numpy as np
import pytest
import torch

from oracle import rope_q4 as Q
from oracle import rope_q8 as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6


@pytest.fixture(scope="module")
def B():
    from paged_decode_attention_attn_gb300 import build
    build.build()
    from paged_decode_attention_attn_gb300 import binding
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return binding


class Step:
    """One ragged append: lengths of new tokens and positions, fused qkv."""

    def __init__(self, new, past, hq=6, hkv=2, d=128, rot=None, inter=False, pad=0, seed=0,
                 fused=True, spare=3, norm=True, eps=EPS, has_q=True):
        rot = d if rot is None else rot
        rng = np.random.default_rng(seed)
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.new, self.past = np.asarray(new), np.asarray(past)
        self.hq, self.hkv, self.d, self.inter, self.eps = hq, hkv, d, inter, eps
        cu = np.concatenate([[0], np.cumsum(self.new)])
        self.n = int(cu[-1])
        n = self.n + pad
        qkv = torch.randn(n, hq + 2 * hkv, d, generator=g, device=DEV) * \
            torch.exp(torch.randn(1, hq + 2 * hkv, d, generator=g, device=DEV))
        self.q, self.k, self.v = qkv.bfloat16().split([hq, hkv, hkv], 1)
        if not fused:
            self.q, self.k, self.v = (t.contiguous() for t in (self.q, self.k, self.v))
        if not has_q:
            self.q = None
        w = torch.exp(0.5 * torch.randn(2, d, generator=g, device=DEV))
        w[:, 3] *= -1
        self.qw, self.kw = (w[0], w[1]) if norm else (None, None)
        half = rot // 2
        self.inv = (10000.0 ** (-np.arange(half) / max(1, half))).astype(np.float32)
        ends = self.past + self.new
        width = int(max(1, -(-int(ends.max()) // 64)))
        used = [range(int(p) // 64, -(-int(e) // 64)) if e > p else [] for p, e in zip(past, ends)]
        self.pages = sum(len(u) for u in used) + spare
        perm = rng.permutation(self.pages)
        table = np.zeros((len(new), width), np.int32)
        at = 0
        for b, u in enumerate(used):
            for p in u:
                table[b, p] = perm[at]
                at += 1
        places = R.token_places(cu, self.past, table)
        rows = np.array([p[3] for p in places], dtype=np.int64)
        self.pos = np.array([p[2] for p in places], dtype=np.int64)
        self.page, self.row = (torch.from_numpy(x).to(DEV) for x in (rows // 64, rows % 64))
        self.table = torch.from_numpy(table).to(DEV)
        self.positions = torch.from_numpy(self.past.astype(np.int32)).to(DEV)
        self.cu = None if np.all(self.new == 1) and not pad else \
            torch.from_numpy(cu.astype(np.int32)).to(DEV)
        self.inv_dev = torch.from_numpy(self.inv).to(DEV) if half else None
        self.q_out = torch.full((n, hq, d), 7.0, device=DEV).bfloat16() if has_q else None
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def q4_pool(self, seed=1):
        g = torch.Generator(device=DEV).manual_seed(seed)
        shape = (self.pages, 2 * self.hkv, 64)
        return [torch.randint(0, 256, shape + (n,), generator=g, device=DEV, dtype=torch.uint8)
                for n in (self.d // 2, self.d // 32)]

    def append_q4(self, B, pool, scales, **kw):
        B.kv_append_rope_q4(self.q, self.k, self.v, pool, scales, self.table, self.positions,
                            self.inv_dev, self.q_out, cu_tokens=self.cu, interleaved=self.inter,
                            q_weight=self.qw if self.q is not None else None, k_weight=self.kw,
                            eps=self.eps, status=self.status, **kw)

    def append(self, B, pool, **kw):
        B.kv_append_norm_rope(self.q, self.k, self.v, pool, self.table, self.positions,
                              self.inv_dev, self.qw if self.q is not None else None, self.kw,
                              self.q_out, cu_tokens=self.cu, interleaved=self.inter, eps=self.eps,
                              status=self.status, **kw)

    def exact(self, name):
        """(normed and rotated float64 [n][h][d], allowance u)."""
        x = getattr(self, name)[:self.n].double().cpu().numpy()
        w = self.qw if name == "q" else self.kw
        by = 4e-7
        if w is not None:
            x = Q.norm(x, w.double().cpu().numpy(), self.eps)
            by += 2.0 ** -20
        half = len(self.inv)
        u = np.abs(x) * (0.0 if w is None else 2.0 ** -20)
        lo, hi = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if self.inter
                  else (slice(0, half), slice(half, 2 * half)))
        u[..., lo] = u[..., hi] = by * (np.abs(x[..., lo]) + np.abs(x[..., hi]))
        return R.rotate(x, self.pos, self.inv, self.inter), u

    def check_bf16(self, got, name):
        y, u = self.exact(name)
        assert np.all(np.abs(got.double().cpu().numpy() - y) <= u + np.abs(y) * 2.0 ** -8), name

    def check_q(self):
        if self.q is not None:
            self.check_bf16(self.q_out[:self.n], "q")
            assert torch.all(self.q_out[self.n:] == 7.0), "padding rows written"

    def check_k_q4(self, codes, scales):
        """codes [n][hkv][d / 2], scales [n][hkv][d / 32] of the new keys."""
        y, u = self.exact("k")
        g, ug = (a.reshape(a.shape[:-1] + (-1, 32)) for a in (y, u))
        e = scales.astype(np.int64)
        top = np.max(np.abs(g) + ug, -1)
        low = np.max(np.abs(g) - ug, -1)
        s = 2.0 ** (e - 127.0)
        assert np.all((e >= 67) & (low <= 6 * s) & ((e == 67) | (top > 3 * s)))
        a = np.abs(g) / s[..., None]
        half = np.where(a < 2, 0.25, np.where(a < 4, 0.5, 1.0)) * s[..., None]
        got = Q.values(codes, scales).reshape(g.shape)
        assert np.all(np.abs(got - g) <= half + ug)


CASES = [
    dict(new=[1], past=[0]),
    dict(new=[1] * 37, past=list(range(0, 37 * 29, 29)), hq=24, hkv=4, d=256),
    dict(new=[0, 5, 0, 1, 64, 17], past=[3, 62, 0, 127, 15, 4090], hq=32, hkv=8, rot=64, inter=True,
         pad=3),
    dict(new=[130, 1, 2], past=[1, 200000, 63], hq=7, hkv=1, d=256, rot=72, pad=1),
    dict(new=[3, 40], past=[9, 0], hq=4, hkv=4, rot=0),
    dict(new=[1100, 700], past=[5, 64], hq=4, hkv=2, rot=40, inter=True, pad=7),
    dict(new=[2050, 0, 3], past=[0, 8, 11], hq=8, hkv=1, d=256, fused=False),
    dict(new=[33, 4], past=[40, 1 << 20], hq=5, hkv=5, rot=104, has_q=False, pad=2),
    dict(new=[700], past=[60], hq=3, hkv=3, d=256, rot=24),
]
IDS = ["one", "decode37", "ragged-interleaved", "far-partial", "no-rotation", "prompts", "long",
       "no-q", "odd-heads"]


@pytest.mark.parametrize("kw", CASES + [dict(new=[9, 1], past=[60, 0], hq=3, hkv=3, d=64, rot=32),
                                        dict(new=[1, 1], past=[0, 9], hq=17, hkv=1, d=64, rot=24)],
                         ids=IDS + ["d64", "d64-odd"])
def test_normed_append(B, kw):
    s = Step(**kw)
    pool = torch.randn(s.pages, 64, 2 * s.hkv * s.d, device=DEV).bfloat16()
    before = pool.clone()
    s.append(B, pool)
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0
    s.check_q()
    got = pool[s.page, s.row].view(s.n, 2 * s.hkv, s.d)
    s.check_bf16(got[:, :s.hkv], "k")
    assert torch.equal(got[:, s.hkv:], s.v[:s.n])
    pool[s.page, s.row] = before[s.page, s.row]
    assert torch.equal(pool, before)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("kw", CASES, ids=IDS)
def test_q4_append_and_gather(B, kw, norm):
    s = Step(norm=norm, **kw)
    pool, scales = s.q4_pool()
    before = pool.clone(), scales.clone()
    s.append_q4(B, pool, scales)
    out = torch.full((s.n + kw.get("pad", 0), 2 * s.hkv * s.d), 7.0, device=DEV).bfloat16()
    B.kv_gather_q4(pool, scales, s.table, s.positions, s.cu, out, status=s.status)
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0
    s.check_q()
    codes, sc = (t[s.page, :, s.row].cpu().numpy() for t in (pool, scales))
    s.check_k_q4(codes[:, :s.hkv], sc[:, :s.hkv])
    v = s.v[:s.n].double().cpu().numpy()
    want = Q.values(*Q.quantise(v))
    assert np.array_equal(Q.values(codes[:, s.hkv:], sc[:, s.hkv:]), want)
    assert np.array_equal(sc[:, s.hkv:], Q.quantise(v)[1])
    assert np.array_equal(out[:s.n].double().cpu().numpy(), Q.values(codes, sc).reshape(s.n, -1))
    assert torch.all(out[s.n:] == 7.0)
    for now, was in zip((pool, scales), before):      # nothing else is touched
        now[s.page, :, s.row] = was[s.page, :, s.row]
        assert torch.equal(now, was)


def test_without_norm_both_pools_get_the_same_rotation(B):
    """q of the 4-bit append is q of the plain rotated append, bit for bit."""
    s = Step([70, 3], [5, 900], hq=8, hkv=2, d=256, norm=False)
    pool, scales = s.q4_pool()
    s.append_q4(B, pool, scales)
    want = torch.empty_like(s.q_out)
    rows = torch.zeros(s.pages, 64, 2 * s.hkv * s.d, device=DEV).bfloat16()
    B.kv_append_rope(s.q, s.k, s.v, rows, s.table, s.positions, s.inv_dev, want, cu_tokens=s.cu)
    torch.cuda.synchronize()
    assert torch.equal(s.q_out, want)


@pytest.mark.parametrize("size", [3e38, 1e30, 1e-20, 1e-38])
def test_norms_of_very_large_and_very_small_heads(B, size):
    s = Step([5, 1], [3, 64], hq=4, hkv=2, eps=2.0 ** -60 if size < 1 else EPS)
    s.q = (s.q.float() / s.q.float().abs().amax() * size).bfloat16()
    s.k = (s.k.float() / s.k.float().abs().amax() * size).bfloat16()
    s.k[1, 0] = 0                                      # and a head of zeros
    pool = torch.zeros(s.pages, 64, 2 * s.hkv * s.d, device=DEV).bfloat16()
    s.append(B, pool)
    torch.cuda.synchronize()
    y, u = s.exact("q")
    tiny = 2.0 ** -133                                 # a step of bf16's subnormals
    assert np.all(np.abs(s.q_out.double().cpu().numpy() - y) <= u + np.abs(y) * 2.0 ** -8 + tiny)
    y, u = s.exact("k")
    got = pool[s.page, s.row].view(s.n, 4, s.d)[:, :2].double().cpu().numpy()
    assert np.all(np.abs(got - y) <= u + np.abs(y) * 2.0 ** -8 + tiny)
    assert np.all(got[1, 0] == 0)


def test_values_that_are_not_finite(B):
    s = Step([3], [10], hq=2, hkv=2, rot=0, norm=False)
    s.k, s.v = s.k.clone(), s.v.clone()
    s.k[0, 0, 5] = float("nan")
    s.v[1, 1, 64] = float("inf")
    s.v[2, 0, 127] = float("-inf")
    pool, scales = s.q4_pool()
    s.append_q4(B, pool, scales)
    torch.cuda.synchronize()
    sc = scales[s.page, :, s.row].cpu().numpy()
    bad = np.zeros(sc.shape, bool)
    bad[0, 0, 0] = bad[1, 3, 2] = bad[2, 2, 3] = True
    assert np.array_equal(sc == 255, bad)
    # with norms a NaN takes its head, and an infinity its own value while the others are 0
    s = Step([2], [10], hq=2, hkv=2, rot=0)
    s.q, s.k = s.q.clone(), s.k.clone()
    s.q[0, 0, 5], s.k[1, 1, 100] = float("nan"), float("inf")
    s.append_q4(B, pool, scales)
    rows = torch.zeros(s.pages, 64, 2 * s.hkv * s.d, device=DEV).bfloat16()
    s.append(B, rows)
    torch.cuda.synchronize()
    assert s.q_out[0, 0].isnan().all() and s.q_out[0, 1].isfinite().all()
    got = rows[s.page, s.row].view(2, 4, s.d)
    assert got[1, 1, 100].isnan() and int(got[1, 1].isnan().sum()) == 1
    assert int((got[1, 1] == 0).sum()) == s.d - 1 and got[0].isfinite().all()
    sc = scales[s.page, :, s.row].cpu().numpy()
    assert (sc[1, 1] == 255).tolist() == [False, False, False, True]
    assert not (sc[0] == 255).any() and not (sc[1, 0] == 255).any()


def test_frequencies_that_are_not_finite(B):
    s = Step([2], [7], hq=2, hkv=1, norm=False)
    s.inv_dev[3] = float("inf")
    pool, scales = s.q4_pool()
    s.append_q4(B, pool, scales)
    torch.cuda.synchronize()
    assert s.q_out[:, :, [3, 67]].isnan().all()
    sc = scales[s.page, :, s.row].cpu().numpy()
    assert (sc[:, 0] == 255).tolist() == [[True, False, True, False]] * 2
    assert not (sc[:, 1] == 255).any()


@pytest.mark.parametrize("norm", [False, True])
def test_bad_places_are_reported_and_left_alone(B, norm):
    s = Step([2, 1, 3], [0, 0, 0], hq=4, hkv=2, norm=norm)
    s.table[0, 0] = s.pages
    s.table[1, 0] = -1
    s.positions[2] = 62                                # rows 62, 63, and one behind the table
    pool, scales = s.q4_pool()
    before = pool.clone(), scales.clone()
    s.append_q4(B, pool, scales)
    torch.cuda.synchronize()
    assert int(s.status.item()) == B.PA_STATUS_BAD_ROW
    page = int(s.table[2, 0])
    changed = (pool != before[0]).any(-1).any(1)
    assert changed.nonzero().tolist() == [[page, 62], [page, 63]]
    assert not torch.any(s.q_out == 7.0)               # q is turned all the same
    s.status.zero_()
    out = torch.zeros(6, 2 * s.hkv * s.d, device=DEV).bfloat16()
    B.kv_gather_q4(pool, scales, s.table, s.positions, s.cu, out, status=s.status)
    torch.cuda.synchronize()
    assert int(s.status.item()) == B.PA_STATUS_BAD_ROW
    assert out.isnan().all(1).tolist() == [True, True, True, False, False, True]
    rows = torch.zeros(s.pages, 64, 2 * s.hkv * s.d, device=DEV).bfloat16()
    if norm:
        s.status.zero_()
        s.append(B, rows)
        torch.cuda.synchronize()
        assert int(s.status.item()) == B.PA_STATUS_BAD_ROW
        assert (rows != 0).any(-1).nonzero().tolist() == [[page, 62], [page, 63]]


def test_in_place_on_another_stream_and_captured(B):
    s = Step([40, 7, 0, 1], [3, 100, 5, 63], hq=24, hkv=4, d=256)
    pool, scales = s.q4_pool()
    rows = torch.zeros(s.pages, 64, 2 * s.hkv * s.d, device=DEV).bfloat16()
    s.append_q4(B, pool, scales)
    torch.cuda.synchronize()
    want = s.q_out.clone(), pool.clone(), scales.clone()
    q = s.q.clone()
    side = torch.cuda.Stream()
    s.q_out = s.q                                      # q itself, strided
    pool.zero_(), scales.zero_()
    side.wait_stream(torch.cuda.current_stream())
    s.append_q4(B, pool, scales, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(s.q, want[0])
    written = pool[s.page, :, s.row], scales[s.page, :, s.row]
    assert torch.equal(written[0], want[1][s.page, :, s.row])
    assert torch.equal(written[1], want[2][s.page, :, s.row])
    s.q.copy_(q)
    s.q_out = torch.zeros_like(want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.append_q4(B, pool, scales)
        s.append(B, rows)
    for _ in range(2):
        pool.zero_(), rows.zero_(), s.q_out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s.q_out, want[0])
        assert torch.equal(pool[s.page, :, s.row], want[1][s.page, :, s.row])
        s.check_bf16(rows[s.page, s.row].view(s.n, -1, s.d)[:, :s.hkv], "k")


def test_binding_checks_shapes(B):
    s = Step([1], [0], hq=2, hkv=2)
    pool, scales = s.q4_pool()
    with pytest.raises(ValueError, match="scales"):
        s.append_q4(B, pool, scales[..., :2].contiguous())
    with pytest.raises(ValueError, match="pool"):
        s.append_q4(B, pool[:, :3].contiguous(), scales[:, :3].contiguous())
    with pytest.raises(ValueError, match="pool is for"):
        s.append_q4(B, pool[:, :2].contiguous(), scales[:, :2].contiguous())
    s.kw = s.kw[:64]
    with pytest.raises(ValueError, match="k_weight"):
        s.append_q4(B, pool, scales)
    s.kw = None
    with pytest.raises(ValueError, match="k_weight"):
        s.append_q4(B, pool, scales)
    out = torch.zeros(1, 2 * s.hkv * s.d - 1, device=DEV).bfloat16()
    with pytest.raises(ValueError, match="out"):
        B.kv_gather_q4(pool, scales, s.table, s.positions, None, out)
