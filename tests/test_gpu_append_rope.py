"""Appends with the position rotation (bf16 and 8-bit pools) and the gather of
8-bit rows, against the float64 oracle.

Tolerances.  With u = 4e-7 (|x1| + |x2|) for the FP32 evaluation of a rotated
value (sine and cosine within 1.5e-7, two products and a sum within 1.5 steps
of 2^-24 each), a bf16 result is within u plus half a step (2^-8 relative) of
the exact value; an e4m3 value within u plus half a step: 2^-4 relative, or
2^-10 scales where the code is subnormal.  Unrotated values are exact bits.
"""

import numpy as np
import pytest
import torch

from oracle import rope_q8 as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def B():
    from paged_decode_attention_attn_gb300 import build
    build.build()
    from paged_decode_attention_attn_gb300 import binding
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return binding


class Step:
    """One ragged append: lengths of new tokens and positions, fused qkv."""

    def __init__(self, new, past, hq=6, hkv=2, d=128, rot=None, interleaved=False, pad=0, seed=0,
                 fused=True, spare=3, base=10000.0):
        rot = d if rot is None else rot
        rng = np.random.default_rng(seed)
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.new, self.past = np.asarray(new), np.asarray(past)
        self.hq, self.hkv, self.d, self.inter = hq, hkv, d, interleaved
        self.cu = np.concatenate([[0], np.cumsum(self.new)])
        n = int(self.cu[-1]) + pad
        self.qkv = torch.randn(n, hq + 2 * hkv, d, generator=g, device=DEV).bfloat16()
        if fused:
            self.q, self.k, self.v = self.qkv.split([hq, hkv, hkv], 1)
        else:
            self.q, self.k, self.v = (t.contiguous() for t in self.qkv.split([hq, hkv, hkv], 1))
        half = rot // 2
        self.inv = (base ** (-np.arange(half) / max(1, half))).astype(np.float32)
        ends = self.past + self.new
        width = int(max(1, -(-int(ends.max()) // 64)))
        used = [range(int(p) // 64, -(-int(e) // 64)) if e > p else [] for p, e in zip(past, ends)]
        self.pages = sum(len(u) for u in used) + spare
        perm = rng.permutation(self.pages)
        self.table = np.zeros((len(new), width), np.int32)
        at = 0
        for b, u in enumerate(used):
            for p in u:
                self.table[b, p] = perm[at]
                at += 1
        self.places = R.token_places(self.cu, self.past, self.table)
        self.rows = np.array([p[3] for p in self.places], dtype=np.int64)
        self.pos = np.array([p[2] for p in self.places], dtype=np.int64)
        self.n = int(self.cu[-1])
        self.t = dict(table=torch.from_numpy(self.table).to(DEV),
                      pos=torch.from_numpy(self.past.astype(np.int32)).to(DEV),
                      cu=torch.from_numpy(self.cu.astype(np.int32)).to(DEV),
                      inv=torch.from_numpy(self.inv).to(DEV) if half else None)

    def exact(self, name):
        """(rotated float64 [n][h][d], allowance u of the FP32 evaluation)."""
        x = getattr(self, name)[:self.n].double().cpu().numpy()
        y = R.rotate(x, self.pos, self.inv, self.inter)
        half = len(self.inv)
        u = np.zeros_like(x)
        lo, hi = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if self.inter
                  else (slice(0, half), slice(half, 2 * half)))
        u[..., lo] = u[..., hi] = 4e-7 * (np.abs(x[..., lo]) + np.abs(x[..., hi]))
        return y, u

    def check_q(self, q_out, before):
        got = q_out.double().cpu().numpy()
        y, u = self.exact("q")
        assert np.all(np.abs(got[:self.n] - y) <= u + np.abs(y) * 2.0 ** -8)
        assert torch.equal(q_out[self.n:], before[self.n:]), "padding rows written"


CASES = [
    dict(new=[1], past=[0]),
    dict(new=[1] * 37, past=list(range(0, 37 * 29, 29)), hq=24, hkv=4, d=256),
    dict(new=[0, 5, 0, 1, 64, 17], past=[3, 62, 0, 127, 15, 4090], hq=32, hkv=8, rot=64,
         interleaved=True, pad=3),
    dict(new=[130, 1, 2], past=[1, 200000, 63], hq=7, hkv=1, d=256, rot=72, pad=1),
    dict(new=[3, 40], past=[9, 0], hq=4, hkv=4, d=128, rot=0),
    dict(new=[1100, 700], past=[5, 64], hq=4, hkv=2, d=128, rot=40, interleaved=True, pad=7),
    dict(new=[2050, 0, 3], past=[0, 8, 11], hq=8, hkv=1, d=256, fused=False),
]
IDS = ["one", "decode37", "ragged-interleaved", "far-partial", "no-rotation", "prompts", "long"]


@pytest.mark.parametrize("kw", CASES + [dict(new=[9, 1], past=[60, 0], hq=3, hkv=3, d=64, rot=32)],
                         ids=IDS + ["d64"])
def test_bf16_append(B, kw):
    s = Step(**kw)
    pool = torch.randn(s.pages, 64, 2 * s.hkv * s.d, device=DEV).bfloat16()
    before = pool.clone()
    q_out = torch.full_like(s.q, 7.0, memory_format=torch.contiguous_format)
    q_before = q_out.clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    cu = None if np.all(s.new == 1) and not kw.get("pad") else s.t["cu"]
    B.kv_append_rope(s.q, s.k, s.v, pool, s.t["table"], s.t["pos"], s.t["inv"], q_out,
                     cu_tokens=cu, interleaved=s.inter, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    s.check_q(q_out, q_before)
    rows = torch.from_numpy(s.rows).to(DEV)
    got = pool.view(-1, 2 * s.hkv, s.d)
    y, u = s.exact("k")
    assert np.all(np.abs(got[rows, :s.hkv].double().cpu().numpy() - y)
                  <= u + np.abs(y) * 2.0 ** -8)
    assert torch.equal(got[rows, s.hkv:], s.v[:s.n])
    other = torch.ones(len(got), dtype=torch.bool, device=DEV)
    other[rows] = False
    assert torch.equal(got[other], before.view(-1, 2 * s.hkv, s.d)[other])


def _filled(s, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    codes = torch.randint(0, 256, (s.pages, 64, 2 * s.hkv * s.d), generator=g, device=DEV,
                          dtype=torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x11
    e = torch.randint(-12, -6, (s.pages, 2 * s.hkv, 4), generator=g, device=DEV)
    return codes.view(E4M3), torch.exp2(e.float())


def _by_block(scales):
    return scales.double().cpu().numpy().transpose(0, 2, 1).reshape(-1, scales.shape[1])


@pytest.mark.parametrize("kw", CASES, ids=IDS)
def test_q8_append_and_gather(B, kw):
    s = Step(**kw)
    pool, scales = _filled(s)
    heads = 2 * s.hkv
    codes0 = pool.view(torch.uint8).cpu().numpy().reshape(-1, heads, s.d)
    scales0 = _by_block(scales)
    q_out = torch.full_like(s.q, 7.0, memory_format=torch.contiguous_format)
    q_before = q_out.clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    cu = None if np.all(s.new == 1) and not kw.get("pad") else s.t["cu"]
    B.kv_append_rope_q8(s.q, s.k, s.v, pool, scales, s.t["table"], s.t["pos"], s.t["inv"], q_out,
                        cu_tokens=cu, interleaved=s.inter, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    s.check_q(q_out, q_before)
    y, u = s.exact("k")
    v = s.v[:s.n].double().cpu().numpy()
    want_codes, want_scales = R.append_q8(codes0.copy(), scales0.copy(), s.places, y, v)
    got_codes = pool.view(torch.uint8).cpu().numpy().reshape(-1, heads, s.d)
    got_scales = _by_block(scales)
    # a block's scale may differ only where its largest key meets a border
    # between two scales within the FP32 allowance; none does in these draws
    assert np.array_equal(got_scales, want_scales)
    # every row that is not new: older rows requantised, others untouched
    new = np.zeros(len(got_codes), bool)
    new[s.rows] = True
    assert np.array_equal(got_codes[~new], want_codes[~new])
    # new rows: values are exact nearest codes, keys within half a code
    assert np.array_equal(got_codes[s.rows, s.hkv:], want_codes[s.rows, s.hkv:])
    val = R.pool_values(got_codes, got_scales)[s.rows, :s.hkv]
    sc = got_scales[s.rows // 16][:, :s.hkv, None]
    assert np.all(np.abs(val - y) <= u + np.maximum(np.abs(y) / 16, sc * 2.0 ** -10))
    # the gather gives those values, exactly
    out = torch.full((s.qkv.shape[0], heads * s.d), 7.0, device=DEV, dtype=torch.bfloat16)
    B.kv_gather_q8(pool, scales, s.t["table"], s.t["pos"], s.t["cu"] if s.qkv.shape[0] != s.n
                   else cu, out, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    want = R.pool_values(got_codes, got_scales)[s.rows].reshape(s.n, -1)
    assert np.array_equal(out[:s.n].double().cpu().numpy(), want)
    assert torch.all(out[s.n:] == 7.0)


def test_q8_append_token_by_token_equals_at_once(B):
    """A block filled in pieces of any size holds the scale of the whole; codes
    differ from the at-once append only where a code became subnormal."""
    whole = Step([45], [0], hq=2, hkv=2, d=256, seed=5)
    p1, s1 = _filled(whole, 2)
    p2, s2 = p1.view(torch.uint8).clone().view(E4M3), s1.clone()
    grow = torch.linspace(0.1, 30, 45, device=DEV)[:, None, None]
    k, v = (whole.k * grow).bfloat16(), (whole.v * grow).bfloat16()
    B.kv_append_rope_q8(None, k, v, p1, s1, whole.t["table"], whole.t["pos"], whole.t["inv"],
                        cu_tokens=whole.t["cu"])
    at = 0
    for n in (1, 1, 1, 5, 10, 1, 13, 13):
        pos = torch.tensor([at], dtype=torch.int32, device=DEV)
        cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
        B.kv_append_rope_q8(None, k[at:at + n], v[at:at + n], p2, s2, whole.t["table"], pos,
                            whole.t["inv"], cu_tokens=cu)
        at += n
    torch.cuda.synchronize()
    assert torch.equal(s1, s2)
    a, b = (p.view(torch.uint8).to(torch.int32) for p in (p1, p2))
    normal = (a & 0x7F) >= 16          # two binades above the subnormals' end
    assert torch.equal(a[normal], b[normal])
    assert int((a - b).abs().max()) <= 1


@pytest.mark.parametrize("q8", [False, True])
def test_rotation_in_place_and_on_another_stream(B, q8):
    s = Step([3, 1, 30], [5, 70, 1000], hq=8, hkv=2, d=256, seed=3)
    side = torch.cuda.Stream()
    results = []
    for in_place in (False, True):
        t = Step([3, 1, 30], [5, 70, 1000], hq=8, hkv=2, d=256, seed=3)
        q_out = t.q if in_place else torch.empty_like(t.q)
        pool, scales = _filled(t)
        if not q8:
            pool = torch.zeros(t.pages, 64, 2 * t.hkv * t.d, device=DEV, dtype=torch.bfloat16)
        torch.cuda.synchronize()
        if q8:
            B.kv_append_rope_q8(t.q, t.k, t.v, pool, scales, t.t["table"], t.t["pos"], t.t["inv"],
                                q_out, cu_tokens=t.t["cu"], stream=side)
        else:
            B.kv_append_rope(t.q, t.k, t.v, pool, t.t["table"], t.t["pos"], t.t["inv"], q_out,
                             cu_tokens=t.t["cu"], stream=side)
        side.synchronize()
        results.append((q_out.clone(), pool.view(torch.uint8).clone(), scales.clone()))
        assert torch.equal(t.k, s.k) and torch.equal(t.v, s.v)
    for a, b in zip(*results):
        assert torch.equal(a, b)


@pytest.mark.parametrize("q8", [False, True])
def test_rows_outside_the_table_or_pool_are_reported_and_skipped(B, q8):
    """Requests 0 and 2 are good; 1 has a negative position, 3 runs behind the
    table and 4 names pages outside the pool.  Their q is rotated all the same."""
    s = Step([4, 3, 20, 5, 2], [0, 0, 30, 60, 0], hq=4, hkv=2, d=128, seed=9)
    s.table = s.table[:, :1].copy()
    s.past[1] = -2
    s.table[4, 0] = s.pages + 5
    s.places = [(r, b, p, row if b in (0, 2) and 0 <= p < 64 else -1)
                for r, b, p, row in R.token_places(s.cu, s.past, s.table)]
    # request 1's third token has position 0, request 3's first four fit the table
    for i, (r, b, p, _) in enumerate(s.places):
        if (b == 1 and p >= 0) or (b == 3 and p < 64):
            s.places[i] = (r, b, p, int(s.table[b, 0]) * 64 + p)
    s.pos = np.array([p[2] for p in s.places])
    table = torch.from_numpy(s.table).to(DEV)
    pos = torch.from_numpy(s.past.astype(np.int32)).to(DEV)
    pool, scales = _filled(s)
    if not q8:
        pool = torch.randn(s.pages, 64, 2 * s.hkv * s.d, device=DEV).bfloat16()
    before = pool.view(torch.uint8).clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    q_out = torch.zeros(s.qkv.shape[0], s.hq, s.d, device=DEV, dtype=torch.bfloat16)
    if q8:
        want = R.append_q8(before.cpu().numpy().reshape(-1, 2 * s.hkv, s.d), _by_block(scales),
                           s.places, s.exact("k")[0], s.v.double().cpu().numpy())
        B.kv_append_rope_q8(s.q, s.k, s.v, pool, scales, table, pos, s.t["inv"], q_out,
                            cu_tokens=s.t["cu"], status=status)
    else:
        B.kv_append_rope(s.q, s.k, s.v, pool, table, pos, s.t["inv"], q_out,
                         cu_tokens=s.t["cu"], status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == B.PA_STATUS_BAD_ROW
    s.check_q(q_out, q_out)
    rows = np.array([p[3] for p in s.places])
    kept = np.ones(s.pages * 64, bool)
    kept[rows[rows >= 0]] = False
    width = (1 if q8 else 2) * 2 * s.hkv * s.d
    after = pool.view(torch.uint8).reshape(-1, width).cpu().numpy()
    if q8:
        assert np.array_equal(_by_block(scales), want[1])
        assert np.array_equal(after[kept], want[0].reshape(-1, width)[kept])
        vals = after.reshape(-1, 2 * s.hkv, s.d)[rows[rows >= 0], s.hkv:]
        assert np.array_equal(vals, want[0][rows[rows >= 0], s.hkv:])
    else:
        assert np.array_equal(after[kept], before.reshape(-1, width).cpu().numpy()[kept])
        got = pool.view(-1, 2 * s.hkv, s.d)[torch.from_numpy(rows[rows >= 0]).to(DEV), s.hkv:]
        assert torch.equal(got, s.v[torch.from_numpy(rows >= 0).to(DEV)])


def test_gather_fills_bad_rows_with_nan(B):
    s = Step([4, 4], [60, 0], hq=2, hkv=1, d=128)
    pool, scales = _filled(s)
    table = torch.full((2, 1), -1, dtype=torch.int32, device=DEV)
    table[0, 0] = 0
    out = torch.zeros(8, 256, device=DEV, dtype=torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.kv_gather_q8(pool, scales, table, torch.tensor([62, 0], dtype=torch.int32, device=DEV),
                   torch.tensor([0, 4, 8], dtype=torch.int32, device=DEV), out, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == B.PA_STATUS_BAD_ROW
    assert torch.all(out[:2].isfinite()) and torch.all(out[2:].isnan())


def test_non_finite_values_are_stored_as_nan_and_set_no_scale(B):
    s = Step([20], [0], hq=2, hkv=1, d=128, rot=0)
    v = s.v.clone()
    v[3, 0, 5], v[4, 0, 6], v[17, 0, 0] = float("inf"), float("nan"), float("-inf")
    k = torch.zeros_like(v)
    pool, scales = _filled(s)
    B.kv_append_rope_q8(None, k, v, pool, scales, s.t["table"], s.t["pos"], None,
                        cu_tokens=s.t["cu"])
    torch.cuda.synchronize()
    page = int(s.table[0, 0])
    vd = v.double().cpu().numpy()[:, 0]
    sc = scales[page].cpu().numpy()
    assert sc[1, 0] == R.need_scale(vd[:16]) and sc[1, 1] == R.need_scale(vd[16:])
    assert sc[0, 0] == 2.0 ** -60                     # zeros take the smallest scale
    codes = pool.view(torch.uint8)[page].cpu().numpy()
    want = R.e4m3_encode(vd / np.repeat(sc[1, :2], [16, 4])[:, None])
    got = codes[:20, 128:]
    nan = ~np.isfinite(vd)
    assert np.all(got[nan] & 0x7F == 0x7F) and np.array_equal(got[~nan], want[~nan])
    assert np.all(codes[:20, :128] == 0)


def test_far_positions_keep_their_angles(B):
    """Positions up to 2^31 - 1 (fp32 holds no integers there): a float64
    product is within 2^-21 of the angle, inside the bf16 half step used here."""
    n = 8
    s = Step([1] * n, [0] * n, hq=2, hkv=1, d=128)
    pos = np.array([2 ** 24 + 1, 2 ** 28 + 3, 2 ** 31 - 1, 16777217, 123456789, 1, 0, 2 ** 30 + 7])
    s.pos, s.past = pos, pos
    table = torch.zeros(n, 1, dtype=torch.int32, device=DEV)
    pool = torch.zeros(1, 64, 256, device=DEV, dtype=torch.bfloat16)
    q_out = torch.empty(n, 2, 128, device=DEV, dtype=torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.kv_append_rope(s.q, s.k, s.v, pool, table,
                     torch.from_numpy(pos.astype(np.int32)).to(DEV), s.t["inv"], q_out,
                     status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == B.PA_STATUS_BAD_ROW      # the table holds one page
    y, u = s.exact("q")
    got = q_out.double().cpu().numpy()
    assert np.all(np.abs(got - y) <= u + np.abs(y) * 2.0 ** -8 + 2.0 ** -19)


@pytest.mark.parametrize("q8", [False, True])
def test_captured_append_replays_with_new_inputs(B, q8):
    s = Step([1] * 9, list(range(9)), hq=4, hkv=2, d=128)
    pool, scales = _filled(s)
    if not q8:
        pool = torch.zeros(s.pages, 64, 2 * s.hkv * s.d, device=DEV, dtype=torch.bfloat16)
    q_out = torch.empty(9, 4, 128, device=DEV, dtype=torch.bfloat16)

    def call(pool, scales, q_out):
        if q8:
            B.kv_append_rope_q8(s.q, s.k, s.v, pool, scales, s.t["table"], s.t["pos"],
                                s.t["inv"], q_out)
        else:
            B.kv_append_rope(s.q, s.k, s.v, pool, s.t["table"], s.t["pos"], s.t["inv"], q_out)

    call(pool, scales, q_out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(pool, scales, q_out)
    pool2, scales2 = pool.view(torch.uint8).clone().view(pool.dtype), scales.clone()
    for step in range(3):
        s.qkv.normal_()
        s.t["pos"].fill_(5 + step)
        graph.replay()
        q2 = torch.empty_like(q_out)
        call(pool2, scales2, q2)
        torch.cuda.synchronize()
        assert torch.equal(q2, q_out)
        assert torch.equal(pool2.view(torch.uint8), pool.view(torch.uint8))
        assert torch.equal(scales2, scales)


@pytest.mark.parametrize("kw", [
    dict(new=[1] * 1100, past=[i * 7 % 150 for i in range(1100)], hq=2, hkv=1, d=128, pad=2),
    dict(new=[i % 9 for i in range(400)], past=[i * 11 % 90 for i in range(400)], hq=2, hkv=1,
         d=128, rot=64),
    dict(new=[0] * 300 + [1300] + [0] * 200, past=[0] * 300 + [7] + [0] * 200, hq=2, hkv=1, d=256),
], ids=["single-tokens", "short", "one-among-empty"])
def test_q8_appends_of_many_requests(B, kw):
    """More rows than are given a CTA each, in requests of few tokens or none."""
    test_q8_append_and_gather(B, kw)


@pytest.mark.parametrize("q8", [False, True])
def test_pages_past_4_gib_of_pool(B, q8):
    """The same pages at the top of a 5.4 GB pool: the same bits are stored, and
    read back."""
    s = Step([70, 1, 300], [5, 63, 0], hq=4, hkv=4, d=256, seed=21)
    row = 2 * s.hkv * s.d
    small, sc_small = _filled(s)
    if not q8:
        small = torch.randn(s.pages, 64, row, device=DEV).bfloat16()
    pages = 5_400_000_000 // (64 * row * small.element_size())
    lift = pages - s.pages
    assert lift * 64 * row * small.element_size() > 1 << 32
    big = torch.zeros(pages, 64, row, dtype=torch.uint8 if q8 else torch.bfloat16, device=DEV)
    big = big.view(E4M3) if q8 else big
    raw = (lambda t: t.view(torch.uint8)) if q8 else (lambda t: t)
    raw(big)[lift:] = raw(small)
    sc_big = torch.ones(pages, 2 * s.hkv, 4, device=DEV)
    sc_big[lift:] = sc_small
    table = s.t["table"] + lift
    for pool, scales, tab in ((small, sc_small, s.t["table"]), (big, sc_big, table)):
        if q8:
            B.kv_append_rope_q8(None, s.k, s.v, pool, scales, tab, s.t["pos"], s.t["inv"],
                                cu_tokens=s.t["cu"])
        else:
            B.kv_append_rope(None, s.k, s.v, pool, tab, s.t["pos"], s.t["inv"],
                             cu_tokens=s.t["cu"])
    torch.cuda.synchronize()
    bits = (lambda t: t.view(torch.uint8)) if q8 else (lambda t: t.view(torch.int16))
    assert torch.equal(bits(big[lift:]), bits(small))
    assert not raw(big)[:64].any()
    if q8:
        assert torch.equal(sc_big[lift:], sc_small)
        outs = []
        for pool, scales, tab in ((small, sc_small, s.t["table"]), (big, sc_big, table)):
            outs.append(torch.empty(s.n, row, dtype=torch.bfloat16, device=DEV))
            B.kv_gather_q8(pool, scales, tab, s.t["pos"], s.t["cu"], outs[-1])
        torch.cuda.synchronize()
        assert torch.equal(*outs)


def test_padded_requests_of_a_captured_step(B):
    """A graph captured for more requests than a step has: the spare ones hold
    position -1, store nothing and say so; the others are as in a call of their
    own."""
    s = Step([1] * 6, [0, 15, 16, 63, 64, 500], hq=4, hkv=2, d=128, seed=22)
    pool, scales = _filled(s)
    want_pool, want_scales = pool.view(torch.uint8).clone().view(E4M3), scales.clone()
    n = 11
    q = torch.cat([s.q, s.q[:n - 6]])
    k, v = torch.cat([s.k, s.k[:n - 6]]), torch.cat([s.v, s.v[:n - 6]])
    table = torch.cat([s.t["table"], s.t["table"][:n - 6]])
    pos = torch.cat([s.t["pos"], torch.full((n - 6,), -1, dtype=torch.int32, device=DEV)])
    q_out = torch.empty_like(q)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        B.kv_append_rope_q8(q, k, v, pool, scales, table, pos, s.t["inv"], q_out, status=status)
    graph.replay()
    want_q = torch.empty_like(s.q, memory_format=torch.contiguous_format)
    B.kv_append_rope_q8(s.q, s.k, s.v, want_pool, want_scales, s.t["table"], s.t["pos"],
                        s.t["inv"], want_q)
    torch.cuda.synchronize()
    assert int(status.item()) == B.PA_STATUS_BAD_ROW
    assert torch.equal(pool.view(torch.uint8), want_pool.view(torch.uint8))
    assert torch.equal(scales, want_scales) and torch.equal(q_out[:6], want_q)
