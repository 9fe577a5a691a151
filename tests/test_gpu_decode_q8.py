"""Decode attention over the 8-bit pool against the float64 oracle, which
attends the values that codes and scales stand for.

Tolerances.  With A = scale max_j sum_d |q_d k_jd| over a row, an FP32 score
(sums over head_dim, the scaling) is within 8 steps of 2^-24 of A, so a
probability is within e = 2^-21 A + 2^-18 relative, the second term for the
exponential (2^-22) and for the parts a probability is held in: 2^-16 at worst
for one key, a quarter of that on the root mean square of several.  The output
is then within (e + 2^-16) max |V| (a row may hang on one key), the log-sum-exp
within e + 2^-22 |lse|.
"""

import numpy as np
import pytest
import torch

import oracle
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


def check_request(K, V, q, tiles, scale, out, lse, merged, merged_lse, what):
    """One request's tiles and merge against the oracle over K, V float64
    [tokens][Hkv][D]."""
    q = q.double().cpu().numpy()
    outs, lses = oracle.tile_attention(q, K, V, tiles, scale)
    want = list(zip(outs, lses)) + [oracle.lse_merge(outs, lses)]
    got = [(out[t], lse[t]) for t in range(len(tiles))] + [(merged, merged_lse)]
    G = q.shape[0] // K.shape[1]
    for i, ((o, l), (wo, wl)) in enumerate(zip(got, want)):
        o, l = o.double().cpu().numpy(), l.double().cpu().numpy()
        if np.all(wl == -np.inf):
            assert np.all(o == 0) and np.all(l == -np.inf), (what, i)
            continue
        for h in range(q.shape[0]):
            if not np.isfinite(wl[h]):
                assert np.isnan(o[h]).all() and np.isnan(l[h]), (what, i, h)
                continue
            A = scale * np.max(np.abs(K[:, h // G]) @ np.abs(q[h]))
            e = 2.0 ** -21 * A + 2.0 ** -18
            vmax = np.max(np.abs(V[:, h // G]))
            err = np.max(np.abs(o[h] - wo[h]))
            assert err <= (e + 2.0 ** -16) * vmax, (what, i, h, err, vmax, A)
            assert abs(l[h] - wl[h]) <= e + 2.0 ** -22 * abs(wl[h]), (what, i, h)


class Case:
    def __init__(self, lengths, tiles=None, hq=24, hkv=4, d=256, seed=0, spare=3, scale=None,
                 q_scale=1.0, v_exp=(-8, -5), k_exp=(-8, -5), max_pages=None):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.lengths, self.hq, self.hkv, self.d = list(lengths), hq, hkv, d
        self.scale = d ** -0.5 if scale is None else scale
        n_pages = [-(-n // 64) for n in lengths]
        self.pages = sum(n_pages) + spare
        perm = rng.permutation(self.pages)
        self.table = np.zeros((len(lengths), max_pages or max(1, max(n_pages))), np.int32)
        at = 0
        for b, n in enumerate(n_pages):
            self.table[b, :n] = perm[at:at + n]
            at += n
        tiles = [[(0, n)] for n in lengths] if tiles is None else tiles
        T = max(len(t) for t in tiles)
        self.tiles = np.zeros((len(lengths), T, 2), np.int32)
        for b, tl in enumerate(tiles):
            for i, r in enumerate(tl):
                self.tiles[b, i] = r
        self.q = (torch.randn(len(lengths), hq, d, generator=g, device=DEV) * q_scale).bfloat16()
        x = torch.randn(self.pages, 64, 2 * hkv * d, generator=g, device=DEV) * 64
        self.pool = x.to(E4M3)
        ek = torch.randint(*k_exp, (self.pages, hkv, 4), generator=g, device=DEV)
        ev = torch.randint(*v_exp, (self.pages, hkv, 4), generator=g, device=DEV)
        self.scales = torch.exp2(torch.cat([ek, ev], 1).float())
        # everything no request names, and the rows behind each last token: NaN
        raw = self.pool.view(torch.uint8)
        raw[torch.from_numpy(perm[at:].copy()).to(DEV)] = 0x7F
        for b, n in enumerate(lengths):
            if n % 64:
                raw[int(self.table[b, n // 64]), n % 64:] = 0xFF
        self.table_dev = torch.from_numpy(self.table).to(DEV)
        shape = (len(lengths), T, hq)
        self.out = torch.full(shape + (d,), 7.0, device=DEV)
        self.lse = torch.full(shape, 7.0, device=DEV)
        self.merged = torch.full((len(lengths), hq, d), 7.0, device=DEV)
        self.merged_lse = torch.full((len(lengths), hq), 7.0, device=DEV)
        self.ws = None

    def run(self, B, merged=True, stream=None):
        if self.ws is None:
            self.ws = B.alloc_workspace_q8(len(self.lengths), self.tiles.shape[1], self.hq,
                                           self.hkv, self.d)
            torch.cuda.synchronize()
        B.paged_decode_attn_q8_lse(
            self.q, self.pool, self.scales, self.table_dev, self.tiles, self.scale, self.out,
            self.lse, self.ws, merged_out=self.merged if merged else None,
            merged_lse=self.merged_lse if merged else None, stream=stream)
        torch.cuda.synchronize()
        return int(self.ws[:4].view(torch.int32).item())

    def history(self, b):
        n = self.lengths[b]
        pages = torch.from_numpy(self.table[b, :-(-n // 64)].astype(np.int64)).to(DEV)
        codes = self.pool.view(torch.uint8)[pages].cpu().numpy().reshape(-1, 2 * self.hkv, self.d)
        scales = self.scales[pages].double().cpu().numpy().transpose(0, 2, 1)
        kv = R.pool_values(codes, scales.reshape(-1, 2 * self.hkv))[:n]
        return kv[:, :self.hkv], kv[:, self.hkv:]

    def check(self, requests=None):
        for b in range(len(self.lengths)) if requests is None else requests:
            check_request(*self.history(b), self.q[b], self.tiles[b], self.scale, self.out[b],
                          self.lse[b], self.merged[b], self.merged_lse[b], f"request {b}")


LENGTHS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 192, 193, 1000]


@pytest.mark.parametrize("geo", [(24, 4, 256), (32, 8, 128), (7, 1, 256), (8, 8, 128), (20, 5, 128),
                                 (16, 2, 256)])
def test_lengths_around_blocks_pages_and_steps(B, geo):
    c = Case(LENGTHS, hq=geo[0], hkv=geo[1], d=geo[2], seed=geo[0])
    assert c.run(B) == 0
    c.check()


@pytest.mark.parametrize("d", [128, 256])
def test_tiles_that_start_and_end_anywhere(B, d):
    tiles = [[(0, 1), (1, 700), (699, 700), (3, 3)], [(0, 0)], [(63, 65), (64, 128), (0, 64)],
             [(5, 2001), (130, 131), (1990, 2100), (0, 2100)], [(0, 0), (17, 18)]]
    c = Case([700, 0, 200, 2100, 40], tiles, hq=16, hkv=4, d=d, seed=3)
    assert c.run(B) == 0
    c.check()


@pytest.mark.parametrize("lengths,tile,geo", [
    ([40000], None, (24, 4, 256)), ([30011], 4096, (32, 8, 128)),
    ([9000, 1, 20000, 12345, 64], 8192, (24, 4, 256)), ([5000] * 3, None, (8, 1, 128))])
def test_long_histories_split_over_many_ctas(B, lengths, tile, geo):
    tiles = None if tile is None else [[(s, min(n, s + tile)) for s in range(0, n, tile)]
                                       for n in lengths]
    c = Case(lengths, tiles, hq=geo[0], hkv=geo[1], d=geo[2], seed=len(lengths))
    assert c.run(B) == 0
    c.check()
    first = [t.clone() for t in (c.out, c.lse, c.merged, c.merged_lse)]
    for _ in range(3):                                # the workspace is ready for the next call
        assert c.run(B) == 0
        for a, b in zip(first, (c.out, c.lse, c.merged, c.merged_lse)):
            assert torch.equal(a, b)


def test_many_requests_and_units(B):
    rng = np.random.default_rng(5)
    lengths = [int(n) for n in rng.integers(1, 500, 301)]
    c = Case(lengths, [[(0, n // 2), (n // 2, n)] for n in lengths], hq=16, hkv=4, d=128, seed=6)
    assert c.run(B) == 0
    c.check(requests=list(range(0, 301, 13)) + [300])


def test_without_merge_and_with_one_tile(B):
    c = Case([300, 70], hq=8, hkv=2, d=128, seed=8)
    assert c.run(B, merged=False) == 0
    assert torch.all(c.merged == 7.0) and torch.all(c.merged_lse == 7.0)
    c.run(B)
    assert torch.equal(c.merged, c.out[:, 0]) and torch.equal(c.merged_lse, c.lse[:, 0])


@pytest.mark.parametrize("q_scale,v_exp,k_exp", [
    (8.0, (-8, -5), (-5, -2)),          # scores in the hundreds: one key dominates
    (1.0, (-50, 40), (-8, -5)),         # V scales far apart between blocks
    (1e-3, (-60, -59), (-60, -59)),     # the smallest scales
    (1.0, (95, 100), (-8, -5)), (2.0 ** -60, (-8, -5), (50, 56))])
def test_wide_ranges_of_scales_and_scores(B, q_scale, v_exp, k_exp):
    c = Case([3, 500, 1333], hq=12, hkv=2, d=256, seed=11, q_scale=q_scale, v_exp=v_exp,
             k_exp=k_exp)
    assert c.run(B) == 0
    c.check()


def test_growing_scores_move_the_running_maximum(B):
    """Keys whose scores rise through the history, so the maximum moves in every
    step, and fall again."""
    c = Case([4000], hq=6, hkv=1, d=128, seed=12)
    up = torch.linspace(-12, -1, 4 * c.pages, device=DEV).round()
    order = torch.from_numpy(c.table[0].astype(np.int64)).to(DEV)
    c.scales[order, 0] = torch.exp2(up[:4 * len(order)].view(-1, 4))
    assert c.run(B) == 0
    c.check()


def test_q_with_a_wide_spread_of_magnitudes(B):
    c = Case([777], hq=8, hkv=2, d=256, seed=13)
    c.q *= torch.exp2(torch.randint(-20, 1, c.q.shape, device=DEV).float()).bfloat16()
    c.q[0, 3] = 0                                        # a row of zeros: plain averages
    c.q[0, 4] *= 2.0 ** 20
    assert c.run(B) == 0
    c.check()


def test_scales_that_are_no_powers_of_two(B):
    c = Case([500, 64], hq=8, hkv=2, d=128, seed=14)
    c.scales *= 1 + torch.rand_like(c.scales)
    c.scales[int(c.table[0, 2]), 2:, 1] = 0.0            # V blocks of zeros
    c.scales[int(c.table[0, 3]), :2, 2] = 0.0
    assert c.run(B) == 0
    c.check()


def test_nan_codes_and_scales_inside_a_tile_reach_that_tile_alone(B):
    c = Case([300, 300, 300], [[(0, 150), (150, 300)]] * 3, hq=8, hkv=2, d=128, seed=15)
    raw = c.pool.view(torch.uint8)
    raw[int(c.table[0, 0]), 5, 0] = 0x7F                 # K of kv head 0, tile 0
    raw[int(c.table[1, 4]), 1, 128 * 3 + 7] = 0xFF       # V of kv head 1, tile 1, dim 7
    c.scales[int(c.table[2, 1]), 2, 0] = float("nan")    # V scale of kv head 0, tile 0
    assert c.run(B) == 0
    o, l = c.out, c.lse
    assert o[0, 0, :4].isnan().all() and o[0, 0, 4:].isfinite().all() and o[0, 1].isfinite().all()
    assert o[1, 1, 4:, 7].isnan().all() and o[1, 1, :4].isfinite().all() and o[1, 0].isfinite().all()
    rest = torch.ones(128, dtype=torch.bool, device=DEV)
    rest[7] = False
    assert o[1, 1, 4:][:, rest].isfinite().all() and l[1].isfinite().all()
    assert o[2, 0, :4].isnan().all() and o[2, 0, 4:].isfinite().all() and o[2, 1].isfinite().all()


def test_bad_page_ids_are_reported_and_never_read(B):
    c = Case([200, 200], hq=8, hkv=2, d=256, seed=16)
    good = Case([200, 200], hq=8, hkv=2, d=256, seed=16)
    assert good.run(B) == 0
    c.table_dev[1, 1] = c.pages
    c.table_dev[1, 2] = -7
    assert c.run(B) == B.PA_STATUS_BAD_PAGE
    assert c.out[1].isnan().all() and c.lse[1].isnan().all() and c.merged[1].isnan().all()
    assert torch.equal(c.out[0], good.out[0]) and torch.equal(c.merged[0], good.merged[0])


def test_another_stream_and_a_captured_graph(B):
    c = Case([3000, 17, 500], [[(0, 2000), (2000, 3000)], [(0, 17)], [(0, 500)]], seed=17)
    assert c.run(B) == 0
    want = [t.clone() for t in (c.out, c.lse, c.merged, c.merged_lse)]
    side = torch.cuda.Stream()
    assert c.run(B, stream=side) == 0
    assert all(torch.equal(a, b) for a, b in zip(want, (c.out, c.lse, c.merged, c.merged_lse)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.paged_decode_attn_q8_lse(c.q, c.pool, c.scales, c.table_dev, c.tiles, c.scale, c.out,
                                   c.lse, c.ws, merged_out=c.merged, merged_lse=c.merged_lse)
    for _ in range(3):
        c.out.zero_(), c.merged.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (c.out, c.lse, c.merged, c.merged_lse)))
    c.q.neg_()
    graph.replay()
    torch.cuda.synchronize()
    c.check()


def test_pages_may_sit_anywhere(B):
    """Two pools that differ only in where the pages lie give the same bits."""
    a = Case([1500, 700], hq=24, hkv=4, d=256, seed=18, spare=20)
    assert a.run(B) == 0
    want = a.out.clone()
    perm = torch.randperm(a.pages, device=DEV)
    raw = torch.empty_like(a.pool.view(torch.uint8))
    raw[perm] = a.pool.view(torch.uint8)
    scales = torch.empty_like(a.scales)
    scales[perm] = a.scales
    a.pool, a.scales = raw.view(E4M3), scales
    a.table_dev = perm[a.table_dev.long()].int()
    assert a.run(B) == 0
    assert torch.equal(a.out, want)


@pytest.mark.parametrize("d", [128, 256])
def test_a_step_of_appends_and_attention(B, d):
    """Prompt appended in chunks, then decode steps of one token each, every one
    attended: the cache and the outputs match the oracle's at each step."""
    hq, hkv, inv = 8, 2, 10000.0 ** (-np.arange(d // 2) / (d // 2))
    inv = torch.from_numpy(inv.astype(np.float32)).to(DEV)
    g = torch.Generator(device=DEV).manual_seed(4)
    c = Case([256, 256], hq=hq, hkv=hkv, d=d, seed=19)
    at = [0, 0]
    for new in ([100, 37], [20, 0], [1, 1], [1, 1], [1, 1]):
        n = sum(new)
        qkv = torch.randn(n, hq + 2 * hkv, d, generator=g, device=DEV).bfloat16()
        q = torch.empty(n, hq, d, device=DEV, dtype=torch.bfloat16)
        cu = torch.tensor([0, new[0], n], dtype=torch.int32, device=DEV)
        pos = torch.tensor(at, dtype=torch.int32, device=DEV)
        B.kv_append_rope_q8(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], c.pool, c.scales,
                            c.table_dev, pos, inv, q, cu_tokens=cu)
        at = [a + m for a, m in zip(at, new)]
        if min(new) == 0:
            continue
        c.q = torch.stack([q[new[0] - 1], q[n - 1]])     # each request's newest token
        c.lengths = list(at)
        c.tiles = np.array([[(0, a)] for a in at], np.int32)
        assert c.run(B) == 0
        c.check()


def test_ctas_that_leave_the_merge_to_the_last_one(B):
    """A split unit's CTAs that do not wait for each other give the same bits."""
    c = Case([20000, 9000], hq=24, hkv=4, d=256, seed=20)
    assert c.run(B) == 0
    want = [t.clone() for t in (c.out, c.lse, c.merged, c.merged_lse)]
    B.test_slice_wait(0)
    assert c.run(B) == 0
    assert all(torch.equal(a, b) for a, b in zip(want, (c.out, c.lse, c.merged, c.merged_lse)))


@pytest.mark.parametrize("iteration", [0, 1, 4])
def test_a_wait_that_runs_out_is_reported_and_the_context_survives(B, iteration):
    """One step's loads of CTA 0 stay unarmed; with a 50 ms limit every warp
    gives up, the call reports it, and the next one is right again."""
    c = Case([64000], hq=24, hkv=4, d=256, seed=21)
    assert c.run(B) == 0
    want = c.out.clone()
    B.test_stall(iteration, 50_000_000)
    assert c.run(B) & B.PA_STATUS_TIMEOUT
    c.ws = None
    c.out.zero_()
    assert c.run(B) == 0
    assert torch.equal(c.out, want)


@pytest.mark.parametrize("rotated", [False, True])
def test_the_decode_step_over_an_8_bit_pool(B, rotated):
    """ResidentQ8Decode: the pool holds the bf16 history's nearest codes, the
    step's rotated rows join it, and every layer's outputs match the oracle's
    over what the pool holds; a captured step replays to the same bits."""
    from paged_decode_attention_attn_gb300 import decode, workloads as wl
    w = wl.custom([1500, 1, 65, 640], [[(0, 1000), (1000, 1500)], [(0, 1)], [(0, 65), (64, 65)],
                                       [(0, 640)]], seed=31, n_layers=2)
    t = wl.materialize(w, DEV)
    geo = w.geometry
    inv = torch.from_numpy((10000.0 ** (-np.arange(32) / 32)).astype(np.float32)).to(DEV)
    dec = decode.ResidentQ8Decode(w, t, inv_freq=inv if rotated else None)
    dec.step()
    torch.cuda.synchronize()
    assert dec.kernel_status() == 0
    heads = 2 * geo.n_kv_heads
    for i in range(w.n_layers):
        for r in range(w.batch):
            n = int(w.lengths[r])
            pages = torch.from_numpy(w.page_table[r, :w.pages_of(r)].astype(np.int64)).to(DEV)
            codes = dec.pool[i].view(torch.uint8)[pages].cpu().numpy().reshape(-1, heads, 256)
            scales = dec.scales[i][pages].double().cpu().numpy().transpose(0, 2, 1)
            scales = scales.reshape(-1, heads)
            kv = R.pool_values(codes, scales)[:n]
            want = wl.history_rows(w, t["pool"][i], r).double().cpu().numpy().reshape(n, heads, 256)
            step = np.repeat(scales, 16, 0)[:n, :, None] * 2.0 ** -10
            near = np.abs(kv - want) <= np.maximum(np.abs(want) / 16, step)
            assert near[:n - 1].all()
            new = t["new_rows"][i, r].double().cpu().numpy().reshape(heads, 256)
            if rotated:
                new[:4] = R.rotate(new[None, :4], [n - 1], inv.cpu().numpy())[0]
            slack = 1e-6 * np.max(np.abs(new))
            assert np.all(np.abs(kv[-1] - new) <= slack + np.maximum(np.abs(new) / 16, step[-1]))
            check_request(kv[:, :4], kv[:, 4:], dec.q[i, r], w.tiles[r], geo.scale,
                          dec.o.tile_out[i, r], dec.o.tile_lse[i, r], dec.merged[i, r],
                          dec.merged_lse[i, r], f"layer {i} request {r}")
    want = dec.merged.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dec.step()
    for _ in range(2):
        dec.merged.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert dec.kernel_status() == 0 and torch.equal(dec.merged, want)


def test_two_graphs_with_workspaces_of_their_own_overlap(B):
    """Two captured calls on two streams, each with its workspace, replayed
    together: each gives what it gives alone."""
    cases = [Case([9000, 30, 700], hq=24, hkv=4, d=256, seed=41),
             Case([5000, 2500], hq=32, hkv=8, d=128, seed=42)]
    graphs, wants, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for c in cases:
        assert c.run(B) == 0
        wants.append(c.out.clone())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(20):
                B.paged_decode_attn_q8_lse(c.q, c.pool, c.scales, c.table_dev, c.tiles, c.scale,
                                           c.out, c.lse, c.ws, merged_out=c.merged,
                                           merged_lse=c.merged_lse)
        graphs.append(g)
        c.out.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for c, want in zip(cases, wants):
        assert int(c.ws[:4].view(torch.int32).item()) == 0
        assert torch.equal(c.out, want)


def test_sixty_four_tiles_per_request(B):
    """Many tiles per request, empty and one-token ones among them, merged."""
    rng = np.random.default_rng(64)
    lengths, tiles = [9000, 1, 4097], []
    for n in lengths:
        cuts = np.sort(rng.integers(0, n + 1, 63))
        cuts = [0] + [int(c) for c in cuts] + [n]
        tiles.append(list(zip(cuts[:-1], cuts[1:])))
    c = Case(lengths, tiles, hq=16, hkv=2, d=128, seed=43)
    assert c.run(B) == 0
    c.check()
    whole = Case(lengths, hq=16, hkv=2, d=128, seed=43)
    assert whole.run(B) == 0
    assert float((c.merged - whole.merged).abs().max()) <= 1e-5 * float(whole.merged.abs().max())


def test_requests_without_tokens(B):
    c = Case([0, 5, 0], [[(0, 0), (0, 0)], [(0, 3), (3, 5)], [(0, 0), (0, 0)]], hq=8, hkv=2, d=128,
             seed=44)
    assert c.run(B) == 0
    c.check()
    c = Case([0, 0], hq=8, hkv=1, d=256, seed=45)
    assert c.run(B) == 0
    assert torch.all(c.merged == 0) and torch.all(c.merged_lse == -float("inf"))


def test_q_that_is_not_finite_gives_nan_in_its_head_alone(B):
    c = Case([200], hq=8, hkv=2, d=128, seed=46)
    c.q[0, 1, 3], c.q[0, 6, 0] = float("inf"), float("nan")
    assert c.run(B) == 0
    bad = torch.zeros(8, dtype=torch.bool, device=DEV)
    bad[1] = bad[6] = True
    assert c.out[0, 0][bad].isnan().all() and c.lse[0, 0][bad].isnan().all()
    assert c.out[0, 0][~bad].isfinite().all() and c.lse[0, 0][~bad].isfinite().all()


@pytest.mark.parametrize("n,full,tiles", [(256, 4, 1), (300, 3, 5), (1500, 2, 1), (200, 0, 3)])
def test_many_requests_without_tokens(B, n, full, tiles):
    """Padded batches: units without pages outnumber the others (and the CTAs)."""
    rng = np.random.default_rng(n)
    lengths = [0] * n
    for b in rng.choice(n, full, replace=False):
        lengths[b] = int(rng.integers(1, 900))
    cut = [[(min(x, t * 200), x if t == tiles - 1 else min(x, t * 200 + 200))
            for t in range(tiles)] for x in lengths]
    c = Case(lengths, cut, hq=8, hkv=2, d=256, seed=47)
    for _ in range(2):                      # the workspace is ready for another call
        c.merged.fill_(7.0)
        assert c.run(B) == 0
        c.check([b for b in range(n) if lengths[b]])
        empty = torch.tensor([x == 0 for x in lengths], device=DEV)
        assert torch.all(c.merged[empty] == 0)
        assert torch.all(c.merged_lse[empty] == -float("inf"))
        assert torch.all(c.out[empty] == 0) and torch.all(c.lse[empty] == -float("inf"))


def test_pages_past_4_gib_of_pool(B):
    """The same pages at the top of a 5.4 GB pool: the same bits."""
    c = Case([3000, 777], [[(0, 3000), (100, 2000)], [(0, 777), (777, 777)]], hq=24, hkv=4, d=256,
             seed=48)
    assert c.run(B) == 0
    want = [t.clone() for t in (c.out, c.lse, c.merged, c.merged_lse)]
    pages = 5_400_000_000 // (64 * 2 * c.hkv * c.d)
    lift = pages - c.pages
    pool = torch.full((pages, 64, 2 * c.hkv * c.d), 0x7F, dtype=torch.uint8, device=DEV)
    pool[lift:] = c.pool.view(torch.uint8)
    scales = torch.full((pages, 2 * c.hkv, 4), float("nan"), device=DEV)
    scales[lift:] = c.scales
    c.pool, c.scales, c.table_dev = pool.view(E4M3), scales, c.table_dev + lift
    assert c.run(B) == 0
    for a, b in zip((c.out, c.lse, c.merged, c.merged_lse), want):
        assert torch.equal(a, b)


def test_requests_that_share_pages(B):
    """A prefix common to two requests is stored once: both attend it."""
    c = Case([640, 1000, 700], hq=8, hkv=2, d=128, seed=49)
    for b in (1, 2):
        c.table[b, :6] = c.table[0, :6]
    c.table_dev.copy_(torch.from_numpy(c.table))
    assert c.run(B) == 0
    c.check()


@pytest.mark.parametrize("tiles", [2, 8, 9, 37])
@pytest.mark.parametrize("d", [128, 256])
def test_merge_of_any_number_of_tiles(B, tiles, d):
    """Requests whose tiles are all there, partly empty, all empty, and one with
    a NaN scale in its last tile."""
    step = 70
    lengths = [step * tiles, step * (tiles // 2) + 1, 0, step * tiles]
    cut = [[(min(n, t * step), min(n, t * step + step)) for t in range(tiles)] for n in lengths]
    c = Case(lengths, cut, hq=6, hkv=2, d=d, seed=50)
    last = int(c.table[3, (lengths[3] - 1) // 64])
    c.scales[last, 2 * c.hkv - 1, (lengths[3] - 1) % 64 // 16] = float("nan")   # V of head 1
    assert c.run(B) == 0
    c.check([0, 1])
    assert torch.all(c.merged[2] == 0) and torch.all(c.merged_lse[2] == -float("inf"))
    assert c.merged[3, 3:].isnan().all()
    assert c.merged[3, :3].isfinite().all() and c.merged_lse[3, :3].isfinite().all()


@pytest.mark.parametrize("n,top,geo", [(64, 900, (8, 8, 128)), (200, 300, (6, 2, 256)),
                                       (400, 150, (16, 4, 128)), (170, 2000, (4, 1, 256))])
def test_batches_of_more_units_than_ctas(B, n, top, geo):
    """Units of very different lengths, dealt to CTAs whole and out of order, in
    one launch or several, some of them empty."""
    hq, hkv, d = geo
    rng = np.random.default_rng(n)
    lengths = rng.integers(0, top, n).tolist()
    tiles = [[(0, x // 3), (x // 3, x)] for x in lengths]
    c = Case(lengths, tiles, hq=hq, hkv=hkv, d=d, seed=51)
    assert c.run(B) == 0
    c.check(rng.choice(n, 24, replace=False).tolist() + [int(np.argmax(lengths))])
    want = [t.clone() for t in (c.out, c.lse, c.merged, c.merged_lse)]
    assert c.run(B) == 0
    assert all(torch.equal(a, b) for a, b in zip(want, (c.out, c.lse, c.merged, c.merged_lse)))
