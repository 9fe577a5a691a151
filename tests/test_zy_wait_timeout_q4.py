"""Failure detection in the 4-bit decode without a fault: a page's load that is never
armed runs the waits for it out.  The warps of a page meet at barriers without a time
limit, so one that gives up goes on meeting the others until all have: every CTA returns
within the 50 ms limit, the call reports it, and the next one is right."""

import time

import numpy as np
import pytest
import torch

import oracle
from oracle import rope_q4 as Q

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def B():
    from paged_decode_attention_attn_gb300 import build
    build.build()
    from paged_decode_attention_attn_gb300 import binding
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return binding


def prepared(B, tiles, d, hq, hkv):
    """Requests of one tile each over pages of their own."""
    g = torch.Generator(device=DEV).manual_seed(d)
    n, width = len(tiles), max(-(-e // 64) for _, e in tiles)
    shape = (n * width, 2 * hkv, 64)
    s = dict(pool=torch.randint(0, 256, shape + (d // 2,), generator=g, device=DEV, dtype=torch.uint8),
             scales=torch.randint(124, 127, shape + (d // 32,), generator=g, device=DEV,
                                  dtype=torch.uint8),
             table=torch.arange(n * width, dtype=torch.int32, device=DEV).view(n, width),
             q=torch.randn(n, hq, d, generator=g, device=DEV).bfloat16(),
             tiles=np.array([[t] for t in tiles], np.int32), out=torch.empty(n, 1, hq, d, device=DEV),
             lse=torch.empty(n, 1, hq, device=DEV))

    def run():
        ws = B.alloc_workspace_q4(n, 1, hq, hkv, d)     # a fresh one for every call
        B.paged_decode_attn_q4_lse(s["q"], s["pool"], s["scales"], s["table"], s["tiles"],
                                   d ** -0.5, s["out"], s["lse"], ws)
        torch.cuda.synchronize()
        return int(ws[:4].view(torch.int32).item())
    return s, run


@pytest.mark.parametrize("d", [128, 256])
# the loads of each of a CTA's first pages, of pages after a stage's first use (17 and 9
# stages), and of later segments
@pytest.mark.parametrize("page", [0, 1, 2, 3, 5, 7, 8, 9, 10, 12])
@pytest.mark.parametrize("tiles", [
    [(5, 120011)],                                      # a unit over many CTAs
    [(3 * r % 50, 70 + r % 190) for r in range(600)]])  # several units on a CTA
def test_a_page_that_never_arrives_is_reported(B, d, page, tiles):
    s, run = prepared(B, tiles, d, 8, 2)
    assert run() == 0
    want = s["out"].clone()
    B.test_stall(page, 50_000_000)
    t0 = time.perf_counter()
    status = run()
    assert time.perf_counter() - t0 < 1.5               # the limit of 50 ms, not 2 s
    assert status & B.PA_STATUS_TIMEOUT
    s["out"].zero_()
    assert run() == 0 and torch.equal(s["out"], want)


def test_the_hook_of_the_values_leaves_a_4_bit_call_alone(B):
    """Its load numbers never reach the flag: the call runs and consumes the hook."""
    s, run = prepared(B, [(0, 700)], 256, 8, 2)
    assert run() == 0
    want = s["out"].clone()
    B.test_stall(0, 50_000_000, values=True)
    assert run() == 0 and torch.equal(s["out"], want)


def test_more_kv_heads_than_16_bits_count(B):
    """Three heads of 70,000 against the oracle."""
    hkv, d, n = 70_000, 128, 9
    s, run = prepared(B, [(0, n)], d, hkv, hkv)
    assert run() == 0
    for h in (0, 65_535, hkv - 1):
        kv = Q.values(*(x[0][[h, hkv + h]].cpu().numpy() for x in (s["pool"], s["scales"])))[:, :n]
        o, lse = oracle.tile_attention(s["q"][0, h:h + 1].double().cpu().numpy(), kv[0][:, None],
                                       kv[1][:, None], [(0, n)], d ** -0.5)
        # |q k| sums below 100 / sqrt(128) = 9: scores within 2^-21 of that, probabilities
        # within 2^-17; values at most 6 * 2^-1
        assert np.max(np.abs(s["out"][0, 0, h].double().cpu().numpy() - o[0][0])) <= 3 * 2.0 ** -16
        assert abs(float(s["lse"][0, 0, h]) - float(lse[0][0])) <= 2.0 ** -17 + 2.0 ** -22 * abs(
            float(lse[0][0]))
