"""Failure detection in the 8-bit decode without a fault: a load of V that is
never armed runs the waits for it out, at steps whose tile begins or ends inside
a page, where only some lanes of a warp wait for V (they clear the rows outside
the tile).  Every wait has the 50 ms limit and every lane of a warp gets one
answer, so every CTA returns, the call reports it, and the next one is right."""

import time

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda"
HQ, HKV = 8, 2


@pytest.fixture(scope="module")
def B():
    from paged_decode_attention_attn_gb300 import build
    build.build()
    from paged_decode_attention_attn_gb300 import binding
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return binding


def prepared(B, tiles, d):
    """Requests of one tile each over pages of their own, scales all one."""
    g = torch.Generator(device=DEV).manual_seed(d)
    n, width = len(tiles), max(-(-e // 64) for _, e in tiles)
    s = dict(pool=(torch.randn(n * width, 64, 2 * HKV * d, generator=g, device=DEV) / 4).to(
        torch.float8_e4m3fn), scales=torch.ones(n * width, 2 * HKV, 4, device=DEV),
        table=torch.arange(n * width, dtype=torch.int32, device=DEV).view(n, width),
        q=torch.randn(n, HQ, d, generator=g, device=DEV).bfloat16(),
        tiles=np.array([[t] for t in tiles], np.int32), out=torch.empty(n, 1, HQ, d, device=DEV),
        lse=torch.empty(n, 1, HQ, device=DEV))

    def run():
        ws = B.alloc_workspace_q8(n, 1, HQ, HKV, d)     # a fresh one for every call
        B.paged_decode_attn_q8_lse(s["q"], s["pool"], s["scales"], s["table"], s["tiles"],
                                   d ** -0.5, s["out"], s["lse"], ws)
        torch.cuda.synchronize()
        return int(ws[:4].view(torch.int32).item())
    return s, run


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("step", [0, 1, 2])
@pytest.mark.parametrize("tiles", [
    # 938 pages and 6 of charge per head on 152 CTAs: three steps on CTA 0, the first
    # from inside a page
    [(5, 60011)],
    # about four units on a CTA, every step begins or ends inside a page
    [(3 * r % 50, 70 + r % 190) for r in range(300)]])
def test_values_that_never_arrive_are_reported(B, d, step, tiles):
    s, run = prepared(B, tiles, d)
    assert run() == 0
    want = s["out"].clone()
    B.test_stall(step, 50_000_000, values=True)
    t0 = time.perf_counter()
    assert run() & B.PA_STATUS_TIMEOUT
    assert time.perf_counter() - t0 < 1.5           # the limit of 50 ms, not 2 s
    s["out"].zero_()
    assert run() == 0 and torch.equal(s["out"], want)
    lo, hi = tiles[0]
    kv = s["pool"][:s["table"].shape[1]].float().double().cpu().numpy()
    kv = kv.reshape(-1, 2 * HKV, d)[:hi]
    o, _ = oracle.tile_attention(s["q"][0].double().cpu().numpy(), kv[:, :HKV], kv[:, HKV:],
                                 [(lo, hi)], d ** -0.5)
    # scores within 8 steps of 2^-24 of sum |q k| / sqrt(d) < 16, probabilities of
    # four parts within 2^-18 of themselves, |V| < 2
    err = np.abs(s["out"][0, 0].double().cpu().numpy() - o[0])
    assert err.max() <= 2 * (2.0 ** -21 * 16 + 2.0 ** -18 + 2.0 ** -16)


def test_the_hook_of_the_values_leaves_a_bf16_call_alone(B):
    """Its load numbers never reach the flag: the call runs and consumes the hook."""
    from paged_decode_attention_attn_gb300 import decode, workloads as wl
    w = wl.custom([700], [[(0, 700)]], seed=3, n_spare=1)
    dec = decode.ResidentDecode(w, wl.materialize(w, DEV))
    B.test_stall(0, 50_000_000, values=True)
    dec.layer(0, attention_only=True)
    torch.cuda.synchronize()
    assert dec.kernel_status() == 0
