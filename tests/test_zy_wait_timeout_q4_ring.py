"""The 4-bit decode gives up past the first turn of its ring too (16 stages for eight teams of two
warps at 128 dims, 9 stages for four teams of four at 256): the last loads of the first turn, the
first of the second and later ones, each left unarmed under a limit of 50 ms."""

import time

import pytest
import torch
from test_zy_wait_timeout_q4 import B, prepared  # noqa: F401

pytestmark = pytest.mark.gpu
STAGES = {128: 16, 256: 9}


@pytest.mark.parametrize("d,load", [(d, load) for d, n in STAGES.items()
                                    for load in (n - 2, n - 1, n, n + 1, n + 4, 2 * n - 1, 2 * n,
                                                 2 * n + 1)])
@pytest.mark.parametrize("tiles", [
    [(5, 200011)],                                      # 41 pages and more to a CTA
    [(3 * r % 50, 70 + 7 * r % 700) for r in range(500)]])  # units of 2 to 12 pages, 45 and more
def test_a_page_that_never_arrives_in_a_later_turn(B, d, load, tiles):
    s, run = prepared(B, tiles, d, 8, 2)
    assert run() == 0
    want = s["out"].clone()
    B.test_stall(load, 50_000_000)
    t0 = time.perf_counter()
    status = run()
    assert time.perf_counter() - t0 < 1.5
    assert status & B.PA_STATUS_TIMEOUT
    s["out"].zero_()
    assert run() == 0 and torch.equal(s["out"], want)
