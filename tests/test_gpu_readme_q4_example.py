"""The 4-bit example in README.md runs as written, after the others, and its merged
output for one request matches the oracle over the pool's values."""

import os
import re

import numpy as np
import pytest
import torch

import oracle
from oracle import rope_q4 as Q
from oracle import rope_q8 as R

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_q4_example():
    from paged_decode_attention_attn_gb300 import build
    build.build()
    text = open(os.path.join(ROOT, "README.md")).read()
    blocks = re.findall(r"```py(?:thon)?\n(.*?)```", text, re.S)
    assert len(blocks) == 3
    env = {}
    torch.manual_seed(0)
    for code in blocks:
        exec(compile(code, "README.md", "exec"), env)
    torch.cuda.synchronize()
    assert int(env["ws4"][:4].view(torch.int32).item()) == 0
    r, L, D, Hkv = 1, env["L"], env["D"], env["Hkv"]
    pages = env["table"][r].long()
    kv = Q.values(*(env[n][pages].transpose(1, 2).cpu().numpy() for n in ("pool4", "scales4")))
    kv = kv.reshape(-1, 2 * Hkv, D)[:L]
    inv, w = env["inv_freq"].cpu().numpy(), env["k_weight"].double().cpu().numpy()
    for pos in (0, 777, L - 1):               # prompt rows and the step's own
        x = (env["k"][r * (L - 1) + pos] if pos < L - 1 else env["k8"][r]).double().cpu().numpy()
        x = x * w / np.sqrt(np.mean(x * x, -1, keepdims=True) + 1e-6)
        y = R.rotate(x[None], [pos], inv)[0]
        # half a step of a code: a quarter of the scale, which is below a third of its group's
        # largest value, or at most a quarter of the value
        step = np.repeat(np.abs(y).reshape(Hkv, -1, 32).max(-1) / 12, 32, 1)
        assert np.all(np.abs(kv[pos, :Hkv] - y) <= 1e-5 + np.maximum(np.abs(y) / 4, step)), pos
    q = env["q_rot"][r].double().cpu().numpy()
    tiles = [tuple(x) for x in env["tiles"][r]]
    outs, lses = oracle.tile_attention(q, kv[:, :Hkv], kv[:, Hkv:], tiles, 1 / 16)
    want, want_lse = oracle.lse_merge(outs, lses)
    # scores within 2^-21 of their largest sum of magnitudes (see test_gpu_decode_q4)
    A = max(np.max(np.abs(kv[:, h // (env["Hq"] // Hkv)]) @ np.abs(q[h])) for h in range(len(q)))
    e = 2.0 ** -21 * A / 16 + 2.0 ** -18
    got, got_lse = (env[n][r].double().cpu().numpy() for n in ("merged", "merged_lse"))
    assert np.max(np.abs(got - want)) <= (e + 2.0 ** -16) * np.max(np.abs(kv[:, Hkv:]))
    assert np.max(np.abs(got_lse - want_lse)) <= e + 2.0 ** -22 * np.max(np.abs(want_lse))
