"""The 8-bit example in README.md runs as written, after the first one, and its
merged output for one request matches the oracle over the pool's values."""

import os
import re

import numpy as np
import pytest
import torch

import oracle
from oracle import rope_q8 as R

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_q8_example():
    from paged_decode_attention_attn_gb300 import build
    build.build()
    text = open(os.path.join(ROOT, "README.md")).read()
    blocks = re.findall(r"```python\n(.*?)```", text, re.S)
    assert len(blocks) == 2
    env = {}
    torch.manual_seed(0)
    for code in blocks:
        exec(compile(code, "README.md", "exec"), env)
    torch.cuda.synchronize()
    assert int(env["ws8"][:4].view(torch.int32).item()) == 0
    r, L, D, Hkv = 1, env["L"], env["D"], env["Hkv"]
    pages = env["table"][r].long()
    codes = env["codes"][pages].cpu().numpy().reshape(-1, 2 * Hkv, D)
    scales = env["scales"][pages].double().cpu().numpy().transpose(0, 2, 1)
    kv = R.pool_values(codes, scales.reshape(-1, 2 * Hkv))[:L]
    inv = env["inv_freq"].cpu().numpy()
    for pos in (0, 777, L - 1):               # prompt rows and the step's own
        x = (env["k"][r * (L - 1) + pos] if pos < L - 1 else env["k8"][r]).double().cpu().numpy()
        y = R.rotate(x[None], [pos], inv)[0]
        step = np.repeat(scales.reshape(-1, 2 * Hkv)[pos // 16][:Hkv, None], D, 1) * 2.0 ** -10
        slack = 4e-7 * 2 * np.max(np.abs(x))
        assert np.all(np.abs(kv[pos, :Hkv] - y) <= slack + np.maximum(np.abs(y) / 16, step)), pos
    q = env["q_rot"][r].double().cpu().numpy()
    tiles = [tuple(x) for x in env["tiles"][r]]
    outs, lses = oracle.tile_attention(q, kv[:, :Hkv], kv[:, Hkv:], tiles, 1 / 16)
    want, want_lse = oracle.lse_merge(outs, lses)
    # scores within 2^-21 of their largest sum of magnitudes (see test_gpu_decode_q8)
    A = max(np.max(np.abs(kv[:, h // (env["Hq"] // Hkv)]) @ np.abs(q[h])) for h in range(len(q)))
    e = 2.0 ** -21 * A / 16 + 2.0 ** -18
    got, got_lse = (env[n][r].double().cpu().numpy() for n in ("merged", "merged_lse"))
    assert np.max(np.abs(got - want)) <= (e + 2.0 ** -16) * np.max(np.abs(kv[:, Hkv:]))
    assert np.max(np.abs(got_lse - want_lse)) <= e + 2.0 ** -22 * np.max(np.abs(want_lse))
