"""Keys of the 4-bit append near a border between two codes, against the form in plain FP32
arithmetic that its definition names, written out with elementary torch operations.

Tolerances.  A sine or cosine is the nearest float but for 2.1 in 100,000 (counted over 2
million angles of the whole range), so 8.4 in 100,000 turned values take part in one that is
not.  Such a value is off by at most two steps of 2^-24 of itself, and goes to another code if
a border lies between: seven borders over the octaves that codes span, a share of at most 2 *
2^-24 * 7 = 2^-20.2 of values.  Of 2.7 10^8 values, then, 0.02 go another way, and more than two
hardly ever.  Values chosen as the nearest to a border of 2,048 lie there up to 2,048 times as
often: of 4.2 million 0.6, and more than four once in 2,500 draws."""

import pytest
import torch

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


def sum_of_squares(x):
    t = x * x
    d = x.shape[-1]
    if d == 256:
        t = t[..., :128] + t[..., 128:]
        t = ((t[..., 0::4] + t[..., 1::4]) + t[..., 2::4]) + t[..., 3::4]
    else:
        t = ((t[..., :32] + t[..., 32:64]) + t[..., 64:96]) + t[..., 96:]
    while t.shape[-1] > 1:
        t = t[..., 0::2] + t[..., 1::2]
    return t


def plain(x, pos, inv, inter, weight):
    """The values that the codes of bf16 heads x [n][h][d] at positions pos stand for."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(sum_of_squares(x) / x.shape[-1] + EPS) * weight
    angle = pos.double()[:, None] * inv.double()
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if inter:
        a, b = x[..., 0::2], x[..., 1::2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x.chunk(2, -1)
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    g = y.unflatten(-1, (-1, 32))
    mant, expo = torch.frexp(g.abs().amax(-1, keepdim=True))     # 6 = 0.75 * 2^3
    e = (expo - 3 + (mant > 0.75).int()).clamp(min=-60)
    a = torch.ldexp(g.abs(), -e)
    step = 0.5 + 0.5 * (a >= 2).float() + (a >= 4).float()
    return torch.ldexp(torch.copysign(torch.round(a / step) * step, g), e).flatten(-2)


def differing(B, k, first, inv, inter, weight):
    """Codes of one request's keys k from position `first` (of a page's first token) that are
    not the plain form's."""
    n, hkv, d = k.shape
    pages = -(-n // 64)
    pool = torch.zeros(pages, 2 * hkv, 64, d // 2, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(pages, 2 * hkv, 64, d // 32, dtype=torch.uint8, device=DEV)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    out = torch.empty(n, 2 * hkv * d, dtype=torch.bfloat16, device=DEV)
    # pages ahead of the rows are named, and not touched
    table = torch.zeros(1, first // 64 + pages, dtype=torch.int32, device=DEV)
    table[0, first // 64:] = torch.arange(pages, dtype=torch.int32, device=DEV)
    at = torch.full((1,), first, dtype=torch.int32, device=DEV)
    B.kv_append_rope_q4(None, k, k, pool, scales, table, at, inv, cu_tokens=cu,
                        interleaved=inter, k_weight=weight, eps=EPS)
    B.kv_gather_q4(pool, scales, table, at, cu, out)
    other = 0
    for i in range(0, n, 8192):
        x = k[i:i + 8192]
        want = plain(x, first + i + torch.arange(len(x), device=DEV), inv, inter, weight)
        other += int((out[i:i + 8192, :hkv * d].view(x.shape).float() != want).sum())
    return other


def frequencies(d):
    return (10000.0 ** (-torch.arange(d // 2, device=DEV, dtype=torch.float64) / (d // 2))).float()


@pytest.mark.parametrize("d,inter", [(256, False), (128, True)])
def test_normed_keys_go_as_in_the_plain_form(B, d, inter):
    hkv, n = 4, (1 << 26) // (4 * d)
    g = torch.Generator(device=DEV).manual_seed(d)
    weight = 0.5 + torch.rand(d, generator=g, device=DEV)
    other = sum(differing(B, torch.randn(n, hkv, d, generator=g, device=DEV).bfloat16(), r * n,
                          frequencies(d), inter, weight) for r in range(4))
    assert other <= 2


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("inter", [False, True])
def test_keys_at_borders_go_as_in_the_plain_form(B, d, inter):
    """Of 2,048 pairs, all within 6 in magnitude, the one whose first value comes nearest to a
    border of the scale 1 when it is turned."""
    hkv, n, first = 4, (1 << 21) // (2 * d), 3200
    g = torch.Generator(device=DEV).manual_seed(d + inter)
    inv = frequencies(d)
    angle = (first + torch.arange(n, device=DEV)).double()[:, None] * inv.double()
    c, s = angle.cos().float(), angle.sin().float()
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    pairs = []
    for i in range(0, n, 64):
        shape = (min(64, n - i), hkv, d // 2, 2048)
        a, b = ((8 * torch.rand(shape, generator=g, device=DEV) - 4).bfloat16() for _ in range(2))
        y = (a.float() * c[i:i + 64, None, :, None] - b.float() * s[i:i + 64, None, :, None]).abs()
        near = border[torch.bucketize(y, (border[1:] + border[:-1]) / 2)]
        best = ((y - near).abs() / near).argmin(-1, keepdim=True)
        pairs.append(torch.cat([a.gather(-1, best), b.gather(-1, best)], -1))
    k = torch.cat(pairs)                                 # [n][hkv][d / 2][2]
    k = k.flatten(2) if inter else k.transpose(2, 3).flatten(2)
    assert differing(B, k.contiguous(), first, inv, inter, None) <= 4
