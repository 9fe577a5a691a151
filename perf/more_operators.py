"""The appends with norms and the 4-bit paged cache, as measured cases.

Three operators, each in its plain form (elementary torch operations) and as
the framework's own calls:

  norm_append  a root-mean-square norm of every q and k head and the rotation by
               the positions, with k and v stored in a bf16 paged cache
  append_q4    the same (the norms are optional) into a cache held in 4 bits
               (e2m1 codes, a power of two as the scale of each 32 values of a
               head), and the new rows read back as the values they stand for
  decode_q4    grouped-query decode attention over that cache, per tile of the
               history (normalised output and log-sum-exp) and merged
"""

import torch

own = False

PAGE = 64          # tokens per page
GROUP = 32         # values per scale of the 4-bit cache
MIN_EXP = -60      # log2 of the smallest scale written
EPS = 1e-6
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # One sequence, one new token: the smallest append of a decode step.
        dict(name="norm_append 1 token", op="norm_append", batch=1, new_lo=1, new_hi=1,
             past_lo=31743, past_hi=31743, pad=0, hq=24, hkv=4, d=256, rot=256, inter=False,
             norm=True, shape=1),
        # A decode step of a served batch, one new token each, odd batch size.
        dict(name="norm_append 47 tokens", op="norm_append", batch=47, new_lo=1, new_hi=1,
             past_lo=3, past_hi=9000, pad=0, hq=32, hkv=8, d=128, rot=128, inter=False, norm=True,
             shape=2),
        # Prompts of very different lengths packed one after another, half of
        # each head rotated in adjacent pairs, padding rows behind the last one.
        dict(name="norm_append 13 ragged prompts", op="norm_append", batch=13, new_lo=0,
             new_hi=2100, past_lo=0, past_hi=4000, pad=29, hq=32, hkv=8, d=128, rot=64, inter=True,
             norm=True, shape=3),
        # One new token of one far sequence into the 4-bit cache.
        dict(name="append_q4 1 token", op="append_q4", batch=1, new_lo=1, new_hi=1,
             past_lo=200005, past_hi=200005, pad=0, hq=24, hkv=4, d=256, rot=256, inter=False,
             norm=True, shape=4),
        # A decode step of a served batch into the 4-bit cache, without norms.
        dict(name="append_q4 96 tokens", op="append_q4", batch=96, new_lo=1, new_hi=1, past_lo=0,
             past_hi=9000, pad=0, hq=32, hkv=8, d=128, rot=128, inter=False, norm=False, shape=5),
        # A few proposed tokens for each of a batch, a quarter of each head rotated.
        dict(name="append_q4 17x1-5 tokens", op="append_q4", batch=17, new_lo=1, new_hi=5,
             past_lo=0, past_hi=5000, pad=7, hq=16, hkv=2, d=128, rot=32, inter=True, norm=True,
             shape=6),
        # Two prompt chunks into the 4-bit cache.
        dict(name="append_q4 2 prompts", op="append_q4", batch=2, new_lo=3900, new_hi=4300,
             past_lo=0, past_hi=1000, pad=0, hq=24, hkv=4, d=256, rot=256, inter=False, norm=True,
             shape=7),
        # One short sequence: a single decode launch where latency counts.
        dict(name="decode_q4 1x900", op="decode_q4", batch=1, len_lo=900, len_hi=900, tile=32768,
             hq=24, hkv=4, d=256, shape=8),
        # A served batch of chat-length sequences.
        dict(name="decode_q4 64 to 3000", op="decode_q4", batch=64, len_lo=1, len_hi=3000,
             tile=32768, hq=32, hkv=8, d=128, shape=9),
        # The repository's bench shape: 4 sequences of 31,744 tokens.
        dict(name="decode_q4 4x31744", op="decode_q4", batch=4, len_lo=31744, len_hi=31744,
             tile=32768, hq=24, hkv=4, d=256, shape=10),
        # Ragged long sequences in tiles, some of them empty for the short ones.
        dict(name="decode_q4 9 ragged", op="decode_q4", batch=9, len_lo=700, len_hi=50000,
             tile=11000, hq=16, hkv=2, d=128, shape=11),
        # The repository's long-context shape: 262,144 tokens in 8 tiles.
        dict(name="decode_q4 1x262144", op="decode_q4", batch=1, len_lo=262144, len_hi=262144,
             tile=32768, hq=24, hkv=4, d=256, shape=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["norm_append", "append_q4", "decode_q4"])
    hq, hkv, d = rng.choice([(24, 4, 256), (32, 8, 128), (16, 2, 128), (8, 8, 256), (7, 1, 256),
                             (20, 5, 128), (32, 4, 128)])
    shape = rng.randrange(1 << 20)
    if op == "decode_q4":
        batch = _log_int(rng, 1, 64)
        most = min(250000, (1 << 28) // (hkv * d)) // batch
        top = _log_int(rng, 64, max(64, most))
        return dict(op=op, batch=batch, len_lo=int(top * rng.choice([0.0, 0.02, 0.3, 1.0])),
                    len_hi=top, tile=_log_int(rng, max(64, top // 8), 32768 + top), hq=hq, hkv=hkv,
                    d=d, shape=shape)
    batch = _log_int(rng, 1, 100)
    top = _log_int(rng, 1, max(1, 8000 // batch))
    if op == "norm_append" and d == 128 and rng.random() < 0.3:
        d = 64
    return dict(op=op, batch=batch, new_lo=rng.choice([0, 1, top]), new_hi=top, past_lo=0,
                past_hi=_log_int(rng, 16, 200000 // batch), pad=rng.choice([0, 0, 5]), hq=hq,
                hkv=hkv, d=d, rot=rng.choice([d, d, d // 2, d // 4 + 8]),
                inter=rng.random() < 0.4, norm=op == "norm_append" or rng.random() < 0.6,
                shape=shape)


def _ints(case, lo, hi, salt):
    g = torch.Generator().manual_seed(case["shape"] * 8 + salt)
    n = torch.randint(lo, hi + 1, (case["batch"],), generator=g)
    if lo == 0 and int(n.sum()) == 0:
        n[0] = max(1, hi)
    return n


def _new_tokens(case):
    """New tokens of each sequence (some may have none)."""
    return _ints(case, min(case["new_lo"], case["new_hi"]), case["new_hi"], 0)


def _past_tokens(case):
    return _ints(case, min(case["past_lo"], case["past_hi"]), case["past_hi"], 1)


def _lengths(case):
    return _ints(case, min(case["len_lo"], case["len_hi"]), case["len_hi"], 2)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _tables(lengths, first, gen, dev):
    """Physical pages of the logical pages [first, end) each sequence uses, in
    shuffled order; the pages before `first` are named but never touched."""
    ends = (lengths + PAGE - 1) // PAGE
    width = max(1, int(ends.max()))
    n = int((ends - first).clamp(min=0).sum())
    perm = torch.randperm(n + 2, generator=gen, device=dev).int()
    table = torch.zeros(len(lengths), width, dtype=torch.int32, device=dev)
    at = torch.arange(width)[None]
    table[((at >= first[:, None]) & (at < ends[:, None])).to(dev)] = perm[:n]
    return table, n + 2


def _values(n, h, d, gen, dev, spread=None):
    """bf16 activations as projections give them: unit variance, with channels
    of a larger scale where `spread` is given."""
    x = torch.randn(n, h, d, generator=gen, device=dev)
    return (x if spread is None else x * spread).bfloat16()


def _spread(h, d, gen, dev):
    return torch.exp(0.5 * torch.randn(h, d, generator=gen, device=dev))


def _quantised(x):
    """Codes (two a byte, the lower index in the low bits) and exponents of the
    scales (biased by 127) of finite x [..., d], in 32 bits."""
    g = x.unflatten(-1, (-1, GROUP))
    amax = g.abs().amax(-1)
    mant, expo = torch.frexp(amax)                   # amax = mant 2^expo, 6 = 0.75 2^3
    e = torch.where(amax > 0, expo - 3 + (mant > 0.75).int(), torch.full_like(expo, MIN_EXP))
    e = e.clamp(min=MIN_EXP)
    a = torch.ldexp(g.abs(), -e[..., None])
    step = 0.5 + 0.5 * (a >= 2).float() + (a >= 4).float()
    a = torch.round(a / step) * step                 # ties to even: to the even code
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code | (g < 0).to(torch.uint8) << 3).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, (e + 127).to(torch.uint8)


def _table16(dev, dtype):
    return torch.tensor(E2M1 + [-v for v in E2M1], device=dev, dtype=dtype)


def _dequantised(codes, exps):
    """What codes [..., d / 2] and scales [..., d / 32] stand for, in 32 bits."""
    lut = _table16(codes.device, torch.float32)
    x = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], -1).flatten(-2)
    s = torch.exp2(exps.float() - 127)
    s = torch.where(exps == 255, torch.full_like(s, torch.nan), s)
    return (x.unflatten(-1, (-1, GROUP)) * s[..., None]).flatten(-2)


def _filled(pages, hkv, d, gen, dev):
    """A cache in 4 bits whose every row is there: codes and scales."""
    pool = torch.empty(pages, 2 * hkv, PAGE, d // 2, dtype=torch.uint8, device=dev)
    scales = torch.empty(pages, 2 * hkv, PAGE, d // GROUP, dtype=torch.uint8, device=dev)
    spread = torch.cat([_spread(hkv, d, gen, dev), torch.ones(hkv, d, device=dev)])[:, None]
    step = max(1, (1 << 25) // (PAGE * 2 * hkv * d))
    for p0 in range(0, pages, step):
        n = min(step, pages - p0)
        x = torch.randn(n, 2 * hkv, PAGE, d, generator=gen, device=dev) * spread
        pool[p0:p0 + n], scales[p0:p0 + n] = _quantised(x)
    return pool, scales


def _prepare_decode(case, gen, dev):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    lengths = _lengths(case)
    table, pages = _tables(lengths, torch.zeros_like(lengths), gen, dev)
    pool, scales = _filled(pages, hkv, d, gen, dev)
    # the rows behind each sequence's last token hold what an earlier user of
    # the page left there, scales that are NaN among it
    some = lengths[lengths > 0]
    last = table[(lengths > 0).to(dev)]
    last = last[torch.arange(len(some)), ((some - 1) // PAGE).to(dev)].long()
    behind = (torch.arange(PAGE)[None] > ((some - 1) % PAGE)[:, None]).to(dev)
    scales[last] = torch.where(behind[:, None, :, None], torch.full_like(scales[:1], 255), scales[last])
    n_tiles = max(1, -(-int(lengths.max()) // case["tile"]))
    start = torch.arange(n_tiles)[None] * case["tile"]
    tiles = torch.stack([torch.minimum(start, lengths[:, None]),
                         torch.minimum(start + case["tile"], lengths[:, None])], -1).int()
    state = dict(case=case, q=_values(case["batch"], hq, d, gen, dev), pool=pool, scales=scales,
                 table=table, tiles=tiles.numpy(), tiles_dev=tiles.to(dev), lengths=lengths.to(dev),
                 scale=d ** -0.5, out=torch.empty(case["batch"], n_tiles, hq, d, device=dev),
                 lse=torch.empty(case["batch"], n_tiles, hq, device=dev),
                 merged=torch.empty(case["batch"], hq, d, device=dev),
                 merged_lse=torch.empty(case["batch"], hq, device=dev))
    if own:   # zero-filled once, kept by the program for every call
        from paged_decode_attention_attn_gb300 import binding as B
        state["workspace"] = B.alloc_workspace_q4(case["batch"], n_tiles, hq, hkv, d)
    return state


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    if case["op"] == "decode_q4":
        return _prepare_decode(case, gen, dev)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    new, past = _new_tokens(case), _past_tokens(case)
    ends = past + new
    # the pages that hold the new rows; a program's pool holds the rest too
    table, pages = _tables(torch.where(new > 0, ends, torch.zeros_like(ends)), past // PAGE, gen, dev)
    cu = torch.zeros(case["batch"] + 1, dtype=torch.int64)
    cu[1:] = new.cumsum(0)
    n = int(cu[-1])
    rows = n + case["pad"]
    qkv = torch.cat([_values(rows, hq, d, gen, dev, _spread(hq, d, gen, dev)),
                     _values(rows, hkv, d, gen, dev, _spread(hkv, d, gen, dev)),
                     _values(rows, hkv, d, gen, dev)], 1)     # one projection's output
    of = torch.repeat_interleave(torch.arange(case["batch"]), new)
    pos = past[of] + torch.arange(n) - cu[of]
    half = case["rot"] // 2
    inv = (1.0 / 10000.0 ** (torch.arange(half, dtype=torch.float64) / half)).float().to(dev)
    state = dict(case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], table=table,
                 positions=past.int().to(dev), cu=cu.int().to(dev), one_each=bool((new == 1).all())
                 and case["pad"] == 0, inv=inv, n=n, of=of.to(dev), pos=pos.to(dev),
                 q_out=torch.zeros(rows, hq, d, dtype=torch.bfloat16, device=dev),
                 q_weight=None, k_weight=None)
    if case["norm"]:
        state["q_weight"], state["k_weight"] = _spread(2, d, gen, dev).bfloat16().float()
    if case["op"] == "norm_append":
        state["pool"] = _values(pages * PAGE, 2 * hkv, d, gen, dev).view(pages, PAGE, 2 * hkv * d)
        return state
    state["pool"], state["scales"] = _filled(pages, hkv, d, gen, dev)
    state["back"] = torch.zeros(n, 2 * hkv * d, dtype=torch.bfloat16, device=dev)
    return state


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _turned(x, weight, s):
    """Heads x [n, h, d] normed (unless weight is None) and turned by their
    positions; angles in 64 bits, the rest in 32."""
    half = s["inv"].numel()
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    angle = s["pos"].double()[:, None] * s["inv"].double()[None]
    c, t = angle.cos().float()[:, None], angle.sin().float()[:, None]
    r = x[..., :2 * half]
    if s["case"]["inter"]:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack([a * c - b * t, b * c + a * t], -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        y = torch.cat([a * c - b * t, b * c + a * t], -1)
    return torch.cat([y, x[..., 2 * half:]], -1)


def _places(s):
    """Page and row in it of every new token."""
    return s["table"][s["of"], torch.div(s["pos"], PAGE, rounding_mode="floor")].long(), s["pos"] % PAGE


def _plain_norm_append(s):
    n = s["n"]
    s["q_out"][:n] = _turned(s["q"][:n], s["q_weight"], s).bfloat16()
    k = _turned(s["k"][:n], s["k_weight"], s).bfloat16()
    page, row = _places(s)
    s["pool"][page, row] = torch.cat([k, s["v"][:n]], 1).flatten(1)
    return {"q": s["q_out"], "pool": s["pool"]}


def _plain_append_q4(s):
    n = s["n"]
    s["q_out"][:n] = _turned(s["q"][:n], s["q_weight"], s).bfloat16()
    x = torch.cat([_turned(s["k"][:n], s["k_weight"], s), s["v"][:n].float()], 1)
    page, row = _places(s)
    s["pool"][page, :, row], s["scales"][page, :, row] = _quantised(x)
    s["back"].copy_(_dequantised(s["pool"][page, :, row], s["scales"][page, :, row]).flatten(1))
    return _append_q4_outputs(s)


def _append_q4_outputs(s):
    kd = s["case"]["hkv"] * s["case"]["d"]
    return {"q": s["q_out"], "k": s["back"][:, :kd], "v": s["back"][:, kd:]}


def _plain_decode_q4(s):
    c = s["case"]
    b, hq, hkv, d = c["batch"], c["hq"], c["hkv"], c["d"]
    table = s["table"].long()
    x = _dequantised(s["pool"][table], s["scales"][table])               # [b][page][head][row][d]
    x = x.transpose(1, 2).flatten(2, 3)                                  # [b][head][token][d]
    k, v = x[:, :hkv].transpose(2, 3), x[:, hkv:]
    at = torch.arange(v.shape[2], device=x.device)
    v = torch.where((at[None] < s["lengths"][:, None])[:, None, :, None], v, torch.zeros((), device=x.device))
    scores = torch.matmul(s["q"].float().view(b, hkv, hq // hkv, d), k) * s["scale"]
    tiles = s["tiles_dev"]
    inside = (at >= tiles[..., :1]) & (at < tiles[..., 1:])              # [b][tile][token]
    scores = torch.where(inside[:, :, None, None], scores[:, None], torch.full((), -torch.inf, device=x.device))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top > -torch.inf, top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v[:, None]) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + total.log())[..., 0]
    m = lse.amax(1, keepdim=True)
    m = torch.where(m > -torch.inf, m, torch.zeros_like(m))
    w = torch.exp(lse - m)
    merged = (w[..., None] * out).sum(1) / torch.where(w.sum(1) > 0, w.sum(1), torch.ones_like(m[:, 0]))[..., None]
    t = tiles.shape[1]
    return {"out": out.view(b, t, hq, d), "lse": lse.reshape(b, t, hq), "merged": merged.view(b, hq, d),
            "merged_lse": (m[:, 0] + w.sum(1).log()).view(b, hq)}


def run(state):
    s, op, inter = state, state["case"]["op"], state["case"].get("inter")
    if not own:
        return {"norm_append": _plain_norm_append, "append_q4": _plain_append_q4,
                "decode_q4": _plain_decode_q4}[op](s)
    from paged_decode_attention_attn_gb300 import binding as B
    if op == "decode_q4":
        B.paged_decode_attn_q4_lse(s["q"], s["pool"], s["scales"], s["table"], s["tiles"], s["scale"],
                                   s["out"], s["lse"], s["workspace"], merged_out=s["merged"],
                                   merged_lse=s["merged_lse"])
        return {"out": s["out"], "lse": s["lse"], "merged": s["merged"], "merged_lse": s["merged_lse"]}
    cu = None if s["one_each"] else s["cu"]
    if op == "norm_append":
        B.kv_append_norm_rope(s["q"], s["k"], s["v"], s["pool"], s["table"], s["positions"], s["inv"],
                              s["q_weight"], s["k_weight"], s["q_out"], cu_tokens=cu,
                              interleaved=inter, eps=EPS)
        return {"q": s["q_out"], "pool": s["pool"]}
    B.kv_append_rope_q4(s["q"], s["k"], s["v"], s["pool"], s["scales"], s["table"], s["positions"],
                        s["inv"], s["q_out"], cu_tokens=cu, interleaved=inter,
                        q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS)
    B.kv_gather_q4(s["pool"], s["scales"], s["table"], s["positions"], cu, s["back"])
    return _append_q4_outputs(s)


# --------------------------------------------------------------------------
# the work of one pass, and its results in 64 bits
# --------------------------------------------------------------------------
def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    row = 2 * hkv * (d // 2 + d // GROUP)                      # codes and scales of a token
    if case["op"] == "decode_q4":
        n = int(_lengths(case).sum())
        tiles = max(1, -(-int(_lengths(case).max()) // case["tile"]))
        rows = case["batch"] * hq
        return {"bytes": n * row + rows * d * 2 + rows * (tiles + 1) * (d + 1) * 4,
                "flops": 4.0 * n * hq * d}
    n = int(_new_tokens(case).sum())
    moved = n * 2 * d * (hq + 2 * hkv) + n * 2 * d * hq        # activations read, rotated q written
    flops = n * (hq + hkv) * (3.0 * case["rot"] + (4.0 * d if case["norm"] else 0.0))
    if case["op"] == "norm_append":
        return {"bytes": moved + n * 4 * d * hkv, "flops": flops}
    return {"bytes": moved + 2 * n * row + n * 4 * d * hkv, "flops": flops + 4.0 * n * hkv * d}


def _complex_turn(x, weight, s):
    """Norm and rotation (by complex numbers) in 64 bits."""
    half = s["inv"].numel()
    y = x.double().clone()
    if weight is not None:
        y = y / torch.linalg.vector_norm(torch.cat([y / y.shape[-1] ** 0.5, torch.full_like(
            y[..., :1], EPS ** 0.5)], -1), dim=-1, keepdim=True) * weight.double()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                       s["pos"].double()[:, None] * s["inv"].double())[:, None]
    lo, hi = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if s["case"]["inter"] else \
        (slice(0, half), slice(half, 2 * half))
    z = torch.complex(y[..., lo], y[..., hi]) * turn
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _exact_decode(s):
    c = s["case"]
    g, hkv, d = c["hq"] // c["hkv"], c["hkv"], c["d"]
    values = torch.tensor([v / 2 for v in [0, 1, 2, 3, 4, 6, 8, 12, 0, -1, -2, -3, -4, -6, -8, -12]],
                          dtype=torch.float64, device="cuda")
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -torch.inf, dtype=torch.float64, device="cuda")
    merged, merged_lse = out[:, 0].clone(), lse[:, 0].clone()
    for b, n in enumerate(s["lengths"].tolist()):
        if n == 0:
            continue
        pages = s["table"][b, :-(-n // PAGE)].long()
        for h in range(hkv):
            kv = []
            for j in (h, hkv + h):
                codes = s["pool"][pages, j].view(-1, d // 2)[:n].long()
                x = torch.empty(n, d, dtype=torch.float64, device="cuda")
                x[:, 0::2], x[:, 1::2] = values[codes % 16], values[codes // 16]
                e = s["scales"][pages, j].view(-1, d // GROUP)[:n].double() - 127
                kv.append(x * torch.pow(2.0, e).repeat_interleave(GROUP, 1))
            heads = slice(h * g, (h + 1) * g)
            x = s["q"][b, heads].double() @ kv[0].T * s["scale"]
            parts = [(x, kv[1], merged, merged_lse, (b, heads))]
            for t, (lo, hi) in enumerate(s["tiles"][b].tolist()):
                if hi > lo:
                    parts.append((x[:, lo:hi], kv[1][lo:hi], out, lse, (b, t, heads)))
            for y, v, o, l, at in parts:
                l[at] = y.logsumexp(1)
                o[at] = y.softmax(1) @ v
    return {"out": out, "lse": lse, "merged": merged, "merged_lse": merged_lse}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "decode_q4":
        return _exact_decode(s)
    n, hkv, d = s["n"], case["hkv"], case["d"]
    q = s["q_out"].double()
    q[:n] = _complex_turn(s["q"][:n], s["q_weight"], s)
    if case["op"] == "norm_append":
        pool = s["pool"].double().view(-1, 2 * hkv, d)
        at = s["table"].long()[s["of"], s["pos"] // PAGE] * PAGE + s["pos"] % PAGE
        pool[at, :hkv] = _complex_turn(s["k"][:n], s["k_weight"], s)
        pool[at, hkv:] = s["v"][:n].double()
        return {"q": q, "pool": pool.view(s["pool"].shape)}
    # A rounding to 4 bits turns one way or the other where a rotated value
    # meets a border between two codes, so the keys have no such value; the
    # values, which are not rotated, are the nearest codes exactly.
    x = s["v"][:n].double().view(n, hkv, -1, GROUP)
    scale = torch.ceil(torch.log2(x.abs().amax(-1, keepdim=True) / 6).clamp(min=MIN_EXP)).exp2()
    y = x / scale
    step = torch.floor(torch.log2(y.abs()).clamp(0.0, 2.0)).exp2() / 2     # of the code's octave
    y = torch.round(y / step) * step * scale
    return {"q": q, "k": None, "v": y.view(n, hkv * d)}
