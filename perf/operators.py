"""The rotated appends and the 8-bit paged cache, as measured cases.

Three operators, each in its plain form (elementary torch operations) and as
the framework's own calls:

  append     rotate a step's q and k by their positions and store k and v in a
             bf16 paged cache
  append_q8  the same into a cache held in 8 bits (e4m3 codes, one fp32 scale
             for each 16 tokens and head), and the touched blocks read back as
             the values they stand for
  decode_q8  grouped-query decode attention over that cache, per tile of the
             history (normalised output and log-sum-exp) and merged
"""

import torch

own = False

PAGE = 64          # tokens per page
BLOCK = 16         # tokens per scale of the 8-bit cache
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # One sequence, one new token: the smallest append of a decode step.
        dict(name="append 1 token", op="append", batch=1, new_lo=1, new_hi=1, past_lo=31743,
             past_hi=31743, pad=0, hq=24, hkv=4, d=256, rot=256, inter=False, shape=1),
        # A decode step of a served batch, one new token each, odd batch size.
        dict(name="append 61 tokens", op="append", batch=61, new_lo=1, new_hi=1, past_lo=5,
             past_hi=9000, pad=0, hq=32, hkv=8, d=128, rot=128, inter=False, shape=2),
        # Prompts of very different lengths packed one after another, half of
        # each head rotated in adjacent pairs, padding rows behind the last one.
        dict(name="append 11 ragged prompts", op="append", batch=11, new_lo=0, new_hi=2500,
             past_lo=0, past_hi=4000, pad=37, hq=32, hkv=8, d=128, rot=64, inter=True, shape=3),
        # One new token of one far sequence into the 8-bit cache.
        dict(name="append_q8 1 token", op="append_q8", batch=1, new_lo=1, new_hi=1,
             past_lo=200005, past_hi=200005, pad=0, hq=24, hkv=4, d=256, rot=256, inter=False,
             shape=4),
        # A decode step of a served batch into the 8-bit cache.
        dict(name="append_q8 64 tokens", op="append_q8", batch=64, new_lo=1, new_hi=1, past_lo=0,
             past_hi=9000, pad=0, hq=24, hkv=4, d=256, rot=64, inter=False, shape=5),
        # A few proposed tokens for each of a batch, ending inside blocks.
        dict(name="append_q8 23x1-7 tokens", op="append_q8", batch=23, new_lo=1, new_hi=7,
             past_lo=0, past_hi=5000, pad=9, hq=32, hkv=8, d=128, rot=128, inter=True, shape=6),
        # A prompt chunk into the 8-bit cache.
        dict(name="append_q8 2 prompts", op="append_q8", batch=2, new_lo=3900, new_hi=4200,
             past_lo=0, past_hi=1000, pad=0, hq=24, hkv=4, d=256, rot=256, inter=False, shape=7),
        # One short sequence: a single decode launch where latency counts.
        dict(name="decode_q8 1x700", op="decode_q8", batch=1, len_lo=700, len_hi=700, tile=32768,
             hq=24, hkv=4, d=256, shape=8),
        # A served batch of chat-length sequences.
        dict(name="decode_q8 64 to 2500", op="decode_q8", batch=64, len_lo=1, len_hi=2500,
             tile=32768, hq=32, hkv=8, d=128, shape=9),
        # The repository's bench shape: 4 sequences of 31,744 tokens.
        dict(name="decode_q8 4x31744", op="decode_q8", batch=4, len_lo=31744, len_hi=31744,
             tile=32768, hq=24, hkv=4, d=256, shape=10),
        # Ragged long sequences in tiles, some of them empty for the short ones.
        dict(name="decode_q8 7 ragged", op="decode_q8", batch=7, len_lo=900, len_hi=40000,
             tile=9000, hq=16, hkv=2, d=128, shape=11),
        # The repository's long-context shape: 262,144 tokens in 8 tiles.
        dict(name="decode_q8 1x262144", op="decode_q8", batch=1, len_lo=262144, len_hi=262144,
             tile=32768, hq=24, hkv=4, d=256, shape=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["append", "append_q8", "decode_q8"])
    hq, hkv, d = rng.choice([(24, 4, 256), (32, 8, 128), (16, 2, 128), (8, 8, 256), (7, 1, 256),
                             (20, 5, 128), (32, 4, 128)])
    shape = rng.randrange(1 << 20)
    if op == "decode_q8":
        batch = _log_int(rng, 1, 64)
        most = min(250000, (1 << 28) // (hkv * d)) // batch
        top = _log_int(rng, 64, max(64, most))
        return dict(op=op, batch=batch, len_lo=int(top * rng.choice([0.0, 0.02, 0.3, 1.0])),
                    len_hi=top, tile=_log_int(rng, max(64, top // 8), 32768 + top), hq=hq, hkv=hkv,
                    d=d, shape=shape)
    batch = _log_int(rng, 1, 100)
    top = _log_int(rng, 1, max(1, 8000 // batch))
    return dict(op=op, batch=batch, new_lo=rng.choice([0, 1, top]), new_hi=top, past_lo=0,
                past_hi=_log_int(rng, 16, 200000 // batch), pad=rng.choice([0, 0, 5]), hq=hq,
                hkv=hkv, d=d, rot=rng.choice([d, d, d // 2, d // 4 + 8]),
                inter=rng.random() < 0.4, shape=shape)


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
    used = (ends - first).clamp(min=0)
    n = int(used.sum())
    perm = torch.randperm(n + 2, generator=gen, device=dev).int()
    table = torch.zeros(len(lengths), width, dtype=torch.int32, device=dev)
    at = torch.arange(width)[None]
    mask = (at >= first[:, None]) & (at < ends[:, None])
    table[mask.to(dev)] = perm[:n]
    return table, n + 2


def _values(n, h, d, gen, dev, spread=None):
    """bf16 activations as projections give them: unit variance, with channels
    of a larger scale where `spread` is given."""
    x = torch.randn(n, h, d, generator=gen, device=dev)
    return (x if spread is None else x * spread).bfloat16()


def _spread(h, d, gen, dev):
    return torch.exp(0.5 * torch.randn(h, d, generator=gen, device=dev))


def _filled(pages, hkv, d, gen, dev):
    """A cache in 8 bits whose every block is full: codes and scales."""
    pool = torch.empty(pages, PAGE, 2 * hkv * d, dtype=torch.uint8, device=dev)
    scales = torch.empty(pages, 2 * hkv, PAGE // BLOCK, device=dev)
    spread = torch.cat([_spread(hkv, d, gen, dev), torch.ones(hkv, d, device=dev)])
    step = max(1, (1 << 26) // (PAGE * 2 * hkv * d))
    for p0 in range(0, pages, step):
        n = min(step, pages - p0)
        x = torch.randn(n, PAGE // BLOCK, BLOCK, 2 * hkv, d, generator=gen, device=dev) * spread
        s = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 4)) / E4M3_MAX)))
        pool[p0:p0 + n] = (x / s[:, :, None, :, None]).to(E4M3).view(torch.uint8).reshape(n, PAGE, -1)
        scales[p0:p0 + n] = s.transpose(1, 2)
    return pool.view(E4M3), scales


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "decode_q8":
        lengths = _lengths(case)
        table, pages = _tables(lengths, torch.zeros_like(lengths), gen, dev)
        pool, scales = _filled(pages, hkv, d, gen, dev)
        # the rows behind each sequence's last token hold what an earlier
        # user of the page left there, NaN codes among it
        some = lengths[lengths > 0]
        last = table[(lengths > 0).to(dev)]
        last = last[torch.arange(len(some)), ((some - 1) // PAGE).to(dev)].long()
        rows = torch.arange(PAGE, device=dev)[None] > ((some - 1) % PAGE).to(dev)[:, None]
        raw = pool.view(torch.uint8)
        tail = raw[last]
        tail[rows] = 0x7F
        raw[last] = tail
        n_tiles = max(1, -(-int(lengths.max()) // case["tile"]))
        start = torch.arange(n_tiles)[None] * case["tile"]
        tiles = torch.stack([torch.minimum(start, lengths[:, None]),
                             torch.minimum(start + case["tile"], lengths[:, None])], -1).int()
        state = dict(case=case, q=_values(case["batch"], hq, d, gen, dev), pool=pool, scales=scales,
                     table=table, tiles=tiles.numpy(), tiles_dev=tiles.to(dev),
                     lengths=lengths.to(dev), scale=d ** -0.5,
                     out=torch.empty(case["batch"], n_tiles, hq, d, device=dev),
                     lse=torch.empty(case["batch"], n_tiles, hq, device=dev),
                     merged=torch.empty(case["batch"], hq, d, device=dev),
                     merged_lse=torch.empty(case["batch"], hq, device=dev))
        if own:   # zero-filled once, kept by the program for every call
            from paged_decode_attention_attn_gb300 import binding as B
            state["workspace"] = B.alloc_workspace_q8(case["batch"], n_tiles, hq, hkv, d)
        return state
    new, past = _new_tokens(case), _past_tokens(case)
    ends = past + new
    # the pages that hold the touched blocks; a program's pool holds the rest too
    table, pages = _tables(torch.where(new > 0, ends, torch.zeros_like(ends)), past // PAGE, gen, dev)
    cu = torch.zeros(case["batch"] + 1, dtype=torch.int64)
    cu[1:] = new.cumsum(0)
    n = int(cu[-1]) + case["pad"]
    qkv = torch.cat([_values(n, hq, d, gen, dev), _values(n, hkv, d, gen, dev, _spread(hkv, d, gen, dev)),
                     _values(n, hkv, d, gen, dev)], 1)     # one projection's output
    of = torch.repeat_interleave(torch.arange(case["batch"]), new)
    pos = past[of] + torch.arange(int(cu[-1])) - cu[of]
    half = case["rot"] // 2
    inv = (1.0 / 10000.0 ** (torch.arange(half, dtype=torch.float64) / half)).float().to(dev)
    state = dict(case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], table=table,
                 positions=past.int().to(dev), cu=cu.int().to(dev), one_each=bool((new == 1).all())
                 and case["pad"] == 0, inv=inv, n=int(cu[-1]), of=of.to(dev), pos=pos.to(dev),
                 q_out=torch.zeros(n, hq, d, dtype=torch.bfloat16, device=dev))
    if case["op"] == "append":
        state["pool"] = _values(pages * PAGE, 2 * hkv, d, gen, dev).view(pages, PAGE, 2 * hkv * d)
        return state
    state["pool"], state["scales"] = _filled(pages, hkv, d, gen, dev)
    # what is read back: each sequence's new tokens and the older rows of the
    # block that its first one falls in
    first = past // BLOCK * BLOCK
    back = torch.where(new > 0, ends - first, torch.zeros_like(new))
    back_cu = torch.zeros(case["batch"] + 1, dtype=torch.int64)
    back_cu[1:] = back.cumsum(0)
    back_of = torch.repeat_interleave(torch.arange(case["batch"]), back)
    back_pos = first[back_of] + torch.arange(int(back_cu[-1])) - back_cu[back_of]
    state.update(first=first.int().to(dev), back_cu=back_cu.int().to(dev), back_of=back_of.to(dev),
                 back_pos=back_pos.to(dev),
                 back=torch.zeros(int(back_cu[-1]), 2 * hkv * d, dtype=torch.bfloat16, device=dev))
    return state


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _rotated(x, pos, inv, inter):
    """x [n, h, d] turned by its positions; angles in 64 bits, the rest in 32."""
    half = inv.numel()
    angle = pos.double()[:, None] * inv.double()[None]
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = x.float()
    r = x[..., :2 * half]
    if inter:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y, x[..., 2 * half:]], -1)


def _rows(table, of, pos):
    """Row of the pool that holds token `pos` of sequence `of`."""
    return table[of, torch.div(pos, PAGE, rounding_mode="floor")].long() * PAGE + pos % PAGE


def _plain_append(s):
    n, inter = s["n"], s["case"]["inter"]
    s["q_out"][:n] = _rotated(s["q"][:n], s["pos"], s["inv"], inter).bfloat16()
    k = _rotated(s["k"][:n], s["pos"], s["inv"], inter).bfloat16()
    rows = _rows(s["table"], s["of"], s["pos"])
    s["pool"].view(-1, s["pool"].shape[-1])[rows] = torch.cat([k, s["v"][:n]], 1).flatten(1)
    return {"q": s["q_out"], "pool": s["pool"]}


def _plain_append_q8(s):
    c, n = s["case"], s["n"]
    heads, d = 2 * c["hkv"], c["d"]
    s["q_out"][:n] = _rotated(s["q"][:n], s["pos"], s["inv"], c["inter"]).bfloat16()
    x = torch.cat([_rotated(s["k"][:n], s["pos"], s["inv"], c["inter"]), s["v"][:n].float()], 1)
    raw = s["pool"].view(torch.uint8).view(-1, BLOCK, heads, d)          # a block a row
    scales = s["scales"].transpose(1, 2).reshape(-1, heads)              # [block][head]
    rows = _rows(s["table"], s["of"], s["pos"])
    blocks, at = torch.unique(rows // BLOCK, return_inverse=True)
    first = torch.full((blocks.numel(),), BLOCK, device=x.device)
    first = first.scatter_reduce(0, at, rows % BLOCK, "amin")            # older rows of each block
    amax = torch.zeros(blocks.numel(), heads, device=x.device)
    amax = amax.scatter_reduce(0, at[:, None].expand(-1, heads), x.abs().amax(-1), "amax")
    mant, expo = torch.frexp(amax)                                       # amax = mant 2^expo, 448 = 0.875 2^9
    need = torch.exp2((expo - 9 + (mant > 0.875)).float().clamp(min=-60.0))
    need = torch.where(amax > 0, need, torch.full_like(need, 2.0 ** -60))
    old = scales[blocks]
    new = torch.where((first > 0)[:, None], torch.maximum(old, need), need)
    kept = raw[blocks].view(E4M3).float() * (old / new)[:, None, :, None]
    kept = kept.to(E4M3).view(torch.uint8)
    older = torch.arange(BLOCK, device=x.device)[None] < first[:, None]
    raw[blocks] = torch.where(older[..., None, None], kept, raw[blocks])
    raw.view(-1, heads, d)[rows] = (x / new[at][..., None]).to(E4M3).view(torch.uint8)
    scales[blocks] = new
    s["scales"].copy_(scales.view(-1, PAGE // BLOCK, heads).transpose(1, 2))
    rows = _rows(s["table"], s["back_of"], s["back_pos"])
    back = raw.view(-1, heads, d)[rows].view(E4M3).float() * scales[rows // BLOCK][..., None]
    s["back"].copy_(back.flatten(1))
    return _append_q8_outputs(s)


def _append_q8_outputs(s):
    kd = s["case"]["hkv"] * s["case"]["d"]
    return {"q": s["q_out"], "k": s["back"][:, :kd], "v": s["back"][:, kd:]}


def _plain_decode_q8(s):
    c = s["case"]
    b, hq, hkv, d = c["batch"], c["hq"], c["hkv"], c["d"]
    table = s["table"].long()
    x = s["pool"].view(torch.uint8)[table].view(E4M3).view(b, -1, PAGE // BLOCK, BLOCK, 2 * hkv, d).float()
    x = x * s["scales"][table].transpose(2, 3)[:, :, :, None, :, None]
    x = x.reshape(b, -1, 2 * hkv, d)                                     # [b][token][head][d]
    at = torch.arange(x.shape[1], device=x.device)
    k = x[:, :, :hkv].permute(0, 2, 3, 1)
    v = x[:, :, hkv:].permute(0, 2, 1, 3)
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
    op, c = state["case"]["op"], state["case"]
    if not own:
        return {"append": _plain_append, "append_q8": _plain_append_q8,
                "decode_q8": _plain_decode_q8}[op](state)
    from paged_decode_attention_attn_gb300 import binding as B
    s = state
    if op == "decode_q8":
        B.paged_decode_attn_q8_lse(s["q"], s["pool"], s["scales"], s["table"], s["tiles"], s["scale"],
                                   s["out"], s["lse"], s["workspace"], merged_out=s["merged"],
                                   merged_lse=s["merged_lse"])
        return {"out": s["out"], "lse": s["lse"], "merged": s["merged"], "merged_lse": s["merged_lse"]}
    cu = None if s["one_each"] else s["cu"]
    if op == "append":
        B.kv_append_rope(s["q"], s["k"], s["v"], s["pool"], s["table"], s["positions"], s["inv"],
                         s["q_out"], cu_tokens=cu, interleaved=c["inter"])
        return {"q": s["q_out"], "pool": s["pool"]}
    B.kv_append_rope_q8(s["q"], s["k"], s["v"], s["pool"], s["scales"], s["table"], s["positions"],
                        s["inv"], s["q_out"], cu_tokens=cu, interleaved=c["inter"])
    B.kv_gather_q8(s["pool"], s["scales"], s["table"], s["first"], s["back_cu"], s["back"])
    return _append_q8_outputs(s)


# --------------------------------------------------------------------------
# the work of one pass, and its results in 64 bits
# --------------------------------------------------------------------------
def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "decode_q8":
        n = int(_lengths(case).sum())
        tiles = max(1, -(-int(_lengths(case).max()) // case["tile"]))
        rows = case["batch"] * hq
        return {"bytes": n * 2 * hkv * d + n // BLOCK * 2 * hkv * 4 + rows * d * 2
                + rows * (tiles + 1) * (d + 1) * 4, "flops": 4.0 * n * hq * d}
    new, past = _new_tokens(case), _past_tokens(case)
    n = int(new.sum())
    moved = n * 2 * d * (hq + 2 * hkv) + n * 2 * d * hq        # activations read, rotated q written
    flops = 3.0 * n * case["rot"] * (hq + hkv)
    if case["op"] == "append":
        return {"bytes": moved + n * 4 * d * hkv, "flops": flops}
    back = n + int((past % BLOCK)[new > 0].sum())
    blocks = int(((past + new - 1) // BLOCK - past // BLOCK + 1)[new > 0].sum())
    return {"bytes": moved + n * 2 * d * hkv + 2 * blocks * 2 * hkv * 4 + back * 2 * hkv * d * 3, "flops": flops}


def _turned(x, s):
    """Rotation by complex numbers in 64 bits."""
    half = s["inv"].numel()
    y = x.double().clone()
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
                codes = s["pool"].view(torch.uint8)[pages][:, :, j * d:(j + 1) * d].contiguous().view(E4M3)
                by = s["scales"][pages, j].double().repeat_interleave(BLOCK, 1)
                kv.append((codes.double() * by[..., None]).view(-1, d)[:n])
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
    if case["op"] == "decode_q8":
        return _exact_decode(s)
    n, hkv, d = s["n"], case["hkv"], case["d"]
    q = s["q_out"].double()
    q[:n] = _turned(s["q"][:n], s)
    if case["op"] == "append":
        pool = s["pool"].double().view(-1, 2 * hkv, d)
        at = (s["table"].long()[s["of"], s["pos"] // PAGE], s["pos"] % PAGE)
        at = at[0] * PAGE + at[1]
        pool[at, :hkv] = _turned(s["k"][:n], s)
        pool[at, hkv:] = s["v"][:n].double()
        return {"q": q, "pool": pool.view(s["pool"].shape)}
    # A rounding to 8 bits turns one way or the other where a rotated value
    # meets a border between two codes, so the keys have no such value; the
    # values, which are not rotated, are the nearest codes exactly.
    v = torch.zeros(s["back"].shape[0], hkv, d, dtype=torch.float64, device="cuda")
    cu, past = s["cu"].tolist(), s["positions"].tolist()
    back_cu, first = s["back_cu"].tolist(), s["first"].tolist()
    spans, edges = [], []
    for b in range(case["batch"]):
        if cu[b + 1] == cu[b]:
            continue
        for lo in range(first[b], past[b] + cu[b + 1] - cu[b], BLOCK):
            spans.append((b, lo))
            edges.append((max(lo, past[b]), min(lo + BLOCK, past[b] + cu[b + 1] - cu[b])))
    spans, edges = torch.tensor(spans, device="cuda"), torch.tensor(edges, device="cuda")
    b, lo = spans.T
    pages = s["table"].long()[b, lo // PAGE]
    tok = lo[:, None] + torch.arange(BLOCK, device="cuda")
    fresh = (tok >= edges[:, :1]) & (tok < edges[:, 1:])
    src = (s["cu"].long()[b] - s["positions"].long()[b])[:, None] + tok
    x = s["v"].double()[torch.where(fresh, src, torch.zeros_like(src))] * fresh[..., None, None]
    peak = x.abs().amax((1, 3))
    want = torch.ceil(torch.log2(peak / E4M3_MAX).clamp(min=-60.0)).exp2()
    had = s["scales"].double()[pages, hkv:, lo % PAGE // BLOCK]
    has = tok[:, 0] < edges[:, 0]
    scale = torch.where(has[:, None], torch.maximum(had, want), want)[:, None, :, None]
    codes = s["pool"].view(torch.uint8)[pages[:, None], tok % PAGE].view(-1, BLOCK, 2 * hkv, d)[:, :, hkv:]
    was = codes.contiguous().view(E4M3).double() * had[:, None, :, None]
    x = torch.where(fresh[..., None, None], x, was) / scale
    # nearest multiple of the code's step, ties to even
    step = torch.floor(torch.log2(x.abs()).clamp(min=-6.0)).exp2() / 8
    y = torch.round(x / step) * step * scale
    live = tok < edges[:, 1:]
    v[((torch.tensor(back_cu[:-1], device="cuda") - s["first"].long())[b][:, None] + tok)[live]] = y[live]
    return {"q": q, "k": None, "v": v.flatten(1)}
