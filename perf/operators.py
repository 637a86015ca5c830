"""The full-rank cache held in 8 bits: writing it, reading it back, and attention over it.

A block is 64 tokens of one sequence, KV head and side (keys or values).  It
is quantised once, when its last token arrives: with a = max(max |x|, 2^-100)
and M = 127 (int8) or 448 (e4m3), the codes are M x / a rounded half to even
(to whole numbers, or to e4m3) and a code stands for code * (a / M).  Tokens
of an unfinished block stay as they came, in bf16.

Query i of a sequence of L tokens with n queries stands at position L - n + i
and sees the keys up to there; a query that sees none gives 0.
"""
import math

import torch

own = False

D = 128
BLOCK = 64
TOP = {"int8": 127.0, "e4m3": 448.0}
LEAST = 2.0 ** -100
SCALE = 1.0 / math.sqrt(D)


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one generated token per sequence enters an 8K cache: pure latency
        dict(name="write_token", kind="write", code="int8", B=4, H=8, L=8191, n=1, ragged=True,
             wide=True),
        # a ragged batch of follow-up turns lands in the middle of blocks
        dict(name="write_turns", kind="write", code="e4m3", B=8, H=8, L=4001, n=517, ragged=True,
             wide=True),
        # the prompts of the 32K Llama-shaped layer enter an empty cache
        dict(name="write_prompts_32k", kind="write", code="int8", B=4, H=8, L=0, n=32768,
             ragged=False, wide=False),
        # the end of each sequence is looked at again, exactly
        dict(name="read_recent", kind="read", code="int8", B=2, H=2, L=511, n=129, ragged=True,
             wide=True),
        # the whole 8K cache of the Qwen3-shaped layer is handed to a bf16 consumer
        dict(name="read_all_8k", kind="read", code="e4m3", B=4, H=8, L=8192, n=8192, ragged=False,
             wide=False),
        # one token of a short chat: the call's fixed costs
        dict(name="attend_token_512", kind="attend", code="int8", B=2, H=2, G=4, L=511, n=1,
             ragged=True, token_major=False),
        # one token of the 8K Qwen3-shaped layer
        dict(name="attend_token_8k", kind="attend", code="e4m3", B=4, H=8, G=2, L=8192, n=1,
             ragged=False, token_major=False),
        # one token of the 32K Llama-shaped layer
        dict(name="attend_token_32k", kind="attend", code="int8", B=4, H=8, G=4, L=32769, n=1,
             ragged=False, token_major=False),
        # one token of a full serving batch of unequal lengths
        dict(name="attend_token_batch", kind="attend", code="int8", B=64, H=8, G=2, L=16384, n=1,
             ragged=True, token_major=False),
        # drafted tokens are verified in one call
        dict(name="attend_drafted", kind="attend", code="e4m3", B=8, H=8, G=4, L=16385, n=4,
             ragged=True, token_major=True),
        # a chunk of a long prompt attends to what came before it
        dict(name="attend_chunk", kind="attend", code="int8", B=2, H=8, G=4, L=16384, n=2048,
             ragged=False, token_major=True),
        # a whole prompt at once
        dict(name="attend_prompt_8k", kind="attend", code="e4m3", B=1, H=8, G=4, L=8192, n=8192,
             ragged=False, token_major=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["write", "read", "attend", "attend"])
    case = dict(kind=kind, code=rng.choice(["int8", "e4m3"]), ragged=rng.random() < 0.5)
    H = rng.choice([1, 2, 3, 4, 8])
    if kind == "write":
        n = rng.choice([1, 2, _log(rng, 3, 64), _log(rng, 65, 32768), _log(rng, 65, 32768)])
        L = rng.choice([0, _log(rng, 1, 8192)])
        B = max(1, min(_log(rng, 1, 64), 4 * 8 * 32768 // (H * (n + L))))
        case.update(B=B, H=H, L=L, n=n, wide=rng.random() < 0.5)
    elif kind == "read":
        L = _log(rng, 64, 32768)
        n = rng.choice([L, _log(rng, 1, L)])
        B = max(1, min(_log(rng, 1, 32), 4 * 8 * 8192 // (H * L)))
        case.update(B=B, H=H, L=L, n=n, wide=rng.random() < 0.5)
    else:
        G = rng.choice([1, 2, 4, 5, 8])
        L = _log(rng, 1, 32768)
        n = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 16, 8192)])
        n = min(n, L)
        # no more keys than the largest listed batch, nor more products than the listed prompt
        B = min(_log(rng, 1, 64), 64 * 8 * 12288 // (H * L), 8 * 4 * 4096 * 8192 // (H * G * n * L))
        while B < 1:  # one sequence alone is too much work: fewer queries
            n = max(1, n // 2)
            B = min(1, 8 * 4 * 4096 * 8192 // (H * G * n * L))
        case.update(B=B, H=H, G=G, L=L, n=n, token_major=rng.random() < 0.5)
    return case


def _spread(B, top, ragged, low=0.5):
    """B whole numbers between low * top and top (all top when not ragged)."""
    if not ragged:
        return [top] * B
    return [max(0, int(round(top * (1 - (1 - low) * ((b * 0.6180339887498949) % 1.0)))))
            for b in range(B)]


def _lengths(case):
    """Tokens of each sequence before the call, and its tokens in the call."""
    had = _spread(case["B"], case["L"], case["ragged"])
    n = _spread(case["B"], case["n"], case["ragged"] and case["kind"] != "read")
    if case["kind"] != "write":
        n = [min(x, y) for x, y in zip(n, had)]
    return had, n


# ------------------------------------------------------------------ inputs

def _rows(B, H, n, gen):
    """Rows as models make them: every head has a few channels that are larger."""
    x = torch.randn(B, H, n, D, generator=gen, device="cuda")
    gain = torch.exp(0.4 * torch.randn(1, H, 1, D, generator=gen, device="cuda"))
    return (x * gain).to(torch.bfloat16)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    had, n = _lengths(case)
    B, H, kind = case["B"], case["H"], case["kind"]
    most = max(h + (m if kind == "write" else 0) for h, m in zip(had, n))
    s = dict(kind=kind, code=case["code"], B=B, H=H, most=most, had=_ints(had), n=_ints(n),
             n_most=max(n), dtype=torch.float32 if case.get("wide") else torch.bfloat16)
    # what the cache was written from
    k, v = _rows(B, H, max(max(had), 1), gen), _rows(B, H, max(max(had), 1), gen)
    if kind == "write":
        s["new_k"], s["new_v"] = _rows(B, H, max(n), gen), _rows(B, H, max(n), gen)
    elif kind == "attend":
        G = case["G"]
        q = torch.randn(B, max(n), H * G, D, generator=gen, device="cuda").to(torch.bfloat16)
        s["q"] = q.transpose(1, 2) if case["token_major"] else q.transpose(1, 2).contiguous()
        s["o"] = torch.zeros_like(s["q"])
        s["G"] = G
    if kind != "attend":
        # the call reads back from the first block that it wrote, or the last n tokens
        first = [h // BLOCK * BLOCK if kind == "write" else h - m for h, m in zip(had, n)]
        s["first"] = _ints(first)
        s["n_read"] = max(h + m - f if kind == "write" else m for h, m, f in zip(had, n, first))
        shape = (B, H, s["n_read"], D)
        s["out_k"] = torch.zeros(shape, dtype=s["dtype"], device="cuda")
        s["out_v"] = torch.zeros(shape, dtype=s["dtype"], device="cuda")
    if own:
        from rank_kv_cache_lrkv_b200 import lrkv
        s["cache"] = lrkv.QuantCache(B, H, max(most, 1), code=case["code"])
        if max(had):
            lrkv.quant_append(s["cache"], k, v, n_new=s["had"])
        # a cache can be taken back by up to a block; further back its open rows go too
        s["tail"] = s["cache"].tail.clone() if kind == "write" and max(n) > BLOCK else None
        if kind == "attend":
            s["ws"] = lrkv.quant_attn_workspace(s["cache"], H * case["G"], max(n))
    else:
        # blocks up to the one that the next token goes to
        pad = (most // BLOCK + 1) * BLOCK
        for name, x in (("k", k), ("v", v)):
            x = torch.nn.functional.pad(x, (0, 0, 0, max(0, pad - x.shape[2])))[:, :, :pad]
            codes, scales = _quantise(x, case["code"])
            s[name] = dict(codes=codes, scales=scales, open=_open_block(x, s["had"]))
    return s


# ------------------------------------------------------------- plain forms

def _quantise(x, code):
    """Codes [B, H, blocks, 64, D] and scales [B, H, blocks] of whole blocks."""
    x = x.float().unflatten(2, (-1, BLOCK))
    top = x.abs().amax((3, 4)).clamp_min(LEAST)
    y = x * TOP[code] / top[..., None, None]
    y = y.round().to(torch.int8) if code == "int8" else y.to(torch.float8_e4m3fn)
    return y, top / TOP[code]


def _places(length, most):
    """Positions [B, 64] of the block that each sequence's next token goes to."""
    start = (length.long() // BLOCK * BLOCK).clamp_max(most - BLOCK)
    return start[:, None] + torch.arange(BLOCK, device=length.device)


def _open_block(x, length):
    b = torch.arange(x.shape[0], device=x.device)[:, None]
    return x[b, :, _places(length, x.shape[2])]  # [B, 64, H, D]


def _values(side, length):
    """What the cache holds: [B, H, tokens, D] in 32 bits."""
    y = side["codes"].float() * side["scales"][..., None, None]
    y = y.flatten(2, 3)
    b = torch.arange(y.shape[0], device=y.device)[:, None]
    y[b, :, _places(length, y.shape[2])] = side["open"].float()
    return y


def _plain_write(s):
    had, new = s["had"].long(), s["n"].long()
    length = had + new
    out = []
    for side, rows in ((s["k"], s["new_k"]), (s["v"], s["new_v"])):
        # the rows of the blocks from the one that was open: its rows, then the new ones
        at = had % BLOCK
        t = torch.arange((s["n_most"] + BLOCK) // BLOCK * BLOCK + BLOCK, device="cuda") - at[:, None]
        b = torch.arange(s["B"], device="cuda")[:, None]
        x = rows.float()[b, :, t.clamp(0, s["n_most"] - 1)]
        x = torch.where((t < new[:, None])[..., None, None], x, 0.0)
        old = torch.arange(BLOCK, device="cuda") < at[:, None]
        x[:, :BLOCK] = torch.where(old[..., None, None], side["open"].float(), x[:, :BLOCK])
        x = x.transpose(1, 2)
        codes, scales = _quantise(x, s["code"])
        y = (codes.float() * scales[..., None, None]).flatten(2, 3)
        # the block that is not full yet stays as it came
        full = (length - length % BLOCK) - (had - at)
        whole = torch.arange(x.shape[2], device="cuda") < full[:, None]
        y = torch.where(whole[:, None, :, None], y, x)[:, :, :s["n_read"]]
        seen = torch.arange(s["n_read"], device="cuda") < (length - s["first"])[:, None]
        out.append(torch.where(seen[:, None, :, None], y, 0.0).to(s["dtype"]))
    return {"k": out[0], "v": out[1], "length": length.to(torch.int32)}


def _plain_read(s):
    t = s["first"].long()[:, None] + torch.arange(s["n_read"], device="cuda")
    b = torch.arange(s["B"], device="cuda")[:, None]
    seen = (t < s["had"][:, None]) & (t >= 0)
    out = []
    for name in ("k", "v"):
        y = _values(s[name], s["had"])
        y = y[b, :, t.clamp(0, y.shape[2] - 1)]
        out.append(torch.where(seen[..., None, None], y, 0.0).transpose(1, 2).to(s["dtype"]))
    return {"k": out[0], "v": out[1]}


def _plain_attend(s):
    k, v = _values(s["k"], s["had"]), _values(s["v"], s["had"])
    B, H, G, n = s["B"], s["H"], s["G"], s["n_most"]
    q = s["q"].float().reshape(B, H, G * n, D)
    x = (q @ k.transpose(2, 3)).mul_(SCALE).view(B, H, G, n, -1)
    i = torch.arange(n, device="cuda")
    at = s["had"].long()[:, None] - s["n"].long()[:, None] + i
    seen = torch.arange(k.shape[2], device="cuda") <= at[..., None]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.view(B, H, G * n, -1) @ v).view(B, H, G, n, D) / torch.where(total == 0, 1.0, total)
    asked = i < s["n"][:, None]
    return torch.where(asked[:, None, None, :, None], o, 0.0).view(B, H * G, n, D).to(torch.bfloat16)


def _own(s):
    from rank_kv_cache_lrkv_b200 import lrkv
    c = s["cache"]
    if s["kind"] == "write":
        c.seq_len.copy_(s["had"])  # the pass before is taken back
        if s["tail"] is not None:
            c.tail.copy_(s["tail"])
        lrkv.quant_append(c, s["new_k"], s["new_v"], n_new=s["n"])
    if s["kind"] == "attend":
        return lrkv.quant_attn(c, s["q"], SCALE, s["o"], s["ws"], n_q=s["n"])
    k, v = lrkv.quant_read(c, s["out_k"], s["out_v"], first=s["first"])
    return {"k": k, "v": v, "length": c.seq_len} if s["kind"] == "write" else {"k": k, "v": v}


def run(state):
    if own:
        return _own(state)
    return {"write": _plain_write, "read": _plain_read, "attend": _plain_attend}[state["kind"]](state)


# ------------------------------------------------------------ what it costs

def work(case):
    had, n = _lengths(case)
    H, row = case["H"], 2 * D  # one byte for each element of a token's key and value
    if case["kind"] == "write":
        wide = 4 if case["wide"] else 2
        byte = flop = 0
        for h, m in zip(had, n):
            a, z = h // BLOCK * BLOCK, h + m
            full = z // BLOCK * BLOCK
            # the new rows, the open block's rows, the codes, the rows that stay open; read back
            byte += H * row * (2 * m + (2 * (h - a) if full > a else 0) + 2 * (full - a)
                               + 2 * 2 * (z - max(full, h)) + wide * (z - a))
            flop += H * row * 4 * (full - a)
        return {"bytes": byte, "flops": flop}
    if case["kind"] == "read":
        wide = 4 if case["wide"] else 2
        byte = sum(H * row * m * (1 + wide) for m in n)
        return {"bytes": byte, "flops": sum(H * row * m for m in n)}
    G = case["G"]
    byte = flop = 0
    for h, m in zip(had, n):
        byte += H * row * (h + h % BLOCK) + H * G * m * 2 * D * 2
        seen = sum(range(h - m + 1, h + 1))
        flop += 4 * D * H * G * seen
    return {"bytes": byte, "flops": flop}


# ------------------------------------------------------- the definition, 64

def _stored64(x, length, code):
    """Values in 64 bits of one head's rows x [tokens, D] in a cache of `length`."""
    x = x.double()
    full = length // BLOCK * BLOCK
    y = x[:length].clone()
    if full:
        blocks = y[:full].reshape(-1, BLOCK * D)
        a = torch.maximum(blocks.abs().max(1).values, torch.tensor(LEAST, device=x.device, dtype=x.dtype))
        z = blocks * TOP[code] / a[:, None]
        if code == "int8":
            z = torch.round(z)
        else:
            # e4m3: steps of 2^(e - 3) with e the exponent, at least -6
            e = torch.floor(torch.log2(z.abs().clamp_min(2.0 ** -6)))
            e = torch.where(torch.exp2(e) > z.abs().clamp_min(2.0 ** -6), e - 1, e)
            step = torch.exp2(e - 3)
            z = torch.round(z / step) * step
        y[:full] = (z * (a[:, None] / TOP[code])).reshape(full, D)
    return y


def exact(case, seed):
    global own
    mine, own = own, False
    try:
        gen = torch.Generator(device="cuda").manual_seed(seed)
        had, n = _lengths(case)
        B, H, kind, code = case["B"], case["H"], case["kind"], case["code"]
        rows = max(max(had), 1)
        k, v = _rows(B, H, rows, gen), _rows(B, H, rows, gen)
        if kind == "write":
            nk, nv = _rows(B, H, max(n), gen), _rows(B, H, max(n), gen)
            first = [h // BLOCK * BLOCK for h in had]
            most = max(h + m - f for h, m, f in zip(had, n, first))
            out = torch.zeros(2, B, H, most, D, dtype=torch.float64, device="cuda")
            for b in range(B):
                for h in range(H):
                    for i, (old, new) in enumerate(((k, nk), (v, nv))):
                        x = torch.cat([old[b, h, :had[b]], new[b, h, :n[b]]])
                        # whole blocks before the first are not asked for
                        y = _stored64(x[first[b]:], had[b] + n[b] - first[b], code)
                        out[i, b, h, :y.shape[0]] = y
            return {"k": out[0], "v": out[1], "length": None}
        if kind == "read":
            out = torch.zeros(2, B, H, max(n), D, dtype=torch.float64, device="cuda")
            for b in range(B):
                for h in range(H):
                    for i, x in enumerate((k, v)):
                        out[i, b, h, :n[b]] = _stored64(x[b, h], had[b], code)[had[b] - n[b]:]
            return {"k": out[0], "v": out[1]}
        G, m = case["G"], max(n)
        q = torch.randn(B, m, H * G, D, generator=gen, device="cuda").to(torch.bfloat16)
        o = torch.zeros(B, H * G, m, D, dtype=torch.float64, device="cuda")
        for b in range(B):
            for h in range(H):
                kb, vb = _stored64(k[b, h], had[b], code), _stored64(v[b, h], had[b], code)
                for g in range(h * G, h * G + G):
                    for i in range(0, n[b], 2048):
                        j = min(n[b], i + 2048)
                        x = q[b, i:j, g].double() @ kb.T * SCALE
                        at = had[b] - n[b] + torch.arange(i, j, device="cuda")
                        x[torch.arange(had[b], device="cuda") > at[:, None]] = -math.inf
                        o[b, g, i:j] = torch.softmax(x, 1) @ vb
        return o
    finally:
        own = mine
