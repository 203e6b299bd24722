"""Measured cases of the operators between a decoder layer's linear layers:

  norm       root-mean-square norm of the residual stream plus a layer's
             output, to fp16 or to 8 bits with scales
  rope       rotary positions of queries and keys: halves or neighbouring
             channels paired, part of the head, frequencies scaled for long
             contexts
  cache      quantizing new keys and values into a paged 4-bit cache, and
             reading the touched tokens back
  attention  softmax attention of a batch's newest tokens over that cache

`own` chooses between the plain torch form and this package's kernels.

The 4-bit cache (both forms use it): keys in groups of 32 channels of a token,
values in one group per token and head. A group holds its smallest number lo
and a step s, fp16 each, and codes 0 .. 15; the cached number is
fp16(lo + s * code). Page p, head h of k_codes is [D / 32][P][16] bytes (32
channels of a token adjacent) with k_scales [D / 32][P][2] (s, lo); v_codes is
[P / 32][D][16] (32 tokens of a channel adjacent) with v_scales [2][P] (every
token's s, then every lo). Eight codes fill four bytes, code 2 j in nibble j
and code 2 j + 1 in nibble j + 4. Sequence b holds kv_len[b] tokens, token j in
page block_table[b, j // P]; its newest cu[b + 1] - cu[b] tokens are rows
cu[b] .. of the batch's token tensors.
"""

import math

import torch

own = False

TOP = {"int8": 127.0, "e4m3": 448.0}
FLOOR = 1e-5            # smallest group maximum an 8-bit scale is taken from
EPS = 1e-5
NIBBLES = (0, 2, 4, 6, 1, 3, 5, 7)      # the code of each nibble of a word


def listed():
    return [
        # one decoded token: the attention's output joins the residual stream
        _norm("norm decode 1x4096 residual", 1, 4096, True, "fp16", 0),
        # a decode batch, into 8 bits with one scale a token
        _norm("norm batch 64x8192 residual e4m3", 64, 8192, True, "e4m3", 0),
        # a ragged prompt of an odd width, no residual
        _norm("norm ragged 777x5001", 777, 5001, False, "fp16", 0),
        # a long prompt
        _norm("norm prompt 4096x8192 residual", 4096, 8192, True, "fp16", 0),
        # one decoded token, every head its own keys
        _rope("rope decode 1 token 32 heads", 1, 32, 32, 128, 128, "half", "none", 4096, "positions"),
        # a serving batch at far positions, half of the head rotated, interleaved, scaled
        _rope("rope batch 64 tokens yarn", 64, 64, 8, 128, 64, "interleaved", "yarn", 131072, "batch"),
        # a long prompt with grouped heads
        _rope("rope prompt 8192 tokens", 8192, 32, 8, 128, 128, "half", "wavelength", 16384, "positions"),
        # one decode step of 64 sequences: append a token each
        _cache("cache4 append B=64 H=8", 64, 8, 128, 64, 4096, 1),
        # a long prompt's keys and values
        _cache("cache4 prompt B=4 H=32", 4, 32, 128, 64, 4096, 4096),
        # one decoded token of one short sequence, every head its own keys
        _attention("attention4 decode B=1 L=1000 MHA", 1, 32, 32, 128, 64, 1000, 1, True, 0),
        # a serving batch of ragged sequences with grouped heads
        _attention("attention4 decode B=64 L=8192", 64, 64, 8, 128, 64, 8192, 1, True, 0),
        # a prompt chunk of 2048 tokens behind 2048 cached ones
        _attention("attention4 prefill 2x2048 of 4096", 2, 32, 8, 128, 64, 4096, 2048, True, 0),
    ]


def _norm(name, tokens, width, residual, out, group):
    return {"name": name, "op": "norm", "tokens": tokens, "width": width, "residual": residual, "out": out,
            "group": group}


def _rope(name, tokens, q_heads, heads, dim, rotary, layout, scaling, far, by):
    """far: the trained length's bound; positions go up to it. by: positions
    given as a tensor, or taken from a batch of sequences of one token each."""
    return {"name": name, "op": "rope", "tokens": tokens, "q_heads": q_heads, "heads": heads, "dim": dim,
            "rotary": rotary, "layout": layout, "scaling": scaling, "far": far, "by": by}


def _cache(name, seqs, heads, dim, page, length, new):
    return {"name": name, "op": "cache", "seqs": seqs, "heads": heads, "dim": dim, "page": page, "length": length,
            "new": new}


def _attention(name, seqs, q_heads, heads, dim, page, length, new, causal, window):
    return {"name": name, "op": "attention", "seqs": seqs, "q_heads": q_heads, "heads": heads, "dim": dim,
            "page": page, "length": length, "new": new, "causal": causal, "window": window}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "rope", "cache", "attention"))
    if op == "norm":
        out = rng.choice(("fp16", "fp16", "e4m3", "int8"))
        width = _log(rng, 64, 16384)
        group = rng.choice((0, 0, 32, 64, 128)) if out != "fp16" else 0
        if group:
            width = max(group, width // group * group)
        tokens = _log(rng, 1, max(1, min(8192, 4096 * 8192 // width)))
        case = _norm("", tokens, width, rng.random() < 0.6, out, group)
    elif op == "rope":
        dim = rng.choice((64, 80, 96, 128, 256))
        heads, ratio = rng.choice((1, 2, 5, 8, 32)), rng.choice((1, 2, 4, 8))
        tokens = _log(rng, 1, max(1, min(8192, 8192 * 40 * 128 // (heads * (ratio + 1) * dim))))
        case = _rope("", tokens, heads * ratio, heads, dim, dim // rng.choice((1, 1, 2, 4)),
                     rng.choice(("half", "interleaved")), rng.choice(("none", "linear", "ntk", "yarn", "wavelength")),
                     _log(rng, 64, 1 << 20), rng.choice(("positions", "batch")))
    elif op == "cache":
        heads, dim = rng.choice((1, 2, 5, 8, 16, 32)), rng.choice((64, 96, 128, 192, 256))
        length = _log(rng, 1, 4096)
        new = _log(rng, 1, length)
        seqs = _log(rng, 1, max(1, min(64, 4 * 4096 * 32 * 128 // (max(new, 512) * heads * dim))))
        case = _cache("", seqs, heads, dim, rng.choice((32, 64, 128, 256)), length, new)
    else:
        heads, dim = rng.choice((1, 2, 4, 8, 16)), rng.choice((64, 96, 128, 192, 256))
        ratio = rng.choice((1, 2, 3, 4, 8))
        length = _log(rng, 1, 131072)
        new = 1 if rng.random() < 0.4 else _log(rng, 1, min(length, 2048))
        seqs = _log(rng, 1, max(1, min(64, 2 * 131072 * 8 * 128 // (max(length, 512) * heads * dim))))
        most = 2 * 4096 * 2048 * 32 * 128      # the largest listed product of queries, keys, heads and channels
        new = max(1, min(new, most // (seqs * length * heads * ratio * dim)))
        causal = rng.random() < 0.8
        window = _log(rng, 1, length) if causal and rng.random() < 0.3 else 0
        case = _attention("", seqs, heads * ratio, heads, dim, rng.choice((32, 64, 128, 256)), length, new, causal,
                          window)
    del case["name"]
    return case


def _lengths(case):
    """Tokens in the cache and new tokens of every sequence: the first has the
    case's own, the others spread down to a quarter of it."""
    b = case["seqs"]
    total = [max(1, case["length"] - (case["length"] * 3 * i) // (4 * b)) for i in range(b)]
    new = [min(t, max(1, case["new"] - (case["new"] * i) // (3 * b))) for i, t in enumerate(total)]
    return total, new


# ---------------------------------------------------------------- inputs

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _prepare_norm(case, gen):
    t, k = case["tokens"], case["width"]
    x = _randn(gen, t, k)
    r = _randn(gen, t, k) * 2.0 if case["residual"] else None
    for v in (x, r):
        if v is not None:
            v[:, : max(1, k // 100)] *= 8.0     # the residual stream has a few large channels
    wide = case["out"] == "fp16"
    kind = {"fp16": torch.float16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}[case["out"]]
    return {
        "x": x.half(), "residual": r.half() if r is not None else None,
        "weight": (1.0 + 0.2 * _randn(gen, k)).half(),
        "sum": torch.empty(t, k, dtype=torch.float16, device="cuda") if case["residual"] else None,
        "out": torch.empty(t, k, dtype=kind, device="cuda"),
        "scales": None if wide else torch.empty(t, k // case["group"] if case["group"] else 1, device="cuda"),
    }


# What each scaling takes beside the factor: the trained length is a quarter of
# the far end, the ramps' ends are the usual ones.
FACTOR, BASE = 4.0, 10000.0
RAMP = {"yarn": (1.0, 32.0), "wavelength": (1.0, 4.0)}


def _frequencies(case):
    """Radians per position of every pair, fp64, and the factor that the
    rotated numbers carry."""
    r, kind, c = case["rotary"], case["scaling"], FACTOR
    i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    base = BASE * c ** (r / (r - 2)) if kind == "ntk" else BASE
    f = base ** (-2.0 * i / r)
    length = case["far"] / c
    if kind == "linear":
        f = f / c
    if kind == "yarn":
        slow, fast = RAMP[kind]
        low, high = (r * math.log(length / (2 * math.pi * turns)) / (2 * math.log(base)) for turns in (fast, slow))
        low, high = max(math.floor(low), 0), min(math.ceil(high), r - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        f = f / c * ramp + f * (1 - ramp)
    if kind == "wavelength":
        low, high = RAMP[kind]
        keep = ((length * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = f * keep + f / c * (1 - keep)
    return f, 0.1 * math.log(c) + 1.0 if kind == "yarn" else 1.0


def _prepare_rope(case, gen):
    t, far = case["tokens"], case["far"]
    f, amplitude = _frequencies(case)
    state = {"freqs": f, "amplitude": amplitude,
             "q": _randn(gen, t, case["q_heads"], case["dim"]).half(), "k": _randn(gen, t, case["heads"], case["dim"]).half(),
             "positions": torch.randint(0, far, (t,), generator=gen, device="cuda", dtype=torch.int32)}
    if case["by"] == "batch":       # every token the newest of its own sequence
        state["kv_len"] = state["positions"] + 1
        state["cu"] = torch.arange(t + 1, device="cuda", dtype=torch.int32)
    state["out"] = (torch.empty_like(state["q"]), torch.empty_like(state["k"]))
    return state


def _to_nibbles(codes):
    """[..., 8 n] codes to [..., 4 n] bytes."""
    c = codes.to(torch.uint8).unflatten(-1, (-1, 8))[..., list(NIBBLES)].unflatten(-1, (4, 2))
    return (c[..., 0] | (c[..., 1] << 4)).flatten(-2)


def _from_nibbles(b):
    """[..., 4 n] bytes to [..., 8 n] codes, fp32."""
    c = torch.stack((b & 15, b >> 4), -1).unflatten(-2, (-1, 4)).flatten(-2)
    back = [NIBBLES.index(i) for i in range(8)]
    return c[..., back].flatten(-2).float()


def _groups(x):
    """Codes (as fp32), steps and smallest numbers (fp16) of groups [..., n] of
    fp32. The quotients are in 64 bits: many lie halfway between two codes, or
    are fp16 numbers."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    want = ((hi - lo).double() / 15.0).float()
    s = want.half()
    s = (s.view(torch.int16) - (s.float() > want).to(torch.int16)).view(torch.float16)     # not above
    safe = torch.where(s > 0, s.double(), 1.0)
    codes = torch.where(s > 0, torch.round((x - lo).double() / safe).clamp(0, 15), 0.0).float()
    return codes, s.squeeze(-1), lo.half().squeeze(-1)


def _numbers(codes, s, lo):
    """The cached fp16 numbers, as fp32."""
    return (lo.float().unsqueeze(-1) + s.float().unsqueeze(-1) * codes).half().float()


# [pages, H, P, D] codes <-> the stored orders
def _k_store(c):
    p, h, n, d = c.shape
    return _to_nibbles(c.view(p, h, n, d // 32, 32)).permute(0, 1, 3, 2, 4).contiguous()


def _k_load(b):
    return _from_nibbles(b).permute(0, 1, 3, 2, 4).flatten(-2)


def _v_store(c):
    p, h, n, d = c.shape
    return _to_nibbles(c.view(p, h, n // 32, 32, d).permute(0, 1, 2, 4, 3).contiguous())


def _v_load(b):
    return _from_nibbles(b).permute(0, 1, 2, 4, 3).flatten(2, 3)


def _k_numbers(codes, scales):
    """[n, H, P, D] cached keys of pages' codes and scales."""
    sc = scales.permute(0, 1, 3, 2, 4)          # [n, H, P, D / 32, 2]
    return _numbers(_k_load(codes).unflatten(-1, (-1, 32)), sc[..., 0], sc[..., 1]).flatten(-2)


def _v_numbers(codes, scales):
    return _numbers(_v_load(codes), scales[:, :, 0], scales[:, :, 1])


def _prepare_cache(case, gen, total, new):
    """A filled cache (random values quantized token by token), the table of
    pages in a shuffled order, and the index vectors of the batch."""
    dev = "cuda"
    page, heads, dim = case["page"], case["heads"], case["dim"]
    per = [-(-t // page) for t in total]
    n_pages, most = sum(per) + 3, max(per)
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(total), most), -1, dtype=torch.int32, device=dev)
    first = 0
    for b, n in enumerate(per):
        table[b, :n] = order[first: first + n]
        first += n
    state = {"table": table, "n_pages": n_pages,
             "k_codes": torch.empty(n_pages, heads, dim // 32, page, 16, dtype=torch.uint8, device=dev),
             "v_codes": torch.empty(n_pages, heads, page // 32, dim, 16, dtype=torch.uint8, device=dev),
             "k_scales": torch.empty(n_pages, heads, dim // 32, page, 2, dtype=torch.float16, device=dev),
             "v_scales": torch.empty(n_pages, heads, 2, page, dtype=torch.float16, device=dev)}
    step = max(1, (1 << 26) // (heads * page * dim))
    for at in range(0, n_pages, step):      # in pieces: the fp32 values are eight times the cache
        n = min(step, n_pages - at)
        v = _randn(gen, n, heads, page, dim).half().float()
        v[..., : max(1, dim // 32)] *= 4.0      # a few key channels are larger than the rest, as rotary keys have
        c, s, lo = _groups(v.unflatten(-1, (-1, 32)))
        state["k_codes"][at: at + n] = _k_store(c.flatten(-2))
        state["k_scales"][at: at + n] = torch.stack((s, lo), -1).permute(0, 1, 3, 2, 4)
        c, s, lo = _groups(_randn(gen, n, heads, page, dim).half().float())
        state["v_codes"][at: at + n] = _v_store(c)
        state["v_scales"][at: at + n] = torch.stack((s, lo), 2)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    state["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    state["kv_len"] = torch.tensor(total, dtype=torch.int32, device=dev)
    state["max_new"], state["max_len"], state["tokens"] = max(new), max(total), cu[-1]
    # of every new token: its sequence, its number among the new ones, its position
    state["seq"], state["nth"] = _rows(new)
    state["pos"] = state["kv_len"].long()[state["seq"]] - torch.tensor(new, device=dev)[state["seq"]] + state["nth"]
    return state


def _rows(counts):
    c = torch.tensor(counts, device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(counts), device="cuda"), c)
    nth = torch.arange(int(c.sum()), device="cuda") - (torch.cumsum(c, 0) - c)[seq]
    return seq, nth


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    if case["op"] == "norm":
        return {"case": case, **_prepare_norm(case, gen)}
    if case["op"] == "rope":
        return {"case": case, **_prepare_rope(case, gen)}
    total, new = _lengths(case)
    state = {"case": case, **_prepare_cache(case, gen, total, new)}
    heads, dim, page = case["heads"], case["dim"], case["page"]
    if case["op"] == "cache":
        state["k"] = _randn(gen, state["tokens"], heads, dim)
        state["k"][..., : max(1, dim // 32)] *= 4.0
        state["k"] = state["k"].half()
        state["v"] = _randn(gen, state["tokens"], heads, dim).half()
        # the pages the new tokens touch, read back from their first token on
        back = [t - (t - n) // page * page for t, n in zip(total, new)]
        state["back_seq"], nth = _rows(back)
        start = torch.tensor([t - n for t, n in zip(total, back)], device="cuda")
        state["back_pos"] = start[state["back_seq"]] + nth
        cu = [0]
        for n in back:
            cu.append(cu[-1] + n)
        state["back_cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        state["max_back"] = max(back)
        state["out"] = tuple(torch.empty(cu[-1], heads, dim, dtype=torch.float16, device="cuda") for _ in range(2))
        at = state["table"].long()[state["seq"], state["pos"] // page]
        state["touched"] = torch.unique(at)
    else:
        state["q"] = _randn(gen, state["tokens"], case["q_heads"], dim).half()
        state["scale"] = 1.0 / math.sqrt(dim)
        state["out"] = torch.empty(state["tokens"], case["q_heads"], dim, dtype=torch.float16, device="cuda")
    return state


# ---------------------------------------------------------------- the plain forms

def _plain_norm(s):
    case = s["case"]
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * s["weight"].float() * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    out = {"sum": h.half()} if s["residual"] is not None else {}
    if case["out"] == "fp16":
        return {**out, "y": y.half()}
    top = TOP[case["out"]]
    g = y.unflatten(-1, (-1, case["group"] or case["width"]))
    scale = g.abs().amax(-1, keepdim=True).clamp_min(FLOOR) / top
    c = (g / scale).clamp(-top, top).flatten(-2)
    c = torch.round(c).half() if case["out"] == "int8" else c.to(torch.float8_e4m3fn)
    return {**out, "y": c, "scales": scale.squeeze(-1)}


def _plain_rotate(x, cos, sin, case):
    x, r = x.float(), case["rotary"]
    if case["layout"] == "half":
        a, b = x[..., : r // 2], x[..., r // 2: r]
    else:
        a, b = x[..., 0: r: 2], x[..., 1: r: 2]
    y = (a * cos - b * sin, b * cos + a * sin)
    y = torch.cat(y, -1) if case["layout"] == "half" else torch.stack(y, -1).flatten(-2)
    return torch.cat((y, x[..., r:]), -1).half()


def _plain_rope(s):
    angle = s["positions"].double()[:, None, None] * s["freqs"]
    cos, sin = (s["amplitude"] * torch.cos(angle)).float(), (s["amplitude"] * torch.sin(angle)).float()
    return {"q": _plain_rotate(s["q"], cos, sin, s["case"]), "k": _plain_rotate(s["k"], cos, sin, s["case"])}


def _place(s):
    """The place of every page in s["touched"]."""
    place = torch.zeros(s["n_pages"], dtype=torch.long, device="cuda")
    place[s["touched"]] = torch.arange(s["touched"].numel(), device="cuda")
    return place


def _plain_cache(s):
    page, t, place = s["case"]["page"], s["touched"], _place(s)
    at, slot = place[s["table"].long()[s["seq"], s["pos"] // page]], s["pos"] % page
    c, step, lo = _groups(s["k"].float().unflatten(-1, (-1, 32)))
    held, scales = _k_load(s["k_codes"][t]), s["k_scales"][t]
    held[at, :, slot] = c.flatten(-2)
    scales[at, :, :, slot] = torch.stack((step, lo), -1)
    s["k_codes"][t], s["k_scales"][t] = _k_store(held), scales
    c, step, lo = _groups(s["v"].float())
    held, scales = _v_load(s["v_codes"][t]), s["v_scales"][t]
    held[at, :, slot] = c
    scales[at, :, :, slot] = torch.stack((step, lo), -1)
    s["v_codes"][t], s["v_scales"][t] = _v_store(held), scales
    at, slot = place[s["table"].long()[s["back_seq"], s["back_pos"] // page]], s["back_pos"] % page
    return {"k": _k_numbers(s["k_codes"][t], s["k_scales"][t])[at, :, slot].half(),
            "v": _v_numbers(s["v_codes"][t], s["v_scales"][t])[at, :, slot].half()}


def _plain_gather(numbers, codes, scales, s):
    """[B, H, L, D] values of every sequence; pages past a sequence's end are
    page 0's, and masked."""
    t = s["table"].long().clamp_min(0)
    v = numbers(codes[t.view(-1)], scales[t.view(-1)])
    v = v.view(t.shape[0], t.shape[1], *v.shape[1:]).permute(0, 2, 1, 3, 4)
    return v.reshape(v.shape[0], v.shape[1], -1, v.shape[-1])


def _plain_attention(s):
    case = s["case"]
    b, heads, dim, n = case["seqs"], case["heads"], case["dim"], s["max_new"]
    ratio = case["q_heads"] // heads
    k = _plain_gather(_k_numbers, s["k_codes"], s["k_scales"], s)
    v = _plain_gather(_v_numbers, s["v_codes"], s["v_scales"], s)
    q = torch.zeros(b, n, case["q_heads"], dim, device=k.device)
    q[s["seq"], s["nth"]] = s["q"].float()
    pos = torch.full((b, n), -1, dtype=torch.long, device=k.device)
    pos[s["seq"], s["nth"]] = s["pos"]
    q = q.view(b, n, heads, ratio, dim).permute(0, 2, 3, 1, 4).reshape(b, heads, ratio * n, dim)
    logits = (q @ k.transpose(2, 3).contiguous()) * s["scale"]
    j = torch.arange(k.shape[2], device=k.device)
    seen = (j < s["kv_len"][:, None])[:, None, :].expand(b, n, -1)
    if case["causal"]:
        seen = seen & (j <= pos[..., None])
    if case["window"]:
        seen = seen & (j > pos[..., None] - case["window"])
    seen = seen[:, None, None].expand(b, heads, ratio, n, -1).reshape(logits.shape)
    logits = torch.where(seen, logits, torch.full_like(logits, -3.0e38))
    p = torch.where(seen, torch.exp(logits - logits.amax(-1, keepdim=True)), torch.zeros_like(logits))
    o = (p @ v) / p.sum(-1, keepdim=True).clamp_min(1e-30)
    o = o.view(b, heads, ratio, n, dim).permute(0, 3, 1, 2, 4).reshape(b, n, case["q_heads"], dim)
    return o[s["seq"], s["nth"]].half()


# ---------------------------------------------------------------- the package's calls

def _handles(s):
    """What a serving program keeps: the package, the rotary table, or the
    cache object with the batch's page table and lengths, and a workspace."""
    if "handles" not in s:
        import weight_only_int4_quantize_amd as awq
        case = s["case"]
        if case["op"] == "norm":
            s["handles"] = (awq,)
        elif case["op"] == "rope":
            low, high = RAMP.get(case["scaling"], (None, None))
            rope = awq.Rope(case["rotary"], base=BASE, layout=case["layout"], scaling=case["scaling"], factor=FACTOR,
                            trained_len=case["far"] / FACTOR, low=low, high=high)
            by = {"positions": s["positions"]}
            if case["by"] == "batch":
                table = torch.zeros(case["tokens"], 0, dtype=torch.int32, device="cuda")
                by = {"seqs": awq.KVSeqs(table, s["cu"], s["kv_len"], 1, case["far"])}
            s["handles"] = (awq, rope, by)
        else:
            cache = awq.KVCache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"], "int4")
            seqs = awq.KVSeqs(s["table"], s["cu"], s["kv_len"], s["max_new"], s["max_len"])
            if case["op"] == "cache":
                more = awq.KVSeqs(s["table"], s["back_cu"], s["kv_len"], s["max_back"], s["max_len"])
            else:
                more = awq.kv_attention_workspace(cache, seqs, case["q_heads"])
            s["handles"] = (awq, cache, seqs, more)
    return s["handles"]


def _own(s):
    case = s["case"]
    if case["op"] == "norm":
        awq, = _handles(s)
        fmt = None if case["out"] == "fp16" else case["out"]
        y = awq.awq_rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"], residual_out=s["sum"], fmt=fmt,
                            group_size=case["group"], out=s["out"], scales=s["scales"])
        out = {"sum": s["sum"]} if s["residual"] is not None else {}
        if fmt is None:
            return {**out, "y": y}
        return {**out, "y": y[0].half() if fmt == "int8" else y[0], "scales": y[1]}
    if case["op"] == "rope":
        awq, rope, by = _handles(s)
        q, k = awq.awq_rope(s["q"], s["k"], rope, out=s["out"], **by)
        return {"q": q, "k": k}
    awq, cache, seqs, more = _handles(s)
    if case["op"] == "cache":
        awq.awq_kv_write(cache, seqs, s["k"], s["v"])
        k, v = awq.awq_kv_read(cache, more, out=s["out"])
        return {"k": k, "v": v}
    return awq.awq_kv_attention(s["q"], cache, seqs, scale=s["scale"], causal=case["causal"], window=case["window"],
                                out=s["out"], workspace=more)


def run(state):
    if own:
        return _own(state)
    plain = {"norm": _plain_norm, "rope": _plain_rope, "cache": _plain_cache, "attention": _plain_attention}
    return plain[state["case"]["op"]](state)


# ---------------------------------------------------------------- work and the 64-bit results

def _pairs(case):
    """Visible (query, key) pairs and the keys that any query of a sequence sees."""
    pairs = keys = 0
    for t, n in zip(*_lengths(case)):
        if not case["causal"]:
            pairs, keys = pairs + n * t, keys + t
            continue
        w = case["window"] or t
        pairs += sum(min(p + 1, w) for p in range(t - n, t))
        keys += t - max(0, t - n - w + 1)
    return pairs, keys


def work(case):
    if case["op"] == "norm":
        t, k = case["tokens"], case["width"]
        out = 2 * t * k if case["out"] == "fp16" else t * k + 4 * t * (k // case["group"] if case["group"] else 1)
        return {"bytes": (6 if case["residual"] else 2) * t * k + 2 * k + out, "flops": 6 * t * k}
    if case["op"] == "rope":
        numbers = case["tokens"] * (case["q_heads"] + case["heads"])
        return {"bytes": 4 * numbers * case["dim"] + 4 * case["tokens"] + 4 * case["rotary"],
                "flops": 3 * numbers * case["rotary"]}
    total, new = _lengths(case)
    heads, dim, page = case["heads"], case["dim"], case["page"]
    held = dim + dim // 8 + 4           # of a token and head, keys and values
    if case["op"] == "cache":
        back = sum(t - (t - n) // page * page for t, n in zip(total, new))
        return {"bytes": heads * (4 * dim + held) * (sum(new) + back), "flops": 2 * 4 * heads * dim * (sum(new) + back)}
    pairs, keys = _pairs(case)
    return {"bytes": heads * held * keys + 4 * sum(new) * case["q_heads"] * dim,
            "flops": 4 * dim * case["q_heads"] * pairs}


def _two(e):
    """2^e in fp64, exactly (torch's ldexp goes through a power that is not)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_norm(s):
    case = s["case"]
    h = s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
    y = s["weight"].double() * h / torch.sqrt(h.square().mean(1) + EPS)[:, None]
    out = {"sum": h} if case["residual"] else {}
    if case["out"] == "fp16":
        return {**out, "y": y}
    step = torch.stack([g.abs().amax(1) for g in y.split(case["group"] or case["width"], 1)], 1)
    step = step.clamp_min(FLOOR) / TOP[case["out"]]
    c = y / step.repeat_interleave(y.shape[1] // step.shape[1], 1)
    if case["out"] == "int8":
        c = torch.round(c)
    else:       # e4m3: 4 significant bits, exponents down to 2^-6, ties to even
        _, e = torch.frexp(c.abs().clamp_min(2.0 ** -6))
        unit = _two(e - 4)
        c = torch.round(c / unit) * unit
    return {**out, "y": c, "scales": step}


def _exact_rope(s):
    """Every pair as a complex number, times amplitude * e^(i position f)."""
    case, r = s["case"], s["case"]["rotary"]
    dev, c, length = s["q"].device, FACTOR, s["case"]["far"] / FACTOR
    f = []
    for i in range(r // 2):
        if case["scaling"] == "ntk":
            f.append((BASE * c ** (r / (r - 2.0))) ** (-2.0 * i / r))
            continue
        w = BASE ** (-2.0 * i / r)
        part = 1.0                      # of the frequency that stays
        if case["scaling"] == "linear":
            part = 0.0
        elif case["scaling"] == "wavelength":
            part = min(1.0, max(0.0, (length / (2 * math.pi / w) - RAMP["wavelength"][0]) /
                                (RAMP["wavelength"][1] - RAMP["wavelength"][0])))
        elif case["scaling"] == "yarn":
            first, last = (math.log(length / (2 * math.pi * n)) / math.log(BASE) * r / 2
                           for n in reversed(RAMP["yarn"]))
            first, last = max(0, math.floor(first)), min(r - 1, math.ceil(last))
            part = 1.0 - min(1.0, max(0.0, (i - first) / max(last - first, 0.001)))
        f.append(w * part + w / c * (1.0 - part))
    amplitude = 1.0 + 0.1 * math.log(c) if case["scaling"] == "yarn" else 1.0
    turn = torch.outer(s["positions"].double(), torch.tensor(f, dtype=torch.float64, device=dev))
    turn = torch.polar(torch.full_like(turn, amplitude), turn)[:, None]
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        y = x.clone()
        first = slice(0, r // 2) if case["layout"] == "half" else slice(0, r, 2)
        second = slice(r // 2, r) if case["layout"] == "half" else slice(1, r, 2)
        z = torch.complex(x[..., first], x[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        out[name] = y
    return out


def _exact_codes(b):
    """[..., 16] stored bytes to 32 codes."""
    w = b.to(torch.int64).unflatten(-1, (4, 4))
    w = w[..., 0] + 2 ** 8 * w[..., 1] + 2 ** 16 * w[..., 2] + 2 ** 24 * w[..., 3]
    return torch.stack([w // 16 ** (j // 2 + 4 * (j % 2)) % 16 for j in range(8)], -1).flatten(-2).double()


def _exact_half(v):
    """float64 to the nearest fp16 number (ties to even), as float64."""
    _, e = torch.frexp(v.abs().clamp_min(2.0 ** -14))
    unit = _two(e - 11)
    return torch.round(v / unit) * unit


def _exact_held(s, side, ids, head):
    """The cached numbers of pages `ids` and a head, in order: [len(ids) * P, D]."""
    codes = _exact_codes(s[side + "_codes"][ids, head])
    sc = s[side + "_scales"][ids, head].double()
    if side == "k":         # [n, D / 32, P, 32], sc [n, D / 32, P, 2]
        x = sc[..., 1:] + sc[..., :1] * codes
        x = x.permute(0, 2, 1, 3).flatten(2)
    else:                   # [n, P / 32, D, 32], sc [n, 2, P]
        x = codes.permute(0, 1, 3, 2).flatten(1, 2)
        x = sc[:, 1, :, None] + sc[:, 0, :, None] * x
    return _exact_half(x).flatten(0, 1)


def _exact_group(x):
    """The numbers that groups [..., n] are cached as."""
    lo, span = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True) - x.amin(-1, keepdim=True)
    _, e = torch.frexp((span / 15).clamp_min(2.0 ** -14))
    unit = _two(e - 11)
    step = torch.floor(span / 15 / unit) * unit
    code = torch.where(step > 0, torch.round((x - lo) / step.clamp_min(2.0 ** -24)).clamp(0, 15), 0.0)
    return _exact_half(lo + step * code)


def _exact_cache(s):
    case = s["case"]
    page = case["page"]
    total, new = _lengths(case)
    table, out = s["table"].tolist(), {}
    for side in ("k", "v"):
        x = s[side].double()
        x = _exact_group(x.unflatten(-1, (-1, 32))).flatten(-2) if side == "k" else _exact_group(x)
        rows, at = [], 0
        for b, (t, n) in enumerate(zip(total, new)):
            first = (t - n) // page
            held = t - n - first * page         # old tokens on the first touched page
            if held:
                ids = torch.tensor([table[b][first]], device=x.device)
                rows.append(torch.stack([_exact_held(s, side, ids, h)[:held] for h in range(case["heads"])], 1))
            rows.append(x[at: at + n])
            at += n
        out[side] = torch.cat(rows)
    return out


def _exact_attention(s):
    case = s["case"]
    page, heads = case["page"], case["heads"]
    ratio = case["q_heads"] // heads
    total, new = _lengths(case)
    q, rows, at = s["q"].double(), [], 0
    for b, (t, n) in enumerate(zip(total, new)):
        ids = s["table"][b, : -(-t // page)].long()
        pos = torch.arange(t, device=q.device)
        mine = torch.arange(t - n, t, device=q.device)[:, None]
        hide = torch.zeros(n, t, dtype=torch.bool, device=q.device)
        if case["causal"]:
            hide |= pos > mine
        if case["window"]:
            hide |= pos <= mine - case["window"]
        per_head = []
        for h in range(heads):
            k, v = (_exact_held(s, side, ids, h)[:t] for side in ("k", "v"))
            for r in range(ratio):
                a = (q[at: at + n, h * ratio + r] @ k.t()) / math.sqrt(case["dim"])
                a = torch.softmax(a.masked_fill(hide, float("-inf")), -1)
                per_head.append(a @ v)
        rows.append(torch.stack(per_head, 1))
        at += n
    return torch.cat(rows)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(state)
    if case["op"] == "rope":
        return _exact_rope(state)
    if case["op"] == "cache":
        return _exact_cache(state)
    if case["seqs"] * case["q_heads"] > 8192:
        return None         # one product per sequence and head
    return _exact_attention(state)
