"""Cases for the attention layers' longer contexts: a 4-bit cache, sinks beside a window, positions of several axes.

The cache of a hybrid model's attention layers is what grows with the context.  The operators here are the forms
of ``attn`` that keep it small and its use bounded, and that serve models whose tokens stand in time and space:

* ``attn.kv_append`` into pools of 4-bit codes (two to a byte, an 8-bit scale for each 16 places, a 32-bit one for
  each token and head), and with positions of several axes, each of which turns its share of a head's pairs;
* ``attn.kv_read`` from such pools;
* ``attn.paged_attention`` over such pools;
* ``attn.paged_attention`` under a window with sinks: a sequence's first tokens stay visible, for single tokens,
  draft tokens and pieces of prompts, over pools of any type.

``listed()`` and ``draw()`` give the cases, ``prepare`` what a program has in hand before a call, ``run`` the call,
``exact`` the same from the definitions in float64.
"""
import math
import random

import torch

own = False

CODE_MAX = 6.0           # largest 4-bit value: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives
GROUP = 16               # places that share an 8-bit scale
GROUP_MAX = 448.0        # the largest of those
AMAX_FLOOR = 2.0 ** -96  # rows smaller than this are scaled as if they reached it
EPS = 1e-6

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
_VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def listed():
    return [
        # one token of a video model's answer: a position for time, height and width each; nothing but latency
        {"name": "append_axes_token", "op": "append", "tokens": 1, "pad": 0, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "axes": 3, "mixed": False, "norm": True, "page": 64, "kv": "bf16"},
        # images and text of a padded batch, odd length, the axes' pairs interleaved
        {"name": "append_axes_images", "op": "append", "tokens": 4999, "pad": 129, "hq": 28, "hkv": 4, "d": 128, "rot": 128,
         "interleaved": False, "axes": 3, "mixed": True, "norm": False, "page": 16, "kv": "bf16"},
        # a decode batch of 64 sequences written in 4 bits
        {"name": "append4_batch", "op": "append", "tokens": 64, "pad": 0, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "axes": 1, "mixed": False, "norm": True, "page": 64, "kv": "fp4"},
        # a prompt of 8192 tokens written in 4 bits
        {"name": "append4_prompt", "op": "append", "tokens": 8192, "pad": 0, "hq": 32, "hkv": 4, "d": 128, "rot": 128,
         "interleaved": False, "axes": 1, "mixed": False, "norm": True, "page": 64, "kv": "fp4"},
        # the prefix of one long sequence, read back for the next piece of its prompt
        {"name": "read4_prefix", "op": "read", "batch": 1, "lo": 32768, "hi": 32768, "hkv": 8, "d": 128, "page": 64, "kv": "fp4"},
        # the prefixes of a ragged batch, odd lengths, small pages, narrow heads
        {"name": "read4_ragged", "op": "read", "batch": 13, "lo": 1, "hi": 3001, "hkv": 4, "d": 64, "page": 16, "kv": "fp4"},
        # one short sequence over a 4-bit cache: latency again
        {"name": "attn4_short", "op": "attn", "batch": 1, "new": 1, "lo": 300, "hi": 300, "hq": 32, "hkv": 8, "d": 128,
         "window": 0, "sinks": 0, "page": 64, "kv": "fp4"},
        # one sequence at a long context: few rows, so the length has to be split
        {"name": "attn4_long", "op": "attn", "batch": 1, "new": 1, "lo": 131072, "hi": 131072, "hq": 32, "hkv": 8, "d": 128,
         "window": 0, "sinks": 0, "page": 64, "kv": "fp4"},
        # a full decode batch over a 4-bit cache: the ordinary case of serving
        {"name": "attn4_batch", "op": "attn", "batch": 64, "new": 1, "lo": 4096, "hi": 4096, "hq": 64, "hkv": 8, "d": 128,
         "window": 0, "sinks": 0, "page": 64, "kv": "fp4"},
        # endless streams: whatever their lengths, a window and the first four tokens
        {"name": "sinks_batch", "op": "attn", "batch": 96, "new": 1, "lo": 17, "hi": 16384, "hq": 32, "hkv": 8, "d": 128,
         "window": 1024, "sinks": 4, "page": 32, "kv": "bf16"},
        # a piece of a long prompt under a window with sinks: the products count here
        {"name": "sinks_prompt", "op": "attn", "batch": 1, "new": 4096, "lo": 8192, "hi": 8192, "hq": 32, "hkv": 8, "d": 128,
         "window": 1024, "sinks": 4, "page": 64, "kv": "bf16"},
        # four draft tokens of each sequence, narrow heads, both forms at once, an odd page
        {"name": "sinks4_draft", "op": "attn", "batch": 16, "new": 4, "lo": 5, "hi": 9001, "hq": 32, "hkv": 4, "d": 64,
         "window": 2048, "sinks": 100, "page": 24, "kv": "fp4"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "read", "attn", "attn", "attn", "prompt"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 8, 16] if hkv < 8 else [1, 2, 4, 8])
    page = rng.choice([16, 24, 32, 64, 100, 128])
    kv = rng.choice(["fp4", "fp4", "fp4", "bf16", "bf16", "fp8", "f32"])
    if op == "append":
        tokens = _log_int(rng, 1, 8192)
        axes = rng.choice([1, 2, 3, 3, 4] if kv == "fp4" else [2, 3, 3, 4])
        return {"op": op, "tokens": tokens, "pad": rng.choice([0, 0, tokens // 7]), "hq": min(hq, 32), "hkv": hkv, "d": d,
                "rot": rng.choice([d // 4, d // 2, d, d]), "interleaved": rng.random() < 0.3, "axes": axes,
                "mixed": rng.random() < 0.5, "norm": rng.random() < 0.7, "page": page, "kv": kv}
    if op == "read":
        batch = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, max(1, 32768 // batch))
        return {"op": op, "batch": batch, "lo": rng.choice([1, hi]), "hi": hi, "hkv": hkv, "d": d, "page": page, "kv": "fp4"}
    bounded = kv != "fp4" or rng.random() < 0.4
    window, sinks = (rng.choice([100, 1000, 4096]), rng.choice([1, 4, 64, 300])) if bounded else (0, 0)
    if op == "prompt":
        new = _log_int(rng, 64, 512 if kv == "f32" else 2048)
        return {"op": "attn", "batch": rng.choice([1, 1, 2]), "new": new, "lo": 1, "hi": new + _log_int(rng, 1, 2048),
                "hq": min(hq, 32), "hkv": hkv, "d": d, "window": window, "sinks": sinks, "page": page, "kv": kv}
    batch = _log_int(rng, 1, 128)
    hi = _log_int(rng, 1, max(1, min(131072, 262144 // batch)))
    if kv == "f32":
        hi = max(1, hi // 8)
    return {"op": op, "batch": batch, "new": rng.choice([1, 1, 1, 2, 3, 4, 8]), "lo": rng.choice([1, hi]), "hi": hi, "hq": hq,
            "hkv": hkv, "d": d, "window": window, "sinks": sinks, "page": page, "kv": kv}


def _lens(case):
    """The lengths of a case's sequences: all `hi`, or spread from `lo` to `hi` over their logarithm."""
    if case["lo"] == case["hi"]:
        return [case["hi"]] * case["batch"]
    rng = random.Random("%(batch)d %(lo)d %(hi)d %(page)d" % case)
    return [case["hi"]] + [_log_int(rng, case["lo"], case["hi"]) for _ in range(case["batch"] - 1)]


def _sections(case):
    """Runs of pairs, which go round the axes: a quarter of the pairs to the first axis and the rest shared out, or a
    pair to each axis in turn up to the first axis's rest."""
    pairs, axes = case["rot"] // 2, case["axes"]
    if case["mixed"]:
        turns = axes * max(1, pairs // (axes + 1))
        return (1,) * turns + ((pairs - turns,) if pairs > turns else ())
    first = max(1, pairs // 4)
    rest = [(pairs - first) // (axes - 1)] * (axes - 1)
    rest[-1] += pairs - first - sum(rest)
    return (first, *rest)


def _quantise(rows):
    """Rows [..., d] (float32) as 4-bit codes [..., d / 2], the groups' scales [..., d / 16] and the rows' [...]."""
    size = rows.abs()
    scale = size.amax(-1).clamp(min=AMAX_FLOOR) / (CODE_MAX * GROUP_MAX)
    top = size.unflatten(-1, (-1, GROUP)).amax(-1)
    group = (top / (CODE_MAX * scale[..., None])).clamp(max=GROUP_MAX).to(torch.float8_e4m3fn)
    step = group.float() * scale[..., None]
    x = (rows.unflatten(-1, (-1, GROUP)) / step[..., None]).masked_fill((step == 0)[..., None], 0.0).flatten(-2)
    a = x.abs()
    # the number of halfway points passed; a tie goes to the even code
    n = (a > 0.25).to(torch.uint8)
    n += a >= 0.75
    n += a > 1.25
    n += a >= 1.75
    n += a > 2.5
    n += a >= 3.5
    n += a > 5.0
    n += torch.signbit(x).to(torch.uint8) * 8
    return n[..., 0::2] + n[..., 1::2] * 16, group, scale


def _pools(s, case, g, pages, filled):
    """The cache's two pools [pages, heads, page, d] and what goes with them, keys and values side by side as [2, ...]:
    stale or cached values, as the norm, the rotation and the projections leave them (unit size, keys a little larger)."""
    shape = (2, pages, case["hkv"], case["page"], case["d"])
    dev = "cuda"
    s["scale"] = s["group"] = None
    if case["kv"] == "fp4":
        codes = torch.zeros(shape[:-1] + (case["d"] // 2,), dtype=torch.uint8, device=dev)
        s["group"] = torch.zeros(shape[:-1] + (case["d"] // GROUP,), dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
        s["scale"] = torch.ones(shape[:-1], dtype=torch.float32, device=dev)
        if filled:
            for i, size in enumerate((1.2, 1.0)):
                rows = torch.randn(shape[1:], generator=g, device=dev) * size
                codes[i], group, s["scale"][i] = _quantise(rows)
                s["group"].view(torch.uint8)[i] = group.view(torch.uint8)
                del rows
        s["codes"] = codes
        s["k_cache"], s["v_cache"] = codes.view(torch.float4_e2m1fn_x2).unbind(0)
        s["k_group"], s["v_group"] = s["group"].unbind(0)
        s["k_scale"], s["v_scale"] = s["scale"].unbind(0)
        # what a byte of two codes stands for, as float32 and as 8-bit floating point
        both = torch.tensor([[(-v if n & 8 else v) for n in (b & 15, b >> 4) for v in (_VALUES[n & 7],)] for b in range(256)])
        s["pairs"] = both.to(dev)
        s["pairs8"] = both.to(torch.float8_e4m3fn).view(torch.int16).flatten().to(dev)
        return
    if case["kv"] == "fp8":
        pools, s["scale"] = [], torch.ones(shape[:-1], dtype=torch.float32, device=dev)
        for i, size in enumerate((1.2, 1.0)):
            rows = torch.randn(shape[1:], generator=g, device=dev) * size
            amax = rows.abs().amax(-1)
            s["scale"][i] = amax / 448.0
            pools.append((rows * (448.0 / amax[..., None])).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn))
            del rows
        s["k_cache"], s["v_cache"] = pools
    else:
        pools = [torch.randn(shape[1:], generator=g, device=dev, dtype=_TYPES[case["kv"]]) for _ in range(2)]
        s["k_cache"], s["v_cache"] = pools[0].mul_(1.2 if filled else 0.0), pools[1].mul_(1.0 if filled else 0.0)
    s["k_scale"], s["v_scale"] = s["scale"].unbind(0) if s["scale"] is not None else (None, None)
    s["k_group"] = s["v_group"] = None


def _table(case, lens, g):
    """Page tables [batch, most pages] over a shuffled pool, -1 where a sequence has no page, and the number of pages
    (some are nobody's)."""
    used = [-(-n // case["page"]) for n in lens]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    cols = torch.arange(max(max(used), 1), device="cuda")[None]
    n = torch.tensor(used, device="cuda")[:, None]
    start = torch.cumsum(n, 0) - n
    table = torch.where(cols < n, order[(start + cols).clamp_(max=pages - 1)], order.new_full((), -1))
    return table.contiguous(), pages


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind = torch.float32 if case["kv"] == "f32" else torch.bfloat16
    s = {"case": case, "kind": kind}
    if case["op"] == "append":
        t, hq, hkv, d, rot, axes = case["tokens"], case["hq"], case["hkv"], case["d"], case["rot"], case["axes"]
        # queries, keys and values are views of one projection's output
        qkv = torch.randn((t, (hq + 2 * hkv) * d), generator=g, device="cuda", dtype=kind) * 2
        s["q"] = qkv[:, : hq * d].view(t, hq, d)
        s["k"] = qkv[:, hq * d: (hq + hkv) * d].view(t, hkv, d)
        s["v"] = qkv[:, (hq + hkv) * d:].view(t, hkv, d)
        s["q_weight"] = torch.rand((d,), generator=g, device="cuda") + 0.5 if case["norm"] else None
        s["k_weight"] = torch.rand((d,), generator=g, device="cuda") + 0.5 if case["norm"] else None
        rate = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        angle = torch.arange(t + 4096, device="cuda", dtype=torch.float64)[:, None] * rate
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        first = torch.randint(0, 4096, (), generator=g, device="cuda")
        i = torch.arange(t, device="cuda")
        # frames of 24 x 40 patches after some text: frame, row, column, and the place itself as a fourth axis
        places = torch.stack([i // 960, i // 40 % 24, i % 40, i])[:axes] if axes > 1 else i[None]
        s["positions"] = (first + places).to(torch.int32)
        s["sections"], s["axis"] = None, None
        if axes > 1:
            s["sections"] = _sections(case)
            s["axis"] = torch.tensor([j % axes for j, n in enumerate(s["sections"]) for _ in range(n)], device="cuda")
        else:
            s["positions"] = s["positions"][0]
        pages = -(-t // case["page"]) + 2
        _pools(s, case, g, pages, False)
        order = torch.randperm(pages, generator=g, device="cuda")
        slots = (order[i // case["page"]] * case["page"] + i % case["page"]).to(torch.int32)
        if case["pad"]:
            slots[torch.randperm(t, generator=g, device="cuda")[: case["pad"]]] = -1
        s["slots"] = slots
        s["out"] = torch.zeros((t, hq, d), dtype=kind, device="cuda")  # rows of padding stay as they are
        return s
    lens = _lens(case)
    lens = [lens[i] for i in torch.randperm(len(lens), generator=torch.Generator().manual_seed(seed)).tolist()]
    s["table"], pages = _table(case, lens, g)
    _pools(s, case, g, pages, True)
    if case["op"] == "read":
        s["cu_lens"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
        s["tokens"] = sum(lens)
        return s
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["q"] = torch.randn((case["batch"], case["new"], case["hq"], case["d"]), generator=g, device="cuda").to(kind)
    return s


# ---- the plain forms, in float32 ------------------------------------------------------------


def _plain_rows(x, weight, cos, sin, rot, interleaved):
    """RMS norm over the last axis and rotation of its first `rot` places."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    turn, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = turn[..., : rot // 2], turn[..., rot // 2:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, rest), -1)


def _plain_put(s, i, page, at, rows):
    """Writes rows [n, heads, d] to places (page, at) of the keys' (i = 0) or values' pool."""
    name = "kv"[i]
    if s["case"]["kv"] == "fp4":
        s["codes"][i][page, :, at], group, s["scale"][i][page, :, at] = _quantise(rows)
        s["group"].view(torch.uint8)[i][page, :, at] = group.view(torch.uint8)
    elif s["case"]["kv"] == "fp8":
        size = rows.abs().amax(-1).clamp(min=AMAX_FLOOR) / 448.0
        codes = (rows / size[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        s[name + "_cache"].view(torch.uint8)[page, :, at] = codes.view(torch.uint8)
        s["scale"][i][page, :, at] = size
    else:
        s[name + "_cache"][page, :, at] = rows.to(s["kind"])


def _plain_append(s):
    c = s["case"]
    real = s["slots"] >= 0
    at = s["positions"].long()
    if c["axes"] > 1:
        # [axes, tokens, pairs] -> the row of each pair's own axis
        pick = s["axis"].expand(1, c["tokens"], -1)
        cos, sin = s["cos"][at].gather(0, pick)[0][:, None], s["sin"][at].gather(0, pick)[0][:, None]
    else:
        cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
    q = _plain_rows(s["q"], s["q_weight"], cos, sin, c["rot"], c["interleaved"])
    k = _plain_rows(s["k"], s["k_weight"], cos, sin, c["rot"], c["interleaved"])
    slot = s["slots"][real].long()
    page, at = slot // c["page"], slot % c["page"]
    _plain_put(s, 0, page, at, k[real])
    _plain_put(s, 1, page, at, s["v"][real].float())
    return torch.where(real[:, None, None], q.to(s["kind"]), s["out"])


def _plain_gather(s, i, page, at):
    """The rows at places (page, at) of the keys' or values' pool: [..., heads, d]."""
    if s["case"]["kv"] == "fp4":
        x = s["pairs"][s["codes"][i][page, :, at].int()].flatten(-2)
        x = x.unflatten(-1, (-1, GROUP)) * s["group"].view(torch.uint8)[i][page, :, at].view(torch.float8_e4m3fn).float()[..., None]
        return x.flatten(-2) * s["scale"][i][page, :, at][..., None]
    cache = s["kv"[i] + "_cache"]
    if s["case"]["kv"] == "fp8":
        return cache.view(torch.uint8)[page, :, at].view(torch.float8_e4m3fn).float() * s["scale"][i][page, :, at][..., None]
    return cache[page, :, at].float()


def _plain_read(s):
    c = s["case"]
    i = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(s["cu_lens"].long(), i, right=True) - 1
    pos = i - s["cu_lens"].long()[b]
    page, at = s["table"][b, pos // c["page"]].long(), pos % c["page"]
    return [_plain_gather(s, n, page, at).to(s["kind"]) for n in range(2)]


def _plain_attn(s):
    c = s["case"]
    bn, t, hq, d = s["q"].shape
    hkv, longest = c["hkv"], s["table"].shape[1] * c["page"]
    pos = torch.arange(longest, device="cuda")
    page = s["table"][:, pos // c["page"]].long().clamp(min=0)
    at = (pos % c["page"])[None].expand(bn, -1)
    lens = s["lens"].long()
    k = _plain_gather(s, 0, page, at).permute(0, 2, 3, 1)                                # [b, hkv, d, n]
    q = s["q"].float().view(bn, t, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(bn, hkv, -1, d)
    score = (q @ k).view(bn, hkv, t, hq // hkv, longest) * d ** -0.5
    del k
    last = lens[:, None] - t + torch.arange(t, device="cuda")                            # each row's own place
    seen = pos[None, None] <= last[..., None]
    if c["window"]:
        seen &= (pos[None, None] > last[..., None] - c["window"]) | (pos < c["sinks"])
    seen = seen[:, None, :, None]
    score = score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(torch.isinf(top), 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    v = _plain_gather(s, 1, page, at).permute(0, 2, 1, 3)                                # [b, hkv, n, d]
    v = v.masked_fill((pos[None] >= lens[:, None])[:, None, :, None], 0.0)
    o = (p.view(bn, hkv, -1, longest) @ v).view(bn, hkv, t, hq // hkv, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)[..., 0]
    out = o.permute(0, 2, 1, 3, 4).reshape(bn, t, hq, d).to(s["kind"])
    return [out, lse.permute(0, 2, 1, 3).reshape(bn, t, hq)]


def _framework():
    from state_space_model_gb300 import attn
    return attn


def _own_run(s):
    c, attn = s["case"], _framework()
    pools = dict(k_scale=s["k_scale"], v_scale=s["v_scale"], k_group_scale=s["k_group"], v_group_scale=s["v_group"])
    if c["op"] == "append":
        return attn.kv_append(s["q"], s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], positions=s["positions"],
                              cos=s["cos"], sin=s["sin"], sections=s["sections"], interleaved=c["interleaved"],
                              q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, out=s["out"], **pools)
    if c["op"] == "read":
        return list(attn.kv_read(s["k_cache"], s["v_cache"], s["table"], s["cu_lens"], s["tokens"], dtype=s["kind"], **pools))
    return list(attn.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], window=c["window"],
                                     sinks=c["sinks"], return_lse=True, **pools))


def run(s):
    c = s["case"]
    if own:
        out = _own_run(s)
    else:
        out = (_plain_append if c["op"] == "append" else _plain_read if c["op"] == "read" else _plain_attn)(s)
    if c["op"] != "append":
        return out
    if c["kv"] != "fp4":
        return {"q": out, "k": s["k_cache"], "v": s["v_cache"], "scale": s["scale"]}
    # the codes as the values that they stand for
    values = torch.index_select(s["pairs8"], 0, s["codes"].flatten().int()).view(torch.float8_e4m3fn)
    return {"q": out, "values": values.view(*s["codes"].shape[:-1], c["d"]), "group": s["group"], "scale": s["scale"]}


def work(case):
    d, hkv = case["d"], case["hkv"]
    plain = 4 if case["kv"] == "f32" else 2
    # a cached row: its places, and its scales
    row = {"bf16": 2 * d, "f32": 4 * d, "fp8": d + 4, "fp4": d // 2 + d // GROUP + 4}[case["kv"]]
    held = 2 * hkv * row                                              # a cached token
    few = case["kv"] in ("fp4", "fp8")
    if case["op"] == "append":
        n, hq = case["tokens"] - case["pad"], case["hq"]
        io = (2 * hq + 2 * hkv) * d * plain + held + 4 + 4 * case["axes"] + 4 * case["rot"]
        per = (hq + hkv) * (4 * d * case["norm"] + 3 * case["rot"])
        return {"bytes": n * io, "flops": n * per + 2 * few * n * 2 * hkv * d}
    lens = _lens(case)
    if case["op"] == "read":
        return {"bytes": sum(lens) * (held + 2 * hkv * d * plain) + 4 * sum(-(-n // case["page"]) for n in lens),
                "flops": sum(lens) * 4 * hkv * d}
    t, w, first = case["new"], case["window"], case["sinks"]
    near = [min(n, w + t - 1) if w else n for n in lens]              # cached tokens that some row sees in its window
    seen = sum(m + min(first, n - m) for n, m in zip(lens, near))     # and before it
    rows = [(max(n - t + 1 + i, 0)) for n in lens for i in range(t)]  # what a row would see without a window
    pairs = sum(min(n, w + first) if w else n for n in rows)
    io = case["batch"] * t * case["hq"] * (2 * d * plain + 4)
    return {"bytes": seen * held + io + 4 * sum(-(-m // case["page"]) for m in near), "flops": 4 * d * case["hq"] * pairs}


# ---- the definitions in float64, one sequence or token block at a time ----------------------


def _exact_rows(x, weight, angle, rot, interleaved):
    """angle: unit complex numbers [tokens, 1, rot / 2]."""
    x = x.double()
    if weight is not None:
        x = weight.double() * x / torch.sqrt(torch.sum(x ** 2, -1, keepdim=True) / x.shape[-1] + EPS)
    i = torch.arange(rot // 2, device=x.device)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    z = torch.complex(x[..., first], x[..., second]) * angle
    x = x.clone()
    x[..., first], x[..., second] = z.real, z.imag
    return x


def _exact_codes(rows):
    """The 4-bit values, group scales and row scales that stand for rows [..., d] (float64)."""
    grid = torch.tensor(_VALUES, dtype=torch.float64, device=rows.device)
    scale = torch.clamp(torch.max(torch.abs(rows), -1).values, min=AMAX_FLOOR) / CODE_MAX / GROUP_MAX
    parts = rows.reshape(*rows.shape[:-1], -1, GROUP)
    group = torch.max(torch.abs(parts), -1).values / scale.unsqueeze(-1) / CODE_MAX
    group = torch.clamp(group, max=GROUP_MAX).to(torch.float8_e4m3fn).double()
    x = parts / torch.where(group == 0, math.inf, group * scale.unsqueeze(-1)).unsqueeze(-1)
    # the nearest value of the grid, the even code of two equally near ones
    below = torch.searchsorted(grid, torch.abs(x).clamp(max=CODE_MAX), right=True) - 1
    above = torch.clamp(below + 1, max=7)
    lo, hi = torch.abs(x) - grid[below], grid[above] - torch.abs(x)
    code = torch.where((hi < lo) | ((hi == lo) & (above % 2 == 0)), above, below)
    return (grid[code] * torch.sign(x)).reshape(rows.shape), group, scale


def exact(case, seed):
    s = prepare(case, seed)
    page, d, hkv = case["page"], case["d"], case["hkv"]

    def raw(x, ids):
        """Pages of a pool whose type has no indexing of its own."""
        return x.view(torch.uint8)[ids].view(x.dtype) if x.element_size() == 1 else x[ids]

    if case["op"] == "append":
        rows = [s["positions"]] if case["axes"] == 1 else list(s["positions"])
        angle = torch.zeros((case["tokens"], 1, case["rot"] // 2), dtype=torch.complex128, device="cuda")
        start = 0
        for j, n in enumerate(s["sections"] or [case["rot"] // 2]):
            at = rows[j % len(rows)].long()
            part = slice(start, start + n)
            angle[:, 0, part] = torch.complex(s["cos"][at, part].double(), s["sin"][at, part].double())
            start += n
        q = _exact_rows(s["q"], s["q_weight"], angle, case["rot"], case["interleaved"])
        k = _exact_rows(s["k"], s["k_weight"], angle, case["rot"], case["interleaved"])
        keep = torch.nonzero(s["slots"] >= 0)[:, 0]
        slot = s["slots"][keep].long()
        res = {"q": torch.zeros_like(q).index_copy(0, keep, q[keep])}

        def put(old, new):
            """`new` [n, heads, ...] at the slots of `old` [pages, heads, page, ...]."""
            by_slot = old.double().transpose(1, 2).flatten(0, 1)
            by_slot[slot] = new
            return by_slot.unflatten(0, (-1, page)).transpose(1, 2)

        both = []
        for name, x in (("k", k[keep]), ("v", s["v"].double()[keep])):
            old = s[name + "_cache"]
            if case["kv"] == "fp4":
                values, group, scale = _exact_codes(x)
                zeros = torch.zeros(old.shape[:-1] + (d,), device="cuda")
                both.append((put(zeros, values), put(s[name + "_group"].float(), group), put(s[name + "_scale"], scale)))
            elif case["kv"] == "fp8":
                scale = torch.clamp(torch.max(torch.abs(x), -1).values, min=AMAX_FLOOR) / 448.0
                both.append((put(old.float(), x / scale.unsqueeze(-1)), None, put(s[name + "_scale"], scale)))
            else:
                both.append((put(old, x), None, None))
        if case["kv"] == "fp4":
            res["values"], res["group"], res["scale"] = [torch.stack(x) for x in zip(*both)]
        else:
            res["k"], res["v"] = both[0][0], both[1][0]
            res["scale"] = torch.stack([both[0][2], both[1][2]]) if case["kv"] == "fp8" else None
        return res

    def cached(i, b, lo, hi):
        """Tokens [lo, hi) of sequence b, [heads, hi - lo, d]."""
        ids = s["table"][b, lo // page: -(-hi // page)].long()
        name = "kv"[i]
        if case["kv"] == "fp4":
            byte = s["codes"][i][ids].long()
            grid = torch.tensor(_VALUES + [-v for v in _VALUES], dtype=torch.float64, device="cuda")
            rows = torch.stack((grid[byte % 16], grid[byte // 16]), -1).flatten(-2)
            rows = rows * raw(s[name + "_group"], ids).double().repeat_interleave(GROUP, -1)
        else:
            rows = raw(s[name + "_cache"], ids).float().double()
        if s["scale"] is not None:
            rows = rows * s[name + "_scale"][ids].double().unsqueeze(-1)
        off = lo - lo // page * page
        return rows.transpose(0, 1).reshape(hkv, -1, d)[:, off: off + hi - lo]

    if case["op"] == "read":
        cu = s["cu_lens"].tolist()
        return [torch.cat([cached(i, b, 0, cu[b + 1] - cu[b]).transpose(0, 1) for b in range(case["batch"])]) for i in range(2)]
    group, t = case["hq"] // hkv, case["new"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        k, v = cached(0, b, 0, n), cached(1, b, 0, n)
        for t0 in range(0, t, 64):                     # a block of rows over what any of them sees
            t1 = min(t, t0 + 64)
            hi = n - t + t1
            lo = max(0, n - t + t0 + 1 - case["window"]) if case["window"] else 0
            if hi <= 0:
                continue
            here = torch.cat([torch.arange(min(case["sinks"], lo), device="cuda"), torch.arange(lo, hi, device="cuda")])
            place = n - t + torch.arange(t0, t1, device="cuda")
            gone = here > place[:, None]
            if case["window"]:
                gone = gone | ((place[:, None] - here >= case["window"]) & (here >= case["sinks"]))
            q = s["q"][b, t0:t1].double().view(t1 - t0, hkv, group, d)
            score = torch.einsum("thgd,hnd->hgtn", q, k[:, here]) / math.sqrt(d)
            score = score.masked_fill(gone, -math.inf)
            total = torch.logsumexp(score, -1)
            lse[b, t0:t1] = total.permute(2, 0, 1).flatten(1)
            p = torch.exp(score - torch.where(torch.isinf(total), 0.0, total).unsqueeze(-1))
            out[b, t0:t1] = torch.einsum("hgtn,hnd->thgd", p, v[:, here]).reshape(t1 - t0, case["hq"], d)
    return [out, lse]
