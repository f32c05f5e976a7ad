"""Cases for the attention-layer operators: the key/value cache and what writes and reads it.

A hybrid model's attention layers sit between its state-space layers.  Three operators serve
them next to the mixer and the decode step:

* ``attn.kv_append``: per-head RMS norm and rotation of queries and keys, and the write of keys
  and values into a paged cache (as they are, or quantised to 8 bits with one scale for each
  token and head), for prompts and for single tokens;
* ``attn.kv_read``: the way back, a ragged run of cached tokens as contiguous keys and values;
* ``attn.paged_attention``: attention of one or several new tokens of each sequence over the
  cache, split over its length and joined.

``listed()`` and ``draw()`` give the cases, ``prepare`` what a program has in hand before a call,
``run`` the call, ``exact`` the same from the definitions in float64.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0       # largest finite value of the 8-bit format
AMAX_FLOOR = 2.0 ** -96  # rows smaller than this are scaled as if they reached it
EPS = 1e-6

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}


def listed():
    return [
        # one sequence decodes one token: nothing but latency
        {"name": "append_token", "op": "append", "tokens": 1, "pad": 0, "hq": 32, "hkv": 8, "d": 128,
         "rot": 128, "interleaved": False, "norm": True, "page": 64, "kv": "bf16"},
        # a decode batch of 64 sequences, quantised as it is written
        {"name": "append_batch_fp8", "op": "append", "tokens": 64, "pad": 0, "hq": 64, "hkv": 8, "d": 128,
         "rot": 128, "interleaved": False, "norm": True, "page": 64, "kv": "fp8"},
        # a prompt of 8192 tokens, bf16 cache of small pages
        {"name": "append_prompt", "op": "append", "tokens": 8192, "pad": 0, "hq": 32, "hkv": 8, "d": 128,
         "rot": 128, "interleaved": False, "norm": True, "page": 16, "kv": "bf16"},
        # a padded ragged batch, no norm, half of each head rotated in adjacent pairs, narrow heads
        {"name": "append_ragged_fp8", "op": "append", "tokens": 4999, "pad": 129, "hq": 24, "hkv": 4, "d": 64,
         "rot": 32, "interleaved": True, "norm": False, "page": 32, "kv": "fp8"},
        # a quantised prefix of one long sequence, read back for the next piece of its prompt
        {"name": "read_prefix_fp8", "op": "read", "batch": 1, "lo": 32768, "hi": 32768, "hkv": 8, "d": 128,
         "page": 64, "kv": "fp8"},
        # the prefixes of a ragged batch, odd lengths, small pages, narrow heads
        {"name": "read_ragged", "op": "read", "batch": 13, "lo": 1, "hi": 3001, "hkv": 4, "d": 64,
         "page": 16, "kv": "bf16"},
        # one short sequence: latency again
        {"name": "attn_short", "op": "attn", "batch": 1, "new": 1, "lo": 300, "hi": 300, "hq": 32, "hkv": 8,
         "d": 128, "window": 0, "page": 64, "kv": "bf16"},
        # one sequence at a long context: few rows, so the length has to be split
        {"name": "attn_long", "op": "attn", "batch": 1, "new": 1, "lo": 131072, "hi": 131072, "hq": 32, "hkv": 8,
         "d": 128, "window": 0, "page": 64, "kv": "bf16"},
        # a full decode batch: the ordinary case of serving
        {"name": "attn_batch", "op": "attn", "batch": 64, "new": 1, "lo": 4096, "hi": 4096, "hq": 64, "hkv": 8,
         "d": 128, "window": 0, "page": 64, "kv": "bf16"},
        # a ragged batch over a quantised cache: lengths over three decades
        {"name": "attn_ragged_fp8", "op": "attn", "batch": 96, "new": 1, "lo": 17, "hi": 16384, "hq": 32, "hkv": 8,
         "d": 128, "window": 0, "page": 32, "kv": "fp8"},
        # four draft tokens of each sequence checked together under a sliding window
        {"name": "attn_draft_window", "op": "attn", "batch": 16, "new": 4, "lo": 5, "hi": 9001, "hq": 32, "hkv": 4,
         "d": 128, "window": 2048, "page": 16, "kv": "bf16"},
        # a small model in fp32 with as many key heads as query heads, an odd page
        {"name": "attn_f32", "op": "attn", "batch": 3, "new": 1, "lo": 200, "hi": 1500, "hq": 12, "hkv": 12,
         "d": 64, "window": 0, "page": 24, "kv": "f32"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "attn", "attn"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 8, 16] if hkv < 8 else [1, 2, 4, 8])
    page = rng.choice([16, 24, 32, 64, 100, 128])
    kv = rng.choice(["bf16", "bf16", "fp8", "fp8", "f32"])
    if op == "append":
        tokens = _log_int(rng, 1, 8192)
        return {"op": op, "tokens": tokens, "pad": rng.choice([0, 0, tokens // 7]), "hq": min(hq, 32), "hkv": hkv,
                "d": d, "rot": rng.choice([0, d // 4, d // 2, d, d]), "interleaved": rng.random() < 0.3,
                "norm": rng.random() < 0.7, "page": page, "kv": kv}
    if op == "read":
        batch = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, max(1, 32768 // batch))
        return {"op": op, "batch": batch, "lo": rng.choice([1, hi]), "hi": hi, "hkv": hkv, "d": d, "page": page, "kv": kv}
    batch = _log_int(rng, 1, 128)
    new = rng.choice([1, 1, 1, 2, 3, 4, 8])
    hi = _log_int(rng, 1, max(1, min(131072, 262144 // batch)))
    if kv == "f32":
        hi = max(1, hi // 8)
    return {"op": op, "batch": batch, "new": new, "lo": rng.choice([1, hi]), "hi": hi, "hq": hq, "hkv": hkv, "d": d,
            "window": rng.choice([0, 0, 0, 1000]), "page": page, "kv": kv}


def _lens(case):
    """The lengths of a case's sequences: all `hi`, or spread from `lo` to `hi` over their logarithm."""
    if case["lo"] == case["hi"]:
        return [case["hi"]] * case["batch"]
    rng = random.Random("%(batch)d %(lo)d %(hi)d %(page)d" % case)
    return [case["hi"]] + [_log_int(rng, case["lo"], case["hi"]) for _ in range(case["batch"] - 1)]


def _pool(case, g, pages, filled):
    """Key and value pools [pages, heads, page, d] and their scales: stale or cached values, as the
    norm, the rotation and the projections leave them (unit size, keys a little larger)."""
    shape = (pages, case["hkv"], case["page"], case["d"])
    dev = "cuda"
    pools, scales = [], []
    for size in (1.2, 1.0):
        if case["kv"] == "fp8":
            # rows quantised by their largest value: codes of +-448 are reached, scales vary by row
            p = torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16) if filled else None
            if p is None:
                pools.append(torch.zeros(shape, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn))
                scales.append(torch.ones(shape[:3], dtype=torch.float32, device=dev))
                continue
            amax = p.abs().amax(-1, keepdim=True)
            pools.append((p * (E4M3_MAX / amax)).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn))
            spread = torch.rand(shape[:3], generator=g, device=dev) * 0.5 + 0.75
            scales.append(amax[..., 0].float() * spread * (size / E4M3_MAX))
            del p
        else:
            p = torch.randn(shape, generator=g, device=dev, dtype=_TYPES[case["kv"]])
            pools.append(p.mul_(size) if filled else p.zero_())
            scales.append(None)
    return pools[0], pools[1], scales[0], scales[1]


def _table(case, lens, g):
    """Page tables [batch, most pages] over a shuffled pool, -1 where a sequence has no page, and the
    number of pages (some are nobody's)."""
    page = case["page"]
    used = [-(-n // page) for n in lens]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    most = max(max(used), 1)
    cols = torch.arange(most, device="cuda")[None]
    n = torch.tensor(used, device="cuda")[:, None]
    start = torch.cumsum(n, 0) - n
    table = torch.where(cols < n, order[(start + cols).clamp_(max=pages - 1)], order.new_full((), -1))
    return table.contiguous(), pages


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind = torch.float32 if case["kv"] == "f32" else torch.bfloat16
    s = {"case": case, "kind": kind}
    if own:
        from state_space_model_gb300 import attn
        s["attn"] = attn
    if case["op"] == "append":
        t, hq, hkv, d, rot = case["tokens"], case["hq"], case["hkv"], case["d"], case["rot"]
        # queries, keys and values are views of one projection's output
        qkv = torch.randn((t, (hq + 2 * hkv) * d), generator=g, device="cuda", dtype=kind) * 2
        s["q"] = qkv[:, : hq * d].view(t, hq, d)
        s["k"] = qkv[:, hq * d: (hq + hkv) * d].view(t, hkv, d)
        s["v"] = qkv[:, (hq + hkv) * d:].view(t, hkv, d)
        s["q_weight"] = torch.rand((d,), generator=g, device="cuda") + 0.5 if case["norm"] else None
        s["k_weight"] = torch.rand((d,), generator=g, device="cuda") + 0.5 if case["norm"] else None
        s["cos"] = s["sin"] = s["positions"] = None
        if rot:
            most = t + 4096
            rate = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
            angle = torch.arange(most, device="cuda", dtype=torch.float64)[:, None] * rate
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
            first = torch.randint(0, 4096, (), generator=g, device="cuda")
            s["positions"] = (first + torch.arange(t, device="cuda")).to(torch.int32)
        pages = -(-t // case["page"]) + 2
        s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"] = _pool(case, g, pages, False)
        order = torch.randperm(pages, generator=g, device="cuda")
        i = torch.arange(t, device="cuda")
        slots = (order[i // case["page"]] * case["page"] + i % case["page"]).to(torch.int32)
        if case["pad"]:
            slots[torch.randperm(t, generator=g, device="cuda")[: case["pad"]]] = -1
        s["slots"] = slots
        s["out"] = torch.zeros((t, hq, d), dtype=kind, device="cuda")  # rows of padding stay as they are
        return s
    lens = _lens(case)
    lens = [lens[i] for i in torch.randperm(len(lens), generator=torch.Generator().manual_seed(seed)).tolist()]
    s["table"], pages = _table(case, lens, g)
    s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"] = _pool(case, g, pages, True)
    if case["op"] == "read":
        s["cu_lens"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
        s["tokens"] = sum(lens)
        return s
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["q"] = torch.randn((case["batch"], case["new"], case["hq"], case["d"]), generator=g, device="cuda").to(kind)
    return s


def _plain_rows(x, weight, cos, sin, rot, interleaved):
    """RMS norm over the last axis and rotation of its first `rot` places, in float32."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    if not rot:
        return x
    turn, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = turn[..., : rot // 2], turn[..., rot // 2:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, rest), -1)


def _plain_put(cache, scale, page, at, rows):
    """Writes rows [n, heads, d] to places (page, at) of a pool, quantised where it has scales."""
    if scale is None:
        cache[page, :, at] = rows.to(cache.dtype)
        return
    size = rows.abs().amax(-1).clamp(min=AMAX_FLOOR) / E4M3_MAX
    codes = (rows / size[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    cache.view(torch.uint8)[page, :, at] = codes.view(torch.uint8)
    scale[page, :, at] = size


def _plain_append(s):
    c = s["case"]
    real = s["slots"] >= 0
    cos = sin = None
    if c["rot"]:
        cos, sin = s["cos"][s["positions"].long()][:, None], s["sin"][s["positions"].long()][:, None]
    q = _plain_rows(s["q"], s["q_weight"], cos, sin, c["rot"], c["interleaved"])
    k = _plain_rows(s["k"], s["k_weight"], cos, sin, c["rot"], c["interleaved"])
    slot = s["slots"][real].long()
    page, at = slot // c["page"], slot % c["page"]
    _plain_put(s["k_cache"], s["k_scale"], page, at, k[real])
    _plain_put(s["v_cache"], s["v_scale"], page, at, s["v"][real].float())
    out = torch.where(real[:, None, None], q.to(s["kind"]), s["out"])
    return out


def _plain_gather(cache, scale, page, at):
    """The rows at places (page, at) of a pool, in float32: [..., heads, d]."""
    if scale is None:
        return cache[page, :, at].float()
    return cache.view(torch.uint8)[page, :, at].view(torch.float8_e4m3fn).float() * scale[page, :, at][..., None]


def _plain_read(s):
    c = s["case"]
    i = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(s["cu_lens"].long(), i, right=True) - 1
    pos = i - s["cu_lens"].long()[b]
    page, at = s["table"][b, pos // c["page"]].long(), pos % c["page"]
    return [_plain_gather(s[n + "_cache"], s[n + "_scale"], page, at).to(s["kind"]) for n in "kv"]


def _plain_attn(s):
    c = s["case"]
    bn, t, hq, d = s["q"].shape
    hkv, longest = c["hkv"], s["table"].shape[1] * c["page"]
    pos = torch.arange(longest, device="cuda")
    page = s["table"][:, pos // c["page"]].long().clamp(min=0)
    at = (pos % c["page"])[None].expand(bn, -1)
    lens = s["lens"].long()
    k = _plain_gather(s["k_cache"], s["k_scale"], page, at).permute(0, 2, 3, 1)          # [b, hkv, d, n]
    q = s["q"].float().view(bn, t, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(bn, hkv, -1, d)
    score = (q @ k).view(bn, hkv, t, hq // hkv, longest) * d ** -0.5
    del k
    last = lens[:, None] - t + torch.arange(t, device="cuda")                            # each row's own place
    seen = pos[None, None] <= last[..., None]
    if c["window"]:
        seen &= pos[None, None] > last[..., None] - c["window"]
    seen = seen[:, None, :, None]
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isinf(top), 0.0, top))
    del score
    total = p.sum(-1, keepdim=True)
    v = _plain_gather(s["v_cache"], s["v_scale"], page, at).permute(0, 2, 1, 3)          # [b, hkv, n, d]
    v = v.masked_fill((pos[None] >= lens[:, None])[:, None, :, None], 0.0)
    o = (p.view(bn, hkv, -1, longest) @ v).view(bn, hkv, t, hq // hkv, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)[..., 0]
    out = o.permute(0, 2, 1, 3, 4).reshape(bn, t, hq, d).to(s["kind"])
    return [out, lse.permute(0, 2, 1, 3).reshape(bn, t, hq)]


def run(s):
    c = s["case"]
    if c["op"] == "append":
        if own:
            out = s["attn"].kv_append(s["q"], s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"],
                                      k_scale=s["k_scale"], v_scale=s["v_scale"], positions=s["positions"],
                                      cos=s["cos"], sin=s["sin"], interleaved=c["interleaved"],
                                      q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, out=s["out"])
        else:
            out = _plain_append(s)
        return {"q": out, "k_cache": s["k_cache"], "v_cache": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if c["op"] == "read":
        if own:
            return list(s["attn"].kv_read(s["k_cache"], s["v_cache"], s["table"], s["cu_lens"], s["tokens"],
                                          k_scale=s["k_scale"], v_scale=s["v_scale"], dtype=s["kind"]))
        return _plain_read(s)
    if own:
        return list(s["attn"].paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                              k_scale=s["k_scale"], v_scale=s["v_scale"], window=c["window"],
                                              return_lse=True))
    return _plain_attn(s)


def work(case):
    size = {"bf16": 2, "fp8": 1, "f32": 4}[case["kv"]]
    plain = 4 if case["kv"] == "f32" else 2
    hkv, d = case["hkv"], case["d"]
    held = 2 * hkv * (d * size + (4 if case["kv"] == "fp8" else 0))   # a cached token
    if case["op"] == "append":
        n, hq = case["tokens"] - case["pad"], case["hq"]
        io = (2 * hq + 2 * hkv) * d * plain + held + 4 + (4 + 4 * case["rot"] if case["rot"] else 0)
        per = (hq + hkv) * (4 * d * case["norm"] + 3 * case["rot"])
        return {"bytes": n * io, "flops": n * per + (2 * n * 2 * hkv * d if case["kv"] == "fp8" else 0)}
    lens = _lens(case)
    if case["op"] == "read":
        return {"bytes": sum(lens) * (held + 2 * hkv * d * plain) + 4 * sum(-(-n // case["page"]) for n in lens),
                "flops": sum(lens) * 2 * hkv * d * (case["kv"] == "fp8")}
    t, w = case["new"], case["window"]
    seen = sum(min(n, w + t - 1) if w else n for n in lens)           # each cached token that some row sees
    pairs = sum(min(max(n - t + 1 + i, 0), w or n) for n in lens for i in range(t))
    rows = case["batch"] * t * case["hq"]
    return {"bytes": seen * held + rows * (2 * d * plain + 4) + 4 * sum(-(-n // case["page"]) for n in lens),
            "flops": 4 * d * case["hq"] * pairs}


# ---- the definitions in float64, one sequence or token block at a time ----------------------


def _exact_rows(x, weight, cos, sin, rot, interleaved):
    x = x.double()
    if weight is not None:
        x = weight.double() * x / torch.sqrt(torch.sum(x ** 2, -1, keepdim=True) / x.shape[-1] + EPS)
    if rot:
        first = torch.arange(rot // 2, device=x.device) * 2 if interleaved else torch.arange(rot // 2, device=x.device)
        second = first + (1 if interleaved else rot // 2)
        z = torch.complex(x[..., first], x[..., second]) * torch.complex(cos.double(), sin.double())
        x = x.clone()
        x[..., first], x[..., second] = z.real, z.imag
    return x


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        cos = sin = None
        if case["rot"]:
            at = s["positions"].long()
            cos, sin = s["cos"][at].unsqueeze(1), s["sin"][at].unsqueeze(1)
        q = _exact_rows(s["q"], s["q_weight"], cos, sin, case["rot"], case["interleaved"])
        k = _exact_rows(s["k"], s["k_weight"], cos, sin, case["rot"], case["interleaved"])
        keep = torch.nonzero(s["slots"] >= 0)[:, 0]
        slot = s["slots"][keep].long()
        res = {"q": torch.zeros_like(q).index_copy(0, keep, q[keep])}
        for name, rows in (("k", k[keep]), ("v", s["v"].double()[keep])):
            # pools by slot, [pages * page, heads, d]; 8-bit codes are held to the values that they round
            pool = s[name + "_cache"].float().double().transpose(1, 2).flatten(0, 1)
            res[name + "_scale"] = None
            if case["kv"] == "fp8":
                scale = s[name + "_scale"].double().transpose(1, 2).flatten(0, 1)
                size = torch.clamp(torch.max(torch.abs(rows), -1).values, min=AMAX_FLOOR) / E4M3_MAX
                scale[slot] = size
                res[name + "_scale"] = scale.view(-1, case["page"], case["hkv"]).transpose(1, 2)
                rows = rows / size.unsqueeze(-1)
            pool[slot] = rows
            res[name + "_cache"] = pool.view(-1, case["page"], case["hkv"], case["d"]).transpose(1, 2)
        return res
    page, d = case["page"], case["d"]

    def cached(name, b, lo, hi):
        """Tokens [lo, hi) of sequence b, [heads, hi - lo, d]."""
        ids = s["table"][b, lo // page: -(-hi // page)].long()
        rows = s[name + "_cache"].view(torch.uint8)[ids].view(s[name + "_cache"].dtype) if case["kv"] == "fp8" else s[name + "_cache"][ids]
        rows = rows.float().double()
        if case["kv"] == "fp8":
            rows = rows * s[name + "_scale"][ids].double().unsqueeze(-1)
        off = lo - lo // page * page
        return rows.transpose(0, 1).reshape(case["hkv"], -1, d)[:, off: off + hi - lo]

    if case["op"] == "read":
        cu = s["cu_lens"].tolist()
        return [torch.cat([cached(n, b, 0, cu[b + 1] - cu[b]).transpose(0, 1) for b in range(case["batch"])]) for n in "kv"]
    group, t = case["hq"] // case["hkv"], case["new"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        for i in range(t):
            hi = n - t + 1 + i
            lo = max(0, hi - case["window"]) if case["window"] else 0
            if hi <= 0:
                continue
            k, v = cached("k", b, lo, hi), cached("v", b, lo, hi)
            q = s["q"][b, i].double().view(case["hkv"], group, d)
            score = torch.einsum("hgd,hnd->hgn", q, k) / math.sqrt(d)
            lse[b, i] = torch.logsumexp(score, -1).flatten()
            out[b, i] = torch.einsum("hgn,hnd->hgd", torch.softmax(score, -1), v).reshape(case["hq"], d)
    return [out, lse]
