"""The attention cache's kernels at sizes that take their other paths: prompts (several passes of a
warp), long batches (many tiles of a CTA, across items), pieces of prompts (many row blocks),
many sequences, many heads.

The references are float64 on the GPU, the oracle's formulas on whole tensors; the bounds are those that
test_attn_gpu.py derives.
"""
import math

import pytest
import torch

from test_attn_gpu import BF, F8, F32, U, attn, append_inputs, attn_problem, check_attn, new_pools  # noqa: F401

pytestmark = pytest.mark.gpu


# ---- kv_append: two, three and four passes of a warp -----------------------------------


def norm_rotate64(x, weight, cos, sin, interleaved):
    x = x.double()
    if weight is not None:
        x = x * weight.double() / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    if cos is None:
        return x
    half = cos.shape[-1]
    i = torch.arange(half, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c, s = cos.double()[:, None], sin.double()[:, None]
    y = x.clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


# (T, Hq, Hkv, D): warps of 3, 4, 3 and 4 passes in bf16, of 2 in f32; the last CTA not full
SIZES = [(2501, 4, 2, 128), (1003, 32, 8, 128), (1303, 24, 4, 64), (1301, 40, 8, 64)]


@pytest.mark.parametrize("R,interleaved,norm", [(0, False, True), ("D", False, True), (32, False, False),
                                                (48, True, True), ("D", True, False)], ids=str)
@pytest.mark.parametrize("dt,pdt", [(BF, BF), (BF, F8), (F32, F32), (F32, F8)], ids=["bf16", "bf16-fp8", "f32", "f32-fp8"])
@pytest.mark.parametrize("T,Hq,Hkv,D", SIZES, ids=str)
def test_append_prompts(attn, T, Hq, Hkv, D, dt, pdt, R, interleaved, norm):
    R, ps = D if R == "D" else R, 24
    q, k, v, (qw, kw), cos, sin, pos, g = append_inputs(T, Hq, Hkv, D, R, norm, dt, T + R)
    pages = -(-T // ps) + 2
    kc, vc, ks, vs = new_pools(pages, Hkv, ps, D, pdt)
    slots = torch.randperm(pages * ps, generator=g)[:T].to(torch.int32)
    slots[torch.randperm(T, generator=g)[:97]] = -1
    slots[T - 1] = pages * ps                        # padding too
    slots = slots.cuda()
    out = torch.full((T, Hq, D), 5.0, dtype=dt, device="cuda")
    attn.kv_append(q, k, v, slots, kc, vc, k_scale=ks, v_scale=vs, positions=pos, cos=cos, sin=sin,
                   interleaved=interleaved, q_weight=qw, k_weight=kw, out=out)
    real = (slots >= 0) & (slots < pages * ps)
    c, s = (None, None) if not R else (cos[pos.long()], sin[pos.long()])
    ref = norm_rotate64(q, qw, c, s, interleaved)
    top = ref.abs().amax(-1, keepdim=True)
    err = (out.double() - ref).abs()
    assert (err <= U[dt] * ref.abs() + 2.0 ** -17 * top)[real].all()
    assert (out[~real] == 5.0).all()
    at = slots[real].long()
    held = torch.zeros(pages * ps, dtype=torch.bool, device="cuda")
    held[at] = True
    for pool, scale, rows in ((kc, ks, norm_rotate64(k, kw, c, s, interleaved)), (vc, vs, v.double())):
        rows = rows[real]
        p = pool.float().double().transpose(1, 2).reshape(-1, Hkv, D)
        assert (p[~held] == 3.0).all()
        top = rows.abs().amax(-1, keepdim=True)
        if pdt == F8:
            sc = scale.double().transpose(1, 2).reshape(-1, Hkv, 1)
            assert (sc[~held] == 9.0).all()
            want = top.clamp(min=2.0 ** -96) / 448
            assert ((sc[at] - want).abs() <= 2.0 ** -17 * want).all()
            err = (p[at] * sc[at] - rows).abs()
            assert (err <= torch.maximum(2.0 ** -4 * rows.abs(), 2.0 ** -10 * sc[at]) + 2.0 ** -15 * top).all()
        elif pool is vc:
            assert (p[at] == rows).all()
        else:
            assert ((p[at] - rows).abs() <= U[dt] * rows.abs() + 2.0 ** -17 * top).all()


# ---- kv_read: the look-up in global memory, wide tokens, several tokens in flight ----------


@pytest.mark.parametrize("pdt,odt", [(BF, BF), (F8, BF), (F8, F32), (F32, F32)], ids=str)
@pytest.mark.parametrize("B,Hkv,D,most", [(511, 2, 64, 40), (512, 2, 64, 40), (600, 1, 128, 30), (3, 20, 128, 300),
                                          (2, 40, 64, 500), (5, 4, 128, 2000), (4, 2, 64, 9000)], ids=str)
def test_read_of_many(attn, B, Hkv, D, most, pdt, odt):
    ps = 16
    g = torch.Generator().manual_seed(B + Hkv)
    lens = torch.randint(0, most, (B,), generator=g)
    lens[::3] *= (torch.rand(lens[::3].shape, generator=g) < 0.5)        # empty ones among them
    lens[0], lens[-1] = 0, most
    prob = attn_problem(B, 1, Hkv, Hkv, D, ps, lens.tolist(), pdt, seed=B, nan=False)
    _, kc, vc, table, _, ks, vs = prob
    cu = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)])
    T = int(cu[-1])
    got = attn.kv_read(kc, vc, table, cu.to(torch.int32).cuda(), T, k_scale=ks, v_scale=vs, dtype=odt)
    b = torch.repeat_interleave(torch.arange(B), lens).cuda()
    pos = torch.arange(T).cuda() - cu.cuda()[b]
    page, at = table[b, pos // ps].long(), pos % ps
    for x, pool, scale in zip(got, (kc, vc), (ks, vs)):
        if pdt == F8:
            want = (pool.view(torch.uint8)[page, :, at].view(F8).float() * scale[page, :, at][..., None]).to(odt)
        else:
            want = pool[page, :, at]
        assert torch.equal(x, want)


# ---- paged_attention: many tiles of a CTA, many row blocks -----------------------------------


def check_large(attn, prob, pdt, window=0, scale=None):
    """check_attn with its reference on the GPU, a sequence and some rows at a time."""
    q, kc, vc, table, lens, ks, vs = prob
    out, lse = attn.paged_attention(q, kc, vc, table, lens, k_scale=ks, v_scale=vs, window=window, scale=scale,
                                    return_lse=True)
    B, T, Hq, D = q.shape
    Hkv, ps = kc.shape[1], kc.shape[2]
    scale = D ** -0.5 if scale is None else scale
    ut, uo = 2.0 ** -24 if pdt == F32 else 2.0 ** -22, U[q.dtype]
    for b, n in enumerate(lens.tolist()):
        ids = table[b, : -(-n // ps)].long()

        def rows(pool, sc):
            x = (pool.view(torch.uint8)[ids].view(F8) if pdt == F8 else pool[ids]).double()
            x = x if sc is None else x * sc[ids].double()[..., None]
            return x.transpose(0, 1).reshape(Hkv, -1, D)[:, :n]

        K, V = rows(kc, ks), rows(vc, vs)
        for t0 in range(0, T, 128):
            t = torch.arange(t0, min(t0 + 128, T), device="cuda")
            e = n - T + t
            pos = torch.arange(n, device="cuda")
            see = pos <= e[:, None]
            if window:
                see &= pos > e[:, None] - window
            Q = q[b, t].double().view(len(t), Hkv, Hq // Hkv, D).permute(1, 0, 2, 3)
            s = torch.einsum("htgd,hnd->htgn", Q, K) * scale
            mask = see[None, :, None]
            big = (torch.einsum("htgd,hnd->htgn", Q.abs(), K.abs()) * abs(scale)).masked_fill(~mask, 0)
            s = s.masked_fill(~mask, -math.inf)
            seen = see.sum(-1)[None, :, None].double()
            none = (seen == 0).expand(s.shape[:3])
            ref_l = torch.logsumexp(s, -1) if n else torch.full(s.shape[:3], -math.inf, device="cuda", dtype=torch.float64)
            p = torch.exp(s - torch.where(none, 0.0, ref_l)[..., None])
            ref = torch.einsum("htgn,hnd->htgd", p, V)
            smax = big.amax(-1) if n else torch.zeros_like(ref_l)
            vmax = (V.abs().amax(-1)[:, None].masked_fill(~see[None], 0).amax(-1)[..., None] if n
                    else torch.zeros_like(ref_l))
            ds = (D + 8) * ut * smax
            bound = vmax * (2 * ds + (seen + 8) * ut + (0 if pdt == F32 else 2.0 ** -8))
            o = out[b, t].double().view(len(t), Hkv, Hq // Hkv, D).permute(1, 0, 2, 3)
            l = lse[b, t].double().view(len(t), Hkv, Hq // Hkv).permute(1, 0, 2)
            assert (o[none] == 0).all() and torch.isneginf(l[none]).all()
            assert ((o - ref).abs() <= bound[..., None] * (1 + uo) + uo * ref.abs()).all()
            assert ((l - ref_l).abs() <= ds + seen * ut + 2.0 ** -21 * (1 + ref_l.abs()))[~none].all()


def ragged(B, most, seed):
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(1, most, (B,), generator=g)
    lens[1], lens[B // 2], lens[-1] = 0, most, 3
    return lens.tolist()


# (T, Hq, Hkv, D, ps, sequences, longest, window): 20 to 60 tiles of a CTA's share in bf16 and codes, more in f32
LONG = [
    (1, 32, 8, 128, 16, 60, 5000, 0),                # 4 rows
    (4, 16, 8, 64, 100, 40, 12000, 0),               # 8 rows, pages that end inside a tile
    (4, 32, 8, 128, 64, 40, 5000, 0),                # 16 rows
    (3, 64, 8, 128, 24, 40, 4000, 1500),             # 24 rows under a window
    (7, 16, 2, 64, 128, 60, 16000, 0),               # 56 rows
]


@pytest.mark.parametrize("pdt", [BF, F8, F32], ids=["bf16", "fp8", "f32"])
@pytest.mark.parametrize("case", LONG, ids=str)
def test_attention_many_tiles(attn, case, pdt):
    T, Hq, Hkv, D, ps, B, most, window = case
    if pdt == F32:
        B, most = B // 4, most // 4
    prob = attn_problem(B, T, Hq, Hkv, D, ps, ragged(B, most, B), pdt, seed=70 + T)
    check_large(attn, prob, pdt, window)


@pytest.mark.parametrize("pdt", [BF, F8, F32], ids=["bf16", "fp8", "f32"])
@pytest.mark.parametrize("T,Hq,Hkv,D,lens,window", [(500, 8, 2, 64, [500, 1200, 499, 3], 0), (1001, 4, 4, 128, [1001, 1500], 0),
                                                    (700, 16, 2, 128, [2000], 300)], ids=str)
def test_attention_pieces_of_prompts(attn, T, Hq, Hkv, D, lens, window, pdt):
    """Many row blocks, with what went before (or less: the first rows stand before the sequence)."""
    prob = attn_problem(len(lens), T, Hq, Hkv, D, 16, lens, pdt, seed=80 + T)
    check_large(attn, prob, pdt, window)


@pytest.mark.parametrize("pdt", [BF, F8, F32], ids=["bf16", "fp8", "f32"])
@pytest.mark.parametrize("T,Hq", [(1, 8), (3, 16)])
def test_attention_negative_scale(attn, T, Hq, pdt):
    prob = attn_problem(3, T, Hq, 2, 64, 16, [200, 3, 70], pdt, seed=90)
    check_attn(attn, prob, pdt, scale=-0.25)


# ---- the bounds-checked build on the same paths -------------------------------------------------

DEBUG_CHILD = r"""
import ctypes, json, sys
sys.path[:0] = [sys.argv[1], sys.argv[1] + "/tests"]
import test_attn_paths_gpu as t
from state_space_model_gb300 import _native, attn
import torch
assert _native.LIB_PATH.endswith("libssd_gb300_debug.so"), _native.LIB_PATH
for dt, pdt in ((t.BF, t.BF), (t.BF, t.F8), (t.F32, t.F8)):
    t.test_append_prompts(attn, 2501, 4, 2, 128, dt, pdt, 48, True, True)
    t.test_append_prompts(attn, 1301, 40, 8, 64, dt, pdt, "D", False, True)
for pdt, odt in ((t.BF, t.BF), (t.F8, t.F32), (t.F32, t.F32)):
    t.test_read_of_many(attn, 512, 2, 64, 40, pdt, odt)
    t.test_read_of_many(attn, 3, 20, 128, 300, pdt, odt)
    t.test_read_of_many(attn, 5, 4, 128, 2000, pdt, odt)
for pdt in (t.BF, t.F8, t.F32):
    t.test_attention_pieces_of_prompts(attn, 500, 8, 2, 64, [500, 1200, 499, 3], 0, pdt)
    t.test_attention_pieces_of_prompts(attn, 700, 16, 2, 128, [2000], 300, pdt)
    t.test_attention_many_tiles(attn, (4, 32, 8, 128, 64, 40, 1500, 0), pdt)
    t.test_attention_many_tiles(attn, (1, 12, 4, 64, 100, 300, 500, 0), pdt)
lib = _native.load()
st = lib.ssd_device_status(ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
print(json.dumps({"status": st, "detail": lib.ssd_last_error_detail().decode()}))
"""


def test_debug_build_on_every_path(attn):
    import json
    import os
    import subprocess
    import sys
    from state_space_model_gb300 import build
    build.build(debug_bounds=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", DEBUG_CHILD, root], env=dict(os.environ, SSD_DEBUG_BOUNDS="1"),
                       cwd=root, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    out = json.loads(r.stdout.strip().splitlines()[-1])
    assert out["status"] == 0, out["detail"]
