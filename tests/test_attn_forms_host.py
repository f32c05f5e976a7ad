"""Refusals of the attention entry points' further forms, on the host: 4-bit pools with their group
scales, sections and positions of several axes, sinks.  Descriptors point at fake aligned addresses
that nothing dereferences."""
import ctypes

import pytest

from state_space_model_gb300 import _native
from test_attn_host import (ALIGNMENT, BF16, BYTES, F32, F8, I32, INVALID, UNSUPPORTED, Fake, lib,  # noqa: F401
                            ptr, refused)

F4 = _native.SSD_F4E2M1X2
BYTES.setdefault(F4, 1)


def pools(f, dt, Hkv=2, D=64, ps=16, pages=4):
    width = D // 2 if dt == F4 else D
    scaled = dt in (F8, F4)
    kw = {n: f((pages, Hkv, ps, width), dt) for n in ("kc", "vc")}
    kw.update({n: f((pages, Hkv, ps), F32) if scaled else None for n in ("ks", "vs")})
    kw.update({n: f((pages, Hkv, ps, D // 16), F8) if dt == F4 else None for n in ("kg", "vg")})
    return kw


def append_args(dt=F4, T=5, Hq=8, Hkv=2, D=64, R=32, axes=3, sections=(4, 8, 4), x=BF16):
    f = Fake()
    return dict(q=f((T, Hq, D), x), k=f((T, Hkv, D), x), v=f((T, Hkv, D), x), slots=f((T,), I32),
                positions=f((axes, T) if sections else (T,), I32), cos=f((9, R // 2), F32), sin=f((9, R // 2), F32),
                sections=sections, n=None, qw=None, kw=None, eps=1e-6, inter=0, out=f((T, Hq, D), x),
                **pools(f, dt, Hkv, D)), f


def call_append(lib, a):
    s = a["sections"]
    s = (ctypes.c_int32 * len(s))(*s) if s else None
    n = a["n"] if a["n"] is not None else len(a["sections"] or ())
    return lib.ssd_kv_append_ex(*[ptr(a[m]) for m in ("q", "k", "v", "slots", "positions", "cos", "sin")], s, n,
                                ptr(a["qw"]), ptr(a["kw"]), a["eps"], a["inter"],
                                *[ptr(a[m]) for m in ("kc", "vc", "ks", "vs", "kg", "vg", "out")], None)


GROUPS = [
    ("kg", lambda f: None, INVALID, "k_group_scale"),
    ("vg", lambda f: None, INVALID, "v_group_scale"),
    ("kg", lambda f: f((4, 2, 16, 4), F32), INVALID, "k_group_scale"),
    ("kg", lambda f: f((4, 2, 16, 8), F8), INVALID, "k_group_scale"),
    ("vg", lambda f: f((4, 2, 8, 4), F8), INVALID, "v_group_scale"),
    ("kg", lambda f: f((4, 2, 16), F8), INVALID, "k_group_scale"),
    ("kg", lambda f: f((4, 2, 16, 4), F8, shift=2), ALIGNMENT, "k_group_scale"),
    ("kg", lambda f: f((4, 2, 16, 4), F8, strides=[160, 80, 5, 1]), ALIGNMENT, "k_group_scale"),
    ("vg", lambda f: f((4, 2, 16, 4), F8, strides=[256, 128, 8, 2]), INVALID, "v_group_scale"),
    ("vg", lambda f: f((4, 2, 16, 4), F8, strides=[256, 128, 8, 1]), INVALID, "strides"),
    ("ks", lambda f: None, INVALID, "scale"),
    ("kc", lambda f: f((4, 2, 16, 64), F4), INVALID, "v_cache"),
    ("kc", lambda f: f((4, 2, 16, 64), F8), INVALID, "v_cache"),
]


@pytest.mark.parametrize("name,make,status,word", GROUPS, ids=lambda p: p if isinstance(p, str) else "")
@pytest.mark.parametrize("which", ["append", "read", "attention"])
def test_group_scales(lib, which, name, make, status, word):
    make_args, call = {"append": (append_args, call_append), "read": (read_args, call_read),
                       "attention": (attn_args, call_attn)}[which]
    a, f = make_args()
    a[name] = make(f)
    refused(lib, call(lib, a), status, word)


@pytest.mark.parametrize("dt", [BF16, F8])
@pytest.mark.parametrize("which", ["append", "read", "attention"])
def test_group_scales_only_with_4_bit_pools(lib, which, dt):
    make_args, call = {"append": (append_args, call_append), "read": (read_args, call_read),
                       "attention": (attn_args, call_attn)}[which]
    a, f = make_args(dt)
    a["kg"], a["vg"] = (f((4, 2, 16, 4), F8) for _ in range(2))
    refused(lib, call(lib, a), INVALID, "group_scale")


APPEND = [
    (dict(sections=(4, 8, 3)), INVALID, "sections"),
    (dict(sections=(4, 8, 4, 1)), INVALID, "sections[3]"),
    (dict(sections=(4, 0, 12)), INVALID, "sections[1]"),
    (dict(sections=(4, -4, 16)), INVALID, "sections[1]"),
    (dict(sections=(2 ** 31 - 1, 1)), INVALID, "sections[0]"),
    (dict(sections=None, n=3), INVALID, "sections"),
    (dict(n=-1), INVALID, "sections"),
    (dict(axes=1), UNSUPPORTED, "axes"),
    (dict(axes=5), UNSUPPORTED, "axes"),
    (dict(axes=0), UNSUPPORTED, "axes"),
]


@pytest.mark.parametrize("change,status,word", APPEND, ids=str)
def test_sections(lib, change, status, word):
    change = dict(change)
    n = change.pop("n", None)
    a, _ = append_args(**change)
    a["n"] = n
    refused(lib, call_append(lib, a), status, word)


def test_positions_of_several_axes(lib):
    a, f = append_args()
    a["positions"] = f((5,), I32)
    refused(lib, call_append(lib, a), INVALID, "positions")
    a, f = append_args()
    a["positions"] = f((3, 6), I32)
    refused(lib, call_append(lib, a), INVALID, "positions")
    a, f = append_args()
    a["positions"] = f((3, 5), I32, strides=[8, 1])
    refused(lib, call_append(lib, a), INVALID, "positions")
    a, f = append_args(sections=None)
    a["positions"] = f((3, 5), I32)
    refused(lib, call_append(lib, a), INVALID, "positions")
    a, _ = append_args()
    a["positions"] = a["cos"] = a["sin"] = None
    refused(lib, call_append(lib, a), INVALID, "sections")


def test_written_group_scales_share_no_memory(lib):
    a, f = append_args()
    a["vg"] = a["kg"]
    refused(lib, call_append(lib, a), INVALID, "overlaps")
    a, f = append_args()
    a["kg"], a["vg"] = (f((4, 2, 16, 4), F8, strides=[0, 64, 4, 1]) for _ in range(2))
    refused(lib, call_append(lib, a), INVALID, "share memory")
    a, f = append_args()
    a["kg"].data = a["q"].data
    refused(lib, call_append(lib, a), INVALID, "overlaps")


def test_no_tokens_is_no_work(lib):
    for dt in (BF16, F8, F4):
        a, _ = append_args(dt, T=0)
        assert call_append(lib, a) == 0


def read_args(dt=F4, out=BF16, B=3, T=11, Hkv=2, D=64):
    f = Fake()
    return dict(table=f((B, 2), I32), cu=f((B + 1,), I32), starts=f((B,), I32), k=f((T, Hkv, D), out),
                v=f((T, Hkv, D), out), **pools(f, dt, Hkv, D)), f


def call_read(lib, a):
    return lib.ssd_kv_read_ex(*[ptr(a[n]) for n in ("kc", "vc", "ks", "vs", "kg", "vg", "table", "cu", "starts",
                                                    "k", "v")], None)


def test_read(lib):
    a, f = read_args()
    a["k"] = f((11, 2, 32), BF16)
    refused(lib, call_read(lib, a), INVALID, "k")
    a, f = read_args()
    a["v"] = f((11, 2, 64), F32)
    refused(lib, call_read(lib, a), INVALID, "v")
    a, f = read_args()
    a["k"] = a["kg"]
    refused(lib, call_read(lib, a), INVALID, "k")
    a, f = read_args(out=F8)
    refused(lib, call_read(lib, a), INVALID, "k")
    a, f = read_args()
    a["k"].data = a["kg"].data
    refused(lib, call_read(lib, a), INVALID, "overlaps")


def attn_args(dt=F4, B=3, T=2, Hq=8, Hkv=2, D=64):
    f = Fake()
    x = F32 if dt == F32 else BF16
    return dict(q=f((B, T, Hq, D), x), table=f((B, 2), I32), lens=f((B,), I32), scale=0.125, window=0, sinks=0,
                out=f((B, T, Hq, D), x), lse=None, ws=0x7E0000000000, ws_bytes=1 << 34, **pools(f, dt, Hkv, D)), f


def call_attn(lib, a):
    return lib.ssd_paged_attention_ex(*[ptr(a[n]) for n in ("q", "kc", "vc", "ks", "vs", "kg", "vg", "table", "lens")],
                                      a["scale"], a["window"], a["sinks"], ptr(a["out"]), ptr(a["lse"]), a["ws"],
                                      a["ws_bytes"], None)


def test_attention(lib):
    a, f = attn_args()
    a["q"] = a["out"] = None
    refused(lib, call_attn(lib, a), INVALID, "q")
    a, f = attn_args()
    a["q"] = f((3, 2, 8, 64), F32)
    refused(lib, call_attn(lib, a), INVALID, "q")
    a, f = attn_args()
    a["q"] = f((3, 2, 8, 32), BF16)
    refused(lib, call_attn(lib, a), INVALID, "q")
    a, f = attn_args()
    a["sinks"] = -1
    refused(lib, call_attn(lib, a), INVALID, "sinks")
    a, f = attn_args()
    a["window"] = -1
    refused(lib, call_attn(lib, a), INVALID, "window")
    a, f = attn_args()
    a["kc"], a["vc"] = (f((4, 2, 16, 24), F4) for _ in range(2))
    refused(lib, call_attn(lib, a), UNSUPPORTED, "headdim")
    a, f = attn_args()
    a["out"].data = a["vg"].data
    refused(lib, call_attn(lib, a), INVALID, "overlaps")


def test_python_refuses(lib):
    import torch
    from state_space_model_gb300 import attn
    x = torch.zeros(1, 1, 64)
    pool = torch.zeros(2, 1, 4, 64)
    with pytest.raises((ValueError, TypeError), match="sections"):
        attn.kv_append(x, x, x, torch.zeros(1, dtype=torch.int32), pool, pool, sections=())
    with pytest.raises((ValueError, TypeError), match="sections"):
        attn.kv_append(x, x, x, torch.zeros(1, dtype=torch.int32), pool, pool, sections=[1, "a"])
    with pytest.raises((ValueError, TypeError), match="sections"):
        attn.kv_append(x, x, x, torch.zeros(1, dtype=torch.int32), pool, pool, sections=3)
    with pytest.raises(ValueError, match="cannot be read"):
        attn.kv_read(pool.to(torch.float8_e4m3fn), pool, x, x, 1, dtype=torch.float16)
