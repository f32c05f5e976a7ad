"""Refusals of the attention entry points, on the host: every check returns its
status and a text naming the argument before any CUDA call.  Descriptors point
at fake aligned addresses that nothing dereferences."""
import ctypes

import pytest

from state_space_model_gb300 import _native
from state_space_model_gb300._native import SsdTensor

F32, BF16, I32, F8 = 0, 1, 2, 3
BYTES = {F32: 4, BF16: 2, I32: 4, F8: 1}
INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    from state_space_model_gb300 import build
    build.build()
    return _native.load()


class Fake:
    """Descriptors of fake tensors at distinct addresses."""

    def __init__(self):
        self.at = 0x7F0000000000

    def __call__(self, shape, dtype=BF16, strides=None, shift=0):
        d = SsdTensor()
        n = 1
        packed = []
        for s in reversed(shape):
            packed.insert(0, n)
            n *= max(s, 1)
        strides = packed if strides is None else strides
        reach = 1 + sum((s - 1) * st for s, st in zip(shape, strides) if s > 0)
        d.data = self.at + shift
        self.at += (max(reach, 1) * BYTES.get(dtype, 4) + 8191) // 4096 * 4096
        d.dtype, d.ndim = dtype, len(shape)
        for i, (s, st) in enumerate(zip(shape, strides)):
            d.shape[i], d.stride[i] = s, st
        return d


def ptr(t):
    return None if t is None else ctypes.addressof(t)


def append_args(pools=BF16, x=BF16, T=5, Hq=8, Hkv=2, D=64, R=32):
    f = Fake()
    return dict(q=f((T, Hq, D), x), k=f((T, Hkv, D), x), v=f((T, Hkv, D), x), slots=f((T,), I32),
                positions=f((T,), I32), cos=f((9, R // 2), F32), sin=f((9, R // 2), F32), qw=f((D,), F32),
                kw=f((D,), F32), eps=1e-6, inter=0, kc=f((4, Hkv, 16, D), pools), vc=f((4, Hkv, 16, D), pools),
                ks=f((4, Hkv, 16), F32) if pools == F8 else None, vs=f((4, Hkv, 16), F32) if pools == F8 else None,
                out=f((T, Hq, D), x)), f


def call_append(lib, a):
    return lib.ssd_kv_append(*[ptr(a[n]) for n in ("q", "k", "v", "slots", "positions", "cos", "sin", "qw", "kw")],
                             a["eps"], a["inter"], *[ptr(a[n]) for n in ("kc", "vc", "ks", "vs", "out")], None)


def refused(lib, st, want, word):
    text = lib.ssd_last_error_detail().decode()
    assert st == want, (st, text)
    assert word in text, text


APPEND = [
    ("q", lambda f: None, INVALID, "q"),
    ("q", lambda f: f((5, 8, 64), F8), INVALID, "q"),
    ("q", lambda f: f((5, 7, 64)), INVALID, "multiple"),
    ("q", lambda f: f((5, 8, 64), strides=[512, 64, 2]), INVALID, "innermost"),
    ("q", lambda f: f((5, 8, 64), shift=8), ALIGNMENT, "q"),
    ("q", lambda f: f((5, 8, 64), strides=[516, 64, 1]), ALIGNMENT, "q"),
    ("k", lambda f: f((5, 2, 64), F32), INVALID, "k"),
    ("k", lambda f: f((4, 2, 64)), INVALID, "k"),
    ("v", lambda f: f((5, 4, 64)), INVALID, "v"),
    ("slots", lambda f: None, INVALID, "slots"),
    ("slots", lambda f: f((5,), F32), INVALID, "slots"),
    ("positions", lambda f: None, INVALID, "positions"),
    ("positions", lambda f: f((6,), I32), INVALID, "positions"),
    ("cos", lambda f: None, INVALID, "cos"),
    ("sin", lambda f: f((8, 16), F32), INVALID, "sin"),
    ("cos", lambda f: f((9, 12), F32), UNSUPPORTED, "cos"),
    ("cos", lambda f: f((9, 40), F32), UNSUPPORTED, "cos"),
    ("cos", lambda f: f((9, 0), F32), UNSUPPORTED, "cos"),
    ("qw", lambda f: f((32,), F32), INVALID, "q_weight"),
    ("kw", lambda f: f((64,), BF16), INVALID, "k_weight"),
    ("eps", lambda f: -1.0, INVALID, "eps"),
    ("eps", lambda f: float("nan"), INVALID, "eps"),
    ("kc", lambda f: f((4, 2, 16, 64), F32), INVALID, "v_cache"),
    ("kc", lambda f: f((4, 2, 16, 80)), UNSUPPORTED, "headdim"),
    ("kc", lambda f: f((4, 2, 16, 64), I32), INVALID, "k_cache"),
    ("kc", lambda f: f((4, 2, 0, 64)), INVALID, "k_cache"),
    ("kc", lambda f: f((2 ** 27, 2, 16, 64)), UNSUPPORTED, "slots"),
    ("kc", lambda f: f((4, 2, 16, 64), strides=[4096, 2048, 128, 1]), INVALID, "strides"),
    ("vc", lambda f: None, INVALID, "v_cache"),
    ("ks", lambda f: f((4, 2, 16), F32), INVALID, "scale"),
    ("out", lambda f: f((5, 8, 64), F32), INVALID, "q_out"),
    ("out", lambda f: f((5, 8, 64), strides=[512, 0, 1]), INVALID, "q_out"),
]


@pytest.mark.parametrize("name,make,status,word", APPEND, ids=lambda p: p if isinstance(p, str) else "")
def test_append_refusals(lib, name, make, status, word):
    a, f = append_args()
    a[name] = make(f)
    refused(lib, call_append(lib, a), status, word)


def test_append_refuses_overlap_and_pool_types(lib):
    a, f = append_args()
    a["out"] = a["q"]
    refused(lib, call_append(lib, a), INVALID, "overlaps")
    a, f = append_args()
    a["vc"] = a["kc"]
    refused(lib, call_append(lib, a), INVALID, "overlaps")
    a, f = append_args(pools=F32)
    refused(lib, call_append(lib, a), INVALID, "k_cache")
    a, f = append_args(pools=F8)
    a["vs"] = None
    refused(lib, call_append(lib, a), INVALID, "scale")
    a, f = append_args(pools=F8)
    a["vs"] = f((4, 2, 16), F32, strides=[64, 32, 1])
    refused(lib, call_append(lib, a), INVALID, "strides")
    a, f = append_args()
    a["kc"], a["vc"] = (f((4, 2, 16, 64), strides=[0, 1024, 64, 1]) for _ in range(2))
    refused(lib, call_append(lib, a), INVALID, "share memory")


def test_no_tokens_is_no_work(lib):
    a, _ = append_args(T=0)
    assert call_append(lib, a) == 0


def read_args(pools=BF16, out=BF16, B=3, T=11, Hkv=2, D=64):
    f = Fake()
    return dict(kc=f((4, Hkv, 16, D), pools), vc=f((4, Hkv, 16, D), pools),
                ks=f((4, Hkv, 16), F32) if pools == F8 else None, vs=f((4, Hkv, 16), F32) if pools == F8 else None,
                table=f((B, 2), I32), cu=f((B + 1,), I32), starts=f((B,), I32), k=f((T, Hkv, D), out),
                v=f((T, Hkv, D), out)), f


def call_read(lib, a):
    return lib.ssd_kv_read(*[ptr(a[n]) for n in ("kc", "vc", "ks", "vs", "table", "cu", "starts", "k", "v")], None)


READ = [
    ("table", lambda f: None, INVALID, "page_table"),
    ("table", lambda f: f((3,), I32), INVALID, "page_table"),
    ("table", lambda f: f((3, 2), F32), INVALID, "page_table"),
    ("table", lambda f: f((3, 2 ** 28), I32), UNSUPPORTED, "page_table"),
    ("cu", lambda f: f((3,), I32), INVALID, "cu_lens"),
    ("starts", lambda f: f((2,), I32), INVALID, "starts"),
    ("k", lambda f: None, INVALID, "k"),
    ("k", lambda f: f((11, 2, 64), F32), INVALID, "k"),
    ("k", lambda f: f((11, 3, 64)), INVALID, "k"),
    ("v", lambda f: f((10, 2, 64)), INVALID, "v"),
    ("v", lambda f: f((11, 2, 64), strides=[0, 64, 1]), INVALID, "v"),
    ("v", lambda f: f((11, 2, 64), shift=2), ALIGNMENT, "v"),
]


@pytest.mark.parametrize("name,make,status,word", READ, ids=lambda p: p if isinstance(p, str) else "")
def test_read_refusals(lib, name, make, status, word):
    a, f = read_args()
    a[name] = make(f)
    refused(lib, call_read(lib, a), status, word)


def test_read_refuses_overlap_and_types(lib):
    a, _ = read_args()
    a["v"] = a["k"]
    refused(lib, call_read(lib, a), INVALID, "overlaps")
    a, _ = read_args()
    a["k"] = a["v"] = a["kc"]
    refused(lib, call_read(lib, a), INVALID, "k")
    a, f = read_args(pools=F8, out=BF16)
    a["v"] = f((11, 2, 64), F32)
    refused(lib, call_read(lib, a), INVALID, "v")


def attn_args(pools=BF16, B=3, T=2, Hq=8, Hkv=2, D=64):
    f = Fake()
    x = F32 if pools == F32 else BF16
    return dict(q=f((B, T, Hq, D), x), kc=f((4, Hkv, 16, D), pools), vc=f((4, Hkv, 16, D), pools),
                ks=f((4, Hkv, 16), F32) if pools == F8 else None, vs=f((4, Hkv, 16), F32) if pools == F8 else None,
                table=f((B, 2), I32), lens=f((B,), I32), scale=0.125, window=0, out=f((B, T, Hq, D), x),
                lse=f((B, T, Hq), F32), ws=0x7E0000000000, ws_bytes=1 << 34), f


def call_attn(lib, a):
    return lib.ssd_paged_attention(*[ptr(a[n]) for n in ("q", "kc", "vc", "ks", "vs", "table", "lens")], a["scale"],
                                   a["window"], ptr(a["out"]), ptr(a["lse"]), a["ws"], a["ws_bytes"], None)


ATTN = [
    ("q", lambda f: None, INVALID, "q"),
    ("q", lambda f: f((3, 2, 8, 64), F32), INVALID, "q"),
    ("q", lambda f: f((3, 2, 7, 64)), INVALID, "multiple"),
    ("q", lambda f: f((3, 2, 8, 128)), INVALID, "q"),
    ("q", lambda f: f((3, 8, 64)), INVALID, "q"),
    ("q", lambda f: f((3, 70000, 8, 64)), UNSUPPORTED, "65535"),
    ("kc", lambda f: f((4, 2, 16, 96)), UNSUPPORTED, "headdim"),
    ("table", lambda f: f((2, 2), I32), INVALID, "page_table"),
    ("lens", lambda f: f((3,), F32), INVALID, "lens"),
    ("lens", lambda f: None, INVALID, "lens"),
    ("scale", lambda f: float("inf"), INVALID, "scale"),
    ("scale", lambda f: float("nan"), INVALID, "scale"),
    ("window", lambda f: -1, INVALID, "window"),
    ("out", lambda f: f((3, 2, 8, 64), F32), INVALID, "out"),
    ("out", lambda f: f((3, 2, 8, 64), strides=[1024, 0, 64, 1]), INVALID, "out"),
    ("lse", lambda f: f((3, 2, 7), F32), INVALID, "lse"),
    ("lse", lambda f: f((3, 2, 8), F32, strides=[32, 16, 2]), INVALID, "lse"),
]


@pytest.mark.parametrize("name,make,status,word", ATTN, ids=lambda p: p if isinstance(p, str) else "")
def test_attention_refusals(lib, name, make, status, word):
    a, f = attn_args()
    a[name] = make(f)
    refused(lib, call_attn(lib, a), status, word)


def test_attention_refuses_overlap_and_workspace(lib):
    a, _ = attn_args()
    a["out"] = a["q"]
    refused(lib, call_attn(lib, a), INVALID, "overlaps")
    need = ctypes.c_size_t()
    assert lib.ssd_paged_attention_workspace_size(3, 2, 8, 2, 64, BF16, ctypes.byref(need)) == 0
    if need.value:
        a, _ = attn_args()
        a["ws_bytes"] = need.value - 1
        refused(lib, call_attn(lib, a), WORKSPACE, "workspace")
        a, _ = attn_args()
        a["ws"] = None
        refused(lib, call_attn(lib, a), WORKSPACE, "workspace")
        a, _ = attn_args()
        a["ws"] += 64
        refused(lib, call_attn(lib, a), ALIGNMENT, "workspace")
        a, _ = attn_args()
        a["ws"] = a["kc"].data
        refused(lib, call_attn(lib, a), INVALID, "workspace")


@pytest.mark.parametrize("bad,status", [((-1, 1, 8, 2, 64, BF16), INVALID), ((1, 1, 7, 2, 64, BF16), INVALID),
                                        ((1, 1, 8, 0, 64, BF16), INVALID), ((1, 1, 8, 2, 32, BF16), UNSUPPORTED),
                                        ((1, 1, 8, 2, 64, I32), INVALID),
                                        ((1, 60000, 60000, 1, 64, BF16), UNSUPPORTED), ((70000, 1, 8, 2, 64, F8), UNSUPPORTED)])
def test_workspace_size_refusals(lib, bad, status):
    need = ctypes.c_size_t(7)
    assert lib.ssd_paged_attention_workspace_size(*bad, ctypes.byref(need)) == status
    assert need.value == 0
    assert lib.ssd_paged_attention_workspace_size(1, 1, 8, 2, 64, BF16, None) == INVALID


def test_python_names_what_it_is_given():
    import torch
    from state_space_model_gb300 import attn
    q = torch.zeros(1, 1, 4, 64)
    with pytest.raises(ValueError, match="CUDA tensors"):
        attn.paged_attention(q, torch.zeros(2, 2, 4, 64), torch.zeros(2, 2, 4, 64),
                             torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                             workspace=torch.zeros(1, dtype=torch.uint8))
    with pytest.raises(TypeError, match="torch.Tensor"):
        attn.kv_append([1], None, None, None, None, None, out=torch.zeros(1, 4, 64))
