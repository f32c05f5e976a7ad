"""Where the attention entry points' tensors may lie: keys and values of one allocation, outputs
beside inputs.  The host tests use descriptors at fake addresses, as test_attn_host.py does; a call
without tokens passes every check and launches nothing."""
import pytest
import torch

from test_attn_gpu import BF, F8, F32, attn  # noqa: F401
from test_attn_host import BF16, INVALID, append_args, call_append, lib, refused  # noqa: F401
from test_attn_host import F8 as F8_CODE

# (shape of the allocation, strides [pages, heads, slots, places] and offset of the values in it), 4 pages of
# 16 tokens, 2 heads of 64
SHARED = {
    "pages x 2": ([4096, 1024, 64, 1], 2048),
    "pages x 2, tokens first": ([4096, 64, 128, 1], 2048),
    "tokens x 2": ([4096, 64, 256, 1], 128),
    "heads x 2": ([4096, 2048, 64, 1], 1024),
    "rows x 2": ([4096, 2048, 128, 1], 64),
    "2 x pages": ([2048, 1024, 64, 1], 8192),
}


def shared_args(strides, offset, pools=BF16, T=0):
    a, f = append_args(pools=pools, T=T)
    es = 1 if pools == F8_CODE else 2
    a["kc"] = f((4, 2, 16, 64), pools, strides=strides)
    f.at += 4 * 2 * 2 * 16 * 64 * es
    a["vc"] = f((4, 2, 16, 64), pools, strides=strides)
    a["vc"].data = a["kc"].data + offset * es
    return a, f


@pytest.mark.parametrize("pools", [BF16, F8_CODE], ids=["bf16", "fp8"])
@pytest.mark.parametrize("name", SHARED)
def test_append_takes_pools_of_one_allocation(lib, name, pools):
    strides, offset = SHARED[name]
    a, _ = shared_args(strides, offset, pools)
    assert call_append(lib, a) == 0, lib.ssd_last_error_detail().decode()
    a["kc"], a["vc"] = a["vc"], a["kc"]              # values before keys
    assert call_append(lib, a) == 0, lib.ssd_last_error_detail().decode()


@pytest.mark.parametrize("name", SHARED)
def test_append_refuses_pools_that_share_elements(lib, name):
    strides, offset = SHARED[name]
    for wrong in (offset - 8, offset + 8 if offset < 8192 else 8192 - 64, 0):
        a, _ = shared_args(strides, wrong)
        refused(lib, call_append(lib, a), INVALID, "overlaps")


def test_append_outputs_beside_inputs(lib):
    """Queries out into another column range of the buffer that they come from; one column back is an overlap."""
    a, f = append_args(T=5)
    wide = f((5, 24, 64), strides=[24 * 64, 64, 1])
    for shift, meets in ((8, False), (7, True), (16, False), (17, True)):
        a["q"] = f((5, 8, 64), strides=[24 * 64, 64, 1])
        a["q"].data = wide.data
        a["out"] = f((5, 8, 64), strides=[24 * 64, 64, 1])
        a["out"].data = wide.data + shift * 128
        st = call_append(lib, a)                     # past the overlap checks, the fake addresses are refused
        assert st != 0 and ("overlaps" in lib.ssd_last_error_detail().decode()) == meets


def test_overlap_rule_against_addresses(lib):
    """Accepted pools share no address, over many layouts: every element's bytes enumerated."""
    import itertools
    import random
    rng = random.Random(5)
    taken = 0
    for _ in range(400):
        order = rng.sample(range(3), 3)
        sizes, strides, n = (3, 2, 4), [0, 0, 0], 64 * rng.choice([1, 1, 2])
        for i in order:
            strides[i] = n
            n *= sizes[i] * rng.choice([1, 1, 2])
        offset = 8 * rng.randrange(0, n // 4)
        a, f = append_args(T=0)
        for name, at in (("kc", 0), ("vc", offset)):
            a[name] = f((3, 2, 4, 64), BF16, strides=strides + [1])
            a[name].data = 0x7D0000000000 + 2 * at
        cells = [sum(i * s for i, s in zip(x, strides)) for x in itertools.product(range(3), range(2), range(4))]
        used = {c + d for c in cells for d in range(64)}
        apart = not any(c + offset + d in used for c in cells for d in range(64))
        st = call_append(lib, a)
        assert st == 0 or "overlaps" in lib.ssd_last_error_detail().decode()
        assert apart or st != 0
        taken += st == 0
    assert taken > 50


@pytest.mark.gpu
@pytest.mark.parametrize("pdt", [BF, F8, F32], ids=["bf16", "fp8", "f32"])
@pytest.mark.parametrize("layout", ["pages", "tokens", "heads", "rows"])
def test_shared_allocation_gives_the_same_results(attn, layout, pdt):
    """Append, read and attention on halves of one allocation as on two."""
    pages, Hkv, ps, D, T = 5, 2, 8, 64, 33
    dt = F32 if pdt == F32 else BF
    shape, half = {"pages": ((pages, 2, Hkv, ps, D), 1), "tokens": ((pages, ps, 2, Hkv, D), 2),
                   "heads": ((pages, Hkv, 2, ps, D), 2), "rows": ((pages, Hkv, ps, 2, D), 3)}[layout]
    both = torch.zeros(shape, device="cuda").to(pdt)
    kc, vc = both.unbind(half)
    if layout == "tokens":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    ks = vs = None
    if pdt == F8:
        ks, vs = torch.zeros(pages, 2, Hkv, ps, device="cuda").unbind(1)
    apart = [torch.zeros(pages, Hkv, ps, D, device="cuda").to(pdt) for _ in range(2)]
    sapart = [torch.zeros(pages, Hkv, ps, device="cuda") if pdt == F8 else None for _ in range(2)]
    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, 4 + 2 * Hkv, D, generator=g).to(dt).cuda()
    slots = torch.randperm(pages * ps, generator=g)[:T].to(torch.int32).cuda()
    table = torch.randperm(pages, generator=g).to(torch.int32)[None].cuda()
    lens, cu = torch.tensor([37], dtype=torch.int32).cuda(), torch.tensor([0, 37], dtype=torch.int32).cuda()
    got = []
    for k, v, s, t in ((kc, vc, ks, vs), (*apart, *sapart)):
        q = attn.kv_append(x[:, :4], x[:, 4: 4 + Hkv], x[:, 4 + Hkv:], slots, k, v, k_scale=s, v_scale=t)
        o = attn.paged_attention(q[-2:][None], k, v, table, lens, k_scale=s, v_scale=t)
        got.append([q, o, *attn.kv_read(k, v, table, cu, 37, k_scale=s, v_scale=t), k, v])
    for a, b in zip(*got):
        assert torch.equal(a.float(), b.float())
