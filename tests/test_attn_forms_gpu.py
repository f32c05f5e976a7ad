"""The attention cache's further forms on the GPU: pools of 4-bit codes, sinks beside a window,
positions of several axes, and pieces of prompts on the tensor cores' own path.

The references are float64 on the GPU, from the definitions.  Bounds are those that test_attn_gpu.py
derives; a 4-bit element adds nothing to them in attention, its code times its group's scale being
exact in fp16.  For the write: the row's scale within 2^-17, a group's scale one e4m3 rounding (2^-4,
at least half the smallest step, 2^-10) of gmax / (6 scale), a code the nearest to what it stands for
but for the error of keys before it (2^-15 of the row's largest).
"""
import math

import pytest
import torch

from test_attn_gpu import BF, F8, F32, U, append_inputs, attn, rot_tables  # noqa: F401

pytestmark = pytest.mark.gpu

F4 = torch.float4_e2m1fn_x2
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
IDS = {BF: "bf16", F8: "fp8", F32: "f32", F4: "fp4"}
TYPES = pytest.mark.parametrize("pdt", [BF, F8, F32, F4], ids=lambda t: IDS[t])


def raw(x):
    return x.view(torch.uint8) if x.dtype in (F8, F4) else x


class Pools:
    """Key and value pools of any type with their scales; values for use, and arguments for calls."""

    def __init__(self, pages, Hkv, ps, D, pdt, seed=None, token_major=False):
        self.pdt, self.D, self.ps, self.Hkv = pdt, D, ps, Hkv
        g = torch.Generator(device="cuda").manual_seed(0 if seed is None else seed)

        def make(shape, dtype, fill):
            if token_major and len(shape) == 4:
                shape = (shape[0], shape[2], shape[1], shape[3])
            t = fill(shape, dtype)
            return t.transpose(1, 2) if token_major and len(shape) == 4 else t

        rand = lambda shape, dt: torch.randn(shape, generator=g, device="cuda")
        self.pools, self.scales, self.groups = [], [None, None], [None, None]
        for i in range(2):
            shape = (pages, Hkv, ps, D)
            if pdt == F4:
                bits = make((pages, Hkv, ps, D // 2), None, lambda s, _: torch.randint(
                    0, 256, s, generator=g, device="cuda", dtype=torch.uint8))
                self.pools.append(bits.view(F4))
                self.scales[i] = torch.rand((pages, Hkv, ps), generator=g, device="cuda") * 2e-3 + 5e-4
                groups = make((pages, Hkv, ps, D // 16), None, lambda s, _: torch.randint(
                    0x40, 0x78, s, generator=g, device="cuda", dtype=torch.uint8))   # 2 to 224
                self.groups[i] = groups.view(F8)
            elif pdt == F8:
                x = make(shape, None, rand).clamp(-6, 6) * 64
                self.pools.append(x.to(F8))
                self.scales[i] = torch.rand((pages, Hkv, ps), generator=g, device="cuda") * 0.02 + 0.005
            else:
                self.pools.append(make(shape, None, rand).to(pdt))

    @property
    def kw(self):
        return dict(k_scale=self.scales[0], v_scale=self.scales[1], k_group_scale=self.groups[0],
                    v_group_scale=self.groups[1])

    def rows(self, i, page, at):
        """float64 rows [..., Hkv, D] at places (page, at)."""
        x = raw(self.pools[i])[page, :, at]
        if self.pdt == F4:
            grid = torch.tensor(GRID + [-v for v in GRID], dtype=torch.float64, device="cuda")
            x = grid[torch.stack([x % 16, x // 16], -1).long()].flatten(-2)
            x = x * raw(self.groups[i])[page, :, at].view(F8).double().repeat_interleave(16, -1)
        elif self.pdt == F8:
            x = x.view(F8).double()
        x = x.double()
        return x if self.scales[i] is None else x * self.scales[i][page, :, at].double()[..., None]

    def poison(self, page, at, head=slice(None), value_only=False):
        """NaN at places (page, at)."""
        for i in (1,) if value_only else (0, 1):
            if self.pdt == F4:
                raw(self.groups[i])[page, head, at] = 0x7F
            else:
                raw(self.pools[i])[page, head, at] = 0x7F if self.pdt == F8 else float("nan")

    def poison_unused(self, live):
        """NaN and infinite scales in every slot not in `live` [pages, ps]."""
        dead = ~live[:, None].expand(-1, self.Hkv, -1).cuda()
        for i in range(2):
            if self.pdt in (F8, F4):
                t = raw(self.groups[i] if self.pdt == F4 else self.pools[i])
                t[dead] = 0x7F
                self.scales[i][dead] = float("inf")
            else:
                self.pools[i][dead] = float("nan")


def problem(B, T, Hq, Hkv, D, ps, lens, pdt, seed, poison=True, **kw):
    """(q, pools, table, lens): a shuffled table; slots that no sequence uses hold NaN (poison)."""
    g = torch.Generator().manual_seed(seed)
    used = [-(-max(n, 0) // ps) for n in lens]
    pools = Pools(sum(used) + 2, Hkv, ps, D, pdt, seed, **kw)
    table = torch.full((B, max(used + [1])), -1, dtype=torch.int32)
    order = torch.randperm(sum(used) + 2, generator=g).tolist()
    live = torch.zeros(sum(used) + 2, ps, dtype=torch.bool)
    for b, n in enumerate(used):
        for i in range(n):
            table[b, i] = order.pop()
            live[table[b, i], : min(ps, lens[b] - i * ps)] = True
    if poison:
        pools.poison_unused(live)
    q = torch.randn(B, T, Hq, D, generator=g).to(F32 if pdt == F32 else BF).cuda()
    return q, pools, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()


def check(attn, prob, window=0, sinks=0, scale=None, **kw):
    q, pools, table, lens = prob
    out, lse = attn.paged_attention(q, *pools.pools, table, lens, window=window, sinks=sinks, scale=scale,
                                    return_lse=True, **pools.kw, **kw)
    B, T, Hq, D = q.shape
    Hkv, ps, f32 = pools.Hkv, pools.ps, pools.pdt == F32
    scale = D ** -0.5 if scale is None else scale
    ut, uo = 2.0 ** -24 if f32 else 2.0 ** -22, U[q.dtype]
    assert torch.isfinite(out).all() and not torch.isnan(lse).any()
    for b, n in enumerate(lens.tolist()):
        n = max(n, 0)
        pos = torch.arange(min(n, table.shape[1] * ps), device="cuda")
        page = table[b, pos // ps].long()
        there = (page >= 0) & (page < pools.pools[0].shape[0])
        page, at = page.clamp(0, pools.pools[0].shape[0] - 1), pos % ps
        K, V = (pools.rows(i, page, at).masked_fill(~there[:, None, None], 0).transpose(0, 1) for i in (0, 1))
        for t0 in range(0, T, 64):
            t = torch.arange(t0, min(t0 + 64, T), device="cuda")
            e = n - T + t[:, None]
            see = (pos <= e) & there
            if window:
                see &= (pos > e - window) | (pos < sinks)
            # what no row of these sees may be NaN
            some = see.any(0)
            k, v, sn = K[:, some], V[:, some], see[:, some]
            seen = sn.sum(-1)[None, :, None].double()
            Q = q[b, t].double().view(len(t), Hkv, Hq // Hkv, D).permute(1, 0, 2, 3)
            o = out[b, t].double().view(len(t), Hkv, Hq // Hkv, D).permute(1, 0, 2, 3)
            l = lse[b, t].double().view(len(t), Hkv, Hq // Hkv).permute(1, 0, 2)
            none = (seen == 0).expand(l.shape)
            assert (o[none] == 0).all() and torch.isneginf(l[none]).all()
            if not some.any():
                continue
            m = ~sn[None, :, None]
            s = (torch.einsum("htgd,hnd->htgn", Q, k) * scale).masked_fill(m, -math.inf)
            big = (torch.einsum("htgd,hnd->htgn", Q.abs(), k.abs()) * abs(scale)).masked_fill(m, 0).amax(-1)
            rl = torch.logsumexp(s, -1)
            p = torch.exp(s - torch.where(none, 0.0, rl)[..., None])
            ref = torch.einsum("htgn,hnd->htgd", p, v)
            vmax = v.abs().amax(-1)[:, None].masked_fill(~sn[None], 0).amax(-1)[..., None]
            ds = (D + 8) * ut * big
            bound = vmax * (2 * ds + (seen + 8) * ut + (0 if f32 else 2.0 ** -8))
            assert ((o - ref).abs() <= bound[..., None] * (1 + uo) + uo * ref.abs()).all()
            assert ((l - rl).abs() <= ds + seen * ut + 2.0 ** -21 * (1 + rl.abs()))[~none].all()
    return out, lse


# ---- attention: 4-bit pools, sinks -----------------------------------------------------------

CASES = [
    # (T, Hq, Hkv, D, ps, lens, window, sinks)
    (1, 1, 1, 64, 16, [1], 0, 0),
    (1, 4, 4, 128, 64, [1, 2, 127, 128, 129], 0, 0),
    (1, 8, 1, 128, 16, [0, 5, 257, 16], 0, 0),
    (1, 6, 2, 64, 24, [100, 23, 24, 25, 0, 191], 30, 1),
    (1, 20, 4, 128, 7, [333, 1], 0, 0),
    (1, 64, 4, 64, 32, [257, 700], 64, 4),
    (1, 16, 1, 128, 128, [1000, 0, 3], 1, 1),
    (1, 40, 2, 128, 100, [512, 900], 100, 300),      # 20 rows a head; sinks beyond the window's start
    (1, 37, 1, 64, 1, [77, 128], 5, 3),              # 37 rows, pages of one token
    (2, 8, 8, 128, 16, [1, 2, 40, 0], 0, 0),         # rows before the first position
    (3, 24, 4, 64, 48, [2, 300], 40, 10000),         # more sinks than positions
    (4, 32, 4, 128, 16, [3, 65, 400], 32, 128),      # sinks that end with a tile
    (8, 16, 2, 128, 64, [8, 7, 500], 100, 129),
    (5, 70, 7, 64, 16, [150, 4], 0, 0),
    (17, 12, 3, 128, 32, [17, 90, 16, 600], 200, 33),
    (100, 8, 2, 64, 16, [100, 130, 900], 50, 7),     # a piece of a prompt
    (1, 8, 2, 128, 16, [3000, 20, 0, 1, 2000], 50, 4),
    (9, 16, 2, 64, 64, [2000, 9], 128, 128),
]


@TYPES
@pytest.mark.parametrize("case", CASES, ids=str)
def test_attention_matches_definition(attn, case, pdt):
    T, Hq, Hkv, D, ps, lens, window, sinks = case
    check(attn, problem(len(lens), T, Hq, Hkv, D, ps, lens, pdt, 100 + T + Hq), window, sinks)


@TYPES
def test_sinks_without_a_window_or_inside_it_change_nothing(attn, pdt):
    q, pools, table, lens = prob = problem(4, 3, 8, 2, 64, 16, [400, 3, 90, 0], pdt, 7)
    call = lambda **kw: attn.paged_attention(q, *pools.pools, table, lens, **pools.kw, **kw)
    assert torch.equal(call(sinks=50), call())
    assert torch.equal(call(window=10 ** 6, sinks=3), call(window=10 ** 6))
    big = check(attn, prob, 20, 10 ** 12)[0]         # everything is a sink
    err = (big.float() - call().float()).abs().max()
    assert err <= 2.0 ** -6 * call().float().abs().max()


@pytest.mark.parametrize("pdt", [BF, F4], ids=lambda t: IDS[t])
def test_many_tiles_and_items(attn, pdt):
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(1, 6000, (70,), generator=g).tolist()
    lens[3], lens[40], lens[-1] = 0, 9000, 2
    check(attn, problem(70, 1, 32, 8, 128, 64, lens, pdt, 21))
    check(attn, problem(70, 2, 24, 4, 64, 24, lens, pdt, 22), 700, 130)


@TYPES
@pytest.mark.parametrize("T,D", [(1, 128), (5, 64)])
def test_missing_pages(attn, pdt, T, D):
    q, pools, table, lens = prob = problem(3, T, 4, 2, D, 8, [700, 100, 30], pdt, 14, poison=False)
    table[0, 30:80], table[0, 0], table[1, :] = -1, pools.pools[0].shape[0], -7
    table[2, 1] = 2 ** 31 - 1
    lens[2] = 10 ** 6                                # beyond the table: all of its pages' slots are seen
    check(attn, prob)
    check(attn, prob, 100, 50)                       # freed between the sinks and the window
    check(attn, prob, 100, 1)                        # the sinks' page is missing


@TYPES
@pytest.mark.parametrize("D", [64, 128])
def test_unseen_nan_stays_out(attn, pdt, D):
    T, n, ps = 4, 400, 16
    q, pools, table, lens = problem(1, T, 8, 2, D, ps, [n], pdt, 15)
    call = lambda **kw: attn.paged_attention(q, *pools.pools, table, lens, return_lse=True, **pools.kw, **kw)
    kinds = [dict(), dict(window=37), dict(window=37, sinks=20)]
    good = [call(**k) for k in kinds]
    # the last row's own position
    pools.poison(int(table[0, (n - 1) // ps]), (n - 1) % ps)
    for (o, l), k in zip(good, kinds):
        b, lb = call(**k)
        assert torch.equal(b[:, :3], o[:, :3]) and torch.equal(lb[:, :3], l[:, :3])
        assert torch.isnan(b[:, 3]).all()
    # a value between the sinks and every window, and one that only the first row's window holds
    q, pools, table, lens = problem(1, T, 8, 2, D, ps, [n], pdt, 16)
    kw = dict(window=37, sinks=20)
    good = call(**kw)[0]
    pools.poison(int(table[0, 20 // ps]), 20 % ps)
    assert torch.equal(call(**kw)[0], good)
    at = n - T + 1 - 37
    pools.poison(int(table[0, at // ps]), at % ps, value_only=True)
    bad = call(**kw)[0]
    assert torch.equal(bad[:, 1:], good[:, 1:]) and not torch.isfinite(bad[:, 0]).any()


@pytest.mark.parametrize("D", [64, 128])
def test_leftovers_of_other_calls_stay_out(attn, D):
    q, bad, table, lens = problem(64, 1, 8, 2, D, 16, [512] * 64, F4, 30)
    for i in range(2):
        raw(bad.groups[i])[:] = 0x7F
    for T, Hq in ((1, 2), (1, 24), (1, 40), (1, 100), (3, 20)):
        prob = problem(6, T, Hq, 2, D, 16, [1, 5, 16, 17, 33, 49], F4, 31 + Hq)
        attn.paged_attention(q, *bad.pools, table, lens, **bad.kw)
        check(attn, prob)


@pytest.mark.parametrize("T,Hq", [(1, 8), (3, 16), (1, 64)])
@pytest.mark.parametrize("scale", [-0.25, 0.0, 30.0])
def test_scales_of_scores(attn, T, Hq, scale):
    check(attn, problem(3, T, Hq, 2, 64, 16, [200, 3, 70], F4, 90), scale=scale)


def test_extreme_row_scales(attn):
    """Scales of tokens over the whole range of fp32, each row's own."""
    for lo, hi in ((-80, -70), (60, 100), (-60, 60)):
        q, pools, table, lens = prob = problem(2, 1, 8, 2, 128, 16, [150, 64], F4, 40)
        g = torch.Generator(device="cuda").manual_seed(3)
        e = torch.rand(pools.scales[1].shape, generator=g, device="cuda") * (hi - lo) + lo
        pools.scales[1].copy_(torch.exp2(e - 8))
        out = attn.paged_attention(q, *pools.pools, table, lens, **pools.kw)
        for b, n in enumerate(lens.tolist()):
            pos = torch.arange(n, device="cuda")
            K, V = (pools.rows(i, table[b, pos // 16].long(), pos % 16).transpose(0, 1) for i in (0, 1))
            Q = q[b, 0].double().view(2, 4, 128)
            p = torch.softmax(torch.einsum("hgd,hnd->hgn", Q, K) * 128 ** -0.5, -1)
            ref = torch.einsum("hgn,hnd->hgd", p, V).view(8, 128)
            # an fp16 weight errs by 2^-12 of it, at least 2^-25 of the largest (2^8 / 2^8 .. + 2^13), and
            # the sum over n positions by n 2^-22
            most = torch.einsum("hgn,hnd->hgd", p, V.abs()).view(8, 128)
            top = (p * V.abs().amax(-1)[:, None]).amax(-1).view(8, 1)
            bound = (2.0 ** -8 + 2.0 ** -11 + n * 2.0 ** -22 + 2.0 ** -12) * most + n * 2.0 ** -22 * top
            assert ((out[b, 0].double() - ref).abs() <= bound).all()


def test_token_major_pools_and_views(attn):
    """Pools laid out token by token, queries and outputs as views of wider tensors."""
    for D in (64, 128):
        q, pools, table, lens = prob = problem(2, 2, 8, 2, D, 16, [277, 30], F4, 17, token_major=True)
        want, _ = check(attn, prob, 60, 4)
        wide = torch.zeros(2, 2, 12, D + 32, dtype=BF, device="cuda")
        wide[:, :, 2:10, :D] = q
        outw = torch.zeros(2, 3, 8, D + 8, dtype=BF, device="cuda")
        got = attn.paged_attention(wide[:, :, 2:10, :D], *pools.pools, table, lens, window=60, sinks=4,
                                   out=outw[:, :2, :, :D], **pools.kw)
        assert torch.equal(got, want) and (outw[:, 2] == 0).all() and (outw[..., D:] == 0).all()


def test_offsets_beyond_32_bits(attn):
    """4-bit pools of more than 2^32 bytes, the sequence in the last pages."""
    pages, Hkv, ps, D = 8400, 8, 1024, 128
    if torch.cuda.mem_get_info()[0] < 3 * pages * Hkv * ps * D:
        pytest.skip("not enough device memory")
    q, pools, table, lens = problem(1, 1, 8, Hkv, D, ps, [1500], F4, 18)
    want = attn.paged_attention(q, *pools.pools, table, lens, **pools.kw)
    big = [torch.empty(pages, Hkv, ps, D // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    gr = [torch.empty(pages, Hkv, ps, D // 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.empty(pages, Hkv, ps, device="cuda") for _ in range(2)]
    far = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32).cuda()
    for i in range(2):
        for new, old in ((big[i], raw(pools.pools[i])), (gr[i], raw(pools.groups[i])), (sc[i], pools.scales[i])):
            new[far[0].long()] = old[table[0].long()]
    kw = dict(k_scale=sc[0], v_scale=sc[1], k_group_scale=gr[0].view(F8), v_group_scale=gr[1].view(F8))
    views = [b.view(F4) for b in big]
    assert torch.equal(attn.paged_attention(q, *views, far, lens, **kw), want)
    cu = torch.tensor([0, 1500], dtype=torch.int32).cuda()
    near = attn.kv_read(*pools.pools, table, cu, 1500, **pools.kw)
    for a, b in zip(attn.kv_read(*views, far, cu, 1500, **kw), near):
        assert torch.equal(a, b)
    x = torch.randn(2, Hkv, D, device="cuda").to(BF)
    slots = torch.tensor([pages * ps - 1, (pages - 1) * ps], dtype=torch.int32).cuda()
    attn.kv_append(x, x, x, slots, *views, **kw)
    small = Pools(1, Hkv, ps, D, F4)
    attn.kv_append(x, x, x, torch.tensor([ps - 1, 0], dtype=torch.int32).cuda(), *small.pools, **small.kw)
    for i in range(2):
        for a, b in ((big[i], raw(small.pools[i])), (gr[i], raw(small.groups[i])), (sc[i], small.scales[i])):
            assert torch.equal(a[-1, :, [0, ps - 1]], b[0, :, [0, ps - 1]])


# ---- pieces of prompts (enough row blocks for the tensor cores' own path) ------------------------

PROMPTS = [
    # (T, Hq, Hkv, D, ps, lens, window, sinks)
    (500, 8, 2, 64, 16, [500, 1200, 499, 3, 0], 0, 0),
    (1001, 4, 4, 128, 64, [1001, 1500, 1003], 0, 0),
    (700, 16, 2, 128, 24, [2000], 300, 0),
    (700, 16, 2, 128, 24, [2000, 650], 300, 5),
    (300, 40, 8, 64, 7, [1700, 300, 301, 40], 129, 200),
    (130, 8, 8, 128, 1, [130, 257, 128, 640, 129], 128, 1),
    (128, 8, 8, 128, 128, [128, 5000, 1, 127, 200], 1, 1),
    (257, 6, 6, 64, 100, [257, 1300, 256, 255, 30, 4000, 1], 1000, 64),
    (90, 33, 11, 128, 32, [90, 3000, 91, 0], 500, 10000),
    # a whole round of items and halved ones behind it; a half without rows; 16 positions in all
    (1400, 32, 8, 128, 16, [1411], 0, 0),
    (1400, 32, 8, 64, 16, [3000], 400, 20),
    (90, 8, 8, 128, 16, [300] * 12, 0, 0),
    (300, 32, 8, 128, 16, [16], 0, 0),
    (300, 32, 8, 64, 32, [70, 64, 1], 33, 7),
]


@pytest.mark.parametrize("case", PROMPTS, ids=str)
def test_pieces_of_prompts(attn, case):
    T, Hq, Hkv, D, ps, lens, window, sinks = case
    check(attn, problem(len(lens), T, Hq, Hkv, D, ps, lens, BF, 200 + T), window, sinks)


@pytest.mark.parametrize("scale", [-0.25, 0.0, 30.0])
def test_pieces_of_prompts_scales(attn, scale):
    check(attn, problem(5, 300, 8, 4, 128, 16, [300, 900, 301, 20, 555], BF, 77), 200, 9, scale=scale)


@pytest.mark.parametrize("D", [64, 128])
def test_pieces_of_prompts_missing_pages(attn, D):
    q, pools, table, lens = prob = problem(4, 300, 16, 4, D, 8, [1700, 1000, 310, 600], BF, 14, poison=False)
    table[0, 30:80], table[0, 0], table[1, :], table[3, 70] = -1, pools.pools[0].shape[0], -7, -1
    table[2, 1] = 2 ** 31 - 1
    lens[2] = 1700                                   # beyond what its table names, the last page's slots included
    check(attn, prob)
    check(attn, prob, 100, 50)
    check(attn, prob, 100, 1)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 0), (200, 9)])
def test_pieces_of_prompts_unseen_values_stay_out(attn, D, bad, window, sinks):
    """An infinity or NaN among the values reaches the rows that see it, and no others."""
    T, Hq, Hkv, ps, n = 300, 32, 8, 16, 900
    for at in (0, 3, 400, 401, 550, 700, 898, 899):
        q, pools, table, lens = problem(3, T, Hq, Hkv, D, ps, [n, 640, 300], BF, 15)
        call = lambda: attn.paged_attention(q, *pools.pools, table, lens, window=window, sinks=sinks)
        good = call()
        pools.pools[1][int(table[0, at // ps]), 2, at % ps, 7] = bad
        got = call()
        e = n - T + torch.arange(T, device="cuda")
        see = e >= at
        if window:
            see &= (at > e - window) | (at < sinks)
        G = Hq // Hkv
        hit = torch.zeros(got.shape, dtype=torch.bool, device="cuda")
        hit[0, :, 2 * G: 3 * G, 7] = see[:, None]
        assert torch.equal(got[~hit], good[~hit])
        assert not torch.isfinite(got[hit]).any()


def test_pieces_of_prompts_repeat_bit_for_bit(attn):
    q, pools, table, lens = problem(3, 400, 16, 4, 128, 16, [1500, 400, 900], BF, 19)
    call = lambda **kw: attn.paged_attention(q, *pools.pools, table, lens, window=500, sinks=4, return_lse=True, **kw)
    want, lw = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            got, lg = call()
            s.synchronize()
            assert torch.equal(got, want) and torch.equal(lg, lw)


def test_pieces_of_prompts_two_streams_at_once(attn):
    probs = [problem(3, 400, 16, 4, D, 16, [1500, 400, 900], BF, 19 + D) for D in (64, 128)]
    call = lambda p: attn.paged_attention(p[0], *p[1].pools, p[2], p[3], window=500, sinks=4)
    want = [call(p) for p in probs]
    streams = [torch.cuda.Stream() for _ in probs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(call(probs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_pieces_of_prompts_views(attn):
    q, pools, table, lens = problem(2, 300, 16, 4, 64, 16, [1500, 300], BF, 23, token_major=True)
    want, _ = check(attn, (q, pools, table, lens), 500, 4)
    wide = torch.zeros(2, 300, 20, 96, dtype=BF, device="cuda")
    wide[:, :, 2:18, :64] = q
    outw = torch.zeros(2, 301, 16, 72, dtype=BF, device="cuda")
    got = attn.paged_attention(wide[:, :, 2:18, :64], *pools.pools, table, lens, window=500, sinks=4,
                               out=outw[:, :300, :, :64])
    assert torch.equal(got, want) and (outw[:, 300] == 0).all() and (outw[..., 64:] == 0).all()


@pytest.mark.parametrize("size", [1e2, 1e4, 1e10, 1e17])
@pytest.mark.parametrize("D", [64, 128])
def test_pieces_of_prompts_huge_scores_are_one_hot(attn, size, D):
    """Finite scores so large that one position has all the weight: the output is its value (rounded to
    16 bits at most twice, as a weight and as the result), whatever the size.  Rows of keys that are
    powers of two apart, so that a row's largest score is its next one's double."""
    T, Hq, Hkv, n = 1300, 32, 8, 1500
    q, pools, table, lens = problem(1, T, Hq, Hkv, D, 16, [n], BF, 61)
    k = raw(pools.pools[0])
    g = torch.Generator(device="cuda").manual_seed(3)
    # position j's key: +-2^(j % 12) in one place, the same place as the queries' only one
    flat = table[0].long()
    j = torch.arange(n, device="cuda")
    order = torch.rand(n, generator=g, device="cuda")
    keys = torch.zeros(n, D, device="cuda", dtype=BF)
    keys[:, 3] = torch.exp2(j % 12).to(BF) * torch.where(order < 0.5, -1.0, 1.0).to(BF)
    k[flat[j // 16], :, j % 16] = keys[:, None]
    q.zero_()
    q[..., 3] = size
    out, lse = attn.paged_attention(q, *pools.pools, table, lens, scale=1.0, window=200, sinks=7, return_lse=True)
    own = n - T + torch.arange(T, device="cuda")
    see = (j <= own[:, None]) & ((j > own[:, None] - 200) | (j < 7))
    score = torch.where(see, keys[:, 3].double(), -torch.inf)
    top = score.amax(1, keepdim=True)
    weight = (score == top).double()
    weight = weight / weight.sum(1, keepdim=True)
    v = pools.rows(1, flat[j // 16], j % 16)                       # [n, Hkv, D]
    want = torch.einsum("tj,jhd->thd", weight, v).repeat_interleave(Hq // Hkv, 1)
    assert ((out[0].double() - want).abs() <= 2.0 ** -7 * torch.einsum("tj,jhd->thd", weight, v.abs()).repeat_interleave(
        Hq // Hkv, 1) + 1e-30).all()
    ref = top * float(torch.tensor(size).to(BF)) + torch.log((score == top).double().sum(1, keepdim=True))
    assert ((lse[0].double() - ref).abs() <= 2.0 ** -20 * (1 + ref.abs())).all()


def test_pieces_of_prompts_of_shared_pools(attn):
    """Heads that share memory (a stride of 0)."""
    q, pools, table, lens = problem(1, 1300, 32, 1, 128, 16, [1400], BF, 62)
    wide = [x.expand(-1, 8, -1, -1) for x in pools.pools]
    got = attn.paged_attention(q, *wide, table, lens)
    want = attn.paged_attention(q, *[x.contiguous() for x in wide], table, lens)
    top = want.float().abs().amax()
    assert ((got - want).float().abs() <= 2.0 ** -6 * top).all()


@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 5)])
@pytest.mark.parametrize("D", [64, 128])
def test_many_rows_of_batches_of_any_lengths(attn, D, window, sinks):
    """The lengths, which only the device has, tell which kernel takes the call: a batch of equal ones,
    one long one among short ones, empty ones; one captured graph serves them all."""
    B, T, Hq, Hkv = 14, 32, 32, 8
    longest = 9000
    q, pools, table, lens = problem(B, T, Hq, Hkv, D, 16, [longest] + [1500] * (B - 1), BF, 70)
    cases = [[1500] * B, [longest] + [40] * (B - 1), [33] * B, [0] * B, [longest] + [1500] * (B - 1),
             [31, 32, 33, 1, 0] + [1000] * (B - 5)]
    out = torch.empty_like(q)
    ws = torch.empty(max(attn.paged_attention_workspace_size(B, T, Hq, Hkv, D), 1), dtype=torch.uint8, device="cuda")
    call = lambda: attn.paged_attention(q, *pools.pools, table, lens, window=window, sinks=sinks, out=out, workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for n in cases:
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        out.fill_(7.0)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(call(), got)
        check(attn, (q, pools, table, lens), window, sinks)
        assert torch.equal(attn.paged_attention(q, *pools.pools, table, lens, window=window, sinks=sinks), got)
