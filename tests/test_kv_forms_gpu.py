"""kv_append and kv_read over pools of 4-bit codes and with positions of several axes, and the cache's
operators together, against float64 on the GPU.

Bounds: those of test_attn_gpu.py for queries, bf16, f32 and 8-bit pools.  4-bit keys err before they
are coded by less than 2^-17 of the row's largest value; so

* the row's scale is within 2^-17 of max(amax, 2^-96) / 2688,
* a group's scale, against gmax / (6 s) of the stored s: one e4m3 rounding (2^-4 of it, at least half
  the smallest step, 2^-10), and what that error makes of it: 2^-17 * 2688 / 6 < 2^-8, with s's own
  2^-17 of at most 448 twice that: 2^-7,
* an element's distance to its key is that of the nearest code times its stored scales, and twice the
  error, 2^-16 of the row's largest.

Values are not computed before they are coded: their scales, group scales and elements are bit for bit
those of f32 arithmetic, each operation rounded to nearest.
"""
import pytest
import torch

from test_attn_forms_gpu import F4, GRID, IDS, Pools, check, raw
from test_attn_gpu import BF, F8, F32, U, append_inputs, attn, rot_tables  # noqa: F401

pytestmark = pytest.mark.gpu

DEALT = (1,) * 60 + (4,)
FORMS = [
    # (T, Hq, Hkv, D, R, interleaved, norm, ps, dtype, pool dtype, sections, axes)
    (1, 1, 1, 64, 64, False, True, 16, BF, F4, None, 1),
    (67, 32, 8, 128, 128, False, True, 64, BF, F4, None, 1),
    (7, 5, 5, 128, 16, True, False, 7, BF, F4, None, 1),
    (33, 24, 2, 64, 32, True, True, 24, BF, F4, None, 1),
    (65, 6, 3, 128, 64, False, True, 1, F32, F4, None, 1),
    (19, 4, 4, 64, 0, False, True, 16, F32, F4, None, 1),
    (3, 8, 1, 128, 0, False, False, 128, BF, F4, None, 1),
    (5, 96, 32, 128, 96, False, True, 16, BF, F4, None, 1),
    (9, 7, 7, 64, 48, False, True, 16, BF, F4, None, 1),
    (9, 3, 3, 128, 112, False, False, 48, F32, F4, None, 1),
    (9, 3, 3, 128, 80, True, True, 48, BF, F4, None, 1),
    (1700, 16, 4, 128, 128, False, True, 64, BF, F4, None, 1),
    (2051, 12, 4, 64, 64, True, False, 16, BF, F4, None, 1),
    (1, 4, 1, 128, 128, False, False, 16, BF, BF, (16, 24, 24), 3),
    (21, 8, 2, 128, 128, False, True, 16, BF, F8, DEALT, 3),
    (21, 8, 2, 128, 128, True, True, 16, BF, F4, DEALT, 3),
    (5, 4, 4, 64, 32, False, False, 7, F32, F32, (5, 11), 2),
    (6, 4, 2, 64, 64, True, True, 16, BF, F4, (8, 8, 8, 8), 4),
    (6, 6, 2, 64, 16, False, True, 16, F32, F8, (1, 1, 1, 5), 4),
    (4, 2, 1, 128, 96, False, True, 16, BF, F8, (3, 1, 44), 2),
    (8, 4, 4, 128, 128, False, True, 16, BF, BF, (64,), 3),
    (1500, 28, 4, 128, 128, False, False, 16, BF, BF, DEALT, 3),
    (1500, 24, 8, 64, 48, True, True, 24, BF, F4, (7, 9, 8), 3),
]


def f4_values(codes):
    grid = torch.tensor(GRID + [-v for v in GRID], dtype=torch.float64, device=codes.device)
    return grid[torch.stack([codes % 16, codes // 16], -1).long()].flatten(-2)


def normed(x, w, eps=1e-6):
    x = x.double()
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()


def turned(x, cos, sin, R, interleaved):
    """Rows [T, heads, D] with cos and sin [T, R / 2] of their angles."""
    if not R:
        return x
    x = x.clone()
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., : R // 2], x[..., R // 2: R])
    c, s = cos.double()[:, None], sin.double()[:, None]
    a2, b2 = a * c - b * s, a * s + b * c
    a.copy_(a2), b.copy_(b2)
    return x


def columns(table, positions, sections):
    """The angles [T, R / 2] of tokens at positions [A, T], [T] without sections."""
    if sections is None:
        return table[positions.long()]
    axis = torch.tensor([j % positions.shape[0] for j, n in enumerate(sections) for _ in range(n)])
    cols = torch.arange(table.shape[1])
    return table[positions.long()[axis.cuda()].T, cols.cuda()]


def divided(a, b):
    """a / b in f32, rounded to nearest: 53 bits are enough to round the quotient of two f32 twice.
    (Torch multiplies by a number's reciprocal on the GPU.)"""
    return (a.double() / b).float()


def f4_reference(rows):
    """(elements' codes, group scales, scales) of float32 rows, each operation rounded."""
    n = rows.abs()
    scale = n.amax(-1).clamp(min=2.0 ** -96) * float(divided(torch.ones(1), 2688.0))
    group = divided(n.unflatten(-1, (-1, 16)).amax(-1), 6 * scale[..., None]).clamp(max=448).to(F8)
    step = (group.float() * scale[..., None]).repeat_interleave(16, -1)
    x = torch.where(step == 0, torch.zeros_like(rows), divided(rows, step)).double()
    grid = torch.tensor(GRID, dtype=torch.float64, device="cuda")
    d = (x.abs()[..., None] - grid).abs()
    # of two equally near codes the even one
    d = d + torch.tensor([0, 1] * 4, device="cuda") * 1e-12
    return grid[d.argmin(-1)] * x.sign(), group, scale


def check_append(attn, case, pad=(), token_major=False, make=None):
    T, Hq, Hkv, D, R, inter, norm, ps, dt, pdt, sections, axes = case
    q, k, v, (qw, kw), cos, sin, pos, g = append_inputs(T, Hq, Hkv, D, R, norm, dt, T * 100 + Hq)
    if make:
        k, v = make(k), make(v)
    if sections is not None:
        pos = torch.randint(0, 5000, (axes, T), generator=g).to(torch.int32).cuda()
    pages = -(-T // ps) + 2
    pools = Pools(pages, Hkv, ps, D, pdt, seed=T, token_major=token_major)
    state = [raw(x) for x in pools.pools + pools.groups + pools.scales if x is not None]
    before = [x.clone() for x in state]
    slots = torch.randperm(pages * ps, generator=g)[:T].to(torch.int32)
    gone = torch.zeros(T, dtype=torch.bool)
    for i, s in pad:
        if isinstance(s, tuple):
            pos[s] = -1 if i % 2 else 5000
        else:
            slots[i] = s
        gone[i] = True
    out = torch.full((T, Hq, D), 5.0, dtype=dt, device="cuda")
    got = attn.kv_append(q, k, v, slots.cuda(), *pools.pools, positions=pos, cos=cos, sin=sin, sections=sections,
                         interleaved=inter, q_weight=qw, k_weight=kw, out=out, **pools.kw)
    assert got is out
    keep = (~gone).nonzero()[:, 0].cuda()
    assert (out[gone.cuda()] == 5.0).all()
    angles = [None, None]
    if R:
        at = pos[..., keep]
        angles = [columns(x, at, sections) for x in (cos, sin)]
    want = turned(normed(q[keep], qw), *angles, R, inter)
    top = want.abs().amax(-1, keepdim=True)
    assert ((out[keep].double() - want).abs() <= U[dt] * want.abs() + 2.0 ** -17 * top).all()
    page, at = slots.cuda()[keep].long() // ps, slots.cuda()[keep].long() % ps
    untouched = torch.ones(pages, ps, dtype=torch.bool, device="cuda")
    untouched[page, at] = False
    for new, old in zip(state, before):
        assert torch.equal(new.transpose(1, 2)[untouched], old.transpose(1, 2)[untouched])
    keys = turned(normed(k[keep], kw), *angles, R, inter)
    for i, r in enumerate((keys, v[keep].double())):
        top = r.abs().amax(-1, keepdim=True)
        if pdt == F4:
            s = pools.scales[i][page, :, at].double()[..., None]
            wide = raw(pools.groups[i])[page, :, at].view(F8)
            gs = wide.double()
            codes = f4_values(raw(pools.pools[i])[page, :, at])
            if i == 1:
                x, ref_g, ref_s = f4_reference(v[keep].float())
                assert torch.equal(s[..., 0].float(), ref_s) and torch.equal(raw(wide), raw(ref_g))
                assert torch.equal(codes, x)
                continue
            whole = top.clamp(min=2.0 ** -96) / 2688
            assert ((s - whole).abs() <= 2.0 ** -17 * whole).all()
            ideal = r.abs().unflatten(-1, (-1, 16)).amax(-1) / (6 * s)
            assert ((gs - ideal).abs() <= (2.0 ** -4 * ideal).clamp(min=2.0 ** -10) + 2.0 ** -7).all()
            step = (gs * s).repeat_interleave(16, -1)
            grid = torch.tensor(GRID, dtype=torch.float64, device="cuda")
            near = (r.abs()[..., None] - grid * step[..., None]).abs().amin(-1)
            assert ((codes * step - r).abs() <= near + 2.0 ** -16 * top).all()
        elif pdt == F8:
            s = pools.scales[i][page, :, at].double()[..., None]
            x = raw(pools.pools[i])[page, :, at].view(F8).double() * s
            whole = top.clamp(min=2.0 ** -96) / 448
            assert ((s - whole).abs() <= 2.0 ** -17 * whole).all()
            assert ((x - r).abs() <= torch.maximum(2.0 ** -4 * r.abs(), 2.0 ** -10 * s) + 2.0 ** -15 * top).all()
        elif i == 1:
            assert torch.equal(pools.pools[1][page, :, at].double(), r)
        else:
            x = pools.pools[0][page, :, at].double()
            assert ((x - r).abs() <= U[dt] * r.abs() + 2.0 ** -17 * top).all()


@pytest.mark.parametrize("case", FORMS, ids=lambda c: "-".join(str(IDS.get(x, x)) for x in c[:10]) + f"-{c[11]}")
def test_append_matches_definition(attn, case):
    check_append(attn, case)


@pytest.mark.parametrize("pdt", [BF, F8, F4], ids=lambda t: IDS[t])
def test_append_padding_rows_write_nothing(attn, pdt):
    """Slots outside the pools, and a position outside the table on any one axis."""
    case = (40, 8, 2, 128, 128, False, True, 16, BF, pdt, (16, 24, 24), 3)
    check_append(attn, case, pad=[(0, -1), (7, -2 ** 31), (39, 5 * 16), (12, 2 ** 31 - 1), (3, (0, 3)), (4, (1, 4)),
                                  (6, (2, 6)), (9, (2, 9))])


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [64, 128])
def test_append_token_major_pools(attn, D, dt):
    check_append(attn, (21, 8, 4, D, 64, False, True, 16, dt, F4, None, 1), token_major=True)
    check_append(attn, (21, 8, 4, D, 32, True, True, 8, dt, F4, (4, 12), 2), token_major=True)


@pytest.mark.parametrize("dt", [BF, F32])
def test_append_codes_of_rows_of_any_size(attn, dt):
    """Zero rows, rows below the scale's floor, subnormal and huge ones, groups far smaller than their
    row and groups whose scale ends as 0; halfway values (multiples of a quarter of the step)."""
    def rows(x):
        g = torch.Generator(device="cuda").manual_seed(5)
        y = x.clone()
        y[0] = 0
        y[1] *= 2.0 ** -120
        y[2] *= 1e-30
        y[3] *= 1e36
        y[4, :, 16:48] *= 2.0 ** -12
        y[5, :, 32:] *= 2.0 ** -17
        y[6] = torch.randint(-24, 25, y[6].shape, generator=g, device="cuda").to(dt) / 4
        y[6, :, 0] = 6 * 448 * 2.0 ** -9 * 2
        y[7] = 3.0
        y[8] = 0
        y[8, :, 5] = -2.0 ** -133 if dt == BF else 2.0 ** -149
        return y
    check_append(attn, (9, 4, 2, 128, 0, False, False, 4, dt, F4, None, 1), make=rows)


def test_append_rows_with_infinities_and_nan(attn):
    """They read back as NaN and harm no other row."""
    T, Hkv, D = 6, 2, 128
    x = torch.randn(T, Hkv, D, generator=torch.Generator().manual_seed(1))
    x[1, 0, 77], x[2, 1, 3], x[4, 0, 0], x[5, 1, 127] = float("inf"), float("nan"), float("-inf"), float("nan")
    bad = {(1, 0), (2, 1), (4, 0), (5, 1)}
    k = x.to(BF).cuda()
    pools = Pools(2, Hkv, 4, D, F4, 1)
    slots = torch.arange(T, dtype=torch.int32).cuda()
    attn.kv_append(torch.zeros(T, 2, D, dtype=BF, device="cuda"), k, k, slots, *pools.pools, **pools.kw)
    table = torch.tensor([[0, 1]], dtype=torch.int32).cuda()
    cu = torch.tensor([0, T], dtype=torch.int32).cuda()
    for y in attn.kv_read(*pools.pools, table, cu, T, dtype=F32, **pools.kw):
        for t in range(T):
            for h in range(Hkv):
                if (t, h) in bad:
                    assert torch.isnan(y[t, h]).all()
                    continue
                want, group, scale = f4_reference(k[t, h].float())
                assert torch.equal(y[t, h], want.float() * group.float().repeat_interleave(16) * scale)


@pytest.mark.parametrize("odt", [BF, F32], ids=lambda t: IDS[t])
@pytest.mark.parametrize("token_major", [False, True])
@pytest.mark.parametrize("D,ps,lens", [(64, 16, [5, 0, 33, 1]), (128, 7, [50]), (128, 1, [3, 4, 0]),
                                       (64, 100, [257, 300]), (128, 64, [1]), (128, 16, [4100, 17]),
                                       (64, 64, [9000])])
def test_read_bit_for_bit(attn, odt, token_major, D, ps, lens):
    """(code * group scale) * scale, the second product rounded to f32 and then to the rows' dtype;
    rows of no sequence, positions outside the table and missing pages are zeros."""
    Hkv = 3
    used = [-(-n // ps) for n in lens]
    pools = Pools(sum(used) + 2, Hkv, ps, D, F4, D + ps, token_major=token_major)
    order = torch.randperm(sum(used) + 2, generator=torch.Generator().manual_seed(ps)).tolist()
    M = max(used) + 1
    table = torch.full((len(lens), M + 3), -1, dtype=torch.int32)
    for b, n in enumerate(used):
        for i in range(n):
            table[b, i] = order.pop()
    table[-1, max(used[-1] - 1, 0)] = 2 ** 31 - 1     # the last sequence's last page is none
    table = table.cuda()[:, :M]
    starts = [n // 3 for n in lens]
    counts = [n - n // 3 + 2 for n in lens]           # two positions more than the table has pages for
    cu = [sum(counts[:i]) for i in range(len(lens) + 1)]
    T = cu[-1] + 3
    got = attn.kv_read(*pools.pools, table, torch.tensor(cu, dtype=torch.int32).cuda(), T,
                       starts=torch.tensor(starts, dtype=torch.int32).cuda(), dtype=odt, **pools.kw)
    for i, y in enumerate(got):
        want = torch.zeros(T, Hkv, D, dtype=odt, device="cuda")
        for b, n in enumerate(counts):
            p = starts[b] + torch.arange(n, device="cuda")
            page = torch.where(p < M * ps, table[b, (p // ps).clamp(max=M - 1)].long(), -1)
            live = (page >= 0) & (page < sum(used) + 2)
            rows = pools.rows(i, page.clamp(0, sum(used) + 1), p % ps).float().to(odt)
            want[cu[b]: cu[b + 1]] = rows * live[:, None, None]
        assert y.dtype == odt and torch.equal(y, want)


def test_rows_per_call_change_nothing(attn):
    """The same tokens appended at once and one at a time leave the same bits."""
    T, Hq, Hkv, D = 37, 8, 2, 128
    q, k, v, (qw, kw), cos, sin, _, g = append_inputs(T, Hq, Hkv, D, 128, True, BF, 8)
    pos = torch.randint(0, 5000, (3, T), generator=g).to(torch.int32).cuda()
    slots = torch.randperm(48, generator=g)[:T].to(torch.int32).cuda()
    a, b = Pools(3, Hkv, 16, D, F4, 2), Pools(3, Hkv, 16, D, F4, 2)
    kw = dict(cos=cos, sin=sin, q_weight=qw, k_weight=kw, sections=DEALT)
    whole = attn.kv_append(q, k, v, slots, *a.pools, positions=pos, **kw, **a.kw)
    parts = [attn.kv_append(q[t: t + 1], k[t: t + 1], v[t: t + 1], slots[t: t + 1], *b.pools,
                            positions=pos[:, t: t + 1].contiguous(), **kw, **b.kw) for t in range(T)]
    assert torch.equal(whole, torch.cat(parts))
    for x, y in zip(a.pools + a.groups + a.scales, b.pools + b.groups + b.scales):
        assert torch.equal(raw(x), raw(y))


class Layer:
    """An attention layer's calls on a cache: tokens appended with positions of three axes, then seen
    with sinks beside a window."""

    def __init__(self, attn, pdt, D, Hq=8, Hkv=2, ps=16, pages=40, window=50, sinks=4):
        self.attn, self.D, self.Hq, self.Hkv, self.ps = attn, D, Hq, Hkv, ps
        self.pools = Pools(pages, Hkv, ps, D, pdt, 3)
        self.cos, self.sin = (x.cuda() for x in rot_tables(2000, D))
        self.sections = (D // 8, D // 8, D // 4)
        self.window, self.sinks = window, sinks

    def step(self, x, slots, pos, table, lens, out=None, workspace=None, q_out=None):
        """x [B, T, heads, D] -> [B, T, Hq, D]."""
        B, T = x.shape[:2]
        rows = x.flatten(0, 1)
        q, k, v = rows.split([self.Hq, self.Hkv, self.Hkv], 1)
        q = self.attn.kv_append(q, k, v, slots, *self.pools.pools, positions=pos, cos=self.cos, sin=self.sin,
                                sections=self.sections, out=q_out, **self.pools.kw)
        self.q = q.view(B, T, self.Hq, self.D)
        return self.attn.paged_attention(self.q, *self.pools.pools, table, lens, window=self.window,
                                         sinks=self.sinks, out=out, workspace=workspace, **self.pools.kw)


@pytest.mark.parametrize("pdt", [BF, F8, F4], ids=lambda t: IDS[t])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_then_decode_together(attn, pdt, D):
    """A prompt in one piece, then tokens one by one: each step's attention against the definition over
    what the pools hold, the rows read back against the same."""
    layer = Layer(attn, pdt, D)
    B, n = 2, [160, 131]
    table = torch.full((B, 12), -1, dtype=torch.int32)
    order = torch.randperm(40, generator=torch.Generator().manual_seed(4))
    table[0], table[1] = order[:12], order[12:24]
    slot = lambda b, p: int(table[b, p // 16]) * 16 + p % 16
    g = torch.Generator().manual_seed(6)
    x = torch.randn(B, max(n), 12, D, generator=g).to(BF).cuda()
    # rows of tokens that sequence 1 lacks are padding: slot -1, before its first token
    T = max(n)
    first = [T - m for m in n]
    xs = torch.stack([torch.cat([x[b, n[b]:], x[b, : n[b]]]) for b in range(B)])
    slots = torch.tensor([-1 if t < first[b] else slot(b, t - first[b]) for b in range(B) for t in range(T)],
                         dtype=torch.int32).cuda()
    place = torch.tensor([max(t - first[b], 0) for b in range(B) for t in range(T)])
    pos = torch.stack([place, place // 7, place % 7]).to(torch.int32).cuda()
    dev = table.cuda()
    q_out = torch.zeros(B * T, 8, D, dtype=BF, device="cuda")   # padding's rows stay as they were
    layer.step(xs, slots, pos, dev, torch.tensor(n, dtype=torch.int32).cuda(), q_out=q_out)
    lens = torch.tensor(n, dtype=torch.int32).cuda()
    check(attn, (layer.q, layer.pools, dev, lens), 50, 4)
    for step in range(3):
        x1 = torch.randn(B, 1, 12, D, generator=g).to(BF).cuda()
        slots = torch.tensor([slot(b, m) for b, m in enumerate(n)], dtype=torch.int32).cuda()
        place = torch.tensor(n)
        pos = torch.stack([place, place // 7, place % 7]).to(torch.int32).cuda()
        n = [m + 1 for m in n]
        lens = torch.tensor(n, dtype=torch.int32).cuda()
        layer.step(x1, slots, pos, dev, lens)
        check(attn, (layer.q, layer.pools, dev, lens), 50, 4)
    cu = torch.tensor([0, n[0], sum(n)], dtype=torch.int32).cuda()
    for i, y in enumerate(attn.kv_read(*layer.pools.pools, dev, cu, sum(n), **layer.pools.kw)):
        for b in range(B):
            p = torch.arange(n[b], device="cuda")
            want = layer.pools.rows(i, dev[b, p // 16].long(), p % 16).float().to(y.dtype)
            assert torch.equal(y[cu[b]: cu[b + 1]], want)


@pytest.mark.parametrize("pdt", [BF, F4], ids=lambda t: IDS[t])
def test_a_layer_in_a_graph(attn, pdt):
    """Captured once, replayed with other positions, slots and lengths; two graphs share a workspace."""
    D, B = 128, 3
    layer = Layer(attn, pdt, D, window=40, sinks=3)
    x = torch.randn(B, 1, 12, D, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    table = torch.randperm(36, generator=torch.Generator().manual_seed(2)).to(torch.int32).view(3, 12)
    dev = table.cuda()
    slots, lens = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    pos = torch.zeros(3, B, dtype=torch.int32, device="cuda")
    need = attn.paged_attention_workspace_size(B, 1, 8, 2, D, layer.pools.pools[0].dtype)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    outs = [torch.empty(B, 1, 8, D, dtype=BF, device="cuda") for _ in range(2)]
    q_out = torch.empty(B, 8, D, dtype=BF, device="cuda")

    def place(n):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        slots.copy_(torch.tensor([int(table[b, (m - 1) // 16]) * 16 + (m - 1) % 16 for b, m in enumerate(n)]))
        pos.copy_(torch.tensor([[m % 11 for m in n], n, [m % 5 for m in n]], dtype=torch.int32))

    place([100, 180, 1])
    layer.step(x, slots, pos, dev, lens, outs[0], ws, q_out)
    torch.cuda.synchronize()
    graphs = []
    for out in outs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            layer.step(x, slots, pos, dev, lens, out, ws, q_out)
    for n in ([101, 17, 44], [39, 192, 2]):
        place(n)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = layer.step(x, slots, pos, dev, lens, None, ws)
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
        check(attn, (q_out[:, None], layer.pools, dev, lens), 40, 3)


def test_prompts_in_a_graph(attn):
    """The path of many rows captured and replayed with other lengths."""
    from test_attn_forms_gpu import problem
    q, pools, table, lens = problem(1, 1500, 32, 8, 128, 16, [3000], BF, 5, poison=False)
    out = torch.empty_like(q)
    ws = torch.empty(max(attn.paged_attention_workspace_size(1, 1500, 32, 8, 128), 1), dtype=torch.uint8,
                     device="cuda")
    call = lambda: attn.paged_attention(q, *pools.pools, table, lens, window=700, sinks=9, out=out, workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for n in (1700, 200, 0, 3000):
        lens.fill_(n)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(call(), got)


def test_example_over_a_4_bit_cache(attn):
    """The hybrid example's checks (test_attn_gpu.py runs it over the other caches).  Decoding against one
    prompt of the full length: keys and values differ by a layer's bf16 roundings before they are coded,
    so that a code near a halfway point may be its neighbour, a third of its group's largest away at
    most, with its position's weight."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_decode.py")
    spec = importlib.util.spec_from_file_location("hybrid_decode", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    last, apart = mod.main("fp4")
    assert last < 2e-2 and apart < 5e-2


DEBUG_CHILD = r"""
import ctypes, json, sys
sys.path[:0] = [sys.argv[1], sys.argv[1] + "/tests"]
import test_attn_forms_gpu as a
import test_kv_forms_gpu as t
from state_space_model_gb300 import _native, attn
import torch
assert _native.LIB_PATH.endswith("libssd_gb300_debug.so"), _native.LIB_PATH
for case in t.FORMS[:11] + t.FORMS[13:21]:
    t.check_append(attn, case)
t.check_append(attn, (21, 8, 4, 64, 64, False, True, 8, t.BF, t.F4, None, 1), token_major=True)
for D, ps, lens in ((64, 16, [5, 0, 33, 1]), (128, 7, [50]), (128, 16, [4100, 17])):
    for major in (False, True):
        t.test_read_bit_for_bit(attn, t.BF, major, D, ps, lens)
for pdt in (t.BF, t.F8, t.F32, t.F4):
    for D in (64, 128):
        for T, Hq, ps in ((1, 8, 16), (3, 6, 7), (17, 8, 32)):
            prob = a.problem(3, T, Hq, 2, D, ps, [700, 33, 5], pdt, T + D)
            a.check(attn, prob)
            a.check(attn, prob, 60, 5)
for D in (64, 128):
    for case in ((1, 1300, 32, 8, [1300], 0, 0), (2, 700, 32, 8, [2000, 800], 300, 20), (1, 4000, 16, 16, [4001], 0, 0)):
        B, T, Hq, Hkv, lens, window, sinks = case
        prob = a.problem(B, T, Hq, Hkv, D, 16, lens, t.BF, T)
        a.check(attn, prob, window, sinks)
lib = _native.load()
st = lib.ssd_device_status(ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
print(json.dumps({"status": st, "detail": lib.ssd_last_error_detail().decode()}))
"""


def test_debug_build_finds_every_index_in_bounds(attn):
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
