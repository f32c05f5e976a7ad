"""GPU parity of the attention layers' cache (kv_append, kv_read, paged_attention)
against the float64 oracle.

Bounds, derived from the arithmetic (u is the unit roundoff: 2^-24 fp32, 2^-8
bf16, 2^-11 fp16, 2^-4 e4m3):

* queries and keys: norm and rotation in fp32 err by less than 2^-18 of the
  row's largest value before and after rotation (sum of D squares, a reciprocal
  root and three roundings), then one rounding to the stored type;
* a quantised value: that, one e4m3 rounding (2^-4 of the value, at least half
  the smallest step 2^-9 of the scale); the scale itself within 2^-17;
* read: bf16 and f32 bit for bit; codes times scale bit for bit torch's fp32
  product rounded once;
* attention scores: a D-term fp32 sum of exact products errs by at most
  (D + 8) u_t sum |q k| scale =: ds, with u_t = 2^-22 where tensor cores add
  (they may truncate) and 2^-24 elsewhere; a probability is then off by 2 ds
  relative, and by one rounding to 16 bits (bf16 or fp16: 2^-8 covers both); sums
  over n positions in fp32 add n u_t.  So |out error| <= vmax (2 ds + n u_t + [2^-8
  unless f32]) plus one rounding of the result, and |lse error| <= ds + n u_t +
  2^-21 (1 + |lse|).
"""
import numpy as np
import pytest
import torch

from oracle import attn as orc

pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from state_space_model_gb300 import attn as mod, build
    build.build()
    return mod


def np64(t):
    return None if t is None else t.detach().float().cpu().double().numpy()


def rot_tables(S, R):
    ang = torch.arange(S, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, R, 2).double() / R)
    return ang.cos().float(), ang.sin().float()


# ---- kv_append ---------------------------------------------------------------

APPEND = [
    # (T, Hq, Hkv, D, R, interleaved, norm, ps, dtype, pool dtype)
    (1, 1, 1, 64, 64, False, True, 16, BF, BF),
    (1, 32, 8, 128, 128, False, True, 64, BF, F8),
    (7, 5, 5, 128, 16, True, False, 7, BF, F8),
    (33, 24, 2, 64, 32, True, True, 24, BF, BF),
    (65, 6, 3, 128, 64, False, True, 1, F32, F32),
    (19, 4, 4, 64, 0, False, True, 16, F32, F8),
    (130, 40, 8, 128, 128, True, True, 100, BF, F8),
    (3, 8, 1, 128, 0, False, False, 128, BF, BF),
    (5, 96, 32, 128, 96, False, True, 16, BF, BF),
]


def append_inputs(T, Hq, Hkv, D, R, norm, dt, seed):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(T, (Hq + 2 * Hkv) * D, generator=g) * 2).to(dt).cuda()
    q = qkv[:, : Hq * D].view(T, Hq, D)
    k = qkv[:, Hq * D: (Hq + Hkv) * D].view(T, Hkv, D)
    v = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
    w = [(torch.rand(D, generator=g) + 0.5).cuda() if norm else None for _ in range(2)]
    cos = sin = pos = None
    if R:
        cos, sin = (x.cuda() for x in rot_tables(5000, R))
        pos = torch.randint(0, 5000, (T,), generator=g).to(torch.int32).cuda()
    return q, k, v, w, cos, sin, pos, g


def new_pools(pages, Hkv, ps, D, pdt, nhd=False):
    shape = (pages, ps, Hkv, D) if nhd else (pages, Hkv, ps, D)
    make = lambda: torch.full(shape, 3.0, device="cuda").to(pdt)
    kc, vc = make(), make()
    if nhd:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    ks = vs = None
    if pdt == F8:
        ks, vs = (torch.full((pages, Hkv, ps), 9.0, device="cuda") for _ in range(2))
    return kc, vc, ks, vs


def check_append(attn, case, pad=(), nhd=False):
    T, Hq, Hkv, D, R, inter, norm, ps, dt, pdt = case
    q, k, v, (qw, kw), cos, sin, pos, g = append_inputs(T, Hq, Hkv, D, R, norm, dt, T * 100 + Hq)
    pages = -(-T // ps) + 2
    kc, vc, ks, vs = new_pools(pages, Hkv, ps, D, pdt, nhd)
    before = [None if t is None else t.clone() for t in (kc, vc, ks, vs)]
    slots = torch.randperm(pages * ps, generator=g)[:T].to(torch.int32)
    for i, s in pad:
        slots[i] = s
    out = torch.full((T, Hq, D), 5.0, dtype=dt, device="cuda")
    got = attn.kv_append(q, k, v, slots.cuda(), kc, vc, k_scale=ks, v_scale=vs, positions=pos, cos=cos,
                         sin=sin, interleaved=inter, q_weight=qw, k_weight=kw, out=out)
    assert got is out
    ref, held = orc.kv_append(np64(q), np64(k), np64(v), slots.numpy(), pages * ps,
                              None if pos is None else pos.cpu().numpy(), np64(cos), np64(sin), inter,
                              np64(qw), np64(kw))
    o = np64(out)
    for t in range(T):
        if np.isnan(ref[t]).any():
            assert (o[t] == 5.0).all()
            continue
        top = np.abs(ref[t]).max(-1, keepdims=True)
        assert (np.abs(o[t] - ref[t]) <= U[dt] * np.abs(ref[t]) + 2.0 ** -17 * top).all()
    for pool, scale, old, olds, i in ((kc, ks, before[0], before[2], 0), (vc, vs, before[1], before[3], 1)):
        p, o0 = np64(pool), np64(old)
        for s in range(pages * ps):
            at = (s // ps, slice(None), s % ps)
            if s not in held:
                assert (p[at] == o0[at]).all()
                if scale is not None:
                    assert (scale[at] == olds[at]).all()
                continue
            r = held[s][i]
            top = np.abs(r).max(-1, keepdims=True)
            if pdt == F8:
                sc = np64(scale[at])[:, None]
                want = np.array([orc.row_scale(x) for x in r])[:, None]
                assert (np.abs(sc - want) <= 2.0 ** -17 * want).all()
                err = np.abs(p[at] * sc - r)
                assert (err <= np.maximum(2.0 ** -4 * np.abs(r), 2.0 ** -10 * sc) + 2.0 ** -15 * top).all()
            elif i == 1:
                assert (p[at] == r).all()          # values are copied
            else:
                assert (np.abs(p[at] - r) <= U[dt] * np.abs(r) + 2.0 ** -17 * top).all()


@pytest.mark.parametrize("case", APPEND, ids=str)
def test_append_matches_oracle(attn, case):
    check_append(attn, case)


def test_append_padding_rows_write_nothing(attn):
    case = (40, 8, 2, 128, 128, False, True, 16, BF, F8)
    check_append(attn, case, pad=[(0, -1), (7, -2 ** 31), (39, 5 * 16), (12, 2 ** 31 - 1)])


def test_append_position_out_of_table_is_padding(attn):
    q, k, v, (qw, kw), cos, sin, pos, g = append_inputs(4, 4, 2, 64, 64, True, BF, 3)
    pos[1], pos[2] = 5000, -1
    kc, vc, ks, vs = new_pools(2, 2, 4, 64, BF)
    out = torch.full((4, 4, 64), 5.0, dtype=BF, device="cuda")
    attn.kv_append(q, k, v, torch.arange(4, dtype=torch.int32).cuda(), kc, vc, positions=pos, cos=cos,
                   sin=sin, q_weight=qw, k_weight=kw, out=out)
    assert (out[1:3] == 5).all() and not (out[0] == 5).all()
    assert (kc[0, :, 1:3] == 3).all() and (vc[0, :, 1:3] == 3).all() and not (vc[0, :, 3] == 3).all()


@pytest.mark.parametrize("pdt", [BF, F8])
def test_append_token_major_pools(attn, pdt):
    check_append(attn, (21, 8, 4, 64, 64, False, True, 8, BF, pdt), nhd=True)


def test_append_extreme_rows(attn):
    """A zero row reads back as zeros, tiny and huge rows keep their values, a row with an
    infinity or NaN reads back as NaN and harms no other."""
    T, Hkv, D = 6, 2, 128
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, Hkv, D, generator=g)
    x[1] = 0.0
    x[2] *= 1e-30
    x[3] *= 1e30
    x[4, 0, 77] = float("inf")
    x[5, 1, 3] = float("nan")
    k = x.to(BF).cuda()
    kc, vc, ks, vs = new_pools(2, Hkv, 4, D, F8)
    slots = torch.arange(T, dtype=torch.int32).cuda()
    q = torch.zeros(T, 2, D, dtype=BF, device="cuda")
    attn.kv_append(q, k, k, slots, kc, vc, k_scale=ks, v_scale=vs)
    table = torch.tensor([[0, 1]], dtype=torch.int32).cuda()
    cu = torch.tensor([0, T], dtype=torch.int32).cuda()
    for y in attn.kv_read(kc, vc, table, cu, T, k_scale=ks, v_scale=vs, dtype=F32):
        y, r = np64(y), np64(k)
        assert (y[1] == 0).all()
        for t in (0, 2, 3):
            top = np.abs(r[t]).max(-1, keepdims=True)
            err = np.abs(y[t] - r[t])
            assert (err <= np.maximum(2.0 ** -4 * np.abs(r[t]), 2.0 ** -10 / 448 * top) + 2.0 ** -15 * top).all()
        assert np.isnan(y[4, 0]).all() and np.isfinite(y[4, 1]).all()
        assert np.isnan(y[5, 1]).all() and np.isfinite(y[5, 0]).all()


# ---- kv_read -----------------------------------------------------------------


def fill_pools(pages, Hkv, ps, D, pdt, seed):
    g = torch.Generator().manual_seed(seed)
    r = [torch.randn(pages, Hkv, ps, D, generator=g) for _ in range(2)]
    if pdt == F8:
        s = [(torch.rand(pages, Hkv, ps, generator=g) + 0.5).cuda() / 100 for _ in range(2)]
        return [(x * 100).clamp(-448, 448).to(F8).cuda() for x in r] + s
    return [x.to(pdt).cuda() for x in r] + [None, None]


@pytest.mark.parametrize("pdt,odt", [(BF, BF), (F32, F32), (F8, BF), (F8, F32)])
@pytest.mark.parametrize("D,ps,lens", [(64, 16, [5, 0, 33, 1]), (128, 7, [50]), (128, 1, [3, 4, 0]),
                                       (64, 100, [257, 300])])
def test_read_matches_oracle(attn, pdt, odt, D, ps, lens):
    Hkv = 3
    used = [-(-n // ps) for n in lens]
    pages = sum(used) + 1
    kc, vc, ks, vs = fill_pools(pages, Hkv, ps, D, pdt, D + ps)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(ps)).tolist()
    M = max(used) + 1
    table = torch.full((len(lens), M + 3), -1, dtype=torch.int32)
    for b, n in enumerate(used):
        for i in range(n):
            table[b, i] = order.pop()
    table = table.cuda()[:, :M]                       # a view with a longer row stride
    starts = torch.tensor([n // 3 for n in lens], dtype=torch.int32)
    counts = [n - n // 3 for n in lens]
    cu = torch.tensor([sum(counts[:i]) for i in range(len(lens) + 1)], dtype=torch.int32)
    T = sum(counts) + 2                               # two rows of no sequence
    kw = dict(starts=starts.cuda(), k_scale=ks, v_scale=vs, dtype=odt)
    k, v = attn.kv_read(kc, vc, table, cu.cuda(), T, **kw)
    for got, pool, sc in ((k, kc, ks), (v, vc, vs)):
        ref = orc.kv_read(np64(pool), np64(sc), table.cpu().numpy(), cu.numpy(), T, starts.numpy())
        assert got.dtype == odt and got.shape == (T, Hkv, D)
        if pdt == F8:                                 # one fp32 product, rounded once
            want = torch.tensor(ref, dtype=torch.float64).to(torch.float32).to(odt)
            assert (np.abs(np64(got) - ref) <= (U[odt] * 1.001 + 2.0 ** -24) * np.abs(ref)).all()
            assert (got.cpu() == want).float().mean() > 0.999
        else:
            assert (np64(got) == ref).all()


def test_read_missing_pages_are_zero(attn):
    kc, vc, _, _ = fill_pools(4, 2, 8, 64, BF, 9)
    table = torch.tensor([[0, 4, -1, 3], [2 ** 31 - 1, 1, 2, -2 ** 31]], dtype=torch.int32).cuda()
    cu = torch.tensor([0, 40, 70], dtype=torch.int32).cuda()
    starts = torch.tensor([0, -4], dtype=torch.int32)
    k, v = attn.kv_read(kc, vc, table, cu, 70, starts=starts.cuda())
    for got, pool in ((k, kc), (v, vc)):
        assert (np64(got) == orc.kv_read(np64(pool), None, table.cpu().numpy(), [0, 40, 70], 70, [0, -4])).all()
        assert (got[8:24] == 0).all() and (got[32:40] == 0).all() and not (got[24:32] == 0).all()


# ---- paged attention ------------------------------------------------------------


def attn_problem(B, T, Hq, Hkv, D, ps, lens, pdt, seed, spread=1.0, nan=True):
    """Pools in which every slot that no sequence uses holds NaN, and a shuffled table."""
    g = torch.Generator().manual_seed(seed)
    used = [-(-max(n, 0) // ps) for n in lens]
    pages = sum(used) + 2
    kc, vc, ks, vs = fill_pools(pages, Hkv, ps, D, pdt, seed + 1)
    M = max(used + [1])
    table = torch.full((B, M), -1, dtype=torch.int32)
    order = torch.randperm(pages, generator=g).tolist()
    live = torch.zeros(pages, ps, dtype=torch.bool)
    for b, n in enumerate(used):
        for i in range(n):
            table[b, i] = order.pop()
            live[table[b, i], : max(0, min(ps, lens[b] - i * ps))] = True
    if nan:
        dead = ~live[:, None, :].expand(pages, Hkv, ps)
        dead = dead.cuda()
        for p in (kc, vc):
            if pdt == F8:
                p.view(torch.uint8)[dead] = 0x7F
            else:
                p[dead] = float("nan")
        for s in (ks, vs):
            if s is not None:
                s[dead] = float("inf")
    q = (torch.randn(B, T, Hq, D, generator=g) * spread).to(F32 if pdt == F32 else BF).cuda()
    return q, kc, vc, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), ks, vs


def check_attn(attn, prob, pdt, window=0, scale=None, **kw):
    q, kc, vc, table, lens, ks, vs = prob
    out, lse = attn.paged_attention(q, kc, vc, table, lens, k_scale=ks, v_scale=vs, window=window,
                                    scale=scale, return_lse=True, **kw)
    D = q.shape[-1]
    ref, rl, vmax, smax, seen = orc.paged_attention(np64(q), np64(kc), np64(vc), table.cpu().numpy(),
                                                    lens.cpu().numpy(), np64(ks), np64(vs), scale, window)
    ut = 2.0 ** -24 if pdt == F32 else 2.0 ** -22
    ds = (D + 8) * ut * smax
    bound = vmax * (2 * ds + (seen + 8) * ut + (0 if pdt == F32 else 2.0 ** -8))
    uo = U[q.dtype]
    o, l = np64(out), np64(lse)
    none = seen == 0
    assert (o[none] == 0).all() and np.isneginf(l[none]).all()
    assert np.isfinite(o).all() and np.isfinite(l[~none]).all()
    assert (np.abs(o - ref) <= bound[..., None] * (1 + uo) + uo * np.abs(ref)).all()
    dl = np.abs(l[~none] - rl[~none])
    assert (dl <= (ds + seen * ut + 2.0 ** -21 * (1 + np.abs(rl)))[~none]).all()
    return out, lse


ATTN = [
    # (T, Hq, Hkv, D, ps, lens, window)
    (1, 1, 1, 64, 16, [1], 0),
    (1, 4, 4, 128, 64, [1, 2, 63, 64, 65], 0),
    (1, 8, 1, 128, 16, [0, 5, 129, 16], 0),
    (1, 6, 2, 64, 24, [100, 23, 24, 25, 0, 191], 0),
    (1, 20, 4, 128, 7, [333, 1], 0),
    (1, 64, 4, 64, 32, [257], 0),
    (1, 16, 1, 128, 128, [1000, 0, 3], 0),
    (1, 40, 2, 128, 100, [512], 0),                  # 20 rows a head
    (1, 37, 1, 64, 1, [77, 128], 0),                 # 37 rows, pages of one token
    (2, 8, 8, 128, 16, [1, 2, 40, 0], 0),            # rows before the first position
    (3, 24, 4, 64, 48, [2, 300], 0),
    (4, 32, 4, 128, 16, [3, 65, 200], 0),
    (8, 16, 2, 128, 64, [8, 7, 500], 0),
    (5, 70, 7, 64, 16, [150, 4], 0),
    (17, 12, 3, 128, 32, [17, 90, 16], 0),
    (100, 8, 2, 64, 16, [100, 130], 0),              # a piece of a prompt
    (1, 8, 2, 128, 16, [300, 20, 0, 1], 50),
    (1, 4, 1, 64, 16, [300, 64], 1),
    (4, 8, 2, 128, 24, [300, 3, 66], 33),
    (9, 16, 2, 64, 64, [200, 9], 128),
]


@pytest.mark.parametrize("pdt", [BF, F8, F32], ids=["bf16", "fp8", "f32"])
@pytest.mark.parametrize("case", ATTN, ids=str)
def test_attention_matches_oracle(attn, case, pdt):
    T, Hq, Hkv, D, ps, lens, window = case
    prob = attn_problem(len(lens), T, Hq, Hkv, D, ps, lens, pdt, seed=T + Hq + ps)
    check_attn(attn, prob, pdt, window)


@pytest.mark.parametrize("pdt", [BF, F8, F32], ids=["bf16", "fp8", "f32"])
def test_attention_large_scores(attn, pdt):
    """Scores far apart: the running maximum moves, most probabilities vanish."""
    prob = attn_problem(2, 2, 8, 2, 128, 16, [400, 37], pdt, seed=5, spread=12.0)
    check_attn(attn, prob, pdt, scale=0.5)
    prob = attn_problem(2, 2, 8, 2, 128, 16, [400, 37], pdt, seed=6, spread=1e-3)
    check_attn(attn, prob, pdt, scale=0.0)           # every probability alike


@pytest.mark.parametrize("pdt", [BF, F8], ids=["bf16", "fp8"])
def test_attention_long_splits(attn, pdt):
    """Few rows over a long cache: one sequence on many CTAs, its parts joined."""
    prob = attn_problem(1, 1, 2, 1, 128, 64, [9001], pdt, seed=11)
    check_attn(attn, prob, pdt)
    prob = attn_problem(3, 3, 2, 1, 64, 16, [5000, 1, 2500], pdt, seed=12)
    check_attn(attn, prob, pdt)


def test_attention_ragged_batch(attn):
    """Many short sequences and a long one: CTAs that cross sequences."""
    lens = [3000] + [(37 * i) % 150 for i in range(200)]
    prob = attn_problem(len(lens), 1, 4, 2, 64, 16, lens, BF, seed=13)
    check_attn(attn, prob, BF)


@pytest.mark.parametrize("pdt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B", [32, 33, 600])
def test_attention_many_sequences(attn, pdt, B):
    """Either way of finding a CTA's stretch, and more sequences than a CTA has threads."""
    lens = [(7 * i) % 41 for i in range(B)]
    prob = attn_problem(B, 1, 2, 1, 64, 16, lens, pdt, seed=21 + B)
    check_attn(attn, prob, pdt)


@pytest.mark.parametrize("pdt", [BF, F8, F32], ids=["bf16", "fp8", "f32"])
def test_attention_missing_pages(attn, pdt):
    q, kc, vc, table, lens, ks, vs = attn_problem(3, 2, 4, 2, 64, 8, [100, 100, 30], pdt, seed=14, nan=False)
    table[0, 3], table[0, 0], table[1, :] = -1, kc.shape[0], -7
    table[2, 1] = 2 ** 31 - 1
    lens[2] = 10 ** 6                                # beyond the table: only the table's positions are there
    check_attn(attn, (q, kc, vc, table, lens, ks, vs), pdt)


@pytest.mark.parametrize("pdt", [BF, F8, F32], ids=["bf16", "fp8", "f32"])
def test_attention_unseen_nan_stays_out(attn, pdt):
    """A later draft token's NaN key and value do not reach the rows before it, nor does what a
    window has left behind reach the rows after it."""
    T, n = 4, 50
    q, kc, vc, table, lens, ks, vs = attn_problem(1, T, 8, 2, 128, 16, [n], pdt, seed=15)
    good, lg = attn.paged_attention(q, kc, vc, table, lens, k_scale=ks, v_scale=vs, return_lse=True)
    page, at = int(table[0, (n - 1) // 16]), (n - 1) % 16
    for p in (kc, vc):
        (p.view(torch.uint8) if pdt == F8 else p)[page, :, at] = 0x7F if pdt == F8 else float("nan")
    bad, lb = attn.paged_attention(q, kc, vc, table, lens, k_scale=ks, v_scale=vs, return_lse=True)
    assert torch.equal(bad[:, :3], good[:, :3]) and torch.equal(lb[:, :3], lg[:, :3])
    assert torch.isnan(bad[:, 3]).all()
    # position 10 is inside the first row's window (n - 4 - 36 = 10) only
    q, kc, vc, table, lens, ks, vs = attn_problem(1, T, 8, 2, 128, 16, [n], pdt, seed=16)
    kw = dict(k_scale=ks, v_scale=vs, window=37)
    good = attn.paged_attention(q, kc, vc, table, lens, **kw)
    page = int(table[0, 0])
    (vc.view(torch.uint8) if pdt == F8 else vc)[page, :, 10, 5] = 0x7F if pdt == F8 else float("inf")
    bad = attn.paged_attention(q, kc, vc, table, lens, **kw)
    assert torch.equal(bad[:, 1:], good[:, 1:])
    assert not torch.isfinite(bad[:, 0, :, 5]).any()


@pytest.mark.parametrize("pdt", [BF, F8], ids=["bf16", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_leftovers_of_other_calls_stay_out(attn, pdt, D):
    """A call whose cache is NaN leaves NaN in shared memory; short sequences right after it, whose
    tiles are mostly empty, see none of it (1 to 64 query rows a key/value head)."""
    bad = attn_problem(64, 1, 8, 2, D, 16, [512] * 64, pdt, seed=30, nan=False)
    for p in bad[1:3]:
        (p.view(torch.uint8) if pdt == F8 else p)[:] = 0x7F if pdt == F8 else float("nan")
    for T, Hq in ((1, 2), (1, 24), (1, 40), (1, 100), (3, 20)):
        prob = attn_problem(6, T, Hq, 2, D, 16, [1, 5, 16, 17, 33, 49], pdt, seed=31 + Hq)
        attn.paged_attention(*bad[:5], k_scale=bad[5], v_scale=bad[6])
        check_attn(attn, prob, pdt)


def test_attention_strided_and_token_major(attn):
    """Queries and outputs as views of wider tensors, pools laid out token by token."""
    q, kc, vc, table, lens, _, _ = attn_problem(2, 2, 8, 2, 64, 16, [77, 30], BF, seed=17)
    want, _ = check_attn(attn, (q, kc, vc, table, lens, None, None), BF)
    wide = torch.zeros(2, 2, 12, 96, dtype=BF, device="cuda")
    wide[:, :, 2:10, :64] = q
    outw = torch.zeros(2, 3, 8, 72, dtype=BF, device="cuda")
    tok = [p.transpose(1, 2).contiguous().transpose(1, 2) for p in (kc, vc)]
    got = attn.paged_attention(wide[:, :, 2:10, :64], *tok, table, lens, out=outw[:, :2, :, :64])
    assert torch.equal(got, want) and (outw[:, 2] == 0).all() and (outw[..., 64:] == 0).all()


@pytest.mark.parametrize("pdt", [BF, F8])
def test_attention_offsets_beyond_32_bits(attn, pdt):
    """Pools of more than 2^32 elements, the sequence in the last pages."""
    pages, Hkv, ps, D = 4200, 8, 1024, 128           # 4.4e9 elements a pool
    if torch.cuda.mem_get_info()[0] < 5 * pages * Hkv * ps * D:
        pytest.skip("not enough device memory")
    small = attn_problem(1, 1, 8, Hkv, D, ps, [1500], pdt, seed=18)
    q, kc, vc, table, lens, ks, vs = small
    want, _ = check_attn(attn, small, pdt)
    big = [torch.empty(pages, Hkv, ps, D, dtype=p.dtype, device="cuda") for p in (kc, vc)]
    sc = [None if s is None else torch.empty(pages, Hkv, ps, device="cuda") for s in (ks, vs)]
    far = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32).cuda()
    raw = (lambda t: t.view(torch.uint8)) if pdt == F8 else (lambda t: t)
    for i in range(2):
        for p, b in zip((kc, vc), big):
            raw(b)[far[0, i].long()] = raw(p)[table[0, i].long()]
        for s, b in zip((ks, vs), sc):
            if s is not None:
                b[far[0, i].long()] = s[table[0, i].long()]
    kw = dict(k_scale=sc[0], v_scale=sc[1])
    assert torch.equal(attn.paged_attention(q, *big, far, lens, **kw), want)
    cu = torch.tensor([0, 1500], dtype=torch.int32).cuda()
    near = attn.kv_read(kc, vc, table, cu, 1500, k_scale=ks, v_scale=vs)
    for a, b in zip(attn.kv_read(*big, far, cu, 1500, **kw), near):
        assert torch.equal(a, b)
    k, v = (x[:2].contiguous() for x in near)
    slots = torch.tensor([pages * ps - 1, (pages - 1) * ps], dtype=torch.int32).cuda()
    attn.kv_append(q[0].expand(2, 8, D).contiguous(), k, v, slots, *big, **kw)
    cu2, t2 = torch.tensor([0, 1], dtype=torch.int32).cuda(), torch.tensor([[pages - 1]], dtype=torch.int32).cuda()
    back = attn.kv_read(*big, t2, cu2, 1, **kw)[0]
    assert (np.abs(np64(back[0]) - np64(k[1])) <= 2.0 ** -3 * np.abs(np64(k[1])) + 1e-3).all()


def test_results_repeat_bit_for_bit_on_any_stream(attn):
    prob = attn_problem(5, 2, 8, 2, 128, 16, [700, 3, 64, 0, 1200], BF, seed=19)
    q, kc, vc, table, lens, _, _ = prob
    want, lw = attn.paged_attention(q, kc, vc, table, lens, return_lse=True)
    need = attn.paged_attention_workspace_size(5, 2, 8, 2, 128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for fill in (0, 255):                        # the workspace's contents do not matter
            ws = torch.full((max(need, 1),), fill, dtype=torch.uint8, device="cuda")
            got, lg = attn.paged_attention(q, kc, vc, table, lens, return_lse=True, workspace=ws)
            s.synchronize()
            assert torch.equal(got, want) and torch.equal(lg, lw)


def test_operators_in_a_graph(attn):
    """One decode step of an attention layer captured once and replayed with other lengths."""
    q, kc, vc, table, lens, _, _ = attn_problem(3, 1, 8, 2, 64, 16, [40, 90, 7], BF, seed=20, nan=False)
    x = torch.randn(3, 12, 64, device="cuda").to(BF)
    slots = torch.zeros(3, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(attn.paged_attention_workspace_size(3, 1, 8, 2, 64), 1), dtype=torch.uint8, device="cuda")
    qo, out = torch.empty(3, 8, 64, dtype=BF, device="cuda"), torch.empty(3, 1, 8, 64, dtype=BF, device="cuda")

    def step():
        attn.kv_append(x[:, :8], x[:, 8:10], x[:, 10:], slots, kc, vc, out=qo)
        attn.paged_attention(qo[:, None], kc, vc, table, lens, out=out, workspace=ws)

    def place(n):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        t = table.cpu()
        slots.copy_(torch.tensor([int(t[b, (m - 1) // 16]) * 16 + (m - 1) % 16 for b, m in enumerate(n)]))

    place([40, 90, 7])
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    place([33, 89, 1])
    g.replay()
    torch.cuda.synchronize()
    got = out.clone()
    step()
    assert torch.equal(got, out)
    check_attn(attn, (qo[:, None], kc, vc, table, lens, None, None), BF)


def test_empty_calls(attn):
    kc, vc, ks, vs = fill_pools(2, 2, 4, 64, BF, 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    e = torch.empty(0, 4, 64, dtype=BF, device="cuda")
    attn.kv_append(e, e[:, :2], e[:, :2], torch.empty(0, **i32), kc, vc)
    k, v = attn.kv_read(kc, vc, torch.zeros(1, 2, **i32), torch.zeros(2, **i32), 0)
    assert k.shape == (0, 2, 64)
    q = torch.empty(0, 1, 4, 64, dtype=BF, device="cuda")
    assert attn.paged_attention(q, kc, vc, torch.zeros(0, 2, **i32), torch.zeros(0, **i32)).shape == q.shape
    q = torch.ones(2, 1, 4, 64, dtype=BF, device="cuda")   # no table columns: no positions
    out = attn.paged_attention(q, kc, vc, torch.zeros(2, 0, **i32), torch.full((2,), 9, **i32))
    assert (out == 0).all()


@pytest.mark.parametrize("cache", ["fp8", "bf16"])
def test_example_runs_them_together(cache):
    """The hybrid example: its checks compare bf16 results of the same tokens by two paths.  The
    attention check differs by the probabilities' and the output's rounding (2^-8 each, of values
    up to a few times the largest output); decoding against one prompt accumulates a layer's
    bf16 roundings."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_decode.py")
    spec = importlib.util.spec_from_file_location("hybrid_decode", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    last, apart = mod.main(cache)
    assert last < 2e-2 and apart < 2e-2


DEBUG_CHILD = r"""
import ctypes, json, sys
sys.path[:0] = [sys.argv[1], sys.argv[1] + "/tests"]
import test_attn_gpu as t
from state_space_model_gb300 import _native, attn
import torch
assert _native.LIB_PATH.endswith("libssd_gb300_debug.so"), _native.LIB_PATH
for case in t.APPEND[:6]:
    t.check_append(attn, case)
for pdt in (t.BF, t.F8, t.F32):
    for case in t.ATTN[2:16:3]:
        T, Hq, Hkv, D, ps, lens, window = case
        prob = t.attn_problem(len(lens), T, Hq, Hkv, D, ps, lens, pdt, seed=T + Hq + ps)
        t.check_attn(attn, prob, pdt, window)
    prob = t.attn_problem(40, 1, 8, 2, 128, 16, [9 * i for i in range(39)] + [3000], pdt, seed=3)
    t.check_attn(attn, prob, pdt)
    t.test_read_matches_oracle(attn, pdt, t.BF if pdt == t.F8 else pdt, 64, 16, [5, 0, 33, 1])
lib = _native.load()
st = lib.ssd_device_status(ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
print(json.dumps({"status": st, "detail": lib.ssd_last_error_detail().decode()}))
"""


def test_debug_build_finds_every_index_in_bounds(attn):
    """The bounds-checked build runs the same checks, and none of its own fires."""
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
